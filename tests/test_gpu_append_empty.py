"""msa_cache_append without sequences, at the C entry and through ops."""
import pytest
import torch

from block_sparse_gqa_topk_gb300 import _lib, ops
from test_gpu_append import KINDS, inputs, marked, same_pools
from test_gpu_cache import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", range(3))
def test_no_sequences(kind):
    """Three tokens and no sequence: the C call leaves its outputs and the pool as they are (include/msa.h),
    ops, whose outputs are new, gives zeros."""
    H_q, H, Hi, d, di, T = 4, 2, 2, 64, 32, 3
    c, untouched = (marked(4, H, 16, d, di, KINDS[kind]) for _ in "ab")
    rope, x = ops.new_rope(32), inputs(T, H_q, H, Hi, d, di, 3)
    pages, B = ops._pages_arg(c, dev([[0, 1]])[:0], dev([]))
    assert B == 0
    y, yi = torch.full((T, H_q, d), 7.0, device="cuda").bfloat16(), torch.full((T, Hi, di), 7.0, device="cuda").bfloat16()
    a = _lib.APPEND.pack(32, False, 32, 1.0, H_q, Hi, 1, H_q * d, d, H * d, d, H * d, d, Hi * di, di, di)
    cu = dev([0])
    rc = _lib.msa_cache_append(c._c, pages, dev([1]).data_ptr(), cu.data_ptr(), T, a, rope.turns.data_ptr(), None,
                               *(t.data_ptr() for t in x), y.data_ptr(), yi.data_ptr(),
                               torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == _lib.MSA_OK and (y == 7).all() and (yi == 7).all() and same_pools(c, untouched)
    y, yi = ops.msa_cache_append(c, dev([[0, 1]])[:0], dev([]), rope, *x, cu_seqlens=cu)
    assert not y.any() and not yi.any() and same_pools(c, untouched) and ops.device_status() == 0
