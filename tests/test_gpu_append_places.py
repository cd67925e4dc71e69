"""ops.msa_cache_append with tokens that have no place: every byte of the pool, for every kind of cache.  What
should be there is what an append of the other tokens alone leaves (test_gpu_append.py has that against
msa_rope and msa_cache_write)."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_topk_gb300 import _lib, ops
from test_gpu_append import KINDS, inputs, marked, same_pools
from test_gpu_cache import dev

pytestmark = pytest.mark.gpu

TABLE = [[0, 1], [2, 3]]
BAD = [  # page table, lens, cu_seqlens; the tokens with a place, a range a sequence, and the lengths up to them
    ([[0, 9], [2, 3]], [20, 17], [0, 20, 37], (range(16), range(20, 37)), (16, 17)),
    ([[0, -1], [2, 3]], [20, 17], [0, 20, 37], (range(16), range(20, 37)), (16, 17)),
    ([[2 ** 31 - 1, 1], [2, 4]], [20, 17], [0, 20, 37], (range(16, 20), range(20, 36)), (20, 16)),
    (TABLE, [20, 33], [0, 20, 37], (range(20), range(0)), (20, 0)),
    (TABLE, [-3, 17], [0, 20, 37], (range(0), range(20, 37)), (0, 17)),
    (TABLE, [12, 17], [0, 20, 37], (range(8, 20), range(20, 37)), (12, 17)),
    (TABLE, [20, 0], [0, 20, 37], (range(20), range(0)), (20, 0)),
    (TABLE, [20, 2 ** 31 - 1], [0, 20, 37], (range(20), range(0)), (20, 0)),
    (TABLE, [20, 17], [0, 20, 10], (range(20), range(0)), (20, 0)),
    (TABLE, [20, 17], [3, 20, 37], (range(3, 20), range(20, 37)), (20, 17)),
]


@pytest.mark.parametrize("kind", range(3))
@pytest.mark.parametrize("case", range(len(BAD)))
def test_only_tokens_with_a_place_are_written(case, kind):
    table, lens, cu, kept, upto = BAD[case]
    page, H, d, di = 16, 2, 64, 32
    rope, x = ops.new_rope(32), inputs(40, 4, H, 2, d, di, 7)
    c, want = (marked(4, H, page, d, di, KINDS[kind]) for _ in "ab")
    y, yi = ops.msa_cache_append(c, dev(table), dev(lens), rope, *x, cu_seqlens=dev(cu))
    assert ops.device_status() == _lib.MSA_ERR_ARG
    rows = [t for r in kept for t in r]
    at = torch.tensor(rows, device="cuda")
    want_y, want_yi = torch.zeros_like(y), torch.zeros_like(yi)
    new = np.concatenate([[0], np.cumsum([len(r) for r in kept])])
    good = ops.msa_cache_append(want, dev(TABLE), dev(upto), rope, *(z[at] for z in x), cu_seqlens=dev(new))
    assert ops.device_status() == 0
    want_y[at], want_yi[at] = good
    assert torch.equal(y, want_y) and torch.equal(yi, want_yi)
    assert same_pools(c, want)


@pytest.mark.parametrize("kind", range(3))
def test_a_decode_step_with_lost_slots(kind):
    """One token a sequence, four sequences: an id outside the pool, a length past the table, a negative one."""
    page, H, d, di = 16, 2, 128, 64
    rope, x = ops.new_rope(64), inputs(4, 4, H, 2, d, di, 9)
    c, want = (marked(4, H, page, d, di, KINDS[kind]) for _ in "ab")
    y, yi = ops.msa_cache_append(c, dev([[0], [4], [1], [2]]), dev([3, 5, 17, -1]), rope, *x)
    assert ops.device_status() == _lib.MSA_ERR_ARG
    good = ops.msa_cache_append(want, dev([[0]]), dev([3]), rope, *(z[:1] for z in x))
    assert torch.equal(y[:1], good[0]) and torch.equal(yi[:1], good[1]) and not y[1:].any() and not yi[1:].any()
    assert same_pools(c, want) and ops.device_status() == 0
