"""Coded caches written and read in one call against many small ones, at sizes where a CTA takes from one token to
32, in one wave of CTAs or several: every byte of the pool, and every row read back."""
import pytest
import torch

from block_sparse_gqa_topk_gb300 import ops
from test_gpu_append import KINDS, marked, same_pools
from test_gpu_cache import dev, randn, table_for

pytestmark = pytest.mark.gpu

SIZES = [  # H, d, d_idx, tokens
    (1, 128, 64, 40007), (1, 64, 32, 2501), (1, 64, 0, 311), (2, 128, 64, 3001), (3, 64, 32, 13003), (5, 128, 0, 5003),
    (8, 64, 64, 20011), (8, 128, 64, 9729), (8, 128, 32, 19457), (32, 128, 64, 1303), (300, 64, 32, 157),
]


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("H,d,di,T", SIZES)
def test_one_call_or_many(H, d, di, T, kind):
    page, pieces = 48, 61
    pages = (T + page - 1) // page + 1
    t = dev(table_for([T], page, pages, 5))
    k, v, ki = randn((T, H, d), 1), randn((T, H, d), 2), randn((T, di), 3) if di else None
    a, b = (marked(pages, H, page, d, di, KINDS[kind]) for _ in "ab")
    ops.msa_cache_write(a, t, dev([T]), k, v, ki, cu_seqlens=dev([0, T]))
    step = (T + pieces - 1) // pieces
    cuts = [(i, min(T, i + step)) for i in range(0, T, step)]
    for i, j in cuts:
        ops.msa_cache_write(b, t, dev([j]), k[i:j], v[i:j], None if ki is None else ki[i:j], cu_seqlens=dev([0, j - i]))
    assert same_pools(a, b)
    whole = ops.msa_cache_read(a, t, dev([T]), dev([0, T]), T)
    parts = [ops.msa_cache_read(a, t, dev([j]), dev([0, j - i]), j - i) for i, j in cuts]
    for n, x in enumerate(whole):
        if x is not None:
            assert torch.equal(x, torch.cat([p[n] for p in parts]))
    if di:
        assert torch.equal(whole[2], ki)
    assert ops.device_status() == 0
