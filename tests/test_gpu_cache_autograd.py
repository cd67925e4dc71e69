"""msa_cache_write changes the pool's tensors, and autograd knows it."""
import pytest
import torch

from block_sparse_gqa_topk_gb300 import ops

pytestmark = pytest.mark.gpu


def step(cache, seed=0):
    g = torch.Generator().manual_seed(seed)
    H, d, di = cache.H_kv, cache.d, cache.d_idx
    k, v, ki = (torch.randn(s, generator=g).bfloat16().cuda() for s in ((1, H, d), (1, H, d), (1, di)))
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    ops.msa_cache_write(cache, table, lens, k, v, ki if di else None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d_idx", [0, 32])
def test_a_write_is_a_change_of_every_pool(fp8, d_idx):
    c = ops.new_paged_cache(2, 2, page_size=16, d=64, d_idx=d_idx, fp8=fp8)
    pools = [x for x in (c.k, c.v, c.k_idx, c.k_scale, c.v_scale) if x is not None]
    before = [x._version for x in pools]
    step(c)
    assert all(x._version > n for x, n in zip(pools, before))
    # a call without tokens changes nothing
    before = [x._version for x in pools]
    e = torch.empty(0, dtype=torch.bfloat16, device="cuda")
    ops.msa_cache_write(c, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int32, device="cuda"), e.view(0, 2, 64), e.view(0, 2, 64),
                        e.view(0, d_idx) if d_idx else None,
                        cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert [x._version for x in pools] == before


def test_a_saved_pool_that_was_written_is_noticed():
    c = ops.new_paged_cache(2, 2, page_size=16, d=64, d_idx=32)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = (w * c.k).sum()
    step(c)
    with pytest.raises(RuntimeError):
        y.backward()


def test_pools_of_inference_mode():
    with torch.inference_mode():
        c = ops.new_paged_cache(2, 2, page_size=16, d=64, d_idx=32)
        step(c)
    step(c)
    assert c.k.any() and ops.device_status() == 0
