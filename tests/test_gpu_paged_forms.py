"""Forms of the paged decode that only long caches and far pages take, and infinite values in the
cache.  The reference and its tolerances are those of test_gpu_decode_paged.py."""
import math

import pytest
import torch

from block_sparse_gqa_topk_gb300 import _lib, ops
from test_gpu_decode_paged import SLACK, Batch, check_attention, check_dense, dev, query

pytestmark = pytest.mark.gpu


def dense_and_groups(batch, q):
    """The dense call on a workspace of the test's own, and the number of groups that a CTA served
    side by side: the call leaves it for its join, behind the sequences' work."""
    B, d = q.shape[0], batch.d
    pages = _lib.PAGE_TABLE.pack(batch.table.data_ptr(), B, batch.table.shape[1], batch.table.stride(0))
    n = _lib.msa_decode_paged_workspace_size(batch.cache._c, pages, q.shape[1], 0)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    _lib.check(_lib.msa_decode_paged_dense(
        batch.cache._c, pages, batch.lens_t.data_ptr(), q.shape[1], d ** -0.5, q.data_ptr(), o.data_ptr(),
        lse.data_ptr(), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream), "msa_decode_paged_dense")
    starts = ws[n - (4 * (B + 2) + 255) // 256 * 256:].view(torch.int32)
    return o, lse, int(starts[B + 1])


# lens, page, H_kv, G, d, groups side by side
SIDE_BY_SIDE = [
    ([131072] * 3 + [0, 77], 128, 8, 2, 64, 4),
    ([131072, 1, 131072, 131072, 90001], 64, 6, 3, 64, 2),
    ([60000, 0, 70001, 65, 100000, 16], 48, 8, 4, 128, 4),
    ([131000, 120001, 1, 0], 16, 6, 1, 128, 2),
    ([70000, 33, 0, 69999], 128, 12, 9, 128, 4),
    ([100000, 99, 80016], 256, 6, 16, 128, 2),
    ([131072, 7, 131072, 131001], 32, 8, 16, 64, 4),
    ([100000, 5], 128, 7, 4, 128, 1),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(SIDE_BY_SIDE)))
def test_groups_side_by_side(case, fp8):
    """Caches long enough that the warps of a CTA take 4 or 2 groups (by the number of groups) over
    the same tokens, with short and empty sequences beside them."""
    lens, page, H, G, d, side = SIDE_BY_SIDE[case]
    if fp8 and d == 128:
        lens = [2 * n if n > 1000 else n for n in lens]  # twice the tokens for as much work
    batch = Batch(lens, page, H, d, 0, fp8, seed=70 + case)
    q = query(len(lens), H * G, d, 80 + case)
    o, lse, groups = dense_and_groups(batch, q)
    assert groups == side
    check_dense(batch, q, d ** -0.5, o, lse)
    again = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert ops.device_status() == 0


@SLACK
@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (128, 9)])
@pytest.mark.parametrize("x", [math.inf, -math.inf])
def test_infinite_values_in_the_cache(x, d, G, slack):
    """bf16 pages with an infinite value in one key or value row.  A score of -inf is a key without
    weight, one of +inf makes its output NaN; an infinite value makes its column of the output
    infinite or NaN.  No other sequence, group or column changes."""
    lens = [300, 300]
    batch = Batch(lens, 16, 2, d, 0, False, seed=13, slack=slack)
    q = query(2, 2 * G, d, 14)
    q[1, G:, 3] = (q[1, G:, 3].abs() + 0.25) * (1 if x > 0 else -1)
    before = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    rows = batch.rows(1, 300)

    def put(name, value):
        pool = getattr(batch.cache, name).flatten(0, 1)
        old = pool[rows[217], 1, 3].clone()
        pool[rows[217], 1, 3] = value
        o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
        assert torch.equal(o[0], before[0][0]) and torch.equal(lse[0], before[1][0])
        assert torch.equal(o[1, :G], before[0][1, :G]) and torch.equal(lse[1, :G], before[1][1, :G])
        pool[rows[217], 1, 3] = old
        return o, lse

    o, lse = put("v", x)
    assert not torch.isfinite(o[1, G:, 3]).any() and torch.equal(lse, before[1])
    keep = [c for c in range(d) if c != 3]
    assert torch.equal(o[1, G:, keep], before[0][1, G:, keep])
    o, lse = put("k", x)  # scores of +inf
    assert torch.isnan(o[1, G:]).all() and not torch.isfinite(lse[1, G:]).any()
    o, lse = put("k", -x)
    check_attention(batch, 1, q, o, lse, lambda g: rows if g == 0 else torch.cat([rows[:217], rows[218:]]), d ** -0.5)
    assert ops.device_status() == 0


@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (128, 9)])
@pytest.mark.parametrize("L", [300, 20000])
def test_parts_without_a_finite_score(L, d, G):
    """Scores that are -inf for a run of keys longer than a CTA's part: the others' are the result;
    -inf for all keys: no weights, so NaN, and lse = -inf."""
    batch = Batch([L, 200], 16, 2, d, 0, False, seed=15, slack=8192 // 16 + 1)
    q = query(2, 2 * G, d, 16)
    q[..., 0] = q[..., 0].abs() + 0.25
    rows = batch.rows(0, L)
    k = batch.cache.k.flatten(0, 1)
    k[rows[L // 5:], :, 0] = -math.inf
    k[batch.rows(1, 200), 1, 0] = -math.inf
    o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    check_attention(batch, 0, q, o, lse, lambda g: rows[:L // 5], d ** -0.5)
    assert torch.isnan(o[1, G:]).all() and (lse[1, G:] == -math.inf).all()
    assert torch.isfinite(o[1, :G]).all() and torch.isfinite(lse[1, :G]).all()
    assert ops.device_status() == 0


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_far_pages_of_every_pool(fp8, wide):
    """Pages past 2^31 values of the key, value and index-key pools, in the short form and in the
    one of long caches."""
    page, H, d, di = 256, 1, 64, 64
    P = (1 << 31) // (page * d) + 3
    n = 4 * page - 29
    small = Batch([n, 130], page, H, d, di, fp8, seed=18, slack=8192 // page + 1 if wide else 0)
    c = small.cache
    at = [P - 1, 1, P - 3, P - 2, 0]  # of the pages that are held, in the table's order
    held = small.t[small.t >= 0].tolist()
    new = {p: a for p, a in zip(held, at)}
    pools = []
    for x in (c.k, c.v, c.k_idx, c.k_scale, c.v_scale):
        y = None if x is None else torch.empty((P, *x.shape[1:]), dtype=x.dtype, device="cuda")
        for p, a in new.items():
            if y is not None:
                y[a] = x[p]
        pools.append(y)
    far = ops.PagedCache(*pools)
    table = dev([[new.get(int(p), -1) for p in r] for r in small.t])
    q, qi = query(2, 4, d, 19), query(2, H, di, 20)
    for a, b in zip(ops.msa_decode_paged_dense(q, far, table, small.lens_t),
                    ops.msa_decode_paged_dense(q, c, small.table, small.lens_t)):
        assert torch.equal(a, b)
    for a, b in zip(ops.msa_decode_paged(q, qi, far, table, small.lens_t, 4),
                    ops.msa_decode_paged(q, qi, c, small.table, small.lens_t, 4)):
        assert torch.equal(a, b)
    assert ops.device_status() == 0
