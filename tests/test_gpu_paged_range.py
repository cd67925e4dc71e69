"""Decode over a paged cache at the ends of its values' range: queries, weights and scales far
apart, infinities.  The reference and its tolerances are those of test_gpu_decode_paged.py: the
bounds there are relative to the terms of each sum, so a term that is lost shows wherever the
larger ones are zero."""
import math

import pytest
import torch

from block_sparse_gqa_topk_gb300 import ops
from test_gpu_decode_paged import SLACK, Batch, check_attention, check_dense, query

pytestmark = pytest.mark.gpu


def both_forms(batch, q, qi, topk, check):
    """check(o, lse, tokens) for the dense call, and for the sparse one with the blocks it took."""
    o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    check(o, lse, lambda b, g: batch.rows(b, batch.lens[b]))
    sets, o, lse = ops.msa_decode_paged(q, qi, batch.cache, batch.table, batch.lens_t, topk)
    host = sets.cpu()

    def taken(b, g):
        rows = batch.rows(b, batch.lens[b])
        return torch.cat([rows[:0]] + [rows[c * 128:(c + 1) * 128] for c in host[b, g].tolist() if c >= 0])

    check(o, lse, taken)
    assert ops.device_status() == 0


@SLACK
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (64, 12), (128, 9)])
def test_infinite_queries(d, G, fp8, slack):
    """A query with an infinite value has scores of infinities and NaN only: its output is NaN, and
    every other head's is what it was."""
    lens = [300, 129]
    batch = Batch(lens, 16, 2, d, 32, fp8, seed=1, slack=slack)
    q, qi = query(2, 2 * G, d, 2), query(2, 2, 32, 3)
    bad = [(0, 1, math.inf), (1, 2 * G - 1, -math.inf)]
    for b, h, x in bad:
        q[b, h, 5] = x

    def check(o, lse, tokens):
        finite = torch.ones(o.shape[:2], dtype=torch.bool, device="cuda")
        for b, h, _ in bad:
            assert torch.isnan(o[b, h]).all() and not torch.isfinite(lse[b, h])
            finite[b, h] = False
        assert torch.isfinite(o[finite]).all() and torch.isfinite(lse[finite]).all()
        clean = torch.where(finite[..., None], q, 0)
        for b in range(2):
            got, gl = o[b].clone(), lse[b].clone()
            for h in (~finite[b]).nonzero().flatten().tolist():  # a zero query instead: the mean
                rows = tokens(b, h // G)
                got[h] = batch.values("v", rows, h // G).mean(0).bfloat16()
                gl[h] = math.log(len(rows))
            check_attention(batch, b, clean, got[None].expand(2, -1, -1), gl[None].expand(2, -1),
                            lambda g, b=b: tokens(b, g), d ** -0.5)

    both_forms(batch, q, qi, 2, check)


@SLACK
@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (64, 12), (128, 9)])
@pytest.mark.parametrize("power", [0, 6, 9, 12, 15, 24, 31, 40, 90, 120, -100])
def test_queries_with_an_outlier_channel(power, d, G, slack):
    """E4M3 pages: a channel of the query 2^power times the others, where every key is zero, does
    not decide the softmax and takes no bits from the others.  power < 0: a channel far below them."""
    batch = Batch([300, 129], 16, 2, d, 32, True, seed=4, slack=slack)
    batch.cache.k[..., 7] = 0
    q, qi = query(2, 2 * G, d, 5), query(2, 2, 32, 6)
    q[..., 7] *= 2.0 ** power
    if G == 4:
        q[:, 1] = query(2, 1, d, 7)[:, 0]  # and a head without one

    def check(o, lse, tokens):
        for b in range(2):
            check_attention(batch, b, q, o, lse, lambda g, b=b: tokens(b, g), d ** -0.5)

    both_forms(batch, q, qi, 2, check)


@SLACK
@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (64, 12), (128, 9)])
@pytest.mark.parametrize("power", [100, 118, -100, -118])
def test_queries_and_key_scales_far_from_one(power, d, G, slack):
    """E4M3 pages whose key scales undo a power of two in the queries."""
    batch = Batch([300, 129], 16, 2, d, 32, True, seed=4, slack=slack)
    batch.cache.k_scale.mul_(2.0 ** -power)
    q, qi = (query(2, 2 * G, d, 5).double() * 2.0 ** power).bfloat16(), query(2, 2, 32, 6)

    def check(o, lse, tokens):
        for b in range(2):
            check_attention(batch, b, q, o, lse, lambda g, b=b: tokens(b, g), d ** -0.5)

    both_forms(batch, q, qi, 2, check)


@SLACK
@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (64, 12), (128, 9)])
def test_a_huge_query_beside_small_ones(d, G, slack):
    """E4M3 pages: a query of 2^110 with a value far below it, in a group of queries near 2^-100."""
    batch = Batch([300, 129], 16, 2, d, 32, True, seed=4, slack=slack)
    batch.cache.k[..., 7] = 0
    batch.cache.k_scale.mul_(2.0 ** 100)
    q, qi = (query(2, 2 * G, d, 5).double() * 2.0 ** -100).bfloat16(), query(2, 2, 32, 6)
    q[:, 1] = 0
    q[:, 1, 7], q[:, 1, 8] = 2.0 ** 110, 2.0 ** -100

    def check(o, lse, tokens):
        for b in range(2):
            check_attention(batch, b, q, o, lse, lambda g, b=b: tokens(b, g), d ** -0.5)

    both_forms(batch, q, qi, 2, check)


@SLACK
@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (64, 12), (128, 9)])
@pytest.mark.parametrize("nats", [12, 16, 20])
def test_one_key_far_above_the_others(nats, d, G, slack):
    """E4M3 pages: a key `nats` above all others whose value is zero in half of the columns: there
    the others' values are the output."""
    n = 300
    batch = Batch([n], 16, 1, d, 0, True, seed=8, slack=slack)
    c, rows = batch.cache, batch.rows(0, n)
    g = torch.Generator(device="cuda").manual_seed(9)
    k = torch.randn(n, d, generator=g, device="cuda") * 0.1
    k[:, 0] = 0
    k[77, 0] = 1
    v = torch.rand(n, d, generator=g, device="cuda") + 0.5
    v[77, ::2] = 0
    for name, x in (("k", k), ("v", v)):
        codes, scale = ops.msa_quantize_kv_fp8(x.bfloat16().view(1, n, 1, d))
        getattr(c, name).flatten(0, 1)[rows] = codes[0]
        getattr(c, name + "_scale").flatten(0, 1)[rows] = scale[0]
    q = query(1, G, d, 10)
    q[..., 0] = nats * d ** 0.5
    o, lse = ops.msa_decode_paged_dense(q, c, batch.table, batch.lens_t)
    check_dense(batch, q, d ** -0.5, o, lse)
    assert ops.device_status() == 0


@SLACK
@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (64, 12), (128, 9)])
def test_subnormal_value_scales(d, G, slack):
    """E4M3 rows so small that their scales are subnormal float32 numbers count like any other."""
    batch = Batch([23, 300], 16, 2, d, 0, True, seed=11, slack=slack)
    batch.cache.v_scale.mul_(2.0 ** -120)
    scales = batch.cache.v_scale.flatten(0, 1)[batch.rows(1, 300)]
    assert float(scales.max()) < 2.0 ** -126 and float(scales.min()) > 0
    q = query(2, 2 * G, d, 12)
    o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    check_dense(batch, q, d ** -0.5, o, lse)
    # beside rows of ordinary size, and a row of zeros
    batch.cache.v_scale.flatten(0, 1)[batch.rows(1, 300)[100:]] *= 2.0 ** 120
    batch.cache.v_scale.flatten(0, 1)[batch.rows(0, 23)[5]] = 0
    o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    check_dense(batch, q, d ** -0.5, o, lse)
    assert ops.device_status() == 0


@SLACK
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (64, 12), (128, 9)])
@pytest.mark.parametrize("power", [8, 16, 24, 32, 60, 100])
def test_scores_of_any_size(power, d, G, fp8, slack):
    """Scores of 2^power and more, far apart: one key takes all, and its value is the output."""
    batch = Batch([300, 129], 16, 2, d, 32, fp8, seed=31, slack=slack)
    one = 0x38 if fp8 else 1.0  # E4M3 code of 1
    best = [17, 128]
    for b, n in enumerate(batch.lens):
        rows = batch.rows(b, n)
        k = batch.cache.k.flatten(0, 1)
        k[rows] = 0
        k[rows[best[b]], :, 0] = one
        if fp8:
            batch.cache.k_scale.flatten(0, 1)[rows] = 1
    q, qi = query(2, 2 * G, d, 32), query(2, 2, 32, 33)
    q[..., 0] = 2.0 ** power * d ** 0.5

    def check(o, lse, tokens):
        for b in range(2):
            for g in range(2):
                v = batch.values("v", batch.rows(b, batch.lens[b])[best[b]][None], g)
                h = slice(g * G, (g + 1) * G)
                # the weight: 2^-11 (fp16) or 2^-16 (two bf16 parts); the result's rounding: 2^-8
                assert ((o[b, h].double() - v).abs() <= (2.0 ** -8 + 2.0 ** -11) * v.abs()).all()
                score = q[b, h, 0].double() * d ** -0.5
                assert ((lse[b, h].double() / score - 1).abs() <= 2.0 ** -20).all()

    both_forms(batch, q, qi, 3, check)  # three blocks: all of them


def test_a_cache_without_heads_is_refused():
    with pytest.raises(ValueError):
        ops.new_paged_cache(2, 0, page_size=16, d=64, d_idx=32)
