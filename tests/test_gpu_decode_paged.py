"""Decode over a paged cache (ops.msa_decode_paged_dense, ops.msa_decode_paged) against
attention in 64 bits over the rows that the page table names.

Tolerances, by arithmetic.  A score is a sum of d products of bf16 values in float32: its
error is at most e_s = (d + 4) 2^-23 scale sum_i |q_i k_i| (products exact, one rounding or
truncation an addition, and the scalings), taken at its largest over the keys.  A weight's
relative error is then at most e_s + 2^-21 (the exponential and the sums), and one part more
from its own rounding for the product with v: 2^-16 from the two bf16 parts, 2^-11 from fp16
(E4M3 cache).  o = sum w v / sum w moves by at most twice that times sum w |v| / sum w, and
its rounding to bf16 by 2^-8 of it.  lse moves by at most e_s and 2^-22 of its size."""
import math

import numpy as np
import pytest
import torch

from block_sparse_gqa_topk_gb300 import _lib, ops

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def dev(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


WIDE = "wide"  # a table for more than 8192 tokens: the form of long caches, however short these are
SLACK = pytest.mark.parametrize("slack", [1, WIDE])


class Batch:
    """Random pages, a shuffled table, and what no sequence holds filled with NaN."""

    def __init__(self, lens, page, H, d, di, fp8, seed=0, spare=2, slack=1):
        g = gen(seed)
        self.lens, self.page, self.H, self.d = list(lens), page, H, d
        need = [(n + page - 1) // page for n in lens]
        if slack is WIDE:
            slack = 8192 // page + 1
        P = sum(need) + spare
        order = np.random.default_rng(seed).permutation(P)
        t = np.full((len(lens), max(need + [0]) + slack), -1, dtype=np.int32)
        at = 0
        held = torch.zeros(P * page, dtype=torch.bool)
        for b, n in enumerate(need):
            t[b, :n] = order[at:at + n]
            at += n
            for i in range(n):
                r = int(t[b, i]) * page
                held[r:r + min(page, lens[b] - i * page)] = True
        self.t, self.table = t, dev(t)
        held = held.cuda().view(P, page)
        randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        k, v = randn(P, page, H, d).bfloat16(), randn(P, page, H, d).bfloat16()
        ki = randn(P, page, di).bfloat16() if di else None
        ks = vs = None
        if fp8:
            k, ks = ops.msa_quantize_kv_fp8(k)
            v, vs = ops.msa_quantize_kv_fp8(v)
            k[~held], v[~held] = 0x7F, 0x7F  # NaN codes
            ks[~held], vs[~held] = float("nan"), float("nan")
        else:
            k[~held], v[~held] = float("nan"), float("nan")
        if di:
            ki[~held] = float("nan")
        self.cache = ops.PagedCache(k, v, ki, ks, vs)
        self.lens_t = dev(lens)

    def rows(self, b, n):
        ids = torch.from_numpy(self.t[b, :(n + self.page - 1) // self.page].astype(np.int64)).cuda()
        return (ids[:, None] * self.page + torch.arange(self.page, device="cuda")).flatten()[:n]

    def values(self, name, rows, g):
        x = getattr(self.cache, name).flatten(0, 1)[rows, g]
        if self.cache.fp8:
            s = getattr(self.cache, name + "_scale").flatten(0, 1)[rows, g].double()
            return x.view(torch.float8_e4m3fn).double() * s[:, None]
        return x.double()


def check_attention(batch, b, q, o, lse, tokens, scale):
    """Row b against 64 bits: tokens(g) gives the pool rows that group g attends."""
    H, d = batch.H, batch.d
    G = q.shape[1] // H
    for g in range(H):
        h = slice(g * G, (g + 1) * G)
        rows = tokens(g)
        if len(rows) == 0:
            assert not o[b, h].any() and (lse[b, h] == -math.inf).all()
            continue
        k, v, qq = batch.values("k", rows, g), batch.values("v", rows, g), q[b, h].double()
        s = scale * (qq @ k.T)
        want = torch.logsumexp(s, -1)
        w = torch.exp(s - want[:, None])
        e_s = (d + 4) * 2.0 ** -23 * scale * (qq.abs() @ k.abs().T).amax(-1, keepdim=True)
        e_w = e_s + 2.0 ** -21 + (2.0 ** -11 if batch.cache.fp8 else 2.0 ** -16)
        tol = 2 * e_w * (w @ v.abs()) + 2.0 ** -8 * (w @ v).abs()
        off = (o[b, h].double() - w @ v).abs()
        assert (off <= tol).all(), (b, g, float((off - tol).max()))
        assert ((lse[b, h].double() - want).abs() <= e_s[:, 0] + 2.0 ** -22 * want.abs().clamp(min=1)).all()


def check_dense(batch, q, scale, o, lse, lens=None):
    for b, n in enumerate(batch.lens if lens is None else lens):
        check_attention(batch, b, q, o, lse, lambda g, n=n, b=b: batch.rows(b, n), scale)


def query(B, H_q, d, seed):
    return torch.randn(B, H_q, d, generator=gen(seed), device="cuda").bfloat16()


DENSE = [  # lens, page, H_kv, G, d
    ([1], 16, 1, 1, 64),
    ([0], 16, 1, 2, 64),
    ([15, 16, 17, 63, 64, 65, 0, 1], 16, 2, 3, 64),
    ([700], 16, 2, 4, 64),
    ([129, 1, 0, 5000, 333], 48, 3, 5, 128),
    ([128, 127, 2048], 128, 4, 8, 128),
    ([1000, 40], 256, 1, 12, 128),
    ([513, 0, 77], 64, 2, 16, 64),
    ([70001], 128, 1, 16, 128),
    ([1] * 300 + [0] * 20 + [200] * 30, 32, 2, 1, 64),
    ([64 * (i % 7) + i for i in range(140)], 16, 4, 2, 128),
    ([97, 1, 513, 0, 1100] * 5, 16, 3, 7, 64),
    ([97, 1, 513, 0, 400] * 8, 64, 4, 9, 128),
    ([97, 1, 200, 0, 65] * 30, 32, 4, 16, 64),
    ([4000], 32, 1, 16, 128),
]


@SLACK
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(DENSE)))
def test_dense(case, fp8, slack):
    lens, page, H, G, d = DENSE[case]
    batch = Batch(lens, page, H, d, 0, fp8, seed=case, slack=slack)
    q = query(len(lens), H * G, d, 100 + case)
    for scale in (None, 0.3):
        o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t, scale=scale)
        assert ops.device_status() == 0
        check_dense(batch, q, d ** -0.5 if scale is None else scale, o, lse)
        again = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t, scale=scale)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def check_selection(batch, b, n, q_idx, sets, topk):
    """The set in the oracle's order, where the border's scores are further apart than their
    own error: e = (d_idx + 4) 2^-23 sum |q k|, at its largest."""
    if n == 0:
        assert (sets == -1).all()
        return
    own = (n - 1) // 128
    M = min(topk - 1, own)
    k = batch.cache.k_idx.flatten(0, 1)[batch.rows(b, n)[:own * 128]].double()
    for g in range(batch.H):
        got = sets[g].tolist()
        assert got[M] == own and all(x == -1 for x in got[M + 1:]) and got[:M + 1] == sorted(set(got[:M + 1]))
        if M == 0:
            continue
        z = (k @ q_idx[g].double()).view(own, 128).amax(-1)
        best = torch.sort(z, dim=-1, descending=True, stable=True).indices[:M].tolist()
        if sorted(best) != got[:M]:
            e = (q_idx.shape[-1] + 4) * 2.0 ** -23 * float((k.abs() @ q_idx[g].double().abs()).max())
            border = float(z[best].min())
            assert all(float(z[c]) >= border - 2 * e for c in got[:M]), (b, g, got, best)


SPARSE = [  # lens, page, H_kv, G, d, d_idx, topk
    ([1], 16, 1, 1, 64, 32, 1),
    ([128, 129, 256, 257, 0, 1], 16, 2, 2, 64, 32, 2),
    ([2048], 128, 2, 4, 64, 32, 4),
    ([5000, 333, 129, 0], 48, 3, 5, 128, 64, 16),
    ([20001, 4096, 640], 64, 4, 8, 128, 64, 16),
    ([3000, 2561], 256, 24, 2, 64, 64, 20),
    ([9000], 128, 2, 16, 128, 32, 32),
    ([131, 5, 700] * 40, 16, 1, 12, 64, 64, 3),
    ([4000, 3969, 1100, 130], 16, 3, 4, 128, 64, 16),
    ([2000, 129, 0, 777] * 6, 48, 4, 16, 64, 32, 5),
    ([1000, 129, 0, 777] * 30, 32, 2, 8, 128, 32, 3),
    ([4096, 4095, 4050, 4049], 16, 4, 3, 64, 64, 32),
]


@SLACK
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(SPARSE)))
def test_sparse(case, fp8, slack):
    lens, page, H, G, d, di, topk = SPARSE[case]
    batch = Batch(lens, page, H, d, di, fp8, seed=50 + case, slack=0 if max(lens) == 4096 and slack == 1 else slack)
    q = query(len(lens), H * G, d, 200 + case)
    qi = query(len(lens), H, di, 300 + case)
    sets, o, lse = ops.msa_decode_paged(q, qi, batch.cache, batch.table, batch.lens_t, topk)
    assert ops.device_status() == 0
    host = sets.cpu()
    for b, n in enumerate(lens):
        check_selection(batch, b, n, qi[b], host[b], topk)

        def tokens(g, b=b, n=n):
            rows = batch.rows(b, n)
            return torch.cat([rows[:0]] + [rows[c * 128:(c + 1) * 128] for c in host[b, g].tolist() if c >= 0])

        check_attention(batch, b, q, o, lse, tokens, d ** -0.5)
    again = ops.msa_decode_paged(q, qi, batch.cache, batch.table, batch.lens_t, topk)
    assert all(torch.equal(x, y) for x, y in zip((sets, o, lse), again))


@pytest.mark.parametrize("fp8", [False, True])
def test_long_caches_and_many_sequences(fp8):
    """Long enough that groups are served side by side (1, 2 and 4 of them), enough sequences that
    a warp's lanes hold several, more blocks than the attention kernel selects from, more than the
    ranks hold, and scores that tie across them."""
    for lens, H in (([200001, 64], 6), ([150000, 99], 4), ([40000] * 6, 8)):
        batch = Batch(lens, 16, H, 64, 0, fp8, seed=61)
        q = query(len(lens), H * 2, 64, 62)
        o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
        check_dense(batch, q, 0.125, o, lse)
    lens = [(7 * i) % 190 for i in range(1500)]
    batch = Batch(lens, 16, 2, 64, 32, fp8, seed=63)
    q, qi = query(1500, 2, 64, 64), query(1500, 2, 32, 65)
    o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    sets, o2, lse2 = ops.msa_decode_paged(q, qi, batch.cache, batch.table, batch.lens_t, 2)  # all blocks
    for b in range(0, 1500, 37):
        check_attention(batch, b, q, o, lse, lambda g, b=b: batch.rows(b, lens[b]), 0.125)
        check_attention(batch, b, q, o2, lse2, lambda g, b=b: batch.rows(b, lens[b]), 0.125)
    empty = batch.lens_t == 0
    assert (lse[~empty] > -math.inf).all() and (lse[empty] == -math.inf).all() and not o[empty].any()
    assert torch.equal((sets >= 0).sum(-1), ((batch.lens_t + 127) // 128)[:, None].expand(-1, 2).long())
    for n, topk in ((140000, 16), (600000, 32)):  # 1094 and 4688 blocks
        batch = Batch([n, 1000], 128, 1, 64, 32, fp8, seed=66)
        ki = batch.cache.k_idx.flatten(0, 1)
        rows = batch.rows(0, n)
        ki[rows[5 * 128:9 * 128]] = ki[rows[128:256]].repeat(4, 1)  # five blocks that tie
        q, qi = query(2, 3, 64, 67), query(2, 1, 32, 68)
        qi[0, 0] = ki[rows[130]]  # and are among the best
        sets, o, lse = ops.msa_decode_paged(q, qi, batch.cache, batch.table, batch.lens_t, topk)
        host = sets.cpu()
        for b, m in enumerate((n, 1000)):
            check_selection(batch, b, m, qi[b], host[b], topk)

            def tokens(g, b=b, m=m):
                r = batch.rows(b, m)
                return torch.cat([r[:0]] + [r[c * 128:(c + 1) * 128] for c in host[b, g].tolist() if c >= 0])

            check_attention(batch, b, q, o, lse, tokens, 0.125)
    assert ops.device_status() == 0


@pytest.mark.parametrize("L", [4096, 8192])
@pytest.mark.parametrize("fp8", [False, True])
def test_contiguous_cache_as_pages_agrees_with_msa_decode(fp8, L):
    """msa_decode's cache [B, Lmax] is a paged cache with pages 0, 1, 2, ...: the same sets
    (exact ties among them, lower block first) and, within both roundings, the same output."""
    B, H, G, d, di, topk = 2, 2, 4, 128, 64, 6
    g = gen(7)
    k, v = (torch.randn(B, L, H, d, generator=g, device="cuda").bfloat16() for _ in "kv")
    # blocks that are block 0 scaled by 1, 2 or 4: runs of equal pooled scores
    ki = torch.randn(B, 1, 128, di, generator=g, device="cuda").bfloat16()
    ki = (ki * (2.0 ** torch.randint(0, 3, (L // 128,), generator=g, device="cuda"))[None, :, None, None].bfloat16())
    ki = ki.reshape(B, L, di).contiguous()
    q, qi, lens = query(B, H * G, d, 8), query(B, H, di, 9), dev([L, 3001])
    page = 128
    table = dev(np.arange(B * L // page).reshape(B, -1))
    paged = lambda x: x.view(-1, page, *x.shape[2:])  # noqa: E731
    if fp8:
        k, ks = ops.msa_quantize_kv_fp8(k)
        v, vs = ops.msa_quantize_kv_fp8(v)
        want = ops.msa_decode_fp8(q, qi, k, v, ks, vs, ki, lens, topk)
        cache = ops.PagedCache(paged(k), paged(v), paged(ki), paged(ks), paged(vs))
    else:
        want = ops.msa_decode(q, qi, k, v, ki, lens, topk)
        cache = ops.PagedCache(paged(k), paged(v), paged(ki))
    got = ops.msa_decode_paged(q, qi, cache, table, lens, topk)
    assert torch.equal(got[0], want[0])
    # msa_decode rounds its weights to bf16: 2^-8 of sum w |v| < 8 at most
    assert (got[1].float() - want[1].float()).abs().max() <= 2e-2
    assert (got[2] - want[2]).abs().max() <= 1e-3
    # with enough slots for every block, both forms attend the whole cache
    short = dev([1500, 900])
    _, o, lse = ops.msa_decode_paged(q, qi, cache, table, short, 32)
    o2, lse2 = ops.msa_decode_paged_dense(q, cache, table, short)
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -7 * o2.float().abs().max()
    assert (lse - lse2).abs().max() <= 1e-4


@SLACK
def test_value_scales_far_apart_and_small_queries(slack):
    """E4M3 rows whose scales differ by many orders of magnitude, and queries far from 1: the
    fp16 products keep their range."""
    for power, qpower in ((30, 0), (-30, 20), (60, -20), (-60, 0)):
        batch = Batch([300], 16, 1, 64, 0, True, seed=11, slack=slack)
        step = torch.linspace(-abs(power), 0, 16, device="cuda").round()
        batch.cache.v_scale.mul_(2.0 ** (step * (1 if power > 0 else -1))[None, :, None])
        batch.cache.k_scale.mul_(2.0 ** -qpower)
        q = (query(1, 4, 64, 12).float() * 2.0 ** qpower).bfloat16()
        o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
        check_dense(batch, q, 64 ** -0.5, o, lse)
    assert ops.device_status() == 0


@SLACK
def test_large_scores_and_infinite_rows(slack):
    """Scores in the thousands (one key takes all), and an infinite or NaN value in one
    sequence: its outputs are not finite, its neighbours' are untouched."""
    batch = Batch([300, 300], 16, 2, 64, 0, False, seed=13, slack=slack)
    q = (query(2, 4, 64, 14).float() * 200).bfloat16()
    o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    check_dense(batch, q, 64 ** -0.5, o, lse)
    row = int(batch.rows(1, 300)[217])
    batch.cache.v.flatten(0, 1)[row] = float("nan")
    o2, lse2 = ops.msa_decode_paged_dense(q * 0.01, batch.cache, batch.table, batch.lens_t)
    assert torch.isnan(o2[1]).all() and torch.isfinite(lse2).all() and torch.isfinite(o2[0]).all()
    batch.cache.k.flatten(0, 1)[row] = float("nan")
    o3, lse3 = ops.msa_decode_paged_dense(q * 0.01, batch.cache, batch.table, batch.lens_t)
    assert torch.isnan(lse3[1]).all() and torch.equal(o3[0], o2[0])


@pytest.mark.parametrize("slack", [0, WIDE])
@pytest.mark.parametrize("fp8", [False, True])
def test_places_that_do_not_exist(fp8, slack):
    """Bad lengths count as empty slots, bad page ids as zero rows; the status says so."""
    lens = [200, 300, 150]
    batch = Batch(lens, 16, 2, 64, 32, fp8, seed=15, slack=slack)
    q, qi = query(3, 4, 64, 16), query(3, 2, 32, 17)
    for bad in (-1, batch.t.shape[1] * 16 + 1, 2 ** 31 - 1, -(2 ** 31)):
        lt = dev([200, bad, 150])
        o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, lt)
        assert ops.device_status() == _lib.MSA_ERR_ARG
        check_dense(batch, q, 0.125, o, lse, [200, 0, 150])
        sets, o, lse = ops.msa_decode_paged(q, qi, batch.cache, batch.table, lt, 4)
        assert ops.device_status() == _lib.MSA_ERR_ARG
        assert (sets[1] == -1).all() and not o[1].any() and (lse[1] == -math.inf).all()
    P = batch.cache.num_pages
    for bad in (-1, P, 2 ** 31 - 1, -(2 ** 31)):
        t = batch.table.clone()
        t[1, 3] = bad
        o, lse = ops.msa_decode_paged_dense(q, batch.cache, t, batch.lens_t)
        assert ops.device_status() == _lib.MSA_ERR_ARG
        check_attention(batch, 0, q, o, lse, lambda g: batch.rows(0, 200), 0.125)
        rows = batch.rows(1, 300)
        for g in range(2):  # positions 48 .. 63 are rows of zeros
            h = slice(2 * g, 2 * g + 2)
            k, v = batch.values("k", rows, g), batch.values("v", rows, g)
            k[48:64], v[48:64] = 0, 0
            s = 0.125 * (q[1, h].double() @ k.T)
            assert (lse[1, h].double() - torch.logsumexp(s, -1)).abs().max() <= 1e-4
            assert (o[1, h].double() - torch.softmax(s, -1) @ v).abs().max() <= 1e-2
        sets, o, lse = ops.msa_decode_paged(q, qi, batch.cache, t, batch.lens_t, 4)
        assert ops.device_status() == _lib.MSA_ERR_ARG
        assert torch.isfinite(o).all() and torch.isfinite(lse).all() and int(sets.max()) <= 2
    empty = ops.PagedCache(torch.empty(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda"),
                           torch.empty(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda"))
    o, lse = ops.msa_decode_paged_dense(q, empty, dev(np.zeros((3, 0))), dev([0, 0, 0]))
    assert not o.any() and (lse == -math.inf).all() and ops.device_status() == 0
    # a pool without pages: whatever the table says is outside it, and reads as zero rows
    empty = ops.new_paged_cache(0, 2, page_size=16, d=64, d_idx=32, fp8=fp8)
    t = dev(np.zeros((3, batch.t.shape[1])))
    for call in (lambda: ops.msa_decode_paged_dense(q, empty, t, batch.lens_t),
                 lambda: ops.msa_decode_paged(q, qi, empty, t, batch.lens_t, 4)[1:]):
        o, lse = call()
        assert ops.device_status() == _lib.MSA_ERR_ARG and not o.any()
        assert (lse - torch.log(batch.lens_t.float())[:, None]).abs().max() <= 1e-5


def test_offsets_past_32_bits():
    """Pages beyond 2^31 values of the pool."""
    page, H, d = 128, 8, 128
    P = (1 << 31) // (page * H * d) + 3
    k, v = (torch.empty((P, page, H, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    ki = torch.empty((P, page, 64), dtype=torch.bfloat16, device="cuda")
    batch = Batch([300], page, H, d, 64, False, seed=18, slack=0)
    at = [P - 1, 0, P - 3]
    for x, y in ((k, batch.cache.k), (v, batch.cache.v), (ki, batch.cache.k_idx)):
        for i, n in enumerate(batch.t[0]):
            x[at[i]] = y[int(n)]
    cache, table = ops.PagedCache(k, v, ki), dev([at])
    q, qi = query(1, 32, d, 19), query(1, H, 64, 20)
    for a, b in zip(ops.msa_decode_paged_dense(q, cache, table, batch.lens_t),
                    ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)):
        assert torch.equal(a, b)
    for a, b in zip(ops.msa_decode_paged(q, qi, cache, table, batch.lens_t, 2),
                    ops.msa_decode_paged(q, qi, batch.cache, batch.table, batch.lens_t, 2)):
        assert torch.equal(a, b)
    assert ops.device_status() == 0


@SLACK
def test_streams_and_graphs(slack):
    """Two captured calls replayed together on two streams while lengths and queries change
    between replays: each has its own workspace and each gives the eager answer."""
    lens = [3000, 64, 0, 777]
    batches = [Batch(lens, 16, 2, 64, 32, f, seed=21 + f, slack=slack) for f in (False, True)]
    qs, qis = [query(4, 8, 64, 23 + i) for i in range(2)], [query(4, 2, 32, 25 + i) for i in range(2)]
    graphs, outs = [], []
    for i, bt in enumerate(batches):
        ops.msa_decode_paged(qs[i], qis[i], bt.cache, bt.table, bt.lens_t, 4)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append((*ops.msa_decode_paged(qs[i], qis[i], bt.cache, bt.table, bt.lens_t, 4),
                         *ops.msa_decode_paged_dense(qs[i], bt.cache, bt.table, bt.lens_t)))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in batches]
    for step in range(5):
        for i, bt in enumerate(batches):
            bt.lens_t.copy_(dev([max(0, n - 97 * step) for n in lens]))
            qs[i].copy_(query(4, 8, 64, 30 + 2 * step + i))
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for i, bt in enumerate(batches):
            want = (*ops.msa_decode_paged(qs[i], qis[i], bt.cache, bt.table, bt.lens_t, 4),
                    *ops.msa_decode_paged_dense(qs[i], bt.cache, bt.table, bt.lens_t))
            assert all(torch.equal(x, y) for x, y in zip(outs[i], want))
    assert ops.device_status() == 0


def test_refusals():
    batch = Batch([40, 20], 16, 2, 64, 32, False, seed=40)
    c, t, n, q, qi = batch.cache, batch.table, batch.lens_t, query(2, 4, 64, 41), query(2, 2, 32, 42)
    for kw, err in [
        (dict(q=q.cpu()), ValueError), (dict(q=q.float()), TypeError), (dict(q=q[:1]), ValueError),
        (dict(q=q[:, :3].contiguous()), ValueError), (dict(q=q[..., :32].contiguous()), ValueError),
        (dict(q=q.transpose(0, 1)), ValueError), (dict(q=query(2, 34, 64, 1)), ValueError),
        (dict(page_table=t.long()), TypeError), (dict(lens=n[:1]), ValueError), (dict(lens=n.cpu()), ValueError),
        (dict(cache=(c.k, c.v)), TypeError),
    ]:
        args = dict(q=q, cache=c, page_table=t, lens=n)
        args.update(kw)
        with pytest.raises(err):
            ops.msa_decode_paged_dense(**args)
        with pytest.raises(err):
            ops.msa_decode_paged(q_idx=qi, **args)
    for kw in (dict(topk=0), dict(topk=33), dict(q_idx=qi[:1]), dict(q_idx=qi[..., :16].contiguous()),
               dict(cache=ops.PagedCache(c.k, c.v))):
        args = dict(q=q, q_idx=qi, cache=c, page_table=t, lens=n)
        args.update(kw)
        with pytest.raises(ValueError):
            ops.msa_decode_paged(**args)
    for s in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(_lib.MSAError):
            ops.msa_decode_paged_dense(q, c, t, n, scale=s)
    o, lse = ops.msa_decode_paged_dense(q[:0], c, t[:0], n[:0])
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
