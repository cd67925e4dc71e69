"""Decode over a 4-bit paged cache (ops.msa_decode_paged_dense, ops.msa_decode_paged) against
attention in 64 bits over the rows' values.

Tolerances: those of test_gpu_decode_paged.py (e_s, e_w and the rounding of o), as keys and values
enter the products exactly (6 significant bits) and the weights in fp16.  A weight times its value
row's scale is held relative to the largest such product, which is 2^15: below 2^-14 of fp16, 2^-29 of
the largest, it is rounded to a multiple of 2^-24, so by at most 2^-25: 2^-40 of the largest
(times a value's code and block scale).  A code is 0 for one value in eight, so the largest may
well miss a column, and that term is all that is left of it."""
import math

import numpy as np
import pytest
import torch

from oracle import fp4
from oracle.fp8 import e4m3_decode
from block_sparse_gqa_topk_gb300 import _lib, ops
from test_gpu_decode_paged import DENSE, SLACK, SPARSE, WIDE, Batch, check_selection, dev, gen, query

pytestmark = pytest.mark.gpu


TABLES = []  # the oracle's values of E2M1 and E4M3 codes


@pytest.fixture(autouse=True, scope="module")
def tables():
    TABLES[:] = [torch.from_numpy(x).cuda() for x in (fp4.e2m1_decode(np.arange(16)), e4m3_decode(np.arange(256)))]


class Batch4(Batch):
    """A Batch whose rows are random codes and scales; what no sequence holds reads as NaN."""

    def __init__(self, lens, page, H, d, di, seed=0, spare=2, slack=1):
        super().__init__(lens, page, H, d, di, False, seed, spare, slack)
        g = gen(seed + 1000)
        lost = torch.isnan(self.cache.k[..., :1])
        P = self.cache.num_pages
        pools = []
        for _ in "kv":
            codes = torch.randint(0, 256, (P, page, H, d // 2), generator=g, device="cuda", dtype=torch.uint8)
            scale = torch.empty(P, page, H, 4 + d // 16, dtype=torch.uint8, device="cuda")
            row = torch.randint(-9, -6, (P, page, H, 1), generator=g, device="cuda").float()
            scale[..., :4] = torch.exp2(row).view(torch.uint8)
            scale[..., 4:] = torch.randint(0x50, 0x7F, scale[..., 4:].shape, generator=g, device="cuda", dtype=torch.uint8)
            scale[..., 4:] = torch.where(lost, 0x7F, scale[..., 4:])  # NaN
            scale[..., :4] = torch.where(lost, 0xFF, scale[..., :4])
            pools += [codes, scale]
        self.cache = ops.PagedCache(pools[0], pools[2], self.cache.k_idx, pools[1], pools[3])

    def values(self, name, rows, g):
        codes = getattr(self.cache, name).flatten(0, 1)[rows, g]
        scales = getattr(self.cache, name + "_scale").flatten(0, 1)[rows, g]
        x = TABLES[0][torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
        x = x.unflatten(-1, (-1, 16)) * TABLES[1][scales[..., 4:].int()][..., None]
        return x.flatten(-2) * scales[..., :4].contiguous().view(torch.float32).double()

    def check_row(self, b, q, o, lse, tokens, scale):
        """Row b against 64 bits: tokens(g) gives the pool rows that group g attends."""
        G = q.shape[1] // self.H
        for g in range(self.H):
            h = slice(g * G, (g + 1) * G)
            rows = tokens(g)
            if len(rows) == 0:
                assert not o[b, h].any() and (lse[b, h] == -math.inf).all()
                continue
            k, v, qq = self.values("k", rows, g), self.values("v", rows, g), q[b, h].double()
            row = self.cache.v_scale.flatten(0, 1)[rows, g, :4].contiguous().view(torch.float32).double()[:, 0]
            s = scale * (qq @ k.T)
            want = torch.logsumexp(s, -1)
            w = torch.exp(s - want[:, None])
            e_s = (self.d + 4) * 2.0 ** -23 * scale * (qq.abs() @ k.abs().T).amax(-1, keepdim=True)
            e_w = e_s + 2.0 ** -21 + 2.0 ** -11
            least = 2.0 ** -40 * (w * row).amax(-1, keepdim=True) * (v.abs() / row.where(row > 0, 1.0)[:, None]).sum(0)
            tol = 2 * e_w * (w @ v.abs()) + 2.0 ** -8 * (w @ v).abs() + least
            off = (o[b, h].double() - w @ v).abs()
            assert (off <= tol).all(), (b, g, float((off - tol).max()))
            assert ((lse[b, h].double() - want).abs() <= e_s[:, 0] + 2.0 ** -22 * want.abs().clamp(min=1)).all()

    def taken(self, b, g, host):
        rows = self.rows(b, self.lens[b])
        return torch.cat([rows[:0]] + [rows[c * 128:(c + 1) * 128] for c in host[b, g].tolist() if c >= 0])

    def check_dense(self, q, scale, o, lse):
        for b, n in enumerate(self.lens):
            self.check_row(b, q, o, lse, lambda g, b=b, n=n: self.rows(b, n), scale)

    def check_sparse(self, q, qi, topk, sets, o, lse):
        host = sets.cpu()
        for b, n in enumerate(self.lens):
            check_selection(self, b, n, qi[b], host[b], topk)
            self.check_row(b, q, o, lse, lambda g, b=b: self.taken(b, g, host), self.d ** -0.5)


@SLACK
@pytest.mark.parametrize("case", range(len(DENSE)))
def test_dense(case, slack):
    lens, page, H, G, d = DENSE[case]
    batch = Batch4(lens, page, H, d, 0, seed=case, slack=slack)
    q = query(len(lens), H * G, d, 100 + case)
    for scale in (None, 0.3):
        o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t, scale=scale)
        assert ops.device_status() == 0
        batch.check_dense(q, d ** -0.5 if scale is None else scale, o, lse)
        again = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t, scale=scale)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@SLACK
@pytest.mark.parametrize("case", range(len(SPARSE)))
def test_sparse(case, slack):
    lens, page, H, G, d, di, topk = SPARSE[case]
    batch = Batch4(lens, page, H, d, di, seed=50 + case, slack=0 if max(lens) == 4096 and slack == 1 else slack)
    q, qi = query(len(lens), H * G, d, 200 + case), query(len(lens), H, di, 300 + case)
    got = ops.msa_decode_paged(q, qi, batch.cache, batch.table, batch.lens_t, topk)
    assert ops.device_status() == 0
    batch.check_sparse(q, qi, topk, *got)
    again = ops.msa_decode_paged(q, qi, batch.cache, batch.table, batch.lens_t, topk)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


LONG = [  # lens, H, page: enough work that a CTA serves 2 and 4 groups side by side
    ([480001, 64], 6, 128),
    ([720007, 1, 0, 16], 4, 16),
    ([351000], 8, 48),
    ([30000 + 17 * i for i in range(12)], 8, 128),
]


@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (64, 16), (128, 11)])
@pytest.mark.parametrize("case", range(len(LONG)))
def test_groups_side_by_side(case, d, G):
    lens, H, page = LONG[case]
    batch = Batch4(lens, page, H, d, 0, seed=61 + case)
    q = query(len(lens), H * G, d, 62)
    o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    batch.check_dense(q, d ** -0.5, o, lse)
    again = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert ops.device_status() == 0


def test_groups_side_by_side_without_a_page():
    """Ids outside the pool, whole runs and a page of half a unit: zero rows, which count in the softmax, as
    the cache with rows of zeros gives them."""
    lens, H, d, page = [360013], 8, 64, 16
    batch = Batch4(lens, page, H, d, 0, seed=71)
    q = query(1, H * 2, d, 72)
    t = batch.t.copy()
    bad = [0, 5, 6, 7, 4000, 22498, 22500]
    t[0, bad] = [-1, batch.cache.num_pages, 2 ** 31 - 1, -2, -1, -1, -1]
    o, lse = ops.msa_decode_paged_dense(q, batch.cache, dev(t), batch.lens_t)
    assert ops.device_status() == _lib.MSA_ERR_ARG
    for i in bad:
        for n in ("k_scale", "v_scale"):
            getattr(batch.cache, n)[int(batch.t[0, i])] = 0
    want = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    batch.check_dense(q, d ** -0.5, o, lse)
    assert ops.device_status() == 0


@SLACK
@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (64, 12), (128, 9)])
def test_ranges(d, G, slack):
    """Row scales far apart, block scales from the least to the largest, queries far from 1 and with
    values that fp16 beside the largest does not hold, scores that one key takes."""
    lens = [300, 129]
    for power, qpower in ((0, 0), (20, 0), (-20, 20), (60, -20), (0, 100), (0, -100)):
        batch = Batch4(lens, 16, 2, d, 32, seed=4, slack=slack)
        c = batch.cache
        rows = torch.linspace(-abs(power), 0, 16, device="cuda").round() * (1 if power > 0 else -1)
        row = c.v_scale[..., :4].contiguous().view(torch.float32) * torch.exp2(rows)[None, :, None, None]
        c.v_scale[..., :4] = row.view(torch.uint8)
        row = c.k_scale[..., :4].contiguous().view(torch.float32) * 2.0 ** -qpower
        c.k_scale[..., :4] = row.view(torch.uint8)
        if power == 0:
            c.k_scale[:, 3::5, :, 4] = 1  # 2^-9
            c.k_scale[:, 4::7, :, 5] = 0x7E  # 448
            c.k_scale[:, 1::9, :, 4:] = 0
        q, qi = (query(2, 2 * G, d, 5).float() * 2.0 ** qpower), query(2, 2, 32, 6)
        if power == 0:
            q[..., 7] *= 2.0 ** -34  # lost in fp16: the group's queries enter as they are
        if power == 20:
            q *= 300
        q = q.bfloat16()
        o, lse = ops.msa_decode_paged_dense(q, c, batch.table, batch.lens_t)
        batch.check_dense(q, d ** -0.5, o, lse)
        got = ops.msa_decode_paged(q, qi, c, batch.table, batch.lens_t, 2)
        batch.check_sparse(q, qi, 2, *got)
        assert ops.device_status() == 0


@SLACK
def test_not_finite(slack):
    """A block of NaN in a key takes its sequence's group, in a value the columns of its block; an
    infinite query takes its head; nothing else moves."""
    batch = Batch4([300, 300], 16, 2, 64, 0, seed=13, slack=slack)
    c = batch.cache
    q = query(2, 4, 64, 14)
    o, lse = ops.msa_decode_paged_dense(q, c, batch.table, batch.lens_t)
    row = int(batch.rows(1, 300)[217])
    kept = c.v_scale.flatten(0, 1)[row, 1, 4 + 2].clone()
    c.v_scale.flatten(0, 1)[row, 1, 4 + 2] = 0x7F
    o2, lse2 = ops.msa_decode_paged_dense(q, c, batch.table, batch.lens_t)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[1, 2:, 32:48] = True
    assert torch.isnan(o2[hit]).all() and torch.equal(o2[~hit], o[~hit]) and torch.equal(lse, lse2)
    c.v_scale.flatten(0, 1)[row, 1, 4 + 2] = kept
    c.k_scale.flatten(0, 1)[row, 0, 4] = 0x7F
    o3, lse3 = ops.msa_decode_paged_dense(q, c, batch.table, batch.lens_t)
    assert torch.isnan(o3[1, :2]).all() and torch.isnan(lse3[1, :2]).all()
    assert torch.equal(o3[0], o[0]) and torch.equal(o3[1, 2:], o[1, 2:])
    q[0, 1, 5] = math.inf
    o4, lse4 = ops.msa_decode_paged_dense(q, c, batch.table, batch.lens_t)
    assert torch.isnan(o4[0, 1]).all() and not torch.isfinite(lse4[0, 1])
    assert torch.isfinite(o4[0, [0, 2, 3]]).all()


@pytest.mark.parametrize("slack", [0, WIDE])
def test_places_that_do_not_exist(slack):
    """Bad lengths count as empty slots, bad page ids as zero rows; the status says so."""
    lens = [200, 300, 150]
    batch = Batch4(lens, 16, 2, 64, 32, seed=15, slack=slack)
    q, qi = query(3, 4, 64, 16), query(3, 2, 32, 17)
    want = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    for bad in (-1, batch.t.shape[1] * 16 + 1, 2 ** 31 - 1):
        o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, dev([200, bad, 150]))
        sets, o2, lse2 = ops.msa_decode_paged(q, qi, batch.cache, batch.table, dev([200, bad, 150]), 2)
        assert ops.device_status() == _lib.MSA_ERR_ARG
        assert not o[1].any() and not o2[1].any() and (lse[1] == -math.inf).all() and (sets[1] == -1).all()
        for b in (0, 2):
            batch.check_row(b, q, o, lse, lambda g, b=b: batch.rows(b, lens[b]), 0.125)
    for bad in (-1, batch.cache.num_pages, 2 ** 30):
        t = batch.t.copy()
        t[1, 3] = bad
        o, lse = ops.msa_decode_paged_dense(q, batch.cache, dev(t), batch.lens_t)
        assert ops.device_status() == _lib.MSA_ERR_ARG
        assert torch.isfinite(o).all() and torch.equal(o[0], want[0][0]) and torch.equal(lse[2], want[1][2])


def test_two_streams_and_two_graphs():
    """Calls on two streams, and two captured ones replayed together, do not share a workspace."""
    batches = [Batch4([3000, 9001, 0], 64, 2, 128, 64, seed=20 + i, slack=WIDE) for i in range(2)]
    qs = [(query(3, 8, 128, 30 + i), query(3, 2, 64, 40 + i)) for i in range(2)]

    def both(i):
        c = (batches[i].cache, batches[i].table, batches[i].lens_t)
        return (*ops.msa_decode_paged_dense(qs[i][0], *c), *ops.msa_decode_paged(*qs[i], *c, 5))

    want = [both(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                out = both(i)
            got.append(out)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(i)
        graphs.append((g, out))
    for _ in range(3):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert ops.device_status() == 0
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(want[i], got[i]))
        assert all(torch.equal(x, y) for x, y in zip(want[i], graphs[i][1]))


def test_far_pages():
    """A pool whose codes pass 2^31 bytes: pages beyond that are read where they are."""
    page, H, d, n = 128, 8, 128, 700
    pages = (2 ** 31) // (page * H * d // 2) + 40
    c = ops.new_paged_cache(pages, H, page_size=page, d=d, d_idx=64, fp4=True)
    table = dev([list(range(pages - 6, pages))])
    k, v, ki = query(n, H, d, 1), query(n, H, d, 2), query(n, 64, 64, 3)[:, 0]
    ops.msa_cache_write(c, table, dev([n]), k, v, ki, cu_seqlens=dev([0, n]))
    near = ops.new_paged_cache(6, H, page_size=page, d=d, d_idx=64, fp4=True)
    ops.msa_cache_write(near, dev([list(range(6))]), dev([n]), k, v, ki, cu_seqlens=dev([0, n]))
    assert torch.equal(c.k[-6:], near.k) and torch.equal(c.v_scale[-6:], near.v_scale)
    q, qi = query(1, 32, d, 4), query(1, H, 64, 5)
    a = ops.msa_decode_paged(q, qi, c, table, dev([n]), 3)
    b = ops.msa_decode_paged(q, qi, near, dev([list(range(6))]), dev([n]), 3)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert ops.device_status() == 0


def test_far_pages_of_a_long_call():
    """The same where the groups come together, for the dense call and for reading back."""
    page, H, d, n = 128, 8, 128, 121003
    own = (n + page - 1) // page
    pages = (2 ** 31) // (page * H * d // 2) + own + 40
    c = ops.new_paged_cache(pages, H, page_size=page, d=d, d_idx=64, fp4=True)
    near = ops.new_paged_cache(own, H, page_size=page, d=d, d_idx=64, fp4=True)
    table, near_table = dev([list(range(pages - own, pages))]), dev([list(range(own))])
    k, v, ki = query(n, H, d, 1), query(n, H, d, 2), query(n, 64, 64, 3)[:, 0]
    ops.msa_cache_write(c, table, dev([n]), k, v, ki, cu_seqlens=dev([0, n]))
    ops.msa_cache_write(near, near_table, dev([n]), k, v, ki, cu_seqlens=dev([0, n]))
    assert torch.equal(c.k[-own:], near.k) and torch.equal(c.v_scale[-own:], near.v_scale)
    q, qi = query(1, 32, d, 4), query(1, H, 64, 5)
    a = (*ops.msa_decode_paged(q, qi, c, table, dev([n]), 3), *ops.msa_decode_paged_dense(q, c, table, dev([n])),
         *ops.msa_cache_read(c, table, dev([n]), dev([0, n]), n))
    b = (*ops.msa_decode_paged(q, qi, near, near_table, dev([n]), 3),
         *ops.msa_decode_paged_dense(q, near, near_table, dev([n])),
         *ops.msa_cache_read(near, near_table, dev([n]), dev([0, n]), n))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert ops.device_status() == 0


@pytest.mark.parametrize("slack", [1, 2000])
def test_a_pool_without_pages(slack):
    """Every id is bad: zero rows, as the status says."""
    c = ops.new_paged_cache(0, 4, page_size=16, d=64, d_idx=32, fp4=True)
    q, qi = query(2, 8, 64, 1), query(2, 4, 32, 2)
    t = dev(np.zeros((2, 20 * slack)))
    o, lse = ops.msa_decode_paged_dense(q, c, t, dev([300, 17]))
    assert ops.device_status() == _lib.MSA_ERR_ARG
    assert not o.any() and torch.allclose(lse, torch.tensor([[300.0], [17.0]], device="cuda").log().expand(2, 8))
    sets, o, lse = ops.msa_decode_paged(q, qi, c, t, dev([300, 17]), 2)
    assert ops.device_status() == _lib.MSA_ERR_ARG and not o.any()


@pytest.mark.parametrize("d,G", [(64, 3), (128, 4), (128, 16)])
def test_three_sets_of_four_groups(d, G):
    """Twelve groups come together four at a time, on pages that end inside a unit."""
    lens, H = [90001, 5, 0, 33], 12
    batch = Batch4(lens, 48, H, d, 0, seed=81)
    q = query(len(lens), H * G, d, 82)
    o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    assert ops.device_status() == 0
    batch.check_dense(q, d ** -0.5, o, lse)


def test_long_calls_on_two_streams_and_in_two_graphs():
    """Calls whose groups come together, at the same time on two streams and replayed together."""
    batches = [Batch4([60000 + 31 * i, 30001], 64, 8, 128, 0, seed=90 + i) for i in range(2)]
    qs = [query(2, 32, 128, 92 + i) for i in range(2)]

    def call(i):
        return ops.msa_decode_paged_dense(qs[i], batches[i].cache, batches[i].table, batches[i].lens_t)

    want = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([call(i) for _ in range(3)])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for out in got[i] for x, y in zip(want[i], out))
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(i)
        graphs.append((g, out))
    for _ in range(3):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(want[i], graphs[i][1]))
    assert ops.device_status() == 0
