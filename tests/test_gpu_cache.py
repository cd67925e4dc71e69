"""The paged cache's writer and reader (ops.msa_cache_write, ops.msa_cache_read) against a
plain walk over the page table: bf16 rows move unchanged, E4M3 codes and scales are those of
the oracle's quantiser bit for bit, and reading back is decode(code) * scale in 64 bits
rounded to bf16 (its float32 product is rounded twice, so it may be one bf16 step away only
where the exact value lies within 2^-24 of a rounding border: compared with half a step plus
2^-24 of the value)."""
import numpy as np
import pytest
import torch

from oracle import fp8 as oracle_fp8
from block_sparse_gqa_topk_gb300 import _lib, ops
from parity import bf16_to_np, f64

pytestmark = pytest.mark.gpu


def randn(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


class Pool:
    """A cache full of marked rows, and the host's copy of what it should hold."""

    def __init__(self, pages, page, H, d, di, fp8, seed=0):
        c = self.cache = ops.new_paged_cache(pages, H, page_size=page, d=d, d_idx=di, fp8=fp8)
        c.k.fill_(0x5A if fp8 else 3.0)
        c.v.fill_(0x5B if fp8 else 5.0)
        if di:
            c.k_idx.fill_(7.0)
        if fp8:
            c.k_scale.fill_(11.0)
            c.v_scale.fill_(13.0)
        self.want = {n: getattr(c, n).flatten(0, 1).cpu() for n in self.names()}

    def names(self):
        return [n for n in ("k", "v", "k_idx", "k_scale", "v_scale") if getattr(self.cache, n) is not None]

    def put(self, row, k, v, ki):
        w = self.want
        if ki is not None:
            w["k_idx"][row] = ki
        for n, x in (("k", k), ("v", v)):
            if self.cache.fp8:
                codes, s = oracle_fp8.quantize_rows(bf16_to_np(x))
                w[n][row], w[n + "_scale"][row] = torch.from_numpy(codes), torch.from_numpy(s)
            else:
                w[n][row] = x

    def check(self):
        for n in self.names():
            got = getattr(self.cache, n).flatten(0, 1).cpu()
            bits = {torch.bfloat16: torch.int16, torch.float32: torch.int32}.get(got.dtype, torch.uint8)
            assert torch.equal(got.view(bits), self.want[n].view(bits)), n


def table_for(lens, page, pages, seed, extra=2):
    """A shuffled page table: [B, max] with -1 past each sequence's pages."""
    need = [(n + page - 1) // page for n in lens]
    assert sum(need) <= pages
    order = np.random.default_rng(seed).permutation(pages)
    t = np.full((len(lens), max(need + [0]) + extra), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t


def dev(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


CASES = [  # page, H, d, d_idx, lens, new tokens
    (16, 1, 64, 32, [1], [1]),
    (16, 2, 64, 0, [40, 17, 16, 1], [40, 1, 16, 1]),
    (48, 3, 128, 64, [130, 48, 1, 97], [33, 48, 0, 2]),
    (128, 8, 128, 64, [700, 1, 128, 129, 0], [300, 1, 1, 129, 0]),
    (256, 5, 128, 32, [513], [257]),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_write_then_read(case, fp8):
    page, H, d, di, lens, new = CASES[case]
    pages = sum((n + page - 1) // page for n in lens) + 2
    pool = Pool(pages, page, H, d, di, fp8)
    t = table_for(lens, page, pages, case)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    k, v = randn((T, H, d), 1), randn((T, H, d), 2)
    if fp8 and T > 1:
        k[0] = 0  # an all-zero row takes scale 1
        v[1, 0] *= 2.0 ** 40
    ki = randn((T, di), 3) if di else None
    ops.msa_cache_write(pool.cache, dev(t), dev(lens), k, v, ki, cu_seqlens=dev(cu))
    assert ops.device_status() == 0
    rows = []
    for b in range(len(lens)):
        for i in range(new[b]):
            pos = lens[b] - new[b] + i
            row = int(t[b, pos // page]) * page + pos % page
            n = int(cu[b]) + i
            rows.append(row)
            pool.put(row, k[n].cpu(), v[n].cpu(), None if ki is None else ki[n].cpu())
    pool.check()
    # back, and two packed rows behind the last sequence
    gk, gv, gi = ops.msa_cache_read(pool.cache, dev(t), dev(lens), dev(cu), T + 2)
    assert ops.device_status() == 0
    assert gk.shape == (T + 2, H, d) and (gi is None) == (di == 0)
    if not fp8:
        assert torch.equal(gk[:T], k) and torch.equal(gv[:T], v)
    else:
        for n, g in (("k", gk), ("v", gv)):
            want = oracle_fp8.dequantize_rows(pool.want[n][rows].numpy(), pool.want[n + "_scale"][rows].numpy())
            off = np.abs(f64(g[:T]) - want)
            assert (off <= np.abs(want) * (2.0 ** -9 * 2 + 2.0 ** -24) + 1e-38).all(), n
    if di:
        assert torch.equal(gi[:T], ki)


def test_quantised_codes_over_all_significands():
    """Every pair of bf16 significands (a value's and its row's amax) over 24 exponents, both
    signs, and rows far below and above the usual range: the codes and scales of the oracle."""
    sig = np.arange(128, dtype=np.uint32)
    rows = []
    for shift in range(24):  # one value per significand of 2^-shift times the amax's binade
        for top in sig:
            x = ((127 - shift) << 7 | sig).astype(np.uint16)
            x[1::2] |= 0x8000
            row = np.concatenate([x, [(127 << 7) | top | (0x8000 if top % 3 == 0 else 0)]])
            rows.append(np.where((row & 0x7FFF) > ((127 << 7) | top), 0x8000, row))  # none above amax
    a = np.stack(rows)
    # rows of 128: the amax takes the place of a value in turn, so none is left out
    x = np.concatenate([np.where(np.arange(128) == k, a[:, 128:], a[:, :128]) for k in (0, 127)])
    extra = []
    for e in (1, 30, 66, 67, 186, 187, 240, 254):  # amax binades, tiny to huge
        extra.append(np.where(x[:256] & 0x7F80, np.clip((x[:256] & 0x7F80).astype(np.int64) + ((e - 127) << 7), 0,
                                                        e << 7) | (x[:256] & 0x807F), x[:256]).astype(np.uint16))
    x = np.concatenate([x] + extra).astype(np.uint16)
    T = len(x)
    page = 128
    c = ops.new_paged_cache((T + page - 1) // page, 1, page_size=page, d=128, d_idx=0, fp8=True)
    k = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16).view(T, 1, 128)
    t = dev(np.arange(c.num_pages)[None])
    ops.msa_cache_write(c, t, dev([T]), k, k, cu_seqlens=dev([0, T]))
    codes, scale = oracle_fp8.quantize_rows(x)
    for n in "kv":
        assert np.array_equal(getattr(c, n).flatten(0, 2)[:T].cpu().numpy(), codes)
        got = getattr(c, n + "_scale").flatten()[:T].cpu().numpy()
        assert np.array_equal(got.view(np.uint32), scale.view(np.uint32))
    assert ops.device_status() == 0


def test_one_token_a_sequence_and_empty_slots():
    """The decode step's write: no cu_seqlens, empty slots skipped, growing page by page."""
    page, H, d, di = 16, 2, 128, 64
    pool = Pool(12, page, H, d, di, True)
    t = table_for([40, 40, 40], page, 12, 4)
    for step, lens in enumerate([[1, 0, 16], [2, 0, 17], [0, 33, 18]]):
        k, v, ki = randn((3, H, d), 10 + step), randn((3, H, d), 20 + step), randn((3, di), 30 + step)
        ops.msa_cache_write(pool.cache, dev(t), dev(lens), k, v, ki)
        for b, n in enumerate(lens):
            if n:
                pool.put(int(t[b, (n - 1) // page]) * page + (n - 1) % page, k[b].cpu(), v[b].cpu(), ki[b].cpu())
    assert ops.device_status() == 0
    pool.check()


def test_strided_inputs_and_a_strided_table():
    """Views of one fused projection, an expanded value, misaligned rows and a table that is a
    slice of a wider one write what their contiguous copies write."""
    page, H, d, di, T = 16, 4, 64, 32, 23
    t = table_for([T], page, 4, 5)
    wide = torch.full((1, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + t.shape[1]] = dev(t)
    table = wide[:, 3:3 + t.shape[1]]
    cu, lens = dev([0, T]), dev([T])
    for pad in (0, 8, 3):
        flat = randn((T, 2 * H * d + di + pad), 6 + pad)
        k, v, ki = (x for x in torch.split(flat[:, pad:], [H * d, H * d, di], -1))
        k, v = k.unflatten(-1, (H, d)), v.unflatten(-1, (H, d))
        for vv in (v, v[:, :1].expand(T, H, d), v.transpose(0, 1).contiguous().transpose(0, 1)):
            for fp8 in (False, True):
                a, b = Pool(4, page, H, d, di, fp8), Pool(4, page, H, d, di, fp8)
                ops.msa_cache_write(a.cache, table, lens, k, vv, ki, cu_seqlens=cu)
                ops.msa_cache_write(b.cache, dev(t), lens, k.contiguous(), vv.contiguous(),
                                    ki.contiguous().clone(), cu_seqlens=cu)
                for n in a.names():
                    assert torch.equal(getattr(a.cache, n).view(torch.uint8), getattr(b.cache, n).view(torch.uint8))
    assert ops.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_places_that_do_not_exist(fp8):
    """Page ids outside the pool, lengths that are negative or past the table, more new tokens
    than length, a broken cu_seqlens: the status says so, those tokens are dropped (zeros when
    read), every other token and row is as it should be."""
    page, H, d, di = 16, 2, 64, 32

    def run(t, lens, cu, good):
        pool = Pool(6, page, H, d, di, fp8)
        T = 20
        k, v, ki = randn((T, H, d), 41), randn((T, H, d), 42), randn((T, di), 43)
        args = dev(t), dev(lens)
        ops.msa_cache_write(pool.cache, *args, k, v, ki, cu_seqlens=dev(cu))
        assert ops.device_status() == _lib.MSA_ERR_ARG
        for n, row in good.items():
            pool.put(row, k[n].cpu(), v[n].cpu(), ki[n].cpu())
        pool.check()
        gk, _, gi = ops.msa_cache_read(pool.cache, *args, dev(cu), T)
        assert ops.device_status() == _lib.MSA_ERR_ARG
        for n in range(T):
            if n in good:
                assert torch.equal(gi[n], ki[n])
            elif n < max(cu):
                assert not gk[n].any() and not gi[n].any()

    # sequence 0: 10 tokens on page 4; sequence 1: 10 tokens over pages 1 and a bad one
    rows = {n: 4 * page + n for n in range(10)}
    rows |= {10 + n: 1 * page + 9 + n for n in range(7)}
    for bad in (-1, 6, 2 ** 31 - 1, -(2 ** 31)):
        run([[4, 0], [1, bad]], [10, 19], [0, 10, 20], rows)
    first = {n: 4 * page + n for n in range(10)}
    run([[4, 0], [1, 2]], [10, 33], [0, 10, 20], first)        # past the table's 32 tokens
    run([[4, 0], [1, 2]], [10, -5], [0, 10, 20], first)        # negative length
    run([[4, 0], [1, 2]], [10, 2 ** 31 - 1], [0, 10, 20], first)
    run([[4, 0], [1, 2]], [10, 8], [0, 10, 20], first | {12 + n: 1 * page + n for n in range(8)})
    # cu_seqlens that starts late: tokens 0..2 belong to nobody
    run([[4, 0], [1, 2]], [7, 10], [3, 10, 20],
        {3 + n: 4 * page + n for n in range(7)} | {10 + n: 1 * page + n for n in range(10)})


def test_offsets_past_32_bits():
    """A pool of more than 2^31 values: its last page is written and read where it is."""
    page, H, d = 128, 8, 128
    pages = (1 << 31) // (page * H * d) + 2
    c = ops.PagedCache(*(torch.empty((pages, page, H, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"))
    t = dev([[pages - 1, 0]])
    k, v = randn((130, H, d), 51), randn((130, H, d), 52)
    cu = dev([0, 130])
    ops.msa_cache_write(c, t, dev([130]), k, v, cu_seqlens=cu)
    assert torch.equal(c.k[-1], k[:128]) and torch.equal(c.v[-1], v[:128])
    assert torch.equal(c.k[0, :2], k[128:])
    gk, gv, gi = ops.msa_cache_read(c, t, dev([130]), cu, 130)
    assert torch.equal(gk, k) and torch.equal(gv, v) and gi is None
    assert ops.device_status() == 0


def test_captured_step_and_special_values():
    """A captured write replays with new lengths and values; infinities and NaN in one row
    stay in that row (an E4M3 row of them has NaN codes, as msa_quantize_kv_fp8 gives)."""
    page, H, d, di = 16, 1, 64, 32
    pool = Pool(4, page, H, d, di, True)
    t = dev(table_for([40], page, 4, 7, extra=0))
    lens = dev([1])
    k, v, ki = randn((1, H, d), 61), randn((1, H, d), 62), randn((1, di), 63)
    ops.msa_cache_write(pool.cache, t, lens, k, v, ki)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.msa_cache_write(pool.cache, t, lens, k, v, ki)
    host = t.cpu().numpy()
    for n in range(1, 40):
        lens.fill_(n)
        for i, x in enumerate((k, v)):
            x.copy_(randn(x.shape, 70 + 2 * n + i))
        graph.replay()
        pool.put(int(host[0, (n - 1) // page]) * page + (n - 1) % page, k[0].cpu(), v[0].cpu(), ki[0].cpu())
    torch.cuda.synchronize()
    # k_idx rows all hold the same captured input
    pool.check()
    k[0, 0, 3] = float("inf")
    v[0, 0, 5] = float("nan")
    lens.fill_(40)
    graph.replay()
    x8, sc = ops.msa_quantize_kv_fp8(torch.cat([k, v]).view(1, 2, 1, d))
    row = int(host[0, 39 // page]) * page + 39 % page
    assert torch.equal(pool.cache.k.flatten(0, 1)[row], x8[0, 0])
    assert torch.equal(pool.cache.v.flatten(0, 1)[row], x8[0, 1])
    assert torch.equal(pool.cache.k_scale.flatten(0, 1)[row].view(torch.int32), sc[0, 0].view(torch.int32))
    assert ops.device_status() == 0


def test_refusals():
    c = ops.new_paged_cache(4, 2, page_size=16, d=64, d_idx=32)
    t, lens = dev([[0, 1]]), dev([1])
    k, v, ki = randn((1, 2, 64), 1), randn((1, 2, 64), 2), randn((1, 32), 3)
    for kw, err in [
        (dict(k=k.cpu()), ValueError), (dict(k=k.float()), TypeError), (dict(k=k[:, :1]), ValueError),
        (dict(v=v[..., :32]), ValueError), (dict(k_idx=None), ValueError), (dict(k_idx=ki[:, :16]), ValueError),
        (dict(page_table=t.long()), TypeError), (dict(page_table=t[0]), ValueError),
        (dict(lens=lens.cpu()), ValueError), (dict(lens=dev([1, 1])), ValueError),
        (dict(cu_seqlens=dev([0])), ValueError), (dict(cu_seqlens=lens.long()), TypeError),
        (dict(k=k.expand(2, 2, 64), v=v.expand(2, 2, 64), k_idx=ki.expand(2, 32)), ValueError),
        (dict(cache=None), TypeError),
    ]:
        args = dict(cache=c, page_table=t, lens=lens, k=k, v=v, k_idx=ki)
        args.update(kw)
        with pytest.raises(err):
            ops.msa_cache_write(**args)
    with pytest.raises(TypeError):
        ops.msa_cache_read(c, t, lens, None, 1)
    with pytest.raises(ValueError):
        ops.msa_cache_read(c, t, lens, dev([0, 1]), -1)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    for args, err in [
        ((z(2, 24, 2, 64), z(2, 24, 2, 64)), ValueError),            # page size
        ((z(2, 16, 2, 96), z(2, 16, 2, 96)), ValueError),            # d
        ((z(2, 16, 2, 64), z(2, 16, 1, 64)), ValueError),
        ((z(2, 16, 2, 64), z(2, 16, 2, 64), z(2, 16, 16)), ValueError),
        ((z(2, 16, 2, 64), z(2, 16, 2, 64), z(1, 16, 32)), ValueError),
        ((z(2, 16, 2, 64, dtype=torch.uint8), z(2, 16, 2, 64, dtype=torch.uint8)), ValueError),  # no scales
        ((z(2, 16, 2, 64), z(2, 16, 2, 64), None, z(2, 16, 2, dtype=torch.float32)), ValueError),
        ((z(2, 16, 2, 128)[..., :64], z(2, 16, 2, 64)), ValueError),
        ((z(2, 16, 2, 64).cpu(), z(2, 16, 2, 64)), ValueError),
    ]:
        with pytest.raises(err):
            ops.PagedCache(*args)


def test_a_cache_is_fixed_and_its_copy_has_its_own_pages():
    import copy
    c = ops.new_paged_cache(2, 1, page_size=16, d=64, d_idx=32, fp8=True)
    with pytest.raises(AttributeError):
        c.k = c.v
    d = copy.deepcopy(c)
    k, v, ki = randn((1, 1, 64), 1), randn((1, 1, 64), 2), randn((1, 32), 3)
    ops.msa_cache_write(d, dev([[0]]), dev([1]), k, v, ki)
    assert not c.k.any() and d.k.any() and torch.equal(d.k_idx[0, 0], ki[0])
