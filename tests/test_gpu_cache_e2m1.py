"""The 4-bit paged cache's writer and reader against the oracle's rows: codes and scales bit for bit,
values back exactly (a value has at most 6 significant bits, which bf16 holds)."""
import numpy as np
import pytest
import torch

from oracle import fp4
from block_sparse_gqa_topk_gb300 import _lib, ops
from parity import bf16_to_np, f64
from test_gpu_cache import CASES, dev, randn, table_for

pytestmark = pytest.mark.gpu

NAMES = ("k", "v", "k_idx", "k_scale", "v_scale")


class Pool:
    """A 4-bit cache full of marked rows, and the host's copy of what it should hold."""

    def __init__(self, pages, page, H, d, di):
        c = self.cache = ops.new_paged_cache(pages, H, page_size=page, d=d, d_idx=di, fp4=True)
        assert c.fp4 and not c.fp8 and c.d == d and c.k.shape == (pages, page, H, d // 2)
        assert c.k_scale.shape == (pages, page, H, 4 + d // 16)
        for i, n in enumerate(self.names()):
            getattr(c, n).fill_(7.0 if n == "k_idx" else 0x5A + i)
        self.want = {n: getattr(c, n).flatten(0, 1).cpu() for n in self.names()}

    def names(self):
        return [n for n in NAMES if getattr(self.cache, n) is not None]

    def put(self, row, k, v, ki):
        if ki is not None:
            self.want["k_idx"][row] = ki
        for n, x in (("k", k), ("v", v)):
            codes, s = fp4.quantize_rows(f64(x))
            self.want[n][row], self.want[n + "_scale"][row] = torch.from_numpy(codes), torch.from_numpy(s)

    def check(self):
        for n in self.names():
            got = getattr(self.cache, n).flatten(0, 1).cpu()
            bits = torch.int16 if n == "k_idx" else torch.uint8
            assert torch.equal(got.view(bits), self.want[n].view(bits)), n


@pytest.mark.parametrize("case", range(len(CASES)))
def test_write_then_read(case):
    page, H, d, di, lens, new = CASES[case]
    pages = sum((n + page - 1) // page for n in lens) + 2
    pool = Pool(pages, page, H, d, di)
    t = table_for(lens, page, pages, case)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    k, v = randn((T, H, d), 1), randn((T, H, d), 2)
    if T > 1:
        k[0] = 0
        v[1, 0] *= 2.0 ** 40
        k[1, 0, 16:32] = 0  # a block of zeros in a row that is not
        k[T - 1, H - 1, :16] *= 2.0 ** -24  # and one far below its row
    ki = randn((T, di), 3) if di else None
    ops.msa_cache_write(pool.cache, dev(t), dev(lens), k, v, ki, cu_seqlens=dev(cu))
    assert ops.device_status() == 0
    rows = []
    for b in range(len(lens)):
        for i in range(new[b]):
            pos = lens[b] - new[b] + i
            rows.append(int(t[b, pos // page]) * page + pos % page)
            n = int(cu[b]) + i
            pool.put(rows[-1], k[n].cpu(), v[n].cpu(), None if ki is None else ki[n].cpu())
    pool.check()
    gk, gv, gi = ops.msa_cache_read(pool.cache, dev(t), dev(lens), dev(cu), T + 2)  # and two rows behind the last
    assert ops.device_status() == 0
    assert gk.shape == (T + 2, H, d) and (gi is None) == (di == 0)
    for n, g in (("k", gk), ("v", gv)):
        want = fp4.dequantize_rows(pool.want[n][rows].numpy(), pool.want[n + "_scale"][rows].numpy())
        assert np.array_equal(f64(g[:T]), want), n
    if di:
        assert torch.equal(gi[:T], ki)


def write_rows(x):
    """A cache of one sequence that holds the rows x [T, d] (bf16 bits, uint16) as keys and values."""
    T, d = x.shape
    c = ops.new_paged_cache((T + 127) // 128, 1, d=d, d_idx=0, fp4=True)
    k = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16).view(T, 1, d)
    ops.msa_cache_write(c, dev(np.arange(c.num_pages)[None]), dev([T]), k, k, cu_seqlens=dev([0, T]))
    assert ops.device_status() == 0
    return c, k


def check_rows(c, k):
    T = len(k)
    codes, scales = fp4.quantize_rows(f64(k)[:, 0])
    for n in "kv":
        got_scales = getattr(c, n + "_scale").flatten(0, 2)[:T].cpu().numpy()
        assert np.array_equal(got_scales, scales)
        got = getattr(c, n).flatten(0, 2)[:T].cpu().numpy()
        fine = np.isfinite(f64(k)[:, 0]).reshape(T, -1, 16).all(-1).repeat(8, -1)  # else: any code
        assert np.array_equal(got[fine], codes[fine])
    return codes, scales


def test_codes_over_all_significands():
    """Every pair of bf16 significands (a value's and its block's largest) over 5 exponents and both
    signs, so every border between two codes; every block largest against the row's, over 20
    exponents, so every border between two block scales; rows over the whole range of bf16."""
    sig = np.arange(128)
    blocks = []
    for shift in range(5):
        for top in sig:
            x = (((127 - shift) << 7) | sig).astype(np.uint16)
            x[1::2] |= 0x8000
            x = np.where((x & 0x7FFF) > ((127 << 7) | top), 0x8000, x).reshape(-1, 8)
            blocks.append(np.concatenate([np.full((16, 1), (127 << 7) | top), x, x[:, ::-1][:, :7] ^ 0x8000], 1))
    x = np.concatenate(blocks).astype(np.uint16).reshape(-1, 128)
    scaled = []
    for shift in range(20):  # blocks of one value each under rows of every significand
        rows = np.zeros((128, 8, 16), dtype=np.uint16)
        rows[:, 0, 3] = (127 << 7) | sig
        for j in range(1, 8):
            rows[:, j, 5] = ((127 - shift) << 7) | (37 * j + 5 * sig) % 128
            rows[:, j, 9] = 0x8000 | ((126 - shift) << 7) | (11 * j + sig) % 128
        scaled.append(rows.reshape(128, 128))
    ends = []
    for e in (0, 1, 5, 11, 12, 13, 14, 60, 200, 242, 243, 244, 245, 253, 254):
        r = x[::97].copy()
        mag = (r & 0x7FFF).astype(np.int64) + ((e - 127) << 7)
        ends.append(np.where(r & 0x7FFF, (r & 0x8000) | np.clip(mag, 0, 0x7F7F), r).astype(np.uint16))
    c, k = write_rows(np.concatenate([x] + scaled + ends))
    check_rows(c, k)


@pytest.mark.parametrize("d", [64, 128])
def test_infinite_and_nan_values(d):
    """A block that holds one reads as NaN; the row's other blocks are what they are without it."""
    x = bf16_to_np(randn((12, d), 9)).astype(np.uint16)
    for r, (i, bits) in enumerate([(0, 0x7F80), (17, 0xFF80), (d - 1, 0x7FC0), (33, 0xFFFF), (16, 0x7F81)]):
        x[r, i] = bits
    c, k = write_rows(x)
    codes, scales = check_rows(c, k)
    back, _, _ = ops.msa_cache_read(c, dev([[0]]), dev([12]), dev([0, 12]), 12)
    want = fp4.dequantize_rows(codes, scales)
    assert np.array_equal(f64(back)[:, 0], want, equal_nan=True)
    assert np.isnan(want).sum() == 5 * 16


def test_one_token_a_sequence_and_empty_slots():
    page, H, d, di = 16, 2, 128, 64
    pool = Pool(12, page, H, d, di)
    t = table_for([40, 40, 40], page, 12, 4)
    for step, lens in enumerate([[1, 0, 16], [2, 0, 17], [0, 33, 18]]):
        k, v, ki = randn((3, H, d), 10 + step), randn((3, H, d), 20 + step), randn((3, di), 30 + step)
        ops.msa_cache_write(pool.cache, dev(t), dev(lens), k, v, ki)
        for b, n in enumerate(lens):
            if n:
                pool.put(int(t[b, (n - 1) // page]) * page + (n - 1) % page, k[b].cpu(), v[b].cpu(), ki[b].cpu())
    assert ops.device_status() == 0
    pool.check()


def test_strided_inputs():
    page, H, d, di, T = 16, 3, 64, 32, 23
    t, cu, lens = dev(table_for([T], page, 4, 5)), dev([0, T]), dev([T])
    for pad in (0, 8, 3):
        flat = randn((T, 2 * H * d + di + pad), 6 + pad)
        k, v, ki = (x for x in torch.split(flat[:, pad:], [H * d, H * d, di], -1))
        k, v = k.unflatten(-1, (H, d)), v.unflatten(-1, (H, d))[:, :1].expand(T, H, d)
        a, b = Pool(4, page, H, d, di), Pool(4, page, H, d, di)
        ops.msa_cache_write(a.cache, t, lens, k, v, ki, cu_seqlens=cu)
        ops.msa_cache_write(b.cache, t, lens, k.contiguous(), v.contiguous(), ki.contiguous().clone(), cu_seqlens=cu)
        for n in a.names():
            assert torch.equal(getattr(a.cache, n).view(torch.uint8), getattr(b.cache, n).view(torch.uint8))
    assert ops.device_status() == 0


def test_places_that_do_not_exist():
    """A page id outside the pool and a length past the table: those tokens are dropped, or zeros."""
    page, H, d, di = 16, 2, 64, 32
    pool = Pool(5, page, H, d, di)
    t = np.array([[0, 9], [1, 2], [3, 4]], dtype=np.int32)
    lens, cu = [20, 40, 17], [0, 20, 25, 42]
    k, v, ki = randn((42, H, d), 1), randn((42, H, d), 2), randn((42, di), 3)
    ops.msa_cache_write(pool.cache, dev(t), dev(lens), k, v, ki, cu_seqlens=dev(cu))
    assert ops.device_status() == _lib.MSA_ERR_ARG
    for i in range(16):
        pool.put(i, k[i].cpu(), v[i].cpu(), ki[i].cpu())
    for i in range(17):
        pool.put((3 + i // page) * page + i % page, k[25 + i].cpu(), v[25 + i].cpu(), ki[25 + i].cpu())
    pool.check()
    gk, gv, gi = ops.msa_cache_read(pool.cache, dev(t), dev(lens), dev(cu), 42)
    assert ops.device_status() == _lib.MSA_ERR_ARG
    assert not gk[16:25].any() and not gv[16:25].any() and not gi[16:25].any()
    assert torch.equal(gi[:16], ki[:16]) and torch.equal(gi[25:], ki[25:]) and gk[:16].any()


def test_refusals():
    k = torch.zeros(2, 16, 2, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2, 16, 2, 8, dtype=torch.uint8, device="cuda")
    assert ops.PagedCache(k, k.clone(), None, s, s.clone()).d == 64
    for scale in (s[..., :4].contiguous(), s[:1].contiguous(), s.float(), s[..., 0].contiguous()):
        with pytest.raises((ValueError, TypeError)):
            ops.PagedCache(k, k, None, s, scale)
    for args in ((k, k), (k, k, None, s), (k[..., :24].contiguous(), k[..., :24].contiguous(), None, s, s),
                 (k, k, None, s, s.cpu()), (k.bfloat16(), k.bfloat16(), None, s, s)):
        with pytest.raises((ValueError, TypeError)):
            ops.PagedCache(*args)
    with pytest.raises(ValueError):
        ops.new_paged_cache(2, 2, fp8=True, fp4=True)
