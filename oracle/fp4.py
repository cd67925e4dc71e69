"""4-bit cache rows (E2M1 codes, an E4M3 scale for each 16 values, a power of two for the row) in
plain numpy.

TEST INFRASTRUCTURE ONLY, like the rest of oracle/: imported by the tests and never by the library
under block_sparse_gqa_topk_gb300/.

The pages name 4-bit formats only as one of the precisions that the MSA attention kernels support
(Flash-MSA / fmha_sm100 paragraph of the MSA summary, 7minutos.es, "El codiseño del kernel"); they
give no recipe.  Reading taken here:
  * E2M1: 1 sign bit, 2 exponent bits (bias 1), 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6; two codes
    a byte, the even value in the low half;
  * row scale s: the smallest power of two >= 2^-126 with amax |x| <= 2688 s (2688 = 6 * 448), or 1
    for a row of zeros; amax over the blocks of 16 without an infinity or a NaN;
  * block scale t: the E4M3 number nearest to (block amax) / (6 s), ties to even, at least 2^-9 and
    at most 448 (320 where s is 2^117); NaN for a block with an infinity or a NaN;
  * code: the E2M1 number nearest to x / (t s), ties to the even code, at most 6; the sign is kept.
A row is d / 2 bytes of codes and 4 + d / 16 bytes of scales: s as float32, then the t of each block.
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_decode, e4m3_encode

_POS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_decode(codes) -> np.ndarray:
    """float64 value of 4-bit codes 0 .. 15."""
    c = np.asarray(codes, dtype=np.int64)
    return np.where(c & 8, -1.0, 1.0) * _POS[c & 7]


def e2m1_encode(x) -> np.ndarray:
    """Nearest code of each value (ties to the even code), at most 6."""
    a = np.minimum(np.abs(x), 6.0)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 7)
    lo = np.maximum(hi - 1, 0)
    up = (_POS[hi] - a < a - _POS[lo]) | ((_POS[hi] - a == a - _POS[lo]) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def quantize_rows(x):
    """x [..., d] (bf16 values as float64) -> codes uint8 [..., d / 2], scales uint8 [..., 4 + d / 16]."""
    x = np.asarray(x, dtype=np.float64)
    blocks = x.reshape(*x.shape[:-1], -1, 16)
    bad = ~np.isfinite(blocks).all(-1)
    clean = np.where(bad[..., None], 0.0, blocks)
    most = np.abs(clean).max(-1)
    amax = most.max(-1)
    m, e = np.frexp(np.where(amax > 0, amax / 2688, 0.25))  # 2688 s >= amax: s = 2^e, or 2^(e - 1) where m is 1/2
    e = np.where(amax > 0, np.maximum(e - (m == 0.5), -126), 0)
    s = np.exp2(e.astype(np.float64))
    t = np.clip(most / s[..., None] / 6, 2.0 ** -9, np.where(e == 117, 320.0, 448.0)[..., None])
    t = e4m3_encode(t)
    codes = e2m1_encode(clean / (e4m3_decode(t) * s[..., None])[..., None]).reshape(x.shape)
    t = np.where(bad, np.uint8(0x7F), t)
    row = s.astype(np.float32)[..., None].view(np.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), np.concatenate([row, t], -1).astype(np.uint8)


def dequantize_rows(codes, scales) -> np.ndarray:
    """float64 values of rows."""
    c = np.stack([codes & 15, codes >> 4], -1)
    x = e2m1_decode(c).reshape(*codes.shape[:-1], -1, 16) * e4m3_decode(scales[..., 4:])[..., None]
    s = np.ascontiguousarray(scales[..., :4]).view(np.float32).astype(np.float64)
    return x.reshape(*codes.shape[:-1], -1) * s
