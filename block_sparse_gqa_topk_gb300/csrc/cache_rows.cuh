// cache_rows.cuh -- rows of a paged cache: where a call's tokens belong, and the codes that a row
// of bf16 values becomes (cache.cu, append.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "paged.cuh"
#include "small_div.cuh"

namespace msa {

// The packed tokens of a call and their pages.
struct TokenMap {
  PageView pages;
  const int32_t* lens;
  const int32_t* cu;  // null: one token a sequence
  int B;
};

constexpr int64_t kNoToken = -1;   // the packed row belongs to no sequence: left as it is
constexpr int64_t kNoPlace = -2;   // its place does not exist: recorded in the status word

// The sequence of packed token t and the token's position there; >= 0 (the position), or kNoToken or
// kNoPlace.
__device__ __forceinline__ int64_t token_position(const TokenMap& p, int t, int* sequence) {
  int b = t, after = 1;
  if (p.cu) {
    int lo = 0, hi = p.B - 1;  // last sequence that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(&p.cu[mid]) <= t) lo = mid; else hi = mid - 1;
    }
    b = lo;
    const int first = __ldg(&p.cu[b]), end = __ldg(&p.cu[b + 1]);
    if (t < first || t >= end) {
      // behind the last sequence is no error; anything else is a broken cu_seqlens
      return t >= first && b == p.B - 1 && end >= first ? kNoToken : kNoPlace;
    }
    after = end - t;
  }
  *sequence = b;
  const int len = __ldg(&p.lens[b]);
  if (!p.cu && len == 0) return kNoToken;  // an empty slot of a padded decode batch
  const int64_t pos = (int64_t)len - after;
  if (pos < 0 || len > (int64_t)p.pages.max_pages * p.pages.page_size) return kNoPlace;
  return pos;
}

// Pool row of packed token t, or kNoToken or kNoPlace.
__device__ __forceinline__ int64_t token_row(const TokenMap& p, int t) {
  int b;
  const int64_t pos = token_position(p, t, &b);
  if (pos < 0) return pos;
  const int64_t row = pool_row(p.pages, b, (int)pos);
  return row < 0 ? kNoPlace : row;
}

__device__ __forceinline__ float2 widen(uint32_t w) {  // two bf16
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// E4M3 codes of four bf16 pairs divided by sc; out of line, for rows at the ends of the range.
static __device__ __noinline__ uint2 divide8(uint4 w, float sc) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t c[2] = {0, 0};
#pragma unroll 1
  for (int e = 0; e < 4; ++e) {
    const uint32_t v = e == 0 ? u[0] : e == 1 ? u[1] : e == 2 ? u[2] : u[3];
    const float2 x = widen(v);
    const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x.x, sc), __fdiv_rn(x.y, sc)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t put = (two & 0xffffu) << (16 * (e & 1));
    if (e < 2) c[0] |= put; else c[1] |= put;
  }
  return make_uint2(c[0], c[1]);
}

// A row's scale amax / 448 (1 for an all-zero row), and its reciprocal r for quantize8: an
// approximate reciprocal with one Newton step.
__device__ __forceinline__ void row_scale(float amax, float* sc, float* r) {
  constexpr float kInv = 1.f / 448.f;
  const float q0 = amax * kInv;
  *sc = amax > 0.f ? fmaf(fmaf(-q0, 448.f, amax), kInv, q0) : 1.f;
  float r0;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(*sc));
  *r = fmaf(r0, fmaf(-*sc, r0, 1.f), r0);
}

// E4M3 codes of eight values at scale sc: the code nearest to the float32 quotient x / sc.  With r
// the rounded reciprocal, q0 = x r and the remainder x - q0 sc, which one fma gives exactly,
// q0 + r (x - q0 sc) is the rounded quotient (Markstein 1990; the scale above likewise); that
// scales and codes are those that division gives is checked over all pairs of bf16 significands.
// Rows whose amax leaves the range in which nothing underflows are divided.
__device__ __forceinline__ uint2 quantize8(uint4 w, float sc, float r) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  const float2 rr = make_float2(r, r), nn = make_float2(-sc, -sc);
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = widen(u[e]);
    const float2 q0 = fmul2(x, rr);
    float2 q = ffma2(ffma2(q0, nn, x), rr, q0);
    q = make_float2(copysignf(q.x, x.x), copysignf(q.y, x.y));  // a zero keeps its sign
    const uint32_t two = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    c[e >> 1] |= (two & 0xffffu) << (16 * (e & 1));
  }
  return make_uint2(c[0], c[1]);
}

// decode(code) * s of eight codes, rounded to bf16.
__device__ __forceinline__ uint4 dequantize8(uint2 c, float s) {
  uint32_t y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)((e < 2 ? c.x : c.y) >> (16 * (e & 1)));
    const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
    y[e] = pack_bf16(v.x * s, v.y * s);
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}


// ---------------------------------------------------------------------------
// 4-bit rows: E2M1 codes, an E4M3 scale for each 16 of them and a power of two for the row.
// ---------------------------------------------------------------------------
// Bytes of a row's scales: the row's (float32), then a block's each.
constexpr int e2m1_scale_bytes(int d) { return 4 + d / 16; }

// An E4M3 code as a float.
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
}

// The largest magnitude of 16 bf16 values; infinite or NaN where one of them is.
__device__ __forceinline__ float block_amax(uint4 lo, uint4 hi) {
  const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t m = u[0];  // magnitudes count, signs are of no account
#pragma unroll
  for (int e = 1; e < 8; ++e) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(u[e]));
  uint32_t h;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(h) : "r"(m), "r"(m >> 16));
  return __uint_as_float(h << 16 & 0x7fffffffu);
}

// The exponent field of a row's scale: of the smallest power of two s >= 2^-126 with amax <= 2688 s
// (2688 = 6 * 448 = 1.3125 * 2^11, the largest value of a block of the largest scale); 1 for amax = 0.
__device__ __forceinline__ int row_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 11 + ((u & 0x7fffffu) > 0x280000u);
  return u == 0 ? 127 : max(e, 1);
}

// Eight E2M1 codes of the values nearest to those of q.
__device__ __forceinline__ uint32_t narrow_e2m1(const float2 (&q)[4]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
  return w;
}

// The same of eight bf16 values x down / bs, divided; out of line, for rows at the ends of the range.
static __device__ __noinline__ uint32_t divide_e2m1(uint4 w, float down, float bs) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  float2 q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = widen(u[k]);
    q[k] = make_float2(__fdiv_rn(x.x * down, bs), __fdiv_rn(x.y * down, bs));
  }
  return narrow_e2m1(q);
}

// Codes of 16 bf16 values of largest magnitude amax (of the block) at the row scale 2^(e - 127), and
// their block scale, an E4M3 code:
//   block = E4M3 nearest to amax / 6 / row, at least 2^-9;  code = E2M1 nearest to x / (block row).
// amax / 6 by a product: with the rounded 1/6 (too large by 2^-25 of it) a quotient that lies on the
// border of two E4M3 numbers still rounds to the border, and one that does not is 2^-9 away from it,
// as amax has 8 significant bits.  The other quotient is x (r + s), rounded once, with 1 / block = r + s to 2^-42
// of it (r is at most 3 2^-23 of it too small; s leaves out the square of that, and its own rounding,
// 2^-45): what lies on the border of two codes (block times it has 8 bits) comes out as the border, and
// everything else is 2^-9 away.  r <= 1 / block, so that s is no negative number and a zero keeps its sign.
// A block that holds an infinity or a NaN gets the scale NaN, so that its values read as NaN.  At the
// largest row scale the block's ends at 320: 6 * 320 * 2^117 is the largest value that bf16 holds.
__device__ __forceinline__ uint2 quantize16(uint4 lo, uint4 hi, float amax, int e, uint32_t* block) {
  const float down = __uint_as_float((uint32_t)(254 - e) << 23);  // 1 / row
  const float t = fminf(fmaxf(amax * down * (1.f / 6.f), 0x1p-9f), e == 244 ? 320.f : 448.f);
  const uint32_t code = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
  const float bs = e4m3_value(code);
  *block = amax < INFINITY ? code : 0x7fu;
  // there the factors below leave the range
  if (__any_sync(0xffffffffu, e < 30 || e > 210)) return make_uint2(divide_e2m1(lo, down, bs), divide_e2m1(hi, down, bs));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(bs));
  r = fmaf(r, fmaf(-bs, r, 1.f), r);              // within an ulp
  r = __uint_as_float(__float_as_uint(r) - 2);    // and not above
  const float s = fmaf(-r, bs, 1.f) * r;
  const float2 rr = make_float2(r * down, r * down), ss = make_float2(s * down, s * down);
  const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float2 q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = widen(u[4 * h + k]);
      q[k] = ffma2(x, rr, fmul2(x, ss));
    }
    w[h] = narrow_e2m1(q);
  }
  return make_uint2(w[0], w[1]);
}

// A row of D bf16 values in D / 16 neighbouring lanes of a warp, 16 each, stored as codes (dst: the lane's)
// with the row's scales.  All lanes of the warp come here; those that are not `there` store nothing.
template <int D, int KIND>
__device__ __forceinline__ void store_codes(uint4 lo, uint4 hi, void* dst, uint8_t* scale, bool there) {
  constexpr int LPR = D / 16;
  const int sub = threadIdx.x % LPR;
  if constexpr (KIND == MSA_CACHE_E2M1) {
    const float most = block_amax(lo, hi);
    float amax = most < INFINITY ? most : 0.f;
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int e = row_exponent(amax);
    uint32_t block;
    const uint2 c = quantize16(lo, hi, most, e, &block);
    block <<= 8 * (sub & 3);  // the bytes of four lanes are a word
    block |= __shfl_xor_sync(0xffffffffu, block, 1);
    block |= __shfl_xor_sync(0xffffffffu, block, 2);
    if (!there) return;
    *static_cast<uint2*>(dst) = c;
    uint32_t* words = reinterpret_cast<uint32_t*>(scale);
    if ((sub & 3) == 0) words[1 + sub / 4] = block;
    if (sub == 1) words[0] = (uint32_t)e << 23;
  } else {
    const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 x = widen(u[e]);
      amax = fmax3(amax, fabsf(x.x), fabsf(x.y));
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const bool far = !(amax == 0.f || (amax > 1e-18f && amax < 1e18f));
    uint2 c0, c1;
    float sc;
    if (!__any_sync(0xffffffffu, far)) {
      float r;
      row_scale(amax, &sc, &r);
      c0 = quantize8(lo, sc, r);
      c1 = quantize8(hi, sc, r);
    } else {
      sc = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
      c0 = divide8(lo, sc);
      c1 = divide8(hi, sc);
    }
    if (!there) return;
    *static_cast<uint4*>(dst) = make_uint4(c0.x, c0.y, c1.x, c1.y);
    if (sub == 0) *reinterpret_cast<float*>(scale) = sc;
  }
}

// The keys and values of a call whose rows become codes.
struct CodedRows {
  const __nv_bfloat16* x[2];  // keys, values
  int64_t stride[2][2];       // of token, head
  uint8_t* pool[2];
  uint8_t* scale[2];
  int H;
  uint32_t div_2H;  // magic(2 H)
};

// The rows of tokens t0 .. t0 + nt - 1 by the whole CTA, D / 16 lanes a row: to the pool rows in s_row (negative:
// none), keys after turn(row, token, first value, lo, hi).
template <int D, int KIND, typename Turn>
__device__ __forceinline__ void store_rows(const CodedRows& p, int t0, int nt, const int64_t* s_row, Turn turn) {
  constexpr int LPR = D / 16, BITS = KIND == MSA_CACHE_E2M1 ? 4 : 8;
  constexpr int SCALE = KIND == MSA_CACHE_E2M1 ? e2m1_scale_bytes(D) : 4;
  const int lane = threadIdx.x & 31, rows = nt * 2 * p.H;
  for (int i0 = threadIdx.x - lane; i0 < rows * LPR; i0 += blockDim.x) {  // whole warps
    const int r = (i0 + lane) / LPR, sub = lane % LPR;
    const int tok = min(small_div(r, p.div_2H), nt - 1), hv = r - tok * 2 * p.H;
    const int v = hv >= p.H, h = v ? hv - p.H : hv;
    const int64_t row = s_row[tok];
    const bool there = r < rows && row >= 0;
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    const int64_t cell = there ? row * p.H + h : 0;
    if (there) {
      const __nv_bfloat16* x = p.x[v] + ((t0 + tok) * p.stride[v][0] + h * p.stride[v][1]);
      lo = __ldg(reinterpret_cast<const uint4*>(x + 16 * sub));
      hi = __ldg(reinterpret_cast<const uint4*>(x + 16 * sub + 8));
      if (!v) turn(x, tok, 16 * sub, lo, hi);
    }
    store_codes<D, KIND>(lo, hi, p.pool[v] + (cell * D + 16 * sub) * BITS / 8, p.scale[v] + cell * SCALE, there);
  }
}

// Eight E2M1 codes as four pairs of fp16 (exact).
__device__ __forceinline__ void widen_e2m1(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

// code * s of eight E2M1 codes in bf16 (s a block's scale times its row's: exact).
__device__ __forceinline__ uint4 dequantize_e2m1(uint32_t codes, float s) {
  uint32_t h[4], y[4];
  widen_e2m1(codes, h);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
    y[e] = pack_bf16(v.x * s, v.y * s);
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

}  // namespace msa
