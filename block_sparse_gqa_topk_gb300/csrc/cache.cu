// cache.cu -- tokens into a paged cache and back (see include/msa.h).
//
// A row is one head's key or value of a token (d values), or the token's index key; it
// moves through the lanes of a part of a warp.  An E4M3 cache stores
//   s = amax |x| / 448 (1 for an all-zero row),  code = E4M3 nearest to x / s,
// the rule of msa_quantize_kv_fp8 bit for bit (IEEE divisions), and reads back
// decode(code) * s rounded once to bf16.  Both directions are bound by HBM: every row is
// read once and written once.
#include <cuda_fp8.h>
#include <math.h>

#include "kernels.h"
#include "paged.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;

struct CacheParams {
  PageView pages;
  const int32_t* lens;
  const int32_t* cu;  // null: one token a sequence
  int B, T, H;
  void* k;  // pool
  void* v;
  float* k_scale;
  float* v_scale;
  __nv_bfloat16* k_idx;
  __nv_bfloat16* xk;  // packed rows: read by the write, written by the read
  __nv_bfloat16* xv;
  __nv_bfloat16* xi;
  int64_t sk[2], sv[2], si;  // their strides: token, head; token
  int per;                   // tokens of a warp
  int d_idx;
  int* status;
};

constexpr int64_t kNoToken = -1;   // the packed row belongs to no sequence: left as it is
constexpr int64_t kNoPlace = -2;   // its place does not exist: recorded in the status word

__device__ __forceinline__ int64_t token_row(const CacheParams& p, int t) {
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
  const int len = __ldg(&p.lens[b]);
  if (!p.cu && len == 0) return kNoToken;  // an empty slot of a padded decode batch
  const int64_t pos = (int64_t)len - after;
  if (pos < 0 || len > (int64_t)p.pages.max_pages * p.pages.page_size) return kNoPlace;
  const int64_t row = pool_row(p.pages, b, (int)pos);
  return row < 0 ? kNoPlace : row;
}

__device__ __forceinline__ float2 widen(uint32_t w) {  // two bf16
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// E4M3 codes of four bf16 pairs divided by sc; out of line, for rows at the ends of the range.
__device__ __noinline__ uint2 divide8(uint4 w, float sc) {
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

// A token's keys, and its values, are one run of H D values in the pool; a lane moves 8 values
// of it at a time (16 of E4M3: half the addresses and scales), a warp one token after another.
// Its lanes find the places of all its tokens (at most 32) together, so the chain of lookups
// (sequence, length, page) is paid once, and while it works on STEPS vectors a lane, the next ones
// are on their way.  32K tokens of 8 groups, d 128, with index keys: bf16 41 us each way (6.8
// TB/s), E4M3 write 40 us (bound by instructions: the rounding rule) and read 35 us (6 TB/s).
template <int D, bool F8, bool WRITE>
struct Lanes {
  static constexpr int VALUES = F8 ? 16 : 8;  // of a lane's vector
  static constexpr int LPR = D / VALUES;      // lanes of a head's row
  static constexpr int STEPS = F8 && WRITE ? 1 : 2;
};

// STEPS vectors a lane of one token, loaded; where they go.
template <int D, bool F8, bool WRITE>
struct Batch {
  using L = Lanes<D, F8, WRITE>;
  static constexpr int W = L::VALUES / 8;  // 16-byte vectors of a lane in the packed rows
  uint4 w[L::STEPS][W];                    // (16 codes of the pool: the first)
  float s[L::STEPS];
  uint4* dst[L::STEPS];                    // null: nothing to store
  float* scale[L::STEPS];
};

// As many as the registers of a batch allow; writing E4M3 with a vector a lane on the way and 4
// CTAs is faster than with two vectors and 3 (32K tokens, 8 groups, d 128).
template <bool F8, bool WRITE>
constexpr int kCtasPerSm = F8 && WRITE ? 4 : F8 ? 3 : 4;

template <int D, bool F8, bool WRITE>
__global__ void __launch_bounds__(kThreads, (kCtasPerSm<F8, WRITE>)) cache_kernel(const __grid_constant__ CacheParams p) {
  using L = Lanes<D, F8, WRITE>;
  using B = Batch<D, F8, WRITE>;
  constexpr int W = B::W;
  const int lane = threadIdx.x & 31;
  const int64_t t0 = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * p.per;
  if (t0 >= p.T) return;
  const int n = (int)min((int64_t)p.per, p.T - t0);
  int64_t place = kNoToken;
  if (lane < n) {
    place = token_row(p, (int)t0 + lane);
    if (place == kNoPlace) set_status(p.status, MSA_ERR_ARG);
  }
  const int half = p.H * L::LPR, units = 2 * half;  // vectors of the keys, and of the values too
  int next_i = 0, next_u = 0;                       // token and first vector of the next batch
  auto fetch = [&](B& b) {
    const int64_t row = __shfl_sync(0xffffffffu, place, next_i), t = t0 + next_i;
    const bool there = row >= 0;                     // a missing place reads as zeros
    const bool skip = WRITE ? !there : row == kNoToken;
    const int64_t cell = (there ? row : 0) * p.H;
#pragma unroll
    for (int k = 0; k < L::STEPS; ++k) {
      const int u = next_u + 32 * k + lane;
      const bool v = u >= half;
      const int f = v ? u - half : u, h = f / L::LPR, sub = f % L::LPR;
      __nv_bfloat16* x = v ? p.xv + t * p.sv[0] + h * p.sv[1] : p.xk + t * p.sk[0] + h * p.sk[1];
      uint4* packed = reinterpret_cast<uint4*>(x + sub * L::VALUES);
      void* pool = static_cast<uint8_t*>(v ? p.v : p.k) + (cell * D + f * L::VALUES) * (F8 ? 1 : 2);
      if (F8) b.scale[k] = (v ? p.v_scale : p.k_scale) + cell + h;
#pragma unroll
      for (int e = 0; e < W; ++e) b.w[k][e] = make_uint4(0, 0, 0, 0);
      b.s[k] = 0.f;
      b.dst[k] = nullptr;
      if (u >= units || skip) continue;
      b.dst[k] = WRITE ? static_cast<uint4*>(pool) : packed;
      if (!there) continue;
      if (WRITE) {
#pragma unroll
        for (int e = 0; e < W; ++e) b.w[k][e] = __ldg(packed + e);
      } else {
        b.w[k][0] = *static_cast<const uint4*>(pool);
        if (F8) b.s[k] = *b.scale[k];
      }
    }
    next_u += 32 * L::STEPS;
    if (next_u >= units) {
      next_u = 0;
      ++next_i;
    }
  };
  auto store = [&](const B& b) {
    if constexpr (F8 && WRITE) {
      float amax[L::STEPS];
      bool far = false;
#pragma unroll
      for (int k = 0; k < L::STEPS; ++k) {
        amax[k] = 0.f;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const uint32_t x[4] = {b.w[k][e].x, b.w[k][e].y, b.w[k][e].z, b.w[k][e].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 y = widen(x[c]);
            amax[k] = fmax3(amax[k], fabsf(y.x), fabsf(y.y));
          }
        }
      }
      // a row's lanes are neighbours, and 32 of them hold whole rows
#pragma unroll
      for (int o = L::LPR / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < L::STEPS; ++k) amax[k] = fmaxf(amax[k], __shfl_xor_sync(0xffffffffu, amax[k], o));
#pragma unroll
      for (int k = 0; k < L::STEPS; ++k) far = far || !(amax[k] == 0.f || (amax[k] > 1e-18f && amax[k] < 1e18f));
      uint4 c[L::STEPS];
      float sc[L::STEPS];
      if (!__any_sync(0xffffffffu, far)) {
#pragma unroll
        for (int k = 0; k < L::STEPS; ++k) {
          float r;
          row_scale(amax[k], &sc[k], &r);
          const uint2 lo = quantize8(b.w[k][0], sc[k], r), hi = quantize8(b.w[k][W - 1], sc[k], r);
          c[k] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
      } else {
#pragma unroll
        for (int k = 0; k < L::STEPS; ++k) {
          sc[k] = amax[k] > 0.f ? __fdiv_rn(amax[k], 448.0f) : 1.0f;
          const uint2 lo = divide8(b.w[k][0], sc[k]), hi = divide8(b.w[k][W - 1], sc[k]);
          c[k] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
      }
#pragma unroll
      for (int k = 0; k < L::STEPS; ++k) {
        if (!b.dst[k]) continue;
        *b.dst[k] = c[k];
        if (lane % L::LPR == 0) *b.scale[k] = sc[k];
      }
    } else if constexpr (F8) {
#pragma unroll
      for (int k = 0; k < L::STEPS; ++k) {
        const uint4 c = b.w[k][0];
        const uint4 y0 = dequantize8(make_uint2(c.x, c.y), b.s[k]), y1 = dequantize8(make_uint2(c.z, c.w), b.s[k]);
        // a lane's 32 bytes in two stores would write half sectors each: neighbours swap halves, so
        // that a store writes the 32 bytes of every other lane
        const bool odd = lane & 1;
        const uint4 give = odd ? y0 : y1;
        const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, 1), __shfl_xor_sync(0xffffffffu, give.y, 1),
                                     __shfl_xor_sync(0xffffffffu, give.z, 1), __shfl_xor_sync(0xffffffffu, give.w, 1));
        if (!b.dst[k]) continue;
        uint4* even_dst = b.dst[k] - (odd ? 2 : 0);
        even_dst[odd ? 1 : 0] = odd ? got : y0;
        even_dst[odd ? 3 : 2] = odd ? y1 : got;
      }
    } else {
#pragma unroll
      for (int k = 0; k < L::STEPS; ++k)
        if (b.dst[k]) *b.dst[k] = b.w[k][0];
    }
  };
  if (p.xi) {  // the index keys, d_idx / 8 lanes a token
    const int lanes = p.d_idx >> 3, sub = lane % lanes;
    for (int i0 = 0; i0 < n; i0 += 32 / lanes) {
      const int i = i0 + lane / lanes;
      const int64_t row = __shfl_sync(0xffffffffu, place, min(i, n - 1)), t = t0 + i;
      if (i >= n || row == kNoToken || (WRITE && row < 0)) continue;
      uint4* packed = reinterpret_cast<uint4*>(p.xi + t * p.si + sub * 8);
      uint4* pool = reinterpret_cast<uint4*>(p.k_idx + (row < 0 ? 0 : row) * p.d_idx + sub * 8);
      if (WRITE) *pool = __ldg(packed);
      else *packed = row < 0 ? make_uint4(0, 0, 0, 0) : *pool;
    }
  }
  B now, ahead;
  fetch(now);
  while (true) {  // warp-uniform: next_i is
    const bool more = next_i < n;
    if (more) fetch(ahead);
    store(now);
    if (!more) break;
    const bool again = next_i < n;
    if (again) fetch(now);
    store(ahead);
    if (!again) break;
  }
}

template <int D, bool F8, bool WRITE>
cudaError_t launch_cache(CacheParams& p, int num_sms, cudaStream_t st) {
  // tokens of a warp: as many as let all warps run together
  const int64_t together = (int64_t)num_sms * kCtasPerSm<F8, WRITE> * (kThreads / 32);
  const int64_t want = (p.T + together - 1) / together;
  p.per = (int)(want < 32 ? want : 32);
  const int64_t warps = ((int64_t)p.T + p.per - 1) / p.per;
  const int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
  cache_kernel<D, F8, WRITE><<<(unsigned)grid, kThreads, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <bool WRITE>
int run_cache(const msa_paged_cache_t* c, const msa_page_table_t* pt, const int32_t* lens,
              const int32_t* cu, int total_tokens, void* k, void* v, void* k_idx,
              const int64_t* strides, cudaStream_t stream) {
  int rc = check_cache(c);
  if (rc) return rc;
  PageView pages;
  if ((rc = check_pages(c, pt, &pages))) return rc;
  if (total_tokens < 0) return MSA_ERR_SHAPE;
  if (!cu && total_tokens != pt->B) return MSA_ERR_SHAPE;
  if (pt->B == 0 || total_tokens == 0) return MSA_OK;
  if (!lens || !k || !v) return MSA_ERR_ARG;
  if (k_idx && c->d_idx == 0) return MSA_ERR_SHAPE;
  const void* ptrs[] = {k, v, k_idx};
  for (const void* x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) & 15) return MSA_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(cu)) & 3) return MSA_ERR_ARG;
  CacheParams p = {};
  const int64_t dense[5] = {(int64_t)c->H_kv * c->d, c->d, (int64_t)c->H_kv * c->d, c->d, c->d_idx};
  if (!strides) strides = dense;
  for (int i = 0; i < 5; ++i)
    if ((i < 4 || k_idx) && strides[i] % 8) return MSA_ERR_ARG;  // rows start on 16 bytes
  Ctx cx;
  if ((rc = device_ctx(&cx))) return rc;
  p.pages = pages;
  p.lens = lens;
  p.cu = cu;
  p.B = pt->B;
  p.T = total_tokens;
  p.H = c->H_kv;
  p.k = c->k;
  p.v = c->v;
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.k_idx = static_cast<__nv_bfloat16*>(c->k_idx);
  p.xk = static_cast<__nv_bfloat16*>(k);
  p.xv = static_cast<__nv_bfloat16*>(v);
  p.xi = static_cast<__nv_bfloat16*>(k_idx);
  p.sk[0] = strides[0];
  p.sk[1] = strides[1];
  p.sv[0] = strides[2];
  p.sv[1] = strides[3];
  p.si = strides[4];
  p.d_idx = c->d_idx;
  p.status = cx.status;
  const bool f8 = c->kind == MSA_CACHE_E4M3;
  cudaError_t e;
  if (c->d == 128)
    e = f8 ? launch_cache<128, true, WRITE>(p, cx.num_sms, stream)
           : launch_cache<128, false, WRITE>(p, cx.num_sms, stream);
  else
    e = f8 ? launch_cache<64, true, WRITE>(p, cx.num_sms, stream)
           : launch_cache<64, false, WRITE>(p, cx.num_sms, stream);
  return finish(e);
}

}  // namespace

int check_cache_sizes(const msa_paged_cache_t* c) {
  if (!c) return MSA_ERR_ARG;
  if (c->num_pages < 0 || c->page_size <= 0 || c->H_kv <= 0 || c->d <= 0 || c->d_idx < 0)
    return MSA_ERR_SHAPE;
  if (c->kind != MSA_CACHE_BF16 && c->kind != MSA_CACHE_E4M3) return MSA_ERR_ARG;
  if (c->page_size % 16 != 0 || c->page_size > 65536) return MSA_ERR_UNSUPPORTED;
  if (c->d != 64 && c->d != 128) return MSA_ERR_UNSUPPORTED;
  if (c->d_idx != 0 && c->d_idx != 32 && c->d_idx != 64) return MSA_ERR_UNSUPPORTED;
  if (c->H_kv > 1024) return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

int check_cache(const msa_paged_cache_t* c) {
  const int rc = check_cache_sizes(c);
  if (rc) return rc;
  if (c->num_pages == 0) return MSA_OK;  // no page to address
  const bool f8 = c->kind == MSA_CACHE_E4M3;
  const void* need[] = {c->k, c->v, f8 ? c->k_scale : c->k, f8 ? c->v_scale : c->v,
                        c->d_idx ? c->k_idx : c->k};
  for (const void* x : need)
    if (!x || (reinterpret_cast<uintptr_t>(x) & 15)) return MSA_ERR_ARG;
  return MSA_OK;
}

int check_pages(const msa_paged_cache_t* c, const msa_page_table_t* pt, PageView* out) {
  if (!pt) return MSA_ERR_ARG;
  if (pt->B < 0 || pt->max_pages < 0 || pt->stride < 0) return MSA_ERR_SHAPE;
  if ((int64_t)pt->max_pages * c->page_size > 0x7fffffffLL) return MSA_ERR_UNSUPPORTED;
  if (pt->B > 0 && pt->max_pages > 0 &&
      (!pt->ids || (reinterpret_cast<uintptr_t>(pt->ids) & 3)))
    return MSA_ERR_ARG;
  out->table = pt->ids;
  out->table_stride = pt->stride;
  out->num_pages = c->num_pages;
  out->page_size = c->page_size;
  out->max_pages = pt->max_pages;
  out->shift = page_shift(c->page_size);
  return MSA_OK;
}

}  // namespace msa

using namespace msa;

extern "C" {

int msa_cache_write(const msa_paged_cache_t* c, const msa_page_table_t* pages, const int32_t* lens,
                    const int32_t* cu_seqlens, int total_tokens, const void* k, const void* v,
                    const void* k_idx, const int64_t* strides, cudaStream_t stream) {
  return run_cache<true>(c, pages, lens, cu_seqlens, total_tokens, const_cast<void*>(k),
                         const_cast<void*>(v), const_cast<void*>(k_idx), strides, stream);
}

int msa_cache_read(const msa_paged_cache_t* c, const msa_page_table_t* pages, const int32_t* lens,
                   const int32_t* cu_seqlens, int total_tokens, void* k, void* v, void* k_idx,
                   cudaStream_t stream) {
  if (pages && pages->B > 0 && total_tokens > 0 && !cu_seqlens) return MSA_ERR_ARG;
  return run_cache<false>(c, pages, lens, cu_seqlens, total_tokens, k, v, k_idx, nullptr, stream);
}

}  // extern "C"
