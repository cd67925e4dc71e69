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
  int rows;                  // of a token: 2 H, and the index key's where there is one
  float inv_rows;
  int steps;                 // chunks of a warp
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

// E4M3 codes of eight values at scale sc (amax / 448): the code nearest to the float32
// quotient x / sc.  With r the rounded reciprocal, q0 = x r and the remainder x - q0 sc, which
// one fma gives exactly, q0 + r (x - q0 sc) is the rounded quotient (Markstein 1990); that it
// gives every code that division gives is checked over all pairs of bf16 significands.  Rows
// whose amax leaves the range in which nothing underflows are divided.
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

// Items are the rows of the packed tokens in order: the keys of a token's H heads, the
// values, the index key.  A warp takes `steps` chunks of CHUNK consecutive items; its lanes
// find the places of the (at most 32) tokens among them together, so the chain of lookups
// (sequence, length, page) is paid once, and then move STEPS rows at a time with all their
// loads in flight.
// A lane moves 16 bytes of the pool a row: 8 bf16 values, or 16 codes.
template <int D, bool F8>
struct Lanes {
  static constexpr int VALUES = F8 ? 16 : 8;       // of a lane
  static constexpr int LPR = D / VALUES;           // lanes of a row
  static constexpr int RPS = 32 / LPR;             // rows of a step
  static constexpr int STEPS = F8 ? 2 : 4;         // rows a lane has in flight
  static constexpr int CHUNK = RPS * STEPS;
};

template <int D, bool F8, bool WRITE>
__global__ void __launch_bounds__(kThreads) cache_kernel(const __grid_constant__ CacheParams p) {
  using L = Lanes<D, F8>;
  constexpr int STEPS = L::STEPS;
  constexpr int W = L::VALUES / 8;  // 16-byte vectors of a lane in the packed rows
  const int lane = threadIdx.x & 31, sub = lane % L::LPR;
  const int64_t items = (int64_t)p.T * p.rows;
  const int64_t i0 = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * (L::CHUNK * p.steps);
  if (i0 >= items) return;
  const int n = (int)min((int64_t)L::CHUNK * p.steps, items - i0);
  const int t0 = (int)(i0 / p.rows);
  const int skip = (int)(i0 - (int64_t)t0 * p.rows);
  int64_t place = kNoToken;
  if (lane * p.rows < skip + n) {
    place = token_row(p, t0 + lane);
    if (place == kNoPlace) set_status(p.status, MSA_ERR_ARG);
  }
  for (int c = 0; c < n; c += L::CHUNK) {
    uint4* packed[STEPS];
    uint4* pool[STEPS];
    float* scale[STEPS];
    int kind[STEPS];   // 0: nothing, 1: key or value, 2: index key; negative: its place is missing
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int x = c + i * L::RPS + lane / L::LPR;
      const int y = x + skip;
      const int tok = (int)(((float)y + 0.5f) * p.inv_rows);  // exact: y < 32 rows
      const int r = y - tok * p.rows;
      int64_t row = __shfl_sync(0xffffffffu, place, tok);
      kind[i] = x >= n || row == kNoToken ? 0 : r < 2 * p.H ? 1 : sub * L::VALUES < p.d_idx ? 2 : 0;
      if (row < 0) {
        kind[i] = -kind[i];
        row = 0;
      }
      const int64_t t = t0 + tok;
      const bool v = r >= p.H;
      const int h = v ? r - p.H : r;
      scale[i] = nullptr;
      if (r == 2 * p.H) {
        packed[i] = reinterpret_cast<uint4*>(p.xi + t * p.si + sub * L::VALUES);
        pool[i] = reinterpret_cast<uint4*>(p.k_idx + row * p.d_idx + sub * L::VALUES);
      } else {
        const int64_t cell = row * p.H + h;
        packed[i] = reinterpret_cast<uint4*>((v ? p.xv + t * p.sv[0] + h * p.sv[1]
                                                : p.xk + t * p.sk[0] + h * p.sk[1]) + sub * L::VALUES);
        pool[i] = reinterpret_cast<uint4*>(static_cast<uint8_t*>(v ? p.v : p.k) +
                                           (cell * D + sub * L::VALUES) * (F8 ? 1 : 2));
        if (F8) scale[i] = (v ? p.v_scale : p.k_scale) + cell;
      }
    }
    uint4 w[STEPS][W];
    float s[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
#pragma unroll
      for (int k = 0; k < W; ++k) w[i][k] = make_uint4(0, 0, 0, 0);  // what a missing place reads as
      s[i] = 0.f;
      if (kind[i] <= 0) continue;
      if (!WRITE && F8 && kind[i] == 1) {
        w[i][0] = *pool[i];
        s[i] = *scale[i];
      } else {
#pragma unroll
        for (int k = 0; k < W; ++k) w[i][k] = WRITE ? __ldg(packed[i] + k) : pool[i][k];
      }
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      if constexpr (F8 && WRITE) {
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const uint32_t u[4] = {w[i][k].x, w[i][k].y, w[i][k].z, w[i][k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = widen(u[e]);
            amax = fmax3(amax, fabsf(x.x), fabsf(x.y));
          }
        }
#pragma unroll
        for (int o = L::LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (kind[i] == 1) {
          const float sc = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
          uint2 a, b;
          if (amax > 1e-18f && amax < 1e18f) {
            const float r = __frcp_rn(sc);
            a = quantize8(w[i][0], sc, r);
            b = quantize8(w[i][W - 1], sc, r);
          } else {
            a = divide8(w[i][0], sc);
            b = divide8(w[i][W - 1], sc);
          }
          *pool[i] = make_uint4(a.x, a.y, b.x, b.y);
          if (sub == 0) *scale[i] = sc;
          continue;
        }
      }
      if (WRITE ? kind[i] <= 0 : kind[i] == 0) continue;
      if constexpr (F8 && !WRITE) {
        if (kind[i] == 1 || kind[i] == -1) {
          packed[i][0] = dequantize8(make_uint2(w[i][0].x, w[i][0].y), s[i]);
          packed[i][W - 1] = dequantize8(make_uint2(w[i][0].z, w[i][0].w), s[i]);
          continue;
        }
      }
#pragma unroll
      for (int k = 0; k < W; ++k) (WRITE ? pool[i] : packed[i])[k] = w[i][k];
    }
  }
}

template <int D, bool F8, bool WRITE>
cudaError_t launch_cache(CacheParams& p, int num_sms, cudaStream_t st) {
  constexpr int CHUNK = Lanes<D, F8>::CHUNK;
  const int64_t items = (int64_t)p.T * p.rows;
  // chunks of a warp: as many as let all warps run together (32 or 48 a SM by their registers),
  // while 32 lanes find all of a warp's tokens
  const int64_t together = (int64_t)num_sms * (F8 && WRITE ? 32 : 48);
  const int64_t want = (items + CHUNK * together - 1) / (CHUNK * together);
  const int most = 30 * p.rows / CHUNK > 1 ? 30 * p.rows / CHUNK : 1;
  p.steps = (int)(want < most ? want : most);
  const int64_t warps = (items + CHUNK * p.steps - 1) / (CHUNK * p.steps);
  const int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
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
  p.rows = 2 * c->H_kv + (k_idx ? 1 : 0);
  p.inv_rows = 1.f / (float)p.rows;
  if ((int64_t)total_tokens * p.rows >= (int64_t)1 << 33) return MSA_ERR_UNSUPPORTED;
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
