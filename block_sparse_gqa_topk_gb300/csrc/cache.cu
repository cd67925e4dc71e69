// cache.cu -- tokens into a paged cache and back (see include/msa.h).
//
// A row is one head's key or value of a token (d values), or the token's index key; it
// moves through the lanes of a part of a warp.  An E4M3 cache stores
//   s = amax |x| / 448 (1 for an all-zero row),  code = E4M3 nearest to x / s,
// the rule of msa_quantize_kv_fp8 bit for bit (IEEE divisions), and reads back
// decode(code) * s rounded once to bf16.  An E2M1 cache (quantize16 has its rule) stores 4-bit
// codes with a scale for each 16 of them, and reads back code * block scale * row scale, exactly.
// Either way every row is read once and written once.
#include "cache_rows.cuh"
#include "kernels.h"

#include <algorithm>

namespace msa {
namespace {

constexpr int kThreads = 256;

struct CacheParams {
  TokenMap map;
  int T, H;
  void* k;  // pool
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  __nv_bfloat16* k_idx;
  __nv_bfloat16* xk;  // packed rows: read by the write, written by the read
  __nv_bfloat16* xv;
  __nv_bfloat16* xi;
  int64_t sk[2], sv[2], si;  // their strides: token, head; token
  int per;                   // tokens of a warp (codes: of a CTA)
  int d_idx;
  int* status;
};

// bf16.  A token's keys, and its values, are one run of H D values in the pool; a lane moves 8 values
// of it at a time, a warp one token after another.  Its lanes find the places of all its tokens (at
// most 32) together, so the chain of lookups (sequence, length, page) is paid once, and while it
// works on STEPS vectors a lane, the next ones are on their way.  32K tokens of 8 groups, d 128, with
// index keys, calls back to back: 49 us each way.
template <int D>
struct Lanes {
  static constexpr int LPR = D / 8;  // lanes of a head's row
  static constexpr int STEPS = 2;
};

// STEPS vectors a lane of one token, loaded; where they go.
template <int D>
struct Batch {
  uint4 w[Lanes<D>::STEPS];
  uint4* dst[Lanes<D>::STEPS];  // null: nothing to store
};

constexpr int kCtasPerSm = 4;  // as the registers of a batch allow

template <int D, bool WRITE>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) cache_kernel(const __grid_constant__ CacheParams p) {
  using L = Lanes<D>;
  using B = Batch<D>;
  const int lane = threadIdx.x & 31;
  const int64_t t0 = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * p.per;
  if (t0 >= p.T) return;
  const int n = (int)min((int64_t)p.per, p.T - t0);
  int64_t place = kNoToken;
  if (lane < n) {
    place = token_row(p.map, (int)t0 + lane);
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
      uint4* packed = reinterpret_cast<uint4*>(x + sub * 8);
      uint4* pool = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(v ? p.v : p.k) + cell * D + f * 8);
      b.w[k] = make_uint4(0, 0, 0, 0);
      b.dst[k] = nullptr;
      if (u >= units || skip) continue;
      b.dst[k] = WRITE ? pool : packed;
      if (there) b.w[k] = WRITE ? __ldg(packed) : *pool;
    }
    next_u += 32 * L::STEPS;
    if (next_u >= units) {
      next_u = 0;
      ++next_i;
    }
  };
  auto store = [&](const B& b) {
#pragma unroll
    for (int k = 0; k < L::STEPS; ++k)
      if (b.dst[k]) *b.dst[k] = b.w[k];
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

// Codes.  A CTA takes code_tokens() tokens, and each D / 16 lanes a row at a time.  Bound by instructions and the
// loads in flight, so as many CTAs as the registers allow.  32K tokens of 8 groups, with index keys, calls back
// to back, d 128 (d 64), us:               E4M3 write    4 bits        E4M3 read     4 bits
//   eight CTAs a SM                        38.7 (21.8)   37.6 (21.8)   37.0 (19.6)   34.1 (18.0)
//   six                                    41.1          39.9          39.2          36.8
//   warps that take token after token      40.2 (22.8)   43.8 (23.8)   40.3 (20.1)   34.6 (19.2)
// (the last with the next vectors on their way, as above; a token a sequence takes it 4.8 us, and 3.2 here).
constexpr int kCodeCtas = 8;
constexpr int kMaxCodeTokens = 32;  // as the lanes of their index keys fit a CTA

// Tokens of a CTA: at most `rounds` of its threads' work; in a call of one or two waves of CTAs as many as
// make them even, and where an SM has a CTA all the same, as give all its threads something to do.  E4M3, us:
//   3000 tokens of 2 heads, d 128, written 3.4 and read 3.6 (2 tokens a CTA, 1500 CTAs: 4.8 and 4.8);
//   20000 of 8 heads read 24.6 (8 tokens, a little over two waves: 25.5; 16, a little over one: 28.3);
//   32K of 4 heads read 17.3 in eight rounds, 18.9 in four; 13000 of 8 heads written 17.4 and 16.4.
template <int D, bool WRITE>
int code_tokens(int T, int H, int num_sms) {
  const int items = 2 * H * (D / 16), round = kThreads / items;  // threads' pieces of a token
  const int eight = 8 * kThreads / items, four = 4 * kThreads / items;
  const int rounds = WRITE ? std::max(four, std::min(1024 / D, eight)) : eight;
  const int most = std::max(1, std::min(kMaxCodeTokens, rounds)), together = num_sms * kCodeCtas;
  if (T > 2 * (int64_t)most * together) return most;
  const int wave = T > most * together ? 2 * together : together;
  return std::max(std::max((T + wave - 1) / wave, 1), std::min(std::min((T + num_sms - 1) / num_sms, round), most));
}

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, kCodeCtas)
    cache_code_kernel(const __grid_constant__ CacheParams p, const __grid_constant__ CodedRows rows) {
  __shared__ int64_t s_row[kMaxCodeTokens];
  const int t0 = blockIdx.x * p.per, nt = min(p.per, p.T - t0);
  if (threadIdx.x < nt) {
    const int64_t row = token_row(p.map, t0 + threadIdx.x);
    if (row == kNoPlace) set_status(p.status, MSA_ERR_ARG);
    s_row[threadIdx.x] = row;
  }
  __syncthreads();
  if (p.xi) {  // the index keys, d_idx / 8 lanes a token
    const int lanes = p.d_idx >> 3, tok = threadIdx.x / lanes, sub = threadIdx.x % lanes;
    if (tok < nt && s_row[tok] >= 0)
      reinterpret_cast<uint4*>(p.k_idx + s_row[tok] * p.d_idx)[sub] =
          __ldg(reinterpret_cast<const uint4*>(p.xi + (t0 + tok) * p.si) + sub);
  }
  store_rows<D, KIND>(rows, t0, nt, s_row, [](const __nv_bfloat16*, int, int, uint4&, uint4&) {});
}

// Reading codes, the same way.
template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, kCodeCtas) cache_decode_kernel(const __grid_constant__ CacheParams p, uint32_t div_2H) {
  constexpr int LPR = D / 16, BITS = KIND == MSA_CACHE_E2M1 ? 4 : 8;
  constexpr int SCALE = KIND == MSA_CACHE_E2M1 ? e2m1_scale_bytes(D) : 4;
  __shared__ int64_t s_row[kMaxCodeTokens];
  const int t0 = blockIdx.x * p.per, nt = min(p.per, p.T - t0);
  if (threadIdx.x < nt) {
    const int64_t row = token_row(p.map, t0 + threadIdx.x);
    if (row == kNoPlace) set_status(p.status, MSA_ERR_ARG);
    s_row[threadIdx.x] = row;
  }
  __syncthreads();
  if (p.xi) {
    const int lanes = p.d_idx >> 3, tok = threadIdx.x / lanes, sub = threadIdx.x % lanes;
    if (tok < nt && s_row[tok] != kNoToken)
      reinterpret_cast<uint4*>(p.xi + (t0 + tok) * p.si)[sub] =
          s_row[tok] < 0 ? make_uint4(0, 0, 0, 0) : reinterpret_cast<const uint4*>(p.k_idx + s_row[tok] * p.d_idx)[sub];
  }
  const int lane = threadIdx.x & 31, rows = nt * 2 * p.H, sub = lane % LPR;
  const bool odd = lane & 1;
  for (int i0 = threadIdx.x - lane; i0 < rows * LPR; i0 += kThreads) {  // whole warps
    const int r = (i0 + lane) / LPR, tok = min(small_div(r, div_2H), nt - 1), hv = r - tok * 2 * p.H;
    const int v = hv >= p.H, h = v ? hv - p.H : hv;
    const int64_t row = s_row[tok];
    uint4 y0 = make_uint4(0, 0, 0, 0), y1 = y0;  // a missing place reads as zeros
    if (r < rows && row >= 0) {
      const int64_t cell = row * p.H + h;
      const uint8_t* codes = static_cast<const uint8_t*>(v ? p.v : p.k) + (cell * D + 16 * sub) * BITS / 8;
      const uint8_t* scale = (v ? p.v_scale : p.k_scale) + cell * SCALE;
      float s = *reinterpret_cast<const float*>(scale);
      if constexpr (KIND == MSA_CACHE_E2M1) {
        const uint2 x = *reinterpret_cast<const uint2*>(codes);
        s *= e4m3_value(scale[4 + sub]);
        y0 = dequantize_e2m1(x.x, s);
        y1 = dequantize_e2m1(x.y, s);
      } else {
        const uint4 x = *reinterpret_cast<const uint4*>(codes);
        y0 = dequantize8(make_uint2(x.x, x.y), s);
        y1 = dequantize8(make_uint2(x.z, x.w), s);
      }
    }
    // a lane's 32 bytes in two stores would write half sectors each: neighbours swap halves, so that a store
    // writes the 32 bytes of every other lane
    const uint4 give = odd ? y0 : y1;
    const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, 1), __shfl_xor_sync(0xffffffffu, give.y, 1),
                                 __shfl_xor_sync(0xffffffffu, give.z, 1), __shfl_xor_sync(0xffffffffu, give.w, 1));
    if (r >= rows || row == kNoToken) continue;
    __nv_bfloat16* x = v ? p.xv + (t0 + tok) * p.sv[0] + h * p.sv[1] : p.xk + (t0 + tok) * p.sk[0] + h * p.sk[1];
    uint4* even_dst = reinterpret_cast<uint4*>(x + 16 * (sub & ~1));
    even_dst[odd ? 1 : 0] = odd ? got : y0;
    even_dst[odd ? 3 : 2] = odd ? y1 : got;
  }
}

template <int D, int KIND>
cudaError_t launch_decode(CacheParams& p, int num_sms, cudaStream_t st) {
  p.per = code_tokens<D, false>(p.T, p.H, num_sms);
  cache_decode_kernel<D, KIND><<<(unsigned)(((int64_t)p.T + p.per - 1) / p.per), kThreads, 0, st>>>(p, magic(2 * p.H));
  note_launch();
  return cudaGetLastError();
}

template <int D, int KIND>
cudaError_t launch_codes(CacheParams& p, int num_sms, cudaStream_t st) {
  CodedRows r = {};
  r.x[0] = p.xk;
  r.x[1] = p.xv;
  for (int i = 0; i < 2; ++i) {
    r.stride[0][i] = p.sk[i];
    r.stride[1][i] = p.sv[i];
    r.pool[i] = static_cast<uint8_t*>(i ? p.v : p.k);
    r.scale[i] = i ? p.v_scale : p.k_scale;
  }
  r.H = p.H;
  r.div_2H = magic(2 * p.H);
  p.per = code_tokens<D, true>(p.T, p.H, num_sms);
  cache_code_kernel<D, KIND><<<(unsigned)(((int64_t)p.T + p.per - 1) / p.per), kThreads, 0, st>>>(p, r);
  note_launch();
  return cudaGetLastError();
}

template <int D, bool WRITE>
cudaError_t launch_bf16(CacheParams& p, int num_sms, cudaStream_t st) {
  // tokens of a warp: as many as let all warps run together
  const int64_t together = (int64_t)num_sms * kCtasPerSm * (kThreads / 32);
  const int64_t want = (p.T + together - 1) / together;
  p.per = (int)(want < 32 ? want : 32);
  const int64_t warps = ((int64_t)p.T + p.per - 1) / p.per;
  const int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
  cache_kernel<D, WRITE><<<(unsigned)grid, kThreads, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <int D, bool WRITE>
cudaError_t launch_cache(int kind, CacheParams& p, int num_sms, cudaStream_t st) {
  if (kind == MSA_CACHE_BF16) return launch_bf16<D, WRITE>(p, num_sms, st);
  if (kind == MSA_CACHE_E4M3)
    return WRITE ? launch_codes<D, MSA_CACHE_E4M3>(p, num_sms, st) : launch_decode<D, MSA_CACHE_E4M3>(p, num_sms, st);
  return WRITE ? launch_codes<D, MSA_CACHE_E2M1>(p, num_sms, st) : launch_decode<D, MSA_CACHE_E2M1>(p, num_sms, st);
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
  p.map = {pages, lens, cu, pt->B};
  p.T = total_tokens;
  p.H = c->H_kv;
  p.k = c->k;
  p.v = c->v;
  p.k_scale = reinterpret_cast<uint8_t*>(c->k_scale);
  p.v_scale = reinterpret_cast<uint8_t*>(c->v_scale);
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
  return finish(c->d == 128 ? launch_cache<128, WRITE>(c->kind, p, cx.num_sms, stream)
                            : launch_cache<64, WRITE>(c->kind, p, cx.num_sms, stream));
}

}  // namespace

int check_cache_sizes(const msa_paged_cache_t* c) {
  if (!c) return MSA_ERR_ARG;
  if (c->num_pages < 0 || c->page_size <= 0 || c->H_kv <= 0 || c->d <= 0 || c->d_idx < 0)
    return MSA_ERR_SHAPE;
  if (c->kind != MSA_CACHE_BF16 && c->kind != MSA_CACHE_E4M3 && c->kind != MSA_CACHE_E2M1) return MSA_ERR_ARG;
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
  const bool coded = c->kind != MSA_CACHE_BF16;
  const void* need[] = {c->k, c->v, coded ? c->k_scale : c->k, coded ? c->v_scale : c->v,
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
