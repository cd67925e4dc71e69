// append.cu -- a call's new tokens turned to their positions and stored in a paged cache, in one
// launch (see include/msa.h): what msa_rope and msa_cache_write do, bit for bit, without the turned
// keys' way through memory.
//
//   q_out = R q, q_idx_out = R q_idx;  pool row of the token: k <- R k, v, k_idx <- R k_idx,
// R the rotary turn of the token's position (rope.cu).  A cache of codes codes the turned keys as
// they are in bf16.
#include "cache_rows.cuh"
#include "kernels.h"
#include "rope_items.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens of a CTA
constexpr int kMaxHalf = 64;   // rot_dim / 2 (rot_dim <= d)

// A tensor whose heads are moved item by item.
struct ItemTensor {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;  // packed, or the pool
  int H, parts, rot_parts, d;
  int last;  // items of a token in this tensor and those before it
  int pool;
  uint32_t div_parts, div_H;
  int64_t xs[2];  // strides of token, head
};

struct AppendParams {
  TokenMap map;
  const uint64_t* turns;
  const void* positions;  // null: the token's place in its sequence
  int pos64;
  int64_t ps;
  int T, half, tpb, n;  // tokens; rot_dim / 2; tokens of a CTA; item tensors
  float mscale;
  uint32_t div_half;
  ItemTensor t[5];
  CodedRows rows;  // k, v where the cache holds codes
  int* status;
};

// Values i0 .. i0 + 7 of a head's row, turned as RopeItem turns them.  x: the row; cs: the turns of its token.
template <bool INTER>
__device__ __forceinline__ uint4 turned8(const __nv_bfloat16* x, uint4 w, int i0, int half, const float2* cs) {
  if (i0 >= 2 * half) return w;
  uint32_t u[4] = {w.x, w.y, w.z, w.w};
  if (INTER) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i0 + 2 * e >= 2 * half) break;
      const float2 v = widen(u[e]), c = cs[i0 / 2 + e];
      u[e] = pack_bf16(turned_first(v.x, v.y, c), turned_second(v.x, v.y, c));
    }
  } else if (half % 8 == 0) {
    const bool first = i0 < half;
    const uint4 o = __ldg(reinterpret_cast<const uint4*>(x + (first ? i0 + half : i0 - half)));
    const float2* c = cs + (first ? i0 : i0 - half);
    const uint32_t other[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = widen(u[e]), y = widen(other[e]), c0 = c[2 * e], c1 = c[2 * e + 1];
      u[e] = first ? pack_bf16(turned_first(v.x, y.x, c0), turned_first(v.y, y.y, c1))
                   : pack_bf16(turned_second(y.x, v.x, c0), turned_second(y.y, v.y, c1));
    }
  } else {  // the halves meet within a vector: value by value
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = i0 + e;
      const float2 v = widen(u[e >> 1]);
      const float mine = e & 1 ? v.y : v.x;
      const bool first = i < half;
      f[e] = mine;
      if (i >= 2 * half) continue;
      const float y = __bfloat162float(x[first ? i + half : i - half]);
      const float2 c = cs[first ? i : i - half];
      f[e] = first ? turned_first(mine, y, c) : turned_second(y, mine, c);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// One CTA serves tpb tokens: their sines and cosines and their places in the pool go to shared memory
// once; then the items of q, q_idx and k_idx (and of k and v in a bf16 cache) are spread over the
// threads, and the rows of k and v that become codes over the warps.  Bound by HBM.
template <int D, int KIND, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, 6) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float2 s_cs[kMaxTokens * kMaxHalf];
  __shared__ int64_t s_row[kMaxTokens];
  const int t0 = blockIdx.x * p.tpb, nt = min(p.tpb, p.T - t0);
  if (threadIdx.x < nt) {
    const int64_t row = token_row(p.map, t0 + threadIdx.x);
    if (row == kNoPlace) set_status(p.status, MSA_ERR_ARG);
    s_row[threadIdx.x] = row;
  }
  for (int i = threadIdx.x; i < nt * p.half; i += kThreads) {
    const int tok = small_div(i, p.div_half), pair = i - tok * p.half, t = t0 + tok;
    const uint64_t turns = __ldg(&p.turns[pair]);
    int64_t pos;
    int b;
    if (!p.positions) pos = token_position(p.map, t, &b);
    else if (p.pos64) pos = __ldg(static_cast<const int64_t*>(p.positions) + t * p.ps);
    else pos = __ldg(static_cast<const int32_t*>(p.positions) + t * p.ps);
    s_cs[i] = turn_of(pos, turns, p.mscale);
  }
  __syncthreads();
  const int items = nt * p.t[p.n - 1].last;
  for (int item = threadIdx.x; item < items; item += kThreads) {
    int x = item, ti = 0;
    while (x >= nt * p.t[ti].last) ++ti;
    const ItemTensor& a = p.t[ti];
    if (ti > 0) x -= nt * p.t[ti - 1].last;
    const int r = small_div(x, a.div_parts), part = x - r * a.parts;
    const int tok = small_div(r, a.div_H), h = r - tok * a.H;
    const int64_t row = s_row[tok];
    if (a.pool && row < 0) continue;
    RopeItem<__nv_bfloat16, V> it(part, a.rot_parts, a.rot_parts ? p.half : 0, a.d, INTER);
    it.load(a.x + ((t0 + tok) * a.xs[0] + h * a.xs[1]));
    if (it.turn) it.template rotate<INTER>(s_cs + tok * p.half, part);
    if (row < 0) it.clear();  // no token of a sequence: a zero query
    it.store(a.y + ((a.pool ? row : (int64_t)(t0 + tok)) * a.H + h) * a.d);
  }
  if constexpr (KIND != MSA_CACHE_BF16)
    store_rows<D, KIND>(p.rows, t0, nt, s_row, [&](const __nv_bfloat16* x, int tok, int i0, uint4& lo, uint4& hi) {
      const float2* cs = s_cs + tok * p.half;
      lo = turned8<INTER>(x, lo, i0, p.half, cs);
      hi = turned8<INTER>(x, hi, i0 + 8, p.half, cs);
    });
}

template <int D, int KIND>
cudaError_t launch_append(const AppendParams& p, bool vec, bool inter, cudaStream_t st) {
  const unsigned grid = (unsigned)(((int64_t)p.T + p.tpb - 1) / p.tpb);
  if (vec) {
    if (inter) append_kernel<D, KIND, 8, true><<<grid, kThreads, 0, st>>>(p);
    else append_kernel<D, KIND, 8, false><<<grid, kThreads, 0, st>>>(p);
  } else {
    if (inter) append_kernel<D, KIND, 1, true><<<grid, kThreads, 0, st>>>(p);
    else append_kernel<D, KIND, 1, false><<<grid, kThreads, 0, st>>>(p);
  }
  note_launch();
  return cudaGetLastError();
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" int msa_cache_append(const msa_paged_cache_t* c, const msa_page_table_t* pt, const int32_t* lens,
                                const int32_t* cu_seqlens, int total_tokens, const msa_append_t* a,
                                const uint64_t* turns, const void* positions, const void* q, const void* k,
                                const void* v, const void* q_idx, const void* k_idx, void* q_out, void* q_idx_out,
                                cudaStream_t stream) {
  int rc = check_cache(c);
  if (rc) return rc;
  AppendParams p = {};
  if ((rc = check_pages(c, pt, &p.map.pages))) return rc;
  if (!a) return MSA_ERR_ARG;
  if (total_tokens < 0 || a->H_q < 1 || a->rot_dim < 2 || (a->rot_dim & 1) || a->rot_dim > c->d) return MSA_ERR_SHAPE;
  if (c->d_idx && (a->H_i < 1 || a->rot_dim > c->d_idx)) return MSA_ERR_SHAPE;
  if (a->H_q > 1024 || a->H_i > 1024) return MSA_ERR_UNSUPPORTED;
  if (!cu_seqlens && total_tokens != pt->B) return MSA_ERR_SHAPE;
  if (!isfinite(a->mscale) || (a->positions_bits != 32 && a->positions_bits != 64)) return MSA_ERR_ARG;
  if (pt->B == 0 || total_tokens == 0) return MSA_OK;
  if (!lens || !turns || !q || !k || !v || !q_out) return MSA_ERR_ARG;
  if (c->d_idx && (!q_idx || !k_idx || !q_idx_out)) return MSA_ERR_ARG;
  if (!c->d_idx && (q_idx || k_idx || q_idx_out)) return MSA_ERR_SHAPE;
  auto at = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  if ((at(k) | at(v) | at(k_idx) | at(q_out) | at(q_idx_out)) & 15) return MSA_ERR_ARG;
  if ((at(q) | at(q_idx)) & 1 || (at(lens) | at(cu_seqlens)) & 3 || at(turns) & 7) return MSA_ERR_ARG;
  if (at(positions) % (a->positions_bits / 8)) return MSA_ERR_ARG;
  // rows of what is stored start on 16 bytes
  if ((a->k_stride[0] | a->k_stride[1] | a->v_stride[0] | a->v_stride[1]) & 7 || (c->d_idx && a->k_idx_stride & 7))
    return MSA_ERR_ARG;
  Ctx cx;
  if ((rc = device_ctx(&cx))) return rc;
  // One width for all items: 8 values where the halves of every turned row and the queries' rows start on 16 bytes,
  // else one.  (32K tokens, 32 heads over 8, bf16: 137 us, and 162 by msa_rope and msa_cache_write; one value
  // at a time 468, and 377 by the two, which store whole vectors.  Codes likewise: 410 and 370.)
  bool vec = a->rot_dim % 16 == 0 && ((at(q) | at(q_idx)) & 15) == 0 && ((a->q_stride[0] | a->q_stride[1]) & 7) == 0;
  if (c->d_idx) vec = vec && ((a->q_idx_stride[0] | a->q_idx_stride[1]) & 7) == 0;
  p.map.lens = lens;
  p.map.cu = cu_seqlens;
  p.map.B = pt->B;
  p.turns = turns;
  p.positions = positions;
  p.pos64 = a->positions_bits == 64;
  p.ps = a->positions_stride;
  p.T = total_tokens;
  p.half = a->rot_dim / 2;
  p.div_half = magic(p.half);
  p.mscale = a->mscale;
  const int H = p.rows.H = c->H_kv;
  p.rows.div_2H = magic(2 * H);
  p.status = cx.status;
  const int w = vec ? 8 : 1;
  int all = 0;  // items of a token
  auto add = [&](const void* x, void* y, int H, int d, bool turn, bool pool, int64_t st, int64_t sh) {
    ItemTensor& t = p.t[p.n++];
    t.x = static_cast<const __nv_bfloat16*>(x);
    t.y = static_cast<__nv_bfloat16*>(y);
    t.H = H;
    t.d = d;
    t.rot_parts = turn ? p.half / w : 0;
    t.parts = t.rot_parts + (d - (turn ? a->rot_dim : 0) + 2 * w - 1) / (2 * w);
    t.pool = pool;
    t.div_parts = magic(t.parts);
    t.div_H = magic(H);
    t.xs[0] = st;
    t.xs[1] = sh;
    all += H * t.parts;
    t.last = all;
  };
  add(q, q_out, a->H_q, c->d, true, false, a->q_stride[0], a->q_stride[1]);
  const bool coded = c->kind != MSA_CACHE_BF16;
  if (!coded) {
    add(k, c->k, H, c->d, true, true, a->k_stride[0], a->k_stride[1]);
    add(v, c->v, H, c->d, false, true, a->v_stride[0], a->v_stride[1]);
  }
  if (c->d_idx) {
    add(q_idx, q_idx_out, a->H_i, c->d_idx, true, false, a->q_idx_stride[0], a->q_idx_stride[1]);
    add(k_idx, c->k_idx, 1, c->d_idx, true, true, a->k_idx_stride, 0);
  }
  for (int i = 0; i < 2; ++i) {
    p.rows.x[i] = static_cast<const __nv_bfloat16*>(i ? v : k);
    p.rows.stride[0][i] = a->k_stride[i];
    p.rows.stride[1][i] = a->v_stride[i];
    p.rows.pool[i] = static_cast<uint8_t*>(i ? c->v : c->k);
    p.rows.scale[i] = reinterpret_cast<uint8_t*>(i ? c->v_scale : c->k_scale);
  }
  // tokens of a CTA: up to kMaxTokens while the grid still fills the GPU and an item index stays below
  // 2^18 (small_div)
  p.tpb = kMaxTokens;
  while (p.tpb > 1 && (((int64_t)p.T + p.tpb - 1) / p.tpb < 8 * cx.num_sms || (int64_t)p.tpb * all > (1 << 18))) p.tpb >>= 1;
  const bool inter = a->interleaved != 0;
  cudaError_t e;
  switch (c->kind) {
    case MSA_CACHE_E4M3:
      e = c->d == 128 ? launch_append<128, MSA_CACHE_E4M3>(p, vec, inter, stream)
                      : launch_append<64, MSA_CACHE_E4M3>(p, vec, inter, stream);
      break;
    case MSA_CACHE_E2M1:
      e = c->d == 128 ? launch_append<128, MSA_CACHE_E2M1>(p, vec, inter, stream)
                      : launch_append<64, MSA_CACHE_E2M1>(p, vec, inter, stream);
      break;
    default: e = launch_append<0, MSA_CACHE_BF16>(p, vec, inter, stream); break;
  }
  return finish(e);
}
