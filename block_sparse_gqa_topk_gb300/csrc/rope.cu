// rope.cu -- rotary positions of up to four tensors in one launch.
//
// Pair i of a head's first rot_dim values is a point in the plane, turned by the angle
// a = position * f_i and stretched by mscale:
//   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a);
// the gradient turns the other way (the matrix's transpose).  Values past rot_dim pass
// through.
//
// Angles of far positions: turns[i] is f_i / 2 pi as a 64-bit fixed-point fraction of a
// turn.  position * turns[i] in wrapping 64-bit arithmetic is the angle's fraction of a
// turn without rounding, so position 2^20 is as exact as position 1; its signed value is
// rounded once to float and handed to sincospif.  No table is read or kept.
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRopeTensors = 4;
constexpr int kMaxTokens = 8;    // tokens a CTA computes the angles of
constexpr int kMaxHalf = 256;    // rot_dim / 2

struct RopeTensor {
  const void* x;
  void* y;
  int H, parts, rot_parts, d;  // heads, items of a head, of them rotated
  int last;                    // items of a token in this tensor and those before it
  uint32_t div_parts, div_H;
  int64_t xs[3], ys[3];  // strides of batch, token, head
};

struct RopeParams {
  const uint64_t* turns;
  const void* positions;  // null: the token's index in its sequence
  int pos64;
  int64_t ps[2];  // strides of positions: batch, token
  int64_t tokens;
  int N, half, tpb, n;
  float mscale, sign;
  uint32_t div_half;
  RopeTensor t[kMaxRopeTensors];
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

// V values moved by one load: 16 bytes, or a single value where strides or addresses do
// not allow more.
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
  T v[V];
};

// x / q for 0 <= x < 2^18 and q < 2^14 with m = ceil(2^32 / q): x m / 2^32 exceeds x / q by less
// than 2^18 / 2^32 < 1 / q.  (q = 1 has m = 2^32, which does not fit: m = 0 stands for it.)
__device__ __forceinline__ int small_div(int x, uint32_t m) { return m ? (int)__umulhi((uint32_t)x, m) : x; }
uint32_t magic(int q) { return q == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + q - 1) / q); }

// One CTA serves tpb tokens: their sines and cosines, and where their rows start, go to
// shared memory once; then the items (V pairs of one head, or 2 V values to copy) of all the
// tensors together are spread over the threads.  Bound by HBM: every value is read and written
// once.  One item a thread at a time and 6 CTAs a SM keep the most in flight: a training pass of
// 128K tokens (q 32 x 128, k 8 x 128, q_idx 8 x 64, k_idx, 64 rotated, 5.97 GB) takes 867 us, 6.9
// TB/s; two heads a thread for one load of the angles 971 us, four 1360 us (registers), 8 CTAs
// (spills) 989 us.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, 6) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 s_cs[kMaxTokens * kMaxHalf];
  __shared__ longlong2 s_off[kMaxRopeTensors][kMaxTokens];  // of x and y
  const int64_t t0 = (int64_t)blockIdx.x * p.tpb;
  const int nt = (int)min((int64_t)p.tpb, p.tokens - t0);
  for (int i = threadIdx.x; i < nt * p.half; i += kThreads) {
    const int tok = small_div(i, p.div_half), pair = i - tok * p.half;
    const int64_t t = t0 + tok, b = p.N == p.tokens ? 0 : t / p.N, n = t - b * p.N;
    int64_t pos = n;
    if (p.positions) {
      const int64_t at = b * p.ps[0] + n * p.ps[1];
      pos = p.pos64 ? __ldg(static_cast<const int64_t*>(p.positions) + at)
                    : (int64_t)__ldg(static_cast<const int32_t*>(p.positions) + at);
    }
    const int64_t frac = (int64_t)((uint64_t)pos * __ldg(&p.turns[pair]));
    float s, c;
    sincospif((float)frac * 1.0842021724855044e-19f /* 2^-63: half turns */, &s, &c);
    s_cs[i] = make_float2(c * p.mscale, s * p.mscale * p.sign);
  }
  if (threadIdx.x < p.n * kMaxTokens) {
    const int ti = threadIdx.x / kMaxTokens, tok = threadIdx.x % kMaxTokens;
    const int64_t t = t0 + tok, b = t / p.N, n = t - b * p.N;
    s_off[ti][tok] = make_longlong2(b * p.t[ti].xs[0] + n * p.t[ti].xs[1], b * p.t[ti].ys[0] + n * p.t[ti].ys[1]);
  }
  __syncthreads();
  const int items = nt * p.t[p.n - 1].last;
  for (int item = threadIdx.x; item < items; item += kThreads) {
    int x = item, ti = 0;
    while (x >= nt * p.t[ti].last) ++ti;
    const RopeTensor& a = p.t[ti];
    if (ti > 0) x -= nt * p.t[ti - 1].last;
    const int row = small_div(x, a.div_parts), part = x - row * a.parts;
    const int tok = small_div(row, a.div_H), h = row - tok * a.H;
    const bool turn = part < a.rot_parts;
    // first vector of the item in its head, and the distance of the second one (0: none)
    const int at = turn ? (INTER ? part * 2 * V : part * V) : 2 * p.half + (part - a.rot_parts) * 2 * V;
    const int step = turn ? (INTER ? V : p.half) : at + V < a.d ? V : 0;
    const longlong2 off = s_off[ti][tok];
    const T* src = static_cast<const T*>(a.x) + (off.x + h * a.xs[2] + at);
    T* dst = static_cast<T*>(a.y) + (off.y + h * a.ys[2] + at);
    Pack<T, V> lo = *reinterpret_cast<const Pack<T, V>*>(src), hi;
    if (step) hi = *reinterpret_cast<const Pack<T, V>*>(src + step);
    if (turn) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 w = s_cs[tok * p.half + part * V + e];
        // the pair's two values: the vectors side by side, or neighbours in them
        T* p1 = INTER ? (2 * e < V ? &lo.v[(2 * e) % V] : &hi.v[(2 * e) % V]) : &lo.v[e];
        T* p2 = INTER ? (2 * e + 1 < V ? &lo.v[(2 * e + 1) % V] : &hi.v[(2 * e + 1) % V]) : &hi.v[e];
        const float x1 = to_f(*p1), x2 = to_f(*p2);
        *p1 = from_f<T>(x1 * w.x - x2 * w.y);
        *p2 = from_f<T>(x2 * w.x + x1 * w.y);
      }
    }
    *reinterpret_cast<Pack<T, V>*>(dst) = lo;
    if (step) *reinterpret_cast<Pack<T, V>*>(dst + step) = hi;
  }
}

template <typename T>
cudaError_t launch_rope(const RopeParams& p, bool vec, bool inter, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const unsigned grid = (unsigned)((p.tokens + p.tpb - 1) / p.tpb);
  if (vec) {
    if (inter) rope_kernel<T, V, true><<<grid, kThreads, 0, st>>>(p);
    else rope_kernel<T, V, false><<<grid, kThreads, 0, st>>>(p);
  } else {
    if (inter) rope_kernel<T, 1, true><<<grid, kThreads, 0, st>>>(p);
    else rope_kernel<T, 1, false><<<grid, kThreads, 0, st>>>(p);
  }
  note_launch();
  return cudaGetLastError();
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" int msa_rope(const msa_rope_t* r, const uint64_t* turns, const void* positions,
                        const msa_rope_tensor_t* tensors, int num_tensors, cudaStream_t stream) {
  if (!r || !tensors) return MSA_ERR_ARG;
  if (num_tensors < 1 || num_tensors > kMaxRopeTensors) return MSA_ERR_ARG;
  if (r->B < 0 || r->N < 0 || r->rot_dim < 2 || (r->rot_dim & 1)) return MSA_ERR_SHAPE;
  if (r->rot_dim > 2 * kMaxHalf) return MSA_ERR_UNSUPPORTED;
  if (!isfinite(r->mscale)) return MSA_ERR_ARG;
  if (r->dtype < MSA_DTYPE_BF16 || r->dtype > MSA_DTYPE_F32) return MSA_ERR_ARG;
  if (r->positions_bits != 32 && r->positions_bits != 64) return MSA_ERR_ARG;
  const int size = r->dtype == MSA_DTYPE_F32 ? 4 : 2;
  const int V = 16 / size;
  RopeParams p = {};
  p.tokens = (int64_t)r->B * r->N;
  bool vec = r->rot_dim % (2 * V) == 0;
  for (int i = 0; i < num_tensors; ++i) {
    const msa_rope_tensor_t& t = tensors[i];
    if (t.H < 1 || t.d < r->rot_dim) return MSA_ERR_SHAPE;
    if (t.H > 1024 || t.d > 2 * kMaxHalf) return MSA_ERR_UNSUPPORTED;
    if (p.tokens == 0) continue;
    if (!t.x || !t.y) return MSA_ERR_ARG;
    const uintptr_t ptrs = reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y);
    if (ptrs % size) return MSA_ERR_ARG;
    vec = vec && ptrs % 16 == 0 && t.d % V == 0;
    for (int k = 0; k < 3; ++k) vec = vec && t.x_stride[k] % V == 0 && t.y_stride[k] % V == 0;
  }
  if (p.tokens == 0) return MSA_OK;
  if (!turns || (reinterpret_cast<uintptr_t>(turns) & 7)) return MSA_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(positions) % (r->positions_bits / 8)) return MSA_ERR_ARG;
  Ctx cx;
  const int rc = device_ctx(&cx);
  if (rc) return rc;
  p.turns = turns;
  p.positions = positions;
  p.pos64 = r->positions_bits == 64;
  p.ps[0] = r->positions_stride[0];
  p.ps[1] = r->positions_stride[1];
  p.N = r->N;
  p.half = r->rot_dim / 2;
  p.div_half = magic(p.half);
  p.mscale = r->mscale;
  p.sign = r->inverse ? -1.f : 1.f;
  p.n = num_tensors;
  const int w = vec ? V : 1;
  int all = 0;  // items of a token
  for (int i = 0; i < num_tensors; ++i) {
    const msa_rope_tensor_t& t = tensors[i];
    RopeTensor& a = p.t[i];
    a.x = t.x;
    a.y = t.y;
    a.H = t.H;
    a.d = t.d;
    a.rot_parts = p.half / w;
    const int tail = t.x == t.y ? 0 : t.d - r->rot_dim;  // in place: already there
    a.parts = a.rot_parts + (tail + 2 * w - 1) / (2 * w);
    a.div_parts = magic(a.parts);
    a.div_H = magic(a.H);
    for (int k = 0; k < 3; ++k) {
      a.xs[k] = t.x_stride[k];
      a.ys[k] = t.y_stride[k];
    }
    all += a.H * a.parts;
    a.last = all;
  }
  // tokens a CTA: up to kMaxTokens while the grid still fills the GPU and an item index
  // stays below 2^18
  p.tpb = kMaxTokens;
  while (p.tpb > 1 && ((p.tokens + p.tpb - 1) / p.tpb < 8 * cx.num_sms || (int64_t)p.tpb * all > (1 << 18)))
    p.tpb >>= 1;
  if ((p.tokens + p.tpb - 1) / p.tpb > 0x7fffffffLL) return MSA_ERR_UNSUPPORTED;
  const bool inter = r->interleaved != 0;
  cudaError_t e;
  switch (r->dtype) {
    case MSA_DTYPE_BF16: e = launch_rope<__nv_bfloat16>(p, vec, inter, stream); break;
    case MSA_DTYPE_F16: e = launch_rope<__half>(p, vec, inter, stream); break;
    default: e = launch_rope<float>(p, vec, inter, stream); break;
  }
  return finish(e);
}
