// rope_items.cuh -- the unit of work of a rotary turn (rope.cu, append.cu): V pairs of one head, or
// 2 V values behind the rotated ones.
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "small_div.cuh"

namespace msa {

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

// The sine and cosine of a position's turn of one pair, times mscale.  position * turns in wrapping 64-bit
// arithmetic is the angle's fraction of a turn without rounding.
__device__ __forceinline__ float2 turn_of(int64_t position, uint64_t turns, float mscale) {
  const int64_t frac = (int64_t)((uint64_t)position * turns);
  float s, c;
  sincospif((float)frac * 1.0842021724855044e-19f /* 2^-63: half turns */, &s, &c);
  return make_float2(c * mscale, s * mscale);
}

// A pair's two values turned by w, the same roundings in every kernel: x1 w.x - x2 w.y, x2 w.x + x1 w.y.
__device__ __forceinline__ float turned_first(float x1, float x2, float2 w) {
  return fmaf(x1, w.x, -__fmul_rn(x2, w.y));
}
__device__ __forceinline__ float turned_second(float x1, float x2, float2 w) {
  return fmaf(x1, w.y, __fmul_rn(x2, w.x));
}

// An item of a head (src, dst: where the head starts): its rot_parts turned items come first, then the
// rest, of d values.  cs: the turns of the token's pairs.
template <typename T, int V>
struct RopeItem {
  int at, step;  // first vector of the item in its head, and the distance of the second one (0: none)
  bool turn;
  Pack<T, V> lo, hi;
  __device__ __forceinline__ RopeItem(int part, int rot_parts, int half, int d, bool inter) {
    turn = part < rot_parts;
    at = turn ? (inter ? part * 2 * V : part * V) : 2 * half + (part - rot_parts) * 2 * V;
    step = turn ? (inter ? V : half) : at + V < d ? V : 0;
  }
  __device__ __forceinline__ void load(const T* src) {
    lo = *reinterpret_cast<const Pack<T, V>*>(src + at);
    if (step) hi = *reinterpret_cast<const Pack<T, V>*>(src + at + step);
  }
  template <bool INTER>
  __device__ __forceinline__ void rotate(const float2* cs, int part) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 w = cs[part * V + e];
      // the pair's two values: the vectors side by side, or neighbours in them
      T* p1 = INTER ? (2 * e < V ? &lo.v[(2 * e) % V] : &hi.v[(2 * e) % V]) : &lo.v[e];
      T* p2 = INTER ? (2 * e + 1 < V ? &lo.v[(2 * e + 1) % V] : &hi.v[(2 * e + 1) % V]) : &hi.v[e];
      const float x1 = to_f(*p1), x2 = to_f(*p2);
      *p1 = from_f<T>(turned_first(x1, x2, w));
      *p2 = from_f<T>(turned_second(x1, x2, w));
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < V; ++e) lo.v[e] = hi.v[e] = from_f<T>(0.f);
  }
  __device__ __forceinline__ void store(T* dst) const {
    *reinterpret_cast<Pack<T, V>*>(dst + at) = lo;
    if (step) *reinterpret_cast<Pack<T, V>*>(dst + at + step) = hi;
  }
};

}  // namespace msa
