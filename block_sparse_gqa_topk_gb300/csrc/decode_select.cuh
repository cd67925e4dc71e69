// decode_select.cuh -- the exact top-(k-1) of a row of pooled block scores, by one CTA of 256
// threads (decode.cu, decode_paged.cu).
#pragma once

#include "common.cuh"

namespace msa {

// Block scores as sortable 64-bit keys: larger key = larger score, equal scores -> the
// lower block id first.  Keys of distinct blocks are distinct.
__device__ __forceinline__ uint64_t rank_key(float v, int id) {
  uint32_t u = __float_as_uint(v);
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);  // order-preserving map to unsigned
  return ((uint64_t)u << 32) | (uint32_t)(0x7fffffff - id);
}
__device__ __forceinline__ int key_id(uint64_t key) { return 0x7fffffff - (int)(uint32_t)key; }

// dst[0 .. topk) = the M = min(topk - 1, c_own) best of the blocks 0 .. c_own - 1 (src
// descending, lower id first on ties) and c_own itself, ascending, -1 padded.
//   1. every lane keeps a sorted list of its own best KM >= topk - 1 candidates (registers);
//   2. each warp takes its best M in M rounds of a warp-wide max over the lanes' list
//      heads, into shared memory;
//   3. each of the 8 M survivors counts the survivors above it: rank < M is selected,
//      and the selected ids are placed in ascending order by a second count.
template <int KM>
__device__ __forceinline__ void select_blocks(const float* __restrict__ src, int c_own, int topk,
                                              int32_t* __restrict__ dst) {
  __shared__ uint64_t s_top[8 * KM];  // warp w's best M at [w M, w M + M)
  __shared__ int s_sel[KM];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int M = min(topk - 1, c_own);
  uint64_t top[KM];
#pragma unroll
  for (int s = 0; s < KM; ++s) top[s] = 0;  // below every real key
  for (int c0 = warp * 32 + lane; c0 < c_own; c0 += 4 * 256) {
    float v4[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v4[u] = c0 + 256 * u < c_own ? __ldg(&src[c0 + 256 * u]) : 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (c0 + 256 * u >= c_own) break;
      uint64_t x = rank_key(v4[u], c0 + 256 * u);
      if (x <= top[KM - 1]) continue;
#pragma unroll
      for (int s = 0; s < KM; ++s) {  // sorted insert, descending
        const uint64_t hi = x > top[s] ? x : top[s];
        x = x > top[s] ? top[s] : x;
        top[s] = hi;
      }
    }
  }
  // warp's best M: each round takes the largest list head, as a warp max of the key's
  // high word and then of the low word among the lanes holding that high word
  for (int r = 0; r < M; ++r) {
    const uint32_t hi = (uint32_t)(top[0] >> 32), lo = (uint32_t)top[0];
    const uint32_t mhi = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t mlo = __reduce_max_sync(0xffffffffu, hi == mhi ? lo : 0u);
    const uint64_t best = ((uint64_t)mhi << 32) | mlo;
    if (lane == 0) s_top[warp * M + r] = best;  // 0 when the warp had fewer than M candidates
    if (best != 0 && top[0] == best) {
#pragma unroll
      for (int s = 0; s + 1 < KM; ++s) top[s] = top[s + 1];
      top[KM - 1] = 0;
    }
  }
  __syncthreads();
  // selection among the 8 M survivors, then ascending order of the selected ids
  const int n = 8 * M;
  const int t = threadIdx.x;
  uint64_t mine = 0;
  int above = n;
  if (t < n) {
    mine = s_top[t];
    above = 0;
    for (int u = 0; u < n; ++u) above += s_top[u] > mine ? 1 : 0;
  }
  const bool sel = mine != 0 && above < M;
  if (sel) s_sel[above] = key_id(mine);
  __syncthreads();
  if (t < M) {
    const int id = s_sel[t];
    int pos = 0;
    for (int u = 0; u < M; ++u) pos += s_sel[u] < id ? 1 : 0;
    dst[pos] = id;
  }
  if (t == 0) dst[M] = c_own;  // every selected block lies before the own block
  for (int s = M + 1 + t; s < topk; s += blockDim.x) dst[s] = -1;
}

// The same result for c_own <= PER * 256, by threshold: thread t holds blocks t PER ..
// t PER + PER - 1 as order-preserving integers; the M-th largest value T is built bit by bit
// (the largest T that at least M values reach: one block-wide count a bit), and a scan over
// the threads, whose order is the blocks', places the values above T and the first of those
// equal to it.  Distinct scores are told apart after about 18 counts, which replace the
// lists' insertions and rounds.
template <int PER>
__device__ __forceinline__ void select_blocks_by_threshold(const float* __restrict__ src, int c_own, int topk,
                                                           int32_t* __restrict__ dst) {
  __shared__ int s_count[2][8], s_above[8], s_equal[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int M = min(topk - 1, c_own);
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = tid * PER + i;
    const uint32_t u = c < c_own ? __float_as_uint(__ldg(&src[c])) : 0xffffffffu;
    key[i] = (u & 0x80000000u) ? ~u : (u | 0x80000000u);  // past the end: 0, below every score
  }
  if (M > 0) {
    uint32_t T = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t want = T | (1u << bit);
      int n = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) n += key[i] >= want;
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) s_count[bit & 1][warp] = n;
      __syncthreads();
      n = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) n += s_count[bit & 1][w];
      if (n >= M) T = want;
      if (n == M) {  // exactly the values from T up: no bit below matters
        --T;
        break;
      }
    }
    // places: values above T all count, those equal to T in block order while room is left
    int above = 0, equal = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      above += key[i] > T;
      equal += key[i] == T && tid * PER + i < c_own;
    }
    int sa = above, se = equal;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, sa, o), e = __shfl_up_sync(0xffffffffu, se, o);
      if (lane >= o) {
        sa += a;
        se += e;
      }
    }
    if (lane == 31) {
      s_above[warp] = sa;
      s_equal[warp] = se;
    }
    __syncthreads();
    int total = 0;
    sa -= above;
    se -= equal;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      total += s_above[w];
      if (w < warp) {
        sa += s_above[w];
        se += s_equal[w];
      }
    }
    const int room = M - total;  // equal values that are taken
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = tid * PER + i;
      if (key[i] > T) {
        dst[sa + min(se, room)] = c;
        ++sa;
      } else if (key[i] == T && c < c_own) {
        if (se < room) dst[sa + se] = c;
        ++se;
      }
    }
  }
  if (tid == 0) dst[M] = c_own;
  for (int s = M + 1 + tid; s < topk; s += blockDim.x) dst[s] = -1;
}

}  // namespace msa
