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

// The same result for c_own <= PER * THREADS by counting ranks.  Thread t holds blocks t PER ..
// t PER + PER - 1 as order-preserving integers.
//   1. The M-th best of the threads' best scores bounds the M-th best score from below (M threads
//      hold one at least as good), so at most the PER values of M threads can be taken.
//   2. Each of those counts those above it: rank < M is taken.
//   3. Each taken block counts the taken blocks before it: its place in ascending order.
// Equal scores rank the lower block first throughout.  src: 16-byte aligned, PER a multiple of 4.
template <int PER, int THREADS>
__device__ __forceinline__ void select_blocks_by_rank(const float* __restrict__ src, int c_own, int topk,
                                                      int32_t* __restrict__ dst) {
  constexpr int MOST = 31;  // M <= topk - 1 <= 31
  __shared__ __align__(16) uint32_t s_best[THREADS];
  __shared__ uint64_t s_cand[PER * MOST];
  __shared__ int s_n, s_bound_thread, s_sel[MOST];
  __shared__ uint32_t s_bound;
  const int tid = threadIdx.x;
  const int M = min(topk - 1, c_own);
  if (M > 0) {
    uint32_t key[PER], best = 0;
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const int c = tid * PER + i;
      // blocks of the last vector past c_own are within the row, or padding behind it
      const uint4 w = c < c_own ? __ldg(reinterpret_cast<const uint4*>(src + c)) : make_uint4(0, 0, 0, 0);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t k = (u[e] & 0x80000000u) ? ~u[e] : (u[e] | 0x80000000u);
        key[i + e] = c + e < c_own ? min(max(k, 1u), 0xfffffffeu) : 0u;  // 0: no block
        best = max(best, key[i + e]);
      }
    }
    s_best[tid] = best;
    if (tid == 0) {
      s_n = 0;
      s_bound = 1;  // every block, unless M threads hold one
      s_bound_thread = THREADS;
    }
    __syncthreads();
    // rank of this thread's best: of equal ones the lower thread's is above.  (A short loop:
    // code that runs once is paid for by its size.)
    int rank = 0;
    const uint4* all = reinterpret_cast<const uint4*>(s_best);
#pragma unroll 4
    for (int t = 0; t < THREADS; t += 4) {
      const uint4 x = all[t / 4];
      rank += (x.x + (t < tid) > best) + (x.y + (t + 1 < tid) > best) + (x.z + (t + 2 < tid) > best) +
              (x.w + (t + 3 < tid) > best);
    }
    if (rank == M - 1 && best > 0) {
      s_bound = best;
      s_bound_thread = tid;
    }
    __syncthreads();
    const uint32_t bound = s_bound + (tid <= s_bound_thread ? 0u : 1u);
    if (best >= bound) {
      int mine = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) mine += key[i] >= bound;
      int at = atomicAdd(&s_n, mine);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (key[i] >= bound) s_cand[at++] = ((uint64_t)key[i] << 32) | (uint32_t)(0x7fffffff - (tid * PER + i));
    }
    __syncthreads();
    const int n = s_n;
    for (int x = tid; x < n; x += THREADS) {
      const uint64_t mine = s_cand[x];
      int above = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) above += s_cand[j] > mine ? 1 : 0;
      if (above < M) s_sel[above] = key_id(mine);
    }
    __syncthreads();
    if (tid < M) {
      const int id = s_sel[tid];
      int pos = 0;
      for (int j = 0; j < M; ++j) pos += s_sel[j] < id ? 1 : 0;
      dst[pos] = id;
    }
  }
  if (tid == 0) dst[M] = c_own;
  for (int s = M + 1 + tid; s < topk; s += blockDim.x) dst[s] = -1;
}

}  // namespace msa
