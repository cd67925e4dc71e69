// decode_paged.cuh -- attention of one new token a sequence over a paged cache (see
// include/msa.h): over the whole cache (msa_decode_paged_dense), or over the blocks that the
// index branch selects (msa_decode_paged).  The kernels of all kinds of caches; decode_paged.cu has
// those of bf16 and E4M3, decode_paged_e2m1.cu those of 4 bits (side by side for the compiler's time).
//
// For head h of group g, over the tokens T of the sequence (or of its selected blocks):
//   s_j = scale q_h . k_j,  o = sum_j e^(s_j - m) v_j / l,  l = sum_j e^(s_j - m),
//   lse = m + ln l,  m = max_j s_j,
// in one pass with a running m, l and o, and joined over the parts of a split by
//   lse = ln sum_i e^lse_i,  o = sum_i e^(lse_i - lse) o_i.
//
// The cache is read once and each byte meets 2 G multiply-adds, so HBM sets the pace and the
// products run on mma.sync with the group's heads as the 16 rows (4 bits, where the instructions of
// widening and scaling the codes weigh more than their bytes, with keys as rows).
#pragma once

#include <cuda_fp16.h>
#include <math.h>
#include <atomic>

#include "cache_rows.cuh"
#include "decode_select.cuh"
#include "kernels.h"

namespace msa {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// CTAs over which a call's units are spread: three (four) on each of the 152 SMs.  Each leaves at
// most two partial results (its first and its last (sequence, group)), whatever the batch.
constexpr int kCtas = 152 * 3, kMaxCtas = 152 * 4;  // (four for whole 4-bit caches)
// Blocks a sequence up to which the attention kernel selects for itself, 8 scores a thread: every
// CTA of a (sequence, group) then repeats the counting, which is less than the launch it saves.
constexpr int kSelectPer = 8;

struct PagedDecode {
  PageView pages;
  const __nv_bfloat16* q;      // [B][H G][d]
  const __nv_bfloat16* q_idx;  // [B][H][d_idx]
  const void* k;
  const void* v;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  const __nv_bfloat16* k_idx;
  const int32_t* lens;  // [B]
  int32_t* block_idx;   // [B][H][topk]; null: the whole cache
  float* pooled;        // [B][H][row]
  float* part_o;        // [2 ctas][wh][G][d]
  float* part_lse;      // [2 ctas][wh][G], in bits (log2)
  int* starts;          // [B + 2] first unit of each sequence, their total, wh: for the join
  int* arrive;          // [B][H] parts that are written (selected blocks; zeroed by the pooling)
  __nv_bfloat16* o;
  float* lse;
  int B, H, G, topk;
  int together;    // 4 bits: four groups side by side come by TMA
  int withheld;    // unit of a span whose copies are left out (msa_debug_set); -1: none
  uint64_t wait_ns;  // bound of a wait for it
  int row;         // blocks of the table's length, rounded up to 4
  int cluster;     // CTAs of a (sequence, group) in the small form; 0: the other one
  int ctas;        // of the attention kernel
  int select;      // it selects the blocks itself
  int wh;          // heads (groups) that a CTA may serve side by side
  int keys_shift;  // log2 of a stage's keys
  float scale_log2;  // scale * log2 e: scores in bits
  int* status;
};

namespace {

// Length of sequence b; 0 (an empty slot) where it does not fit the table.
__device__ __forceinline__ int seq_len(const PagedDecode& p, int b) {
  const int n = __ldg(&p.lens[b]);
  if (n < 0 || n > (int64_t)p.pages.max_pages * p.pages.page_size) {
    set_status(p.status, MSA_ERR_ARG);
    return 0;
  }
  return n;
}

// Units of a sequence for one group (wh groups): a unit is a stage of each of the kWarps / wh
// warps that share a group's tokens.
template <bool SPARSE>
__device__ __forceinline__ int seq_units(const PagedDecode& p, int len, int wh) {
  if (SPARSE) {  // the own block, cut at the length, comes last of the selected ones
    const int blocks = (int)(((unsigned)len + 127) / 128);
    len -= max(0, blocks - p.topk) * 128;
  }
  const int shift = p.keys_shift + (wh == 1 ? 2 : wh == 2 ? 1 : 0);
  return (int)(((unsigned)len + (1u << shift) - 1) >> shift);
}

// The work of all (sequence, groups) pairs in order is cut into n runs whose lengths differ by at
// most one: CTA c < n takes total c / n .. total (c + 1) / n - 1.  A pair's work is its units and
// kOverhead more in front of them, about what starting and ending a pair costs a CTA, so that
// CTAs with many short sequences get fewer units.  n is the CTAs, or the multiple of the number of
// pairs next below it where few CTAs are lost (pairs of one length are then cut alike, and no
// CTA has parts of two), and at most total: each run is at least 1 long, so every CTA between
// the first and the last that hold units of a pair holds some.
constexpr int kOverhead = 2;
__device__ __forceinline__ int seq_work(int units) { return units > 0 ? units + kOverhead : 0; }
struct Cut {
  int total, n, q, r;  // total = q n + r
  float inv;           // 1 / n
  __device__ __forceinline__ Cut(int total, int pairs, int ctas) : total(total) {
    const int even = pairs <= ctas ? ctas - ctas % max(1, pairs) : 0;
    n = max(1, min(total, even >= ctas * 9 / 10 ? even : ctas));
    q = total / n;
    r = total - q * n;
    inv = 1.f / (float)n;
  }
  // r cta / n by a float product: (x + 1/2) / n is 0.5 / n from an integer, and x < n^2 < 2^19 moves
  // by at most 2^-4 / n in the roundings
  __device__ __forceinline__ int start(int cta) const {
    return cta >= n ? total : q * cta + (int)(((float)(r * cta) + 0.5f) * inv);
  }
  __device__ __forceinline__ int cta_of(int x) const {  // whose run holds x
    int c = min(n - 1, (int)((float)x * ((float)n / (float)total)));
    while (start(c) > x) --c;
    while (start(c + 1) <= x) ++c;
    return c;
  }
};

// Groups side by side read rows that are neighbours in a page, which HBM serves faster where CTAs
// are not in step (8 groups, one group a CTA against four: 32 x 32K E4M3 d 128 450 / 336 us, d 64
// 398 / 231, bf16 623 / 601; 16 x 60K E4M3 d 64 364 / 212), but they leave wh times the parts to join
// and wait for one another: few pairs, cut alike, lose up to 7 percent (8 x 128K E4M3 d 128 335 / 333,
// d 64 216 / 229, bf16 593 / 598).  They pay from about this much work (of one group) a CTA.
constexpr int kSideBySide = 48;
// 4-bit caches whose groups come together by TMA gain from less work on, as one warp copies for all
// (32 ragged sequences up to 32K, 8 groups: 105 us where they begin at 24 or 48 units a CTA, 82 at 12), but
// not from little: with about 7 units a CTA, 4 groups of 32 ragged sequences up to 8K take 31.2 us apart and 32.2
// together (begun at 3 or 6), 8 groups up to 4K 34.7 and 35.7.
constexpr int kSideBySideTogether = 12;

struct Work {
  Cut cut;
  int wh, HG;   // groups side by side, H / wh
  int b, base;  // the sequence that holds the start of the CTA's run (any if that is empty), and
                // where its work starts
};

// Every warp finds the work for itself, without a barrier.  CTA 0 leaves what the join needs.
template <bool SPARSE>
__device__ __forceinline__ Work find_run(const PagedDecode& p) {
  const int lane = threadIdx.x & 31;
  const int per = (p.B + 31) / 32;
  const int b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
  int mine = 0, side = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = seq_len(p, b);
    mine += seq_work(seq_units<SPARSE>(p, len, 1));
    if (!SPARSE) side += seq_work(seq_units<SPARSE>(p, len, p.wh));
  }
  const int total1 = __reduce_add_sync(0xffffffffu, mine) * p.H;
  const bool sided = !SPARSE && p.wh > 1 && total1 >= (p.together ? kSideBySideTogether : kSideBySide) * p.ctas;
  const int wh = sided ? p.wh : 1, HG = sided ? p.H / p.wh : p.H;
  mine = (sided ? side : mine) * HG;
  int scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += x;
  }
  const int total = __shfl_sync(0xffffffffu, scan, 31);
  int base = scan - mine;  // where the work of this lane's sequences starts
  const Cut cut(total, p.B * HG, p.ctas);
  const int want = cut.start(blockIdx.x);
  const bool first_cta = blockIdx.x == 0 && threadIdx.x < 32;
  const unsigned holds = __ballot_sync(0xffffffffu, want >= base && want < base + mine);
  const int src = holds ? __ffs(holds) - 1 : 0;
  int found = 0, found_base = 0;
  if (first_cta || lane == src) {
    for (int b = b0; b < b1; ++b) {
      const int n = seq_work(seq_units<SPARSE>(p, seq_len(p, b), wh)) * HG;
      if (first_cta) p.starts[b] = base;
      if (want >= base && want < base + n) {
        found = b;
        found_base = base;
      }
      base += n;
    }
  }
  if (first_cta && lane == 0) {
    p.starts[p.B] = total;
    p.starts[p.B + 1] = wh;
  }
  __syncwarp();
  return {cut, wh, HG, __shfl_sync(0xffffffffu, found, src), __shfl_sync(0xffffffffu, found_base, src)};
}

// The parts of one (sequence, groups) pair whose work is first .. first + units + kOverhead - 1.
struct Parts {
  int c0, n, late;
  __device__ __forceinline__ Parts(const Cut& cut, int first, int units) {
    c0 = cut.cta_of(first + kOverhead);  // the CTA that holds the first unit
    n = cut.cta_of(first + kOverhead + units - 1) - c0 + 1;
    late = cut.start(c0) < first;        // it began with another pair
  }
  // part i is slot 0 of CTA c0 + i, except where CTA c0 began with another pair
  __device__ __forceinline__ int64_t slot(int i) const { return 2 * (c0 + i) + (i == 0 ? late : 0); }
};

// D(16x8) += A(16x16, row) * B(16x8, col), fp16
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two E4M3 codes as a pair of fp16 (exact).
__device__ __forceinline__ uint32_t widen_f16(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}

// A pair of fp16 as bf16 (exact for E4M3 values).
__device__ __forceinline__ uint32_t f16_to_bf16(uint32_t two) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&two));
  return pack_bf16(v.x, v.y);
}

// 2^(a - b), 0 for a = -inf whatever b.
__device__ __forceinline__ float weight(float a, float b) { return a == -INFINITY ? 0.f : ex2_fast(a - b); }

// Shared memory of one warp's stage: KEYS key rows and as many value rows (and their scales),
// 8 KB of them for most caches.
//   bf16: rows of 2 D bytes, 16-byte chunks XOR-swizzled for ldmatrix;
//   E4M3: key rows of D bytes whose 64-byte halves are swapped in odd rows, value rows padded
//   by 16 bytes: the fragment loads then fall in distinct banks;
//   E2M1: key rows of D / 2 bytes, value rows padded by 16 bytes, for the same reason; the records of
//   scales lie behind all warps' stages.
template <int D, int KIND, bool WIDE>
struct Stage {
  static constexpr bool CODED = KIND != MSA_CACHE_BF16, F4 = KIND == MSA_CACHE_E2M1;
  static constexpr int KEYS = CODED || D == 64 ? 32 : 16;
  static constexpr int ROW = F4 ? D / 2 : CODED ? D : 2 * D;
  static constexpr int VROW = CODED ? ROW + 16 : ROW;
  static constexpr int BLOCKS = F4 ? D / 16 : 0;         // block scales of a row
  static constexpr int SCALE = CODED ? 4 + BLOCKS : 0;   // bytes of a row's scales in the pool
  static constexpr int V0 = KEYS * ROW;
  static constexpr int S0 = V0 + KEYS * VROW;  // [2][KEYS] scales of E4M3 rows
  static constexpr int BYTES = S0 + (CODED && !F4 ? 2 * KEYS * 4 : 0);
  static constexpr int SCALES = F4 ? 2 * KEYS * SCALE : 0;  // E2M1: a stage's scales, [2][KEYS] records as in the pool
  // CTAs of a SM.  More than 8 heads with d = 128 take more than the 168 registers a thread that
  // three CTAs leave: two with a third stage serve them better (8 x 128K, 16 heads a group, E4M3:
  // 423 -> 392 us), but not with d = 64 (E4M3 269 -> 321 us).
  static constexpr int PER_SM = WIDE && D == 128 ? 2 : 3;
  static constexpr int COUNT = PER_SM == 2 ? 3 : 2;
  // whole 4-bit caches: four, as their products wait for one another (8 x 128K 287 -> 273 us)
  static constexpr int DENSE_PER_SM = F4 && PER_SM == 3 ? 4 : PER_SM;
  static constexpr int HALVES = KEYS / 16;    // runs of 16 tokens, which never straddle a page
  static constexpr int RINGS = kWarps * COUNT * BYTES;           // bytes of all stages without E2M1's scales
  static constexpr int SMEM = RINGS + kWarps * COUNT * SCALES;  // and with them
  // E2M1, four groups of the same tokens together: stages of the CTA, each [2][HALVES] boxes of 16 tokens
  // of keys or values (four groups' codes of a token side by side, 16-byte chunks XOR-swizzled by TMA)
  // and the four groups' scales.
  static constexpr int BOX = 16 * 4 * ROW, TOGETHER = 2 * HALVES * BOX + 4 * SCALES, TOGETHER_COUNT = DENSE_PER_SM == 4 ? 2 : 3;
  static constexpr int SMEM_TOGETHER = TOGETHER_COUNT * TOGETHER + 1024;  // their start is rounded up
  static constexpr int UNIT = KEYS * kWarps;  // tokens of a unit of work
  static constexpr int PER = 128 / UNIT;      // units of a block
  __device__ __forceinline__ static uint32_t key_at(int r, int ch) {  // not of E2M1
    if constexpr (!CODED) return swz<ROW>(r, ch);
    else return r * ROW + ((D == 128 ? ch ^ ((r & 1) << 2) : ch) << 4);
  }
  __device__ __forceinline__ static uint32_t value_at(int r, int ch) {
    if constexpr (!CODED) return V0 + swz<ROW>(r, ch);
    else return V0 + r * VROW + (ch << 4);
  }
};

__device__ __forceinline__ float lg2_fast(float x) {  // relative to 1: about 2^-22; of subnormal x too
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Eight E2M1 codes times their block's scale as four pairs of fp16 (exact: 2 and 4 significant bits,
// 2^-10 .. 2688).
__device__ __forceinline__ void widen_scaled(uint32_t codes, uint32_t scale, uint32_t (&h)[4]) {
  widen_e2m1(codes, h);
#pragma unroll
  for (int e = 0; e < 4; ++e) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[e]) : "r"(h[e]), "r"(scale));
}

constexpr float kWeightBits = 15.f;  // codes: the largest weight of one is 2^15

// One warp's running softmax over its keys.
//   S = Q K^T: rows are heads gq and gq + 8 (WIDE; else idle); columns are keys 8 t + 2 tq + e.
//   O^T = V^T P^T: rows are value columns, columns the heads 8 nt + 2 tq + e, so that the
//   accumulator of at most 8 heads has no idle rows; the fragments of S are those of P^T.
// (gq = lane / 4, tq = lane % 4.)
template <int D, int KIND, bool WIDE>
struct WarpState {
  using St = Stage<D, KIND, WIDE>;
  static constexpr int R = WIDE ? 2 : 1;     // heads of a lane's rows of S
  static constexpr int MT = D / 16;          // tiles of 16 value columns
  static constexpr int KT = St::KEYS / 8;    // tiles of 8 keys
  static constexpr int QS = D / 16;
  static constexpr bool CODED = St::CODED;
  static_assert(!St::F4, "4 bits have their own");
  uint32_t qa[QS][4];       // query fragments
  float o[MT][R][4];
  float m[R], mv[R], l[R];  // max, max with the value scale relative to it (codes), lane's part of the sum
  float fac[R];             // accumulator -> score in bits
  bool far;                 // codes: the queries are bf16, not fp16

  __device__ __forceinline__ void load_q(const PagedDecode& p, int64_t head0, int gq, int tq) {
    bool lost = false, huge[R] = {};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int h = gq + 8 * r;
      const bool ok = h < p.G;
      const __nv_bfloat16* row = p.q + (head0 + (ok ? h : 0)) * D;
      if constexpr (!CODED) {
#pragma unroll
        for (int ks = 0; ks < QS; ++ks)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            qa[ks][r + 2 * half] =
                r < R && ok ? __ldg(reinterpret_cast<const uint32_t*>(row + ks * 16 + half * 8 + 2 * tq)) : 0u;
      } else if (r < R) {
        // lane tq holds values 64 j + 16 tq + 0..15 of the row, in the order in which step() reads
        // the codes of a key: values 4 s + {0, 1} and 4 s + {2, 3} of them are k slots 2 tq.. and
        // 8 + 2 tq.. of k step 4 j + s
        float2 f[D / 64][8];
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint4 w = ok ? __ldg(reinterpret_cast<const uint4*>(row + 64 * j + 16 * tq + 8 * half))
                               : make_uint4(0, 0, 0, 0);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 x = make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u));
              f[j][4 * half + e] = x;
              amax = fmax3(amax, fabsf(x.x), fabsf(x.y));
            }
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // The row enters in fp16, scaled by a power of two to a largest value in [2^14, 2^15):
        // exact for values of at least 2^-31 of the largest.  Where any value is smaller and loses
        // bits (or is NaN), the group's queries enter in bf16 and the codes are widened to that
        // (8 x 128K, d 128: 358 us for 333; 16 heads a group 432 for 392; d 64 246 for 229).
        const int e = max((int)(__float_as_uint(amax) >> 23), 40);
        const float down = __uint_as_float((uint32_t)(268 - e) << 23);  // 2^(141 - e)
        const float up = __uint_as_float((uint32_t)(e - 14) << 23);
        fac[r] = p.scale_log2 * up;
        huge[r] = amax >= 0x1p100f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            const float2 x = f[j][w];
            const uint32_t h2 = pack_f16(x.x * down, x.y * down);
            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            lost = lost || back.x * up != x.x || back.y * up != x.y;
            qa[4 * j + (w >> 1)][r + 2 * (w & 1)] = h2;
          }
      } else {
#pragma unroll
        for (int ks = 0; ks < QS; ++ks) qa[ks][1] = qa[ks][3] = 0u;
      }
    }
    far = CODED && __any_sync(0xffffffffu, lost);
    if constexpr (CODED) {
      if (far) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int h = gq + 8 * r;
          // a query of 2^100 and more enters as 2^-32 of its value, so that no product with a code
          // overflows before the key's scale is applied
          const float down = huge[r] ? 0x1p-32f : 1.f;
          fac[r] = p.scale_log2 / down;
#pragma unroll
          for (int w = 0; w < D / 8; ++w) {
            const int at = 64 * (w >> 3) + 16 * tq + 2 * (w & 7);
            const uint32_t u = h < p.G ? __ldg(reinterpret_cast<const uint32_t*>(p.q + (head0 + h) * D + at)) : 0u;
            qa[w >> 1][r + 2 * (w & 1)] =
                pack_bf16(__uint_as_float(u << 16) * down, __uint_as_float(u & 0xffff0000u) * down);
          }
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) fac[r] = p.scale_log2;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = mv[r] = -INFINITY;
      l[r] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][r][e] = 0.f;
  }

  // O times a factor a head, given for the rows of S (heads gq + 8 r).
  __device__ __forceinline__ void rescale(const float (&alpha)[R], int tq) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float2 a = make_float2(__shfl_sync(0xffffffffu, alpha[r], 8 * tq),
                                   __shfl_sync(0xffffffffu, alpha[r], 8 * tq + 4));
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const float2 x = fmul2(make_float2(o[i][r][0], o[i][r][1]), a);
        const float2 y = fmul2(make_float2(o[i][r][2], o[i][r][3]), a);
        o[i][r][0] = x.x;
        o[i][r][1] = x.y;
        o[i][r][2] = y.x;
        o[i][r][3] = y.y;
      }
    }
  }

  // The keys of a landed stage, of which the first n are the sequence's.
  __device__ __forceinline__ void step(const uint8_t* st, int n, int lane) {
    const int gq = lane >> 2, tq = lane & 3, mi = lane >> 3;
    float sc[KT][4] = {};
    if constexpr (!CODED) {
#pragma unroll
      for (int kp = 0; kp < KT / 2; ++kp) {
        const int row = 16 * kp + (lane & 7) + (mi >> 1) * 8;
#pragma unroll
        for (int ks = 0; ks < QS; ++ks) {
          uint32_t kb[4];
          ldmatrix_x4(kb, st + St::key_at(row, 2 * ks + (mi & 1)));
          mma_bf16_16816(sc[2 * kp], qa[ks], kb[0], kb[1]);
          mma_bf16_16816(sc[2 * kp + 1], qa[ks], kb[2], kb[3]);
        }
      }
    } else {
      // the order of a product's terms is free: lane tq takes values 64 j + 16 tq + 0..15 of
      // key gq as the k slots of steps 4 j .. 4 j + 3, and so do the query fragments
      auto products = [&](bool in_bf16) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            const uint4 c = *reinterpret_cast<const uint4*>(st + St::key_at(8 * t + gq, 4 * j + tq));
            const uint32_t u[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const uint32_t k0 = widen_f16(u[s] & 0xffffu), k1 = widen_f16(u[s] >> 16);
              if (in_bf16) mma_bf16_16816(sc[t], qa[4 * j + s], f16_to_bf16(k0), f16_to_bf16(k1));
              else mma_f16_16816(sc[t], qa[4 * j + s], k0, k1);
            }
          }
      };
      if (far) products(true);
      else products(false);
    }
    // scores in bits; this lane's keys: 8 t + 2 tq + e
    float2 lv[CODED ? KT : 1];  // log2 of the value scales
    if constexpr (CODED) {
      const float* scale = reinterpret_cast<const float*>(st + St::S0);
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const float2 ks = *reinterpret_cast<const float2*>(scale + 8 * t + 2 * tq);
        const float2 vs = *reinterpret_cast<const float2*>(scale + St::KEYS + 8 * t + 2 * tq);
        lv[t] = make_float2(lg2_fast(vs.x), lg2_fast(vs.y));
#pragma unroll
        for (int r = 0; r < R; ++r) {
          sc[t][2 * r] *= ks.x * fac[r];  // one factor: each alone may leave the range
          sc[t][2 * r + 1] *= ks.y * fac[r];
        }
      }
    }
    float alpha[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        float &s0 = sc[t][2 * r], &s1 = sc[t][2 * r + 1];
        if constexpr (!CODED) {
          s0 *= fac[r];
          s1 *= fac[r];
        }
        if (n < St::KEYS) {
          s0 = 8 * t + 2 * tq < n ? s0 : -INFINITY;
          s1 = 8 * t + 2 * tq + 1 < n ? s1 : -INFINITY;
        }
        top = fmax3(top, s0, s1);
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float m_new = fmaxf(m[r], top);
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      const float m_old = m[r];
      alpha[r] = ex2_fast(m_old - m_use);
      m[r] = m_new;
      l[r] *= alpha[r];
      if constexpr (CODED) {
        // o is kept in units of 2^(m + mv - 15), mv the running max of score - m + log2(value scale):
        // the weights of the codes are then at most 2^15, which fp16 holds whatever the scales are.
        // (Relative to m, so that a scale is not lost beside a large score.)
        const float moved = m_old - m_use;
        float topv = -INFINITY;
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          float &s0 = sc[t][2 * r], &s1 = sc[t][2 * r + 1];
          s0 -= m_use;
          s1 -= m_use;
          topv = fmax3(topv, s0 + lv[t].x, s1 + lv[t].y);
        }
        topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, 1));
        topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, 2));
        const float v_new = fmaxf(mv[r] + moved, topv);
        const float v_use = v_new == -INFINITY ? 0.f : v_new, v_unit = v_use - kWeightBits;
        alpha[r] = ex2_fast(mv[r] + moved - v_use);
        mv[r] = v_new;
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          float &s0 = sc[t][2 * r], &s1 = sc[t][2 * r + 1];
          l[r] += ex2_fast(s0) + ex2_fast(s1);
          s0 = ex2_fast(s0 + (lv[t].x - v_unit));
          s1 = ex2_fast(s1 + (lv[t].y - v_unit));
        }
      } else {
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          float &s0 = sc[t][2 * r], &s1 = sc[t][2 * r + 1];
          s0 = ex2_fast(s0 - m_use);
          s1 = ex2_fast(s1 - m_use);
          l[r] += s0 + s1;
        }
      }
    }
    // sc now holds P (codes: times the value scales)
    bool same = alpha[0] == 1.f;
    if constexpr (WIDE) same = same && alpha[R - 1] == 1.f;
    if (!__all_sync(0xffffffffu, same)) rescale(alpha, tq);
#pragma unroll
    for (int kp = 0; kp < KT / 2; ++kp) {  // 16 keys: one k step
      if constexpr (!CODED) {
        // P enters in two bf16 parts (together 2^-17 of its value): the output's own rounding
        // stays its largest error.  (An infinite value makes its column NaN, where one part is 0
        // or below it.)
        uint32_t hi[R][2], lo[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float e0 = sc[2 * kp + t][2 * r], e1 = sc[2 * kp + t][2 * r + 1];
            const uint32_t h = pack_bf16(e0, e1);
            hi[r][t] = h;
            lo[r][t] = pack_bf16(e0 - __uint_as_float(h << 16), e1 - __uint_as_float(h & 0xffff0000u));
          }
        const int row = 16 * kp + (lane & 7) + (mi >> 1) * 8;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          uint32_t va[4];  // V^T: matrix mi covers keys (mi >> 1) * 8.. and columns (mi & 1) * 8..
          ldmatrix_x4_trans(va, st + St::value_at(row, 2 * i + (mi & 1)));
#pragma unroll
          for (int r = 0; r < R; ++r) {
            mma_bf16_16816(o[i][r], va, hi[r][0], hi[r][1]);
            mma_bf16_16816(o[i][r], va, lo[r][0], lo[r][1]);
          }
        }
      } else {
        // weights in fp16: 2^-12 of their value down to 2^-29 of the largest that this warp met (of
        // weight times value scale), below that multiples of 2^-39 of it
        uint32_t pb[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t = 0; t < 2; ++t) pb[r][t] = pack_f16(sc[2 * kp + t][2 * r], sc[2 * kp + t][2 * r + 1]);
        // row gq (+ 8) of tile 4 c + i is value column 64 c + 8 gq + 2 i (+ 1): a lane's 8 codes
        // of each of its four keys serve four tiles, two keys side by side in a register
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint2 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = *reinterpret_cast<const uint2*>(
                st + St::V0 + (16 * kp + (i >> 1) * 8 + 2 * tq + (i & 1)) * St::VROW + 64 * c + 8 * gq);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t va[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // e & 1: column 2 i + 1; e >> 1: keys 8..15
              const uint2 x = w[2 * (e >> 1)], y = w[2 * (e >> 1) + 1];
              const int byte = (2 * i + (e & 1)) & 3;
              va[e] = widen_f16(__byte_perm(i < 2 ? x.x : x.y, i < 2 ? y.x : y.y, byte | ((4 + byte) << 4)));
            }
#pragma unroll
            for (int r = 0; r < R; ++r) mma_f16_16816(o[4 * c + i][r], va, pb[r][0], pb[r][1]);
          }
        }
      }
    }
  }

  // Value column that o[i][.][e] holds; its head is 8 r + 2 tq + (e & 1).
  __device__ __forceinline__ static int column(int i, int e, int gq) {
    return CODED ? (i >> 2) * 64 + 8 * gq + 2 * (i & 3) + (e >> 1) : 16 * i + gq + 8 * (e >> 1);
  }
};

// A matrix of 8 x 8 16-bit values, row gq and columns 2 tq, 2 tq + 1 a lane, turned over.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t t;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(a));
  return t;
}

// The running softmax over 4-bit keys.  Widening the codes takes the ALU (a conversion a pair, 2 cycles) and the
// FMA pipe (a product with the block's scale a pair, 2 cycles), and mma.sync (8 cycles) holds up the
// latter, so its products are few:
//   S^T = K Q^T: rows are keys, columns the heads 8 r + 2 tq + e (no idle rows; heads as rows: 16 of
//   32 products idle, 8 x 128K 38 us more);  O^T = V^T P^T as above, P^T turned over by movmatrix.
// A lane's 4 keys of 32 meet the 2 heads of its columns (with at most 4 heads 2 keys, so that the lanes of the
// other columns have a part too); maxima go over the lanes of a head, which is left out while no score passes
// the running ones.
template <int D, bool WIDE>
struct WarpState<D, MSA_CACHE_E2M1, WIDE> {
  using St = Stage<D, MSA_CACHE_E2M1, WIDE>;
  static constexpr int R = WIDE ? 2 : 1;  // tiles of 8 heads
  static constexpr int MT = D / 16;       // tiles of 16 value columns
  static constexpr int KP = St::KEYS / 16;
  static constexpr int QS = D / 16;
  uint32_t qb[QS][R][2];  // query fragments
  float o[MT][R][4];
  float m[R][2], mv[R][2], l[R][2];  // of heads 8 r + 2 tq + e: as in the form above
  float fac[R][2];
  bool far, few;  // few: at most 4 heads

  __device__ __forceinline__ void load_q(const PagedDecode& p, int64_t head0, int gq, int tq) {
    few = p.G <= 4;
    bool lost = false, huge[R] = {};
    float row_fac[R];  // of heads 8 r + gq
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int h = gq + 8 * r;
      const bool ok = h < p.G;
      const __nv_bfloat16* row = p.q + (head0 + (ok ? h : 0)) * D + D / 4 * tq;
      // lane tq holds values D / 4 tq .. of the row, in the order in which step() reads the codes of a
      // key: of each 16, values 4 s + {0, 1} and 4 s + {2, 3} are k slots 2 tq.. and 8 + 2 tq.. of k step s
      float2 f[D / 64][8];
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint4 w = ok ? __ldg(reinterpret_cast<const uint4*>(row + 16 * j + 8 * half)) : make_uint4(0, 0, 0, 0);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = widen(u[e]);
            f[j][4 * half + e] = x;
            amax = fmax3(amax, fabsf(x.x), fabsf(x.y));
          }
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // fp16 or bf16 by the rule of the form above
      const int e = max((int)(__float_as_uint(amax) >> 23), 40);
      const float down = __uint_as_float((uint32_t)(268 - e) << 23);  // 2^(141 - e)
      const float up = __uint_as_float((uint32_t)(e - 14) << 23);
      row_fac[r] = p.scale_log2 * up;
      huge[r] = amax >= 0x1p100f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float2 x = f[j][w];
          const uint32_t h2 = pack_f16(x.x * down, x.y * down);
          const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h2));
          lost = lost || back.x * up != x.x || back.y * up != x.y;
          qb[4 * j + (w >> 1)][r][w & 1] = h2;
        }
    }
    far = __any_sync(0xffffffffu, lost);
    if (far) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int h = gq + 8 * r;
        const float down = huge[r] ? 0x1p-32f : 1.f;
        row_fac[r] = p.scale_log2 / down;
#pragma unroll
        for (int w = 0; w < D / 8; ++w) {
          const int at = D / 4 * tq + 2 * w;
          const uint32_t u = h < p.G ? __ldg(reinterpret_cast<const uint32_t*>(p.q + (head0 + h) * D + at)) : 0u;
          const float2 x = widen(u);
          qb[w >> 1][r][w & 1] = pack_bf16(x.x * down, x.y * down);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        fac[r][e] = __shfl_sync(0xffffffffu, row_fac[r], 4 * (2 * (few ? tq & 1 : tq) + e));
        m[r][e] = mv[r][e] = -INFINITY;
        l[r][e] = 0.f;
      }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][r][e] = 0.f;
  }

  // Where a lane finds its codes in a stage, and the keys that its rows of the products are.  Of the
  // 16 keys of a run, rows 8 i + gq of S^T and k slots 8 i + 2 tq + s of P^T are keys 8 i + key and 8 i + slot[s].
  // One group's stage: keys in their order.  Four groups': the rows of 8 keys are 128 or 256 bytes apart, and
  // keys in the order 0 2 4 6 1 3 5 7, with the two of a pair changed over in half of the lanes (swap),
  // are what brings a load's chunks into distinct banks.
  template <bool TOGETHER>
  struct Place {
    static constexpr int KEY8 = TOGETHER ? 8 * 4 * St::ROW : 8 * St::ROW;  // bytes of 8 key rows
    static constexpr int VALUE8 = TOGETHER ? KEY8 : 8 * St::VROW;
    static constexpr int RS = (TOGETHER ? 4 : 1) * St::SCALE;  // from a record of scales to the next
    int k, v[2], key, slot[2];
    bool swap;
    __device__ __forceinline__ Place(int lane, int group) {
      const int gq = lane >> 2, tq = lane & 3;
      if constexpr (TOGETHER) {
        auto order = [](int x) { return (x & 3) << 1 | x >> 2; };
        auto at = [&](int row, int byte) {
          const int x = row * 4 * St::ROW + group * St::ROW + byte;
          return x ^ ((x >> 7 & 7) << 4);
        };
        swap = D == 128 ? tq & 1 : tq >> 1;
        key = order(gq);
        k = at(key, tq * (D / 8));
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          slot[s] = order(2 * tq + (s ^ (int)swap));
          v[s] = St::HALVES * St::BOX + at(slot[s], gq * (D / 16));
        }
      } else {
        swap = false;
        key = gq;
        k = gq * St::ROW + tq * (D / 8);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          slot[s] = 2 * tq + s;
          v[s] = St::V0 + slot[s] * St::VROW + gq * (D / 16);
        }
      }
    }
  };

  // From products to weights: sc[k][r][2 i + e] of key key0 + 16 k + 8 i + at.key and head 8 r + 2 tq + e becomes
  // out[k][r][i], turned over for the product with the values.  pairs: lanes tq and tq ^ 2 hold keys of the same
  // heads.
  template <typename P, int K>
  __device__ __forceinline__ void weights(float (&sc)[K][R][4], uint32_t (&out)[K][R][2], const uint8_t* rec,
                                          const P& at, int key0, int n, bool pairs) {
    constexpr int RS = P::RS;
    float lv[K][2];  // log2 of the value rows' scales
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = key0 + 16 * k + 8 * i + at.key;
        const float ks = *reinterpret_cast<const float*>(rec + key * RS);
        lv[k][i] = lg2_fast(*reinterpret_cast<const float*>(rec + (St::KEYS + key) * RS));
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& s = sc[k][r][2 * i + e];
            s *= ks * fac[r][e];  // scores in bits; one factor: each alone may leave the range
            if (n < St::KEYS && key >= n) s = -INFINITY;
          }
      }
    float top[R][2], mu[R][2];
    bool raise = false;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mu[r][e] = m[r][e] == -INFINITY ? 0.f : m[r][e];
        float topv = -INFINITY;
        top[r][e] = -INFINITY;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float s0 = sc[k][r][e], s1 = sc[k][r][2 + e];
          top[r][e] = fmax3(top[r][e], s0, s1);
          topv = fmax3(topv, s0 - mu[r][e] + lv[k][0], s1 - mu[r][e] + lv[k][1]);
        }
        raise = raise || top[r][e] > m[r][e] || topv > mv[r][e];
      }
    if (__any_sync(0xffffffffu, raise)) {  // new maxima: all that was summed takes their units
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          auto all = [&](float x) {  // over the lanes of the head
            if (pairs) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            return x;
          };
          const float m_new = fmaxf(m[r][e], all(top[r][e])), m_use = m_new == -INFINITY ? 0.f : m_new;
          const float moved = m[r][e] - m_use;
          m[r][e] = m_new;
          mu[r][e] = m_use;
          l[r][e] *= ex2_fast(moved);
          // o is kept in units of 2^(m + mv - 15), mv the running max of score - m + log2(value scale)
          float topv = -INFINITY;
#pragma unroll
          for (int k = 0; k < K; ++k)
            topv = fmax3(topv, sc[k][r][e] - m_use + lv[k][0], sc[k][r][2 + e] - m_use + lv[k][1]);
          const float v_new = fmaxf(mv[r][e] + moved, all(topv));
          alpha[e] = ex2_fast(mv[r][e] + moved - (v_new == -INFINITY ? 0.f : v_new));
          mv[r][e] = v_new;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][r][e] *= alpha[e & 1];
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float unit[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) unit[e] = (mv[r][e] == -INFINITY ? 0.f : mv[r][e]) - kWeightBits;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float s = sc[k][r][2 * i + e] - mu[r][e];
            l[r][e] += ex2_fast(s);
            w[e] = ex2_fast(s + (lv[k][i] - unit[e]));
          }
          out[k][r][i] = transpose_8x8(pack_f16(w[0], w[1]));
        }
    }
  }

  // The keys of a landed stage, of which the first n are the sequence's; rec: the first key's record of
  // scales.
  template <bool TOGETHER>
  __device__ __forceinline__ void step(const uint8_t* st, const uint8_t* rec, const Place<TOGETHER>& at, int n,
                                       int lane) {
    using P = Place<TOGETHER>;
    constexpr int RS = P::RS;
    const int gq = lane >> 2, tq = lane & 3;
    float sc[KP][R][4] = {};
    auto products = [&](bool in_bf16) {
      uint32_t u[KP][2][D / 32], scale[KP][2][D / 64];
#pragma unroll
      for (int kp = 0; kp < KP; ++kp)
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // row 8 i + gq
          const uint8_t* codes = st + at.k + (2 * kp + i) * P::KEY8;
          const uint8_t* block = rec + (16 * kp + 8 * i + at.key) * RS + 4 + tq * (D / 64);
          if constexpr (D == 128) {
            const uint4 c = *reinterpret_cast<const uint4*>(codes);
            u[kp][i][0] = c.x, u[kp][i][1] = c.y, u[kp][i][2] = c.z, u[kp][i][3] = c.w;
            const uint32_t two = widen_f16(*reinterpret_cast<const uint16_t*>(block));
            scale[kp][i][0] = __byte_perm(two, two, 0x1010);
            scale[kp][i][1] = __byte_perm(two, two, 0x3232);
          } else {
            const uint2 c = *reinterpret_cast<const uint2*>(codes);
            u[kp][i][0] = c.x, u[kp][i][1] = c.y;
            scale[kp][i][0] = widen_f16(*block * 0x0101u);
          }
        }
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int kp = 0; kp < KP; ++kp) {
          uint32_t k[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) widen_scaled(u[kp][i][w], scale[kp][i][w / 2], k[i]);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            uint32_t a[4] = {k[0][2 * s], k[1][2 * s], k[0][2 * s + 1], k[1][2 * s + 1]};
            if (in_bf16) {
#pragma unroll
              for (int e = 0; e < 4; ++e) a[e] = f16_to_bf16(a[e]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
              if (in_bf16) mma_bf16_16816(sc[kp][r], a, qb[2 * w + s][r][0], qb[2 * w + s][r][1]);
              else mma_f16_16816(sc[kp][r], a, qb[2 * w + s][r][0], qb[2 * w + s][r][1]);
            }
          }
        }
    };
    if (far) products(true);
    else products(false);
    uint32_t pb[KP][R][2];  // the weights times the value scales, in fp16 as in the form above
    if (!WIDE && few) {
      // the lanes of columns 4 .. 7, which no head has, take the second 16 keys of columns 0 .. 3
      float mine[1][R][4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float other = __shfl_xor_sync(0xffffffffu, sc[KP - 1][0][x], 2);
        mine[0][0][x] = tq & 2 ? other : sc[0][0][x];
      }
      uint32_t t[1][R][2];
      weights<P, 1>(mine, t, rec, at, (tq & 2) << 3, n, true);
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // rows 4 .. 7 of the turned matrix are the second 16 keys'
        pb[0][0][i] = t[0][0][i];
        pb[KP - 1][0][i] = __shfl_xor_sync(0xffffffffu, t[0][0][i], 16);
      }
    } else {
      weights<P, KP>(sc, pb, rec, at, 0, n, false);
    }
    if (TOGETHER) {
      const uint32_t order = at.swap ? 0x1032 : 0x3210;
#pragma unroll
      for (int kp = 0; kp < KP; ++kp)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < 2; ++i) pb[kp][r][i] = __byte_perm(pb[kp][r][i], pb[kp][r][i], order);
    }
    // row gq (+ 8) of tile i is value column D / 8 gq + 2 i (+ 1): a lane's D / 8 codes of each of its four
    // keys, one block's, serve all tiles.  The codes of two keys go side by side into a byte, so that
    // they come out as a pair, with the pair of their block's scales.
#pragma unroll
    for (int kp = 0; kp < KP; ++kp) {
      uint32_t w[4][D / 64], scale[2];
      const uint8_t* block = rec + (St::KEYS + 16 * kp) * RS + 4 + gq * (D / 8) / 16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // k slot 8 (i / 2) + 2 tq + i % 2
        const uint8_t* codes = st + at.v[i & 1] + (2 * kp + (i >> 1)) * P::VALUE8;
        if constexpr (D == 128) {
          const uint2 c = *reinterpret_cast<const uint2*>(codes);
          w[i][0] = c.x, w[i][1] = c.y;
        } else {
          w[i][0] = *reinterpret_cast<const uint32_t*>(codes);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        scale[e] = widen_f16(block[(8 * e + at.slot[0]) * RS] | (uint32_t)block[(8 * e + at.slot[1]) * RS] << 8);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t va[4][4];  // [keys 8..15, column 2 i + 1][i], in the order of a fragment's registers
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t x = w[2 * e][c], y = w[2 * e + 1][c];
          widen_scaled((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), scale[e], va[2 * e]);
          widen_scaled(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), scale[e], va[2 * e + 1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a[4] = {va[0][i], va[1][i], va[2][i], va[3][i]};
#pragma unroll
          for (int r = 0; r < R; ++r) mma_f16_16816(o[4 * c + i][r], a, pb[kp][r][0], pb[kp][r][1]);
        }
      }
    }
  }

  __device__ __forceinline__ static int column(int i, int e, int gq) { return D / 8 * gq + 2 * i + (e >> 1); }
};

// o and lse of one (sequence, group) from its few parts (at most 64: those of the selected blocks),
// by the CTA that wrote the last of them: a warp a head, the weights in its lanes.
template <int D>
__device__ __forceinline__ void join_parts(const PagedDecode& p, const Parts& parts, int64_t head0) {
  constexpr int LANES = D / 4, SIDE = 32 / LANES;  // lanes of a part; parts side by side
  const int lane = threadIdx.x & 31, G = p.G, n = parts.n;
  const int sub = lane / LANES, c = 4 * (lane % LANES);
  for (int h = threadIdx.x >> 5; h < G; h += kWarps) {
    float w[2];  // of parts lane, lane + 32
#pragma unroll
    for (int e = 0; e < 2; ++e)
      w[e] = lane + 32 * e < n ? __ldcg(&p.part_lse[parts.slot(lane + 32 * e) * G + h]) : -INFINITY;
    float top = fmaxf(w[0], w[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    w[0] = weight(w[0], top);
    w[1] = weight(w[1], top);
    float l = w[0] + w[1];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    w[0] /= l;
    w[1] /= l;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i0 = 0; i0 < n; i0 += SIDE) {
      const int i = i0 + sub;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) y = __ldcg(reinterpret_cast<const float4*>(p.part_o + (parts.slot(i) * G + h) * D + c));
      const float f = __shfl_sync(0xffffffffu, i0 < 32 ? w[0] : w[1], i & 31);  // 0 from n on
      acc.x = fmaf(f, y.x, acc.x);
      acc.y = fmaf(f, y.y, acc.y);
      acc.z = fmaf(f, y.z, acc.z);
      acc.w = fmaf(f, y.w, acc.w);
    }
    if (SIDE == 2) {
      acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
      acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
      acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
      acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
    }
    if (sub == 0)
      *reinterpret_cast<uint2*>(p.o + (head0 + h) * D + c) =
          make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    if (lane == 0) p.lse[head0 + h] = (top + log2f(l)) * 0.6931471805599453f;
  }
}

// Place<false> of the states that have one.
template <typename State>
struct NoPlace {
  __device__ __forceinline__ NoPlace(int, int) {}
};
template <typename State, bool F4>
struct PlaceIn {
  using Type = NoPlace<State>;
};
template <typename State>
struct PlaceIn<State, true> {
  using Type = typename State::template Place<false>;
};
template <typename State>
using PlaceOf = typename PlaceIn<State, State::St::F4>::Type;

// A warp's part of a span: units u0 .. u0 + n - 1 (n > 0) of group g of sequence b, in unit x the KEYS
// tokens from x unit + my_token on; or (SPARSE) in unit x of the selected blocks, of which lane i
// holds the i-th in blk.
template <int D, int KIND, bool WIDE, bool SPARSE>
__device__ __forceinline__ void attend(const PagedDecode& p, WarpState<D, KIND, WIDE>& ws, uint8_t* smem, int b, int g,
                                       int len, int u0, int n, int blk, int my_token, int unit, bool side_by_side) {
  using St = Stage<D, KIND, WIDE>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, tq = lane & 3;
  uint8_t* ring = smem + warp * St::COUNT * St::BYTES;
  const int64_t head0 = ((int64_t)b * p.H + g) * p.G;
  constexpr int CH = St::ROW / 16;  // 16-byte chunks of a row
  constexpr int RPI = 32 / CH;      // rows of one copy instruction
  const int r0 = lane / CH, ch = lane % CH;
  const int64_t row_step = (int64_t)p.H * St::ROW;
  const int64_t lane_off = r0 * row_step + ch * 16;
  // Page ids of the next 32 half stages sit in the lanes of a register (and those of the 32 after
  // them are on their way), so that no lookup stands in front of a copy.
  // first token of this warp in unit u0 + i
  auto first_token = [&](int i) {
    const int x = u0 + i;
    if (!SPARSE) return x * unit + my_token;
    return __shfl_sync(0xffffffffu, blk, (x / St::PER) & 31) * 128 + (x % St::PER) * St::UNIT + my_token;
  };
  const int32_t* table = p.pages.table + (int64_t)b * p.pages.table_stride;
  constexpr int AHEAD = 32 / St::HALVES;  // units whose page ids a register holds
  auto page_ids = [&](int i) {  // of the halves of units i .. i + AHEAD - 1, one a lane
    const int x = u0 + i + lane / St::HALVES;
    int tok = (lane % St::HALVES) * 16 + my_token;
    if (!SPARSE) tok += x * unit;
    else tok += __shfl_sync(0xffffffffu, blk, (x / St::PER) & 31) * 128 + (x % St::PER) * St::UNIT;
    return i + lane / St::HALVES < n && tok < len ? __ldg(&table[page_of(p.pages, tok)]) : -1;
  };
  int ids = page_ids(0), ids_next = page_ids(AHEAD);
  // 4 bits.  The scales of a run of 16 tokens are chunks of CHUNK bytes, keys' and then values', numbered
  // as they lie in shared memory, 32 an instruction, so that neighbours come from the same cache lines
  // (a copy whose lanes have a line each takes about 27 cycles).
  constexpr bool F4 = St::F4;
  constexpr int CHUNK = D == 64 ? 8 : 4, PER_ROW = F4 ? St::SCALE / CHUNK : 1;
  uint8_t* scales = smem + St::RINGS + warp * St::COUNT * St::SCALES;
  const uint8_t* scale_src[PER_ROW];
  if constexpr (F4) {
#pragma unroll
    for (int j = 0; j < PER_ROW; ++j) {
      const int x = 32 * j + lane, r = x / PER_ROW;
      scale_src[j] = (r >= 16 ? p.v_scale : p.k_scale) + ((int64_t)(r & 15) * p.H + g) * St::SCALE +
                     (x - r * PER_ROW) * CHUNK;
    }
  }
  const uint8_t* k_src = static_cast<const uint8_t*>(p.k) + (int64_t)g * St::ROW + lane_off;
  const uint8_t* v_src = static_cast<const uint8_t*>(p.v) + (int64_t)g * St::ROW + lane_off;
  auto load4 = [&](int i) {
    const uint32_t st = smem_u32(ring) + (i % St::COUNT) * St::BYTES;
    const uint32_t sc = smem_u32(scales) + (i % St::COUNT) * St::SCALES;
    const int pos0 = first_token(i);
#pragma unroll
    for (int hs = 0; hs < St::HALVES; ++hs) {
      const int pos = pos0 + 16 * hs;
      const int id = __shfl_sync(0xffffffffu, ids, (i % AHEAD) * St::HALVES + hs);
      int have = len - pos;  // tokens of the sequence from here on
      const bool good = (unsigned)id < (unsigned)p.pages.num_pages && have > 0;
      if (!good && have > 0) set_status(p.status, MSA_ERR_ARG);
      // any bits are codes, so those of missing rows may be whatever is there: their scales are zeros
      const int64_t row0 = (int64_t)id * p.pages.page_size + (pos - page_of(p.pages, pos) * p.pages.page_size);
      if (good) {
        const uint8_t *kp = k_src + row0 * row_step, *vp = v_src + row0 * row_step;
#pragma unroll
        for (int j = 0; j < 16 / RPI; ++j) {
          const int r = 16 * hs + j * RPI;
          cp_async_16_to(st + r * St::ROW + lane * 16, kp + j * RPI * row_step);
          cp_async_16_to(st + St::V0 + (r + r0) * St::VROW + ch * 16, vp + j * RPI * row_step);
        }
      } else {
        have = 0;
      }
      const int64_t off = good ? row0 * p.H * St::SCALE : 0;
#pragma unroll
      for (int j = 0; j < PER_ROW; ++j) {
        const int x = 32 * j + lane, r = x / PER_ROW;
        cp_async_to<CHUNK>(sc + 16 * hs * St::SCALE + x * CHUNK + (r >= 16 ? (St::KEYS - 16) * St::SCALE : 0),
                           scale_src[j] + off, (r & 15) < have);
      }
    }
  };
  auto load = [&](int i) {
    if (i < n) {
      if (i > 0 && i % AHEAD == 0) {
        ids = ids_next;
        ids_next = page_ids(i + AHEAD);
      }
      if constexpr (F4) {
        load4(i);
      } else {
        uint8_t* st = ring + (i % St::COUNT) * St::BYTES;
        const int pos0 = first_token(i);
#pragma unroll
        for (int hs = 0; hs < St::HALVES; ++hs) {
          const int pos = pos0 + 16 * hs;
          const int id = __shfl_sync(0xffffffffu, ids, (i % AHEAD) * St::HALVES + hs);
          const int have = len - pos;  // tokens of the sequence from here on
          if (hs == 0 && have <= 0) break;  // step() will not look at this stage
          const bool good = (unsigned)id < (unsigned)p.pages.num_pages;
          if (!good && have > 0) set_status(p.status, MSA_ERR_ARG);
          const int64_t row0 =
              good ? (int64_t)id * p.pages.page_size + (pos - page_of(p.pages, pos) * p.pages.page_size) : 0;
          const int64_t at = (row0 * p.H + g) * St::ROW + lane_off;
          const uint8_t* kp = static_cast<const uint8_t*>(p.k) + at;
          const uint8_t* vp = static_cast<const uint8_t*>(p.v) + at;
          const bool full = good && have >= 16;
#pragma unroll
          for (int j = 0; j < 16 / RPI; ++j) {
            const int r = r0 + j * RPI;
            uint8_t* kd = st + St::key_at(16 * hs + r, ch);
            uint8_t* vd = st + St::value_at(16 * hs + r, ch);
            if (full) {
              cp_async_16(kd, kp + j * RPI * row_step);
              cp_async_16(vd, vp + j * RPI * row_step);
            } else {  // else zeros: no stale NaN meets a weight of 0
              const bool ok = good && r < have;
              const int64_t off = ok ? j * RPI * row_step : -lane_off;
              cp_async_16(kd, kp + off, ok);
              cp_async_16(vd, vp + off, ok);
            }
          }
          if constexpr (St::CODED) {  // lanes 0..15 the keys' scales, the others the values'
            const int r = lane & 15;
            const bool ok = good && r < have;
            const uint8_t* src = (lane < 16 ? p.k_scale : p.v_scale) + (ok ? ((row0 + r) * p.H + g) * 4 : 0);
            cp_async_4(st + St::S0 + ((lane < 16 ? 0 : St::KEYS) + 16 * hs + r) * 4, src, ok);
          }
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < St::COUNT - 1; ++i) load(i);
  ws.load_q(p, head0, gq, tq);
  [[maybe_unused]] const PlaceOf<WarpState<D, KIND, WIDE>> place(lane, 0);
  for (int i = 0; i < n; ++i) {
    cp_async_wait<St::COUNT - 2>();
    // unit i has landed for all lanes, and all are done with unit i - 1; heads side by side
    // stay in step, so that what they load together lies together in memory
    if (side_by_side) __syncthreads(); else __syncwarp();
    load(i + St::COUNT - 1);
    const int have = len - first_token(i);
    if (have <= 0) continue;
    const uint8_t* st = ring + (i % St::COUNT) * St::BYTES;
    if constexpr (F4) ws.step(st, scales + (i % St::COUNT) * St::SCALES, place, have, lane);
    else ws.step(st, have, lane);
  }
  cp_async_wait<0>();
}

// The tensor maps of a 4-bit cache's keys and values, [num_pages page_size][H row / 128][128 bytes]; other
// kernels have none.
template <bool SOME>
struct CodeMaps {};
template <>
struct CodeMaps<true> {
  CUtensorMap k, v;
};

// The stages that a CTA fills by TMA: which comes next, and the parity of its barrier's phase.
struct StageRing {
  uint64_t* full;
  int at;
  uint32_t parity;
  template <int COUNT>
  __device__ __forceinline__ void advance() {
    if (++at == COUNT) {
      at = 0;
      parity ^= 1;
    }
  }
};

// attend() for the four warps of a CTA that serve four groups of a 4-bit cache side by side.  They take turns in
// bringing a unit of all four groups: the codes by TMA, 16 tokens a box, and the scales in 16-byte chunks (four
// groups' records are neighbours in the pool; boxes of 48 bytes take TMA longer than those of the codes).  What
// counts beside the products are the instructions of the copies: 8 x 128K, d 128: each warp copying for itself
// 334 us; codes by TMA and a warp's part of the scales by each 273; in turn 269 (the last warp
// to be done with a stage filling it again, without a barrier: 312).
// False, in all threads alike, where a wait ran out: no copy of the CTA is then on its way that was not given
// its time to land, and none follows.
template <int D, bool WIDE>
__device__ __forceinline__ bool attend_together(const PagedDecode& p, const CodeMaps<true>& maps,
                                                WarpState<D, MSA_CACHE_E2M1, WIDE>& ws, uint8_t* smem, StageRing& ring,
                                                int b, int g, int len, int u0, int n) {
  using St = Stage<D, MSA_CACHE_E2M1, WIDE>;
  constexpr int COUNT = St::TOGETHER_COUNT, RECORD = 4 * St::SCALE, SCALES = 2 * St::HALVES * St::BOX;
  constexpr int PER_ROW = RECORD / 16, COPIES = (16 * PER_ROW + 31) / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t head0 = ((int64_t)b * p.H + g) * p.G;
  const int32_t* table = p.pages.table + (int64_t)b * p.pages.table_stride;
  constexpr int AHEAD = 32 / St::HALVES;  // units whose page ids a register holds, one of 16 tokens a lane
  auto page_ids = [&](int i) {
    const int tok = (u0 + i) * St::KEYS + lane * 16;
    return i + lane / St::HALVES < n && tok < len ? __ldg(&table[page_of(p.pages, tok)]) : -1;
  };
  int ids = page_ids(0), ids_next = page_ids(AHEAD);
  const int scale_step = p.H * St::SCALE;
  int chunk_row[COPIES], chunk_off[COPIES];  // chunks 32 j + lane of 16 records (16: none)
#pragma unroll
  for (int j = 0; j < COPIES; ++j) {
    const int x = 32 * j + lane, r = x / PER_ROW;
    chunk_row[j] = x < 16 * PER_ROW ? r : 16;
    chunk_off[j] = r * scale_step + (g & ~3) * St::SCALE + (x - r * PER_ROW) * 16;
  }
  StageRing fill = ring;
  auto load = [&](int i) {  // unit i < n, by warp i % 4
    if (i % AHEAD == 0 && i > 0) {
      ids = ids_next;
      ids_next = page_ids(i + AHEAD);
    }
    if ((i & 3) == warp && i != p.withheld) {
      uint8_t* st = smem + fill.at * St::TOGETHER;
      uint64_t* full = fill.full + fill.at;
      int row[St::HALVES], have[St::HALVES], boxes = 0;  // first row of each half, and its tokens (0: none, or no page)
#pragma unroll
      for (int hs = 0; hs < St::HALVES; ++hs) {
        const int pos = (u0 + i) * St::KEYS + 16 * hs, id = __shfl_sync(0xffffffffu, ids, (i % AHEAD) * St::HALVES + hs);
        have[hs] = len - pos;
        const bool good = (unsigned)id < (unsigned)p.pages.num_pages;
        if (!good && have[hs] > 0) set_status(p.status, MSA_ERR_ARG);
        if (!good || have[hs] < 0) have[hs] = 0;
        row[hs] = have[hs] > 0 ? id * p.pages.page_size + (pos - page_of(p.pages, pos) * p.pages.page_size) : 0;
        boxes += have[hs] > 0 ? 2 : 0;
      }
      if (lane == 0) {
        // any bits are codes: what a missing half leaves in its boxes meets scales of zero
        mbar_arrive_expect_tx(full, boxes * St::BOX);
        const int col = (g & ~3) * St::ROW / 128;
#pragma unroll
        for (int hs = 0; hs < St::HALVES; ++hs) {
          if (have[hs] == 0) continue;
          tma_load_3d(st + hs * St::BOX, &maps.k, full, 0, col, row[hs]);
          tma_load_3d(st + (St::HALVES + hs) * St::BOX, &maps.v, full, 0, col, row[hs]);
        }
      }
      __syncwarp();
      const uint32_t to = smem_u32(st) + SCALES + lane * 16;
#pragma unroll
      for (int hs = 0; hs < St::HALVES; ++hs) {
        const int64_t off = (int64_t)row[hs] * scale_step;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint8_t* from = (v ? p.v_scale : p.k_scale) + off;
#pragma unroll
          for (int j = 0; j < COPIES; ++j)
            if (chunk_row[j] < 16)
              cp_async_to<16>(to + (v * St::KEYS + 16 * hs) * RECORD + 512 * j, from + chunk_off[j], chunk_row[j] < have[hs]);
        }
      }
      cp_async_mbar_arrive(full);
    }
    fill.advance<COUNT>();
  };
  // what the warps left of the span before (and read of it) comes before TMA's writes
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  for (int i = 0; i < min(n, COUNT - 1); ++i) load(i);
  ws.load_q(p, head0, lane >> 2, lane & 3);
  const typename WarpState<D, MSA_CACHE_E2M1, WIDE>::template Place<true> place(lane, g & 3);
  for (int i = 0; i < n; ++i) {
    const bool late = !mbar_wait(ring.full + ring.at, ring.parity, p.wait_ns);
    if (__syncthreads_or(late)) {  // all warps are done with unit i - 1
      set_status(p.status, MSA_ERR_DEVICE_TIMEOUT);
      for (int k = i; k < min(n, i + COUNT - 1); ++k) {  // the units on their way, each in its own phase
        mbar_wait(ring.full + ring.at, ring.parity, p.wait_ns);
        ring.advance<COUNT>();
      }
      return false;
    }
    if (i + COUNT - 1 < n) load(i + COUNT - 1);
    const uint8_t* st = smem + ring.at * St::TOGETHER;
    ws.step(st, st + SCALES + (g & 3) * St::SCALE, place, len - (u0 + i) * St::KEYS, lane);
    ring.advance<COUNT>();
  }
  __syncthreads();  // the sums go where other warps' codes lie
  return true;
}

// What the warps of a CTA leave of a span: running sums in their own stages ([8 R][D + 4] floats),
// the rest here.
struct WarpSums {
  float m[kWarps][16], mv[kWarps][16], l[kWarps][16];
};
template <int D, int KIND, bool WIDE>
__device__ __forceinline__ void leave_sums(const WarpState<D, KIND, WIDE>& ws, uint8_t* smem, WarpSums& s) {
  using St = Stage<D, KIND, WIDE>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, tq = lane & 3;
  __syncwarp();  // the warp is done with its stages
  float* my_o = reinterpret_cast<float*>(smem + warp * St::COUNT * St::BYTES);
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int r = 0; r < ws.R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        my_o[(8 * r + 2 * tq + (e & 1)) * (D + 4) + ws.column(i, e, gq)] = ws.o[i][r][e];
  if constexpr (KIND == MSA_CACHE_E2M1) {
#pragma unroll
    for (int r = 0; r < ws.R; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = ws.l[r][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        if (ws.few) l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int h = 8 * r + 2 * tq + e;  // (few: heads 4 and more are no one's)
        if (gq == 0) {
          s.m[warp][h] = ws.m[r][e];
          s.mv[warp][h] = ws.mv[r][e] - kWeightBits;
          s.l[warp][h] = l;
        }
      }
    return;
  } else {
#pragma unroll
    for (int r = 0; r < ws.R; ++r) {
      float l = ws.l[r];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (tq == 0) {
        s.m[warp][gq + 8 * r] = ws.m[r];
        if (ws.CODED) s.mv[warp][gq + 8 * r] = ws.mv[r] - kWeightBits;
        s.l[warp][gq + 8 * r] = l;
      }
    }
  }
}

// Columns c .. c + 3 of head h, joined over the warps w0, w0 + wh, ... (subs of them), not yet
// divided by l; the maximum (in bits) and l.
template <int D, int KIND, bool WIDE>
__device__ __forceinline__ float4 join_warps(const uint8_t* smem, const WarpSums& s, int h, int c, int w0, int wh,
                                             int subs, float* top_out, float* l_out) {
  using St = Stage<D, KIND, WIDE>;
  float top = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kWarps; ++k)
    if (k < subs) top = fmaxf(top, s.m[w0 + k * wh][h]);
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    if (k >= subs) break;
    const int w = w0 + k * wh;
    l += s.l[w][h] * weight(s.m[w][h], top);
    float4 y = *reinterpret_cast<const float4*>(smem + w * St::COUNT * St::BYTES + (h * (D + 4) + c) * 4);
    float f;
    if constexpr (St::CODED) {  // as its root twice: it underflows where value scales are subnormal
      const float m = s.m[w][h];
      f = m == -INFINITY ? 0.f : ex2_fast(0.5f * (s.mv[w][h] + (m - top)));
      y = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
    } else {
      f = weight(s.m[w][h], top);
    }
    acc.x = fmaf(f, y.x, acc.x);
    acc.y = fmaf(f, y.y, acc.y);
    acc.z = fmaf(f, y.z, acc.z);
    acc.w = fmaf(f, y.w, acc.w);
  }
  *top_out = top;
  *l_out = l;
  return acc;
}

// An empty slot: o = 0, lse = -inf and no blocks for `heads` query heads from head0 on.
template <int D>
__device__ __forceinline__ void write_empty(const PagedDecode& p, int64_t head0, int64_t heads) {
  for (int64_t x = threadIdx.x; x < heads * D; x += kThreads) p.o[head0 * D + x] = __float2bfloat16(0.f);
  for (int64_t x = threadIdx.x; x < heads; x += kThreads) p.lse[head0 + x] = -INFINITY;
}

// One CTA works through its run of units: span after span of one (sequence, wh groups).  Its
// warps take the groups side by side and share each one's tokens, every warp with its own
// stages in shared memory and its own running softmax; they join when a span ends.  A whole
// (sequence, groups) is written out, a part of one goes to the CTA's slot 0 (its first span) or 1.
// Bound by HBM: 8 whole caches of 128K tokens take 594 us in bf16 (4.3 GB, 7.2 TB/s) and 333 us in
// E4M3 (2.2 GB, 6.6 TB/s), 16 blocks of each 19 us after the scores.  Bound by issue: E4M3 with d = 64
// (229 us, 5.0 TB/s) or 16 heads a group (392 us, 5.6 TB/s).  4 bits (262 us, 1.3 GB, 4.9 TB/s; d = 64 184 us)
// fill neither HBM nor a pipe (59 percent of the issue slots, ALU 53): 16 warps a SM wait for the
// latency of their own chains and for one another at a unit's barrier.  With 16 heads a group 8 warps a SM are left,
// and E4M3 is faster (417 us for 392).
template <int D, int KIND, bool WIDE, bool SPARSE>
__global__ void __launch_bounds__(kThreads, (SPARSE ? Stage<D, KIND, WIDE>::PER_SM : Stage<D, KIND, WIDE>::DENSE_PER_SM))
    paged_attn_kernel(const PagedDecode p, const __grid_constant__ CodeMaps<(KIND == MSA_CACHE_E2M1 && !SPARSE)> maps) {
  using St = Stage<D, KIND, WIDE>;
  constexpr bool TOGETHER = St::F4 && !SPARSE;
  extern __shared__ __align__(128) uint8_t smem_start[];
  // TMA's swizzle goes by the address
  uint8_t* smem = TOGETHER ? smem_start + (-smem_u32(smem_start) & 1023) : smem_start;
  __shared__ uint64_t s_full[TOGETHER ? St::TOGETHER_COUNT : 1];
  StageRing stages{s_full, 0, 0};
  if (TOGETHER && p.together) {
    if (threadIdx.x == 0) {
#pragma unroll
      for (int i = 0; i < St::TOGETHER_COUNT; ++i) mbar_init(&s_full[i], 1 + 32);  // TMA's thread, and a warp's copies
      fence_mbar_init();
    }
    __syncthreads();
  }
  __shared__ WarpSums s_sums;
  __shared__ int32_t s_blocks[kMaxSelect];
  __shared__ int s_last;
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Work work = find_run<SPARSE>(p);
  const int wh = SPARSE ? 1 : work.wh, HG = SPARSE ? p.H : work.HG;
  int b = work.b, base = work.base;
  griddep_wait();  // the pooled scores or the selected blocks
  for (int e = blockIdx.x; e < p.B; e += p.ctas) {  // empty slots: o = 0, lse = -inf, no blocks
    if (seq_len(p, e) > 0) continue;
    write_empty<D>(p, (int64_t)e * p.H * p.G, (int64_t)p.H * p.G);
    if (SPARSE && p.select)
      for (int64_t x = tid; x < (int64_t)p.H * p.topk; x += kThreads) p.block_idx[(int64_t)e * p.H * p.topk + x] = -1;
  }
  int u = work.cut.start(blockIdx.x);
  const int u_end = work.cut.start(blockIdx.x + 1);
  // warp w works for head hg wh + w % wh, on the (w / wh)-th run of KEYS tokens of each unit
  const int my_head = warp & (wh - 1), subs = kWarps / wh;
  const int my_token = (wh == 1 ? warp : wh == 2 ? warp >> 1 : 0) * St::KEYS, unit = St::KEYS * subs;
  int slot = 0;  // of the CTA's next part
  while (u < u_end) {
    int len = seq_len(p, b), units = seq_units<SPARSE>(p, len, wh), size = seq_work(units);
    while (base + size * HG <= u) {  // next sequence that has any
      base += size * HG;
      ++b;
      len = seq_len(p, b);
      units = seq_units<SPARSE>(p, len, wh);
      size = seq_work(units);
    }
    const int hg = (u - base) / size, first = base + hg * size;
    const int stop = min(first + size, u_end);
    const int u0 = max(0, u - first - kOverhead);                  // first unit of this span
    const int n = max(0, stop - first - kOverhead) - u0;           // its units
    u = stop;
    if (n == 0) continue;  // only the pair's overhead fell into this run
    const int g = hg * wh + my_head;
    int blk = 0;  // lane i: the i-th selected block
    if constexpr (SPARSE) {
      int32_t* blocks = p.block_idx + ((int64_t)b * p.H + g) * p.topk;
      if (p.select) {
        select_blocks_by_rank<kSelectPer, kThreads>(p.pooled + ((int64_t)b * p.H + g) * p.row, (len - 1) / 128,
                                                    p.topk, s_blocks);
        __syncthreads();
        if (lane < p.topk) blk = s_blocks[lane];
        if (u0 == 0 && tid < p.topk) blocks[tid] = blk;
      } else if (lane < p.topk) {
        blk = __ldg(&blocks[lane]);
      }
    }
    {
      WarpState<D, KIND, WIDE> ws;
      bool done = false;
      if constexpr (TOGETHER) {
        if (wh == 4 && p.together) {
          if (!attend_together<D, WIDE>(p, maps, ws, smem, stages, b, g, len, u0, n)) return;
          done = true;
        }
      }
      if (!done) attend<D, KIND, WIDE, SPARSE>(p, ws, smem, b, g, len, u0, n, blk, my_token, unit, wh > 1);
      leave_sums(ws, smem, s_sums);
    }
    __syncthreads();
    const bool whole = n == units;
    const int64_t part = (int64_t)(2 * blockIdx.x + slot) * wh * p.G;
    const int64_t out0 = ((int64_t)b * p.H + hg * wh) * p.G;  // first of the wh G query heads
    for (int x = tid; x < wh * p.G * (D / 4); x += kThreads) {
      const int row = x / (D / 4), c = 4 * (x % (D / 4));
      const int w0 = wh == 1 ? 0 : row / p.G, h = row - w0 * p.G;
      float top, l;
      float4 acc = join_warps<D, KIND, WIDE>(smem, s_sums, h, c, w0, wh, subs, &top, &l);
      const float inv = whole || l > 0.f ? 1.f / l : 0.f;  // a part of scores that are all -inf
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (whole) {
        *reinterpret_cast<uint2*>(p.o + (out0 + row) * D + c) =
            make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
        if (c == 0) p.lse[out0 + row] = (top + log2f(l)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4*>(p.part_o + (part + row) * D + c) = acc;
        if (c == 0) p.part_lse[part + row] = top + log2f(l);
      }
    }
    slot = 1;
    if (SPARSE && !whole) {
      // the pair's last part to be written joins them all (in their own order)
      const Parts parts(work.cut, first, units);
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(&p.arrive[(int64_t)b * p.H + g], 1) == parts.n - 1;
      __syncthreads();
      if (s_last) {
        __threadfence();
        join_parts<D>(p, parts, out0);
      }
    }
    __syncthreads();  // the stages are free for the next span
  }
}

// ---------------------------------------------------------------------------
// Short caches: one cluster of CTAs per (sequence, group) does the whole call.  The CTAs share the
// units (and the scoring of the blocks) and join through distributed shared memory.  Such a call is
// bound by latency: this is one launch instead of two or three, without a workspace, and no CTA
// has to find its place among the sequences (1 x 700 tokens, 2 groups: 8.0 -> 5.7 us of GPU time,
// 24 -> 16.6 us a call; 2048 tokens, 2 groups, topk 4: 10.5 -> 8.4 and 27 -> 20 us).
// small_cluster() has the limits.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address in CTA `rank` of the cluster that corresponds to this CTA's shared-memory address.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float cluster_ld(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

constexpr int kSmallBlocks = 32;  // blocks of a table that the small form selects from

// Largest score q_idx[b, g] . k_idx[j] over the 128 keys j of block c, in every lane: mma.sync
// fragments of the keys from global memory (as decode_pool_kernel loads them), the query in the
// first of the 8 columns.
template <int DI>
__device__ __forceinline__ float block_score(const PagedDecode& p, int b, int g, int c) {
  constexpr int NP = DI / 32;
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  const int64_t row = lane < 8 ? pool_row(p.pages, b, c * 128 + lane * 16) : 0;
  if (row < 0) set_status(p.status, MSA_ERR_ARG);
  const uint4* qrow = reinterpret_cast<const uint4*>(p.q_idx + ((int64_t)b * p.H + g) * DI);
  uint4 bq[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) bq[j] = gq == 0 ? __ldg(&qrow[j * 4 + tq]) : make_uint4(0, 0, 0, 0);
  float top = -INFINITY;
#pragma unroll 2
  for (int t = 0; t < 8; ++t) {
    const int64_t r = __shfl_sync(0xffffffffu, row, t);
    const uint4* kb = reinterpret_cast<const uint4*>(p.k_idx + (r < 0 ? 0 : r) * DI);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;  // a missing page reads as zero rows
      if (r >= 0) {
        lo = __ldg(&kb[gq * (DI / 8) + j * 4 + tq]);
        hi = __ldg(&kb[(gq + 8) * (DI / 8) + j * 4 + tq]);
      }
      const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
      mma_bf16_16816(acc, a0, bq[j].x, bq[j].y);
      mma_bf16_16816(acc, a1, bq[j].z, bq[j].w);
    }
    top = fmax3(top, acc[0], acc[2]);  // column 0 in the lanes of tq = 0
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  return __shfl_sync(0xffffffffu, top, 0);
}

// The M = min(topk - 1, own) best of blocks 0 .. own - 1 (lane i holds the score of block i; equal
// ones: the lower block) and block `own`: lane i gets the i-th of them, ascending, or -1.
__device__ __forceinline__ int select_in_warp(float score, int own, int topk) {
  const int lane = threadIdx.x & 31, M = min(topk - 1, own);
  const uint32_t u = __float_as_uint(score);
  const uint32_t key = lane < own ? max((u & 0x80000000u) ? ~u : (u | 0x80000000u), 1u) : 0u;
  int above = 0;
#pragma unroll 8
  for (int j = 0; j < 32; ++j) {
    const uint32_t x = __shfl_sync(0xffffffffu, key, j);
    above += x > key || (x == key && j < lane);
  }
  const unsigned taken = __ballot_sync(0xffffffffu, lane < own && above < M) | (1u << own);
  int id = -1;
#pragma unroll 8
  for (int j = 0; j < 32; ++j)
    if ((taken >> j & 1) && __popc(taken & ((1u << j) - 1)) == lane) id = j;
  return id;
}

template <int D, int KIND, bool WIDE, int DI>  // DI = 0: the whole cache
__global__ void __launch_bounds__(kThreads, Stage<D, KIND, WIDE>::PER_SM) paged_small_kernel(const PagedDecode p) {
  using St = Stage<D, KIND, WIDE>;
  constexpr bool SPARSE = DI > 0;
  constexpr int ITEMS = (WIDE ? 16 : 8) * (D / 4) / kThreads;  // of 4 columns, a thread's at most
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ WarpSums s_sums;
  __shared__ float s_lse[16], s_score[kSmallBlocks];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int size = p.cluster, pair = blockIdx.x / size, rank = blockIdx.x - pair * size;
  const int b = pair / p.H, g = pair - b * p.H;
  const int64_t head0 = (int64_t)pair * p.G;
  const int len = seq_len(p, b);
  if (len == 0) {  // the whole cluster's
    if (rank == 0) {
      write_empty<D>(p, head0, p.G);
      if (SPARSE && tid < p.topk) p.block_idx[(int64_t)pair * p.topk + tid] = -1;
    }
    // stay as long as the others would if the length were written meanwhile
    for (int i = 0; i < (SPARSE ? 3 : 2); ++i) cluster_sync();
    return;
  }
  int blk = 0;
  if constexpr (SPARSE) {
    const int own = (len - 1) / 128, warps = size * kWarps;
    for (int c = rank * kWarps + warp; c < own; c += warps) {
      const float top = block_score<DI>(p, b, g, c);
      if (lane == 0) s_score[c] = top;
    }
    cluster_sync();
    float score = 0.f;
    if (lane < own) score = cluster_ld(cluster_addr(&s_score[lane], lane % warps / kWarps));
    blk = select_in_warp(score, own, p.topk);
    if (rank == 0 && tid < p.topk) p.block_idx[(int64_t)pair * p.topk + tid] = blk;
  }
  const int units = seq_units<SPARSE>(p, len, 1);
  const int u0 = units * rank / size, n = units * (rank + 1) / size - u0;
  float4 acc[ITEMS];
  if (n > 0) {
    {
      WarpState<D, KIND, WIDE> ws;
      attend<D, KIND, WIDE, SPARSE>(p, ws, smem, b, g, len, u0, n, blk, warp * St::KEYS, St::UNIT, false);
      leave_sums(ws, smem, s_sums);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int x = tid + k * kThreads, h = x / (D / 4), c = 4 * (x % (D / 4));
      if (h >= p.G) break;
      float top, l;
      acc[k] = join_warps<D, KIND, WIDE>(smem, s_sums, h, c, 0, 1, kWarps, &top, &l);
      const float inv = l > 0.f || size == 1 ? 1.f / l : 0.f;  // a part of scores that are all -inf
      acc[k] = make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv);
      if (c == 0) s_lse[h] = top + log2f(l);
    }
    __syncthreads();  // the warps' sums have been read
    float* part = reinterpret_cast<float*>(smem);  // [G][D]
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int x = tid + k * kThreads;
      if (x < p.G * (D / 4)) *reinterpret_cast<float4*>(part + 4 * x) = acc[k];
    }
  } else if (tid < 16) {
    s_lse[tid] = -INFINITY;
  }
  cluster_sync();
  // this CTA's share of the columns, over the cluster's parts in order
  for (int x = rank * kThreads + tid; x < p.G * (D / 4); x += size * kThreads) {
    const int h = x / (D / 4), c = 4 * (x % (D / 4));
    float top = -INFINITY, l = 0.f;
    for (int r = 0; r < size; ++r) top = fmaxf(top, cluster_ld(cluster_addr(&s_lse[h], r)));
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < size; ++r) {
      const float w = weight(cluster_ld(cluster_addr(&s_lse[h], r)), top);
      if (w == 0.f) continue;  // a CTA without units left no sums
      const float4 y = cluster_ld4(cluster_addr(smem + x * 16, r));
      l += w;
      sum.x = fmaf(w, y.x, sum.x);
      sum.y = fmaf(w, y.y, sum.y);
      sum.z = fmaf(w, y.z, sum.z);
      sum.w = fmaf(w, y.w, sum.w);
    }
    *reinterpret_cast<uint2*>(p.o + (head0 + h) * D + c) =
        make_uint2(pack_bf16(sum.x / l, sum.y / l), pack_bf16(sum.z / l, sum.w / l));
    if (c == 0) p.lse[head0 + h] = (top + log2f(l)) * 0.6931471805599453f;
  }
  cluster_sync();  // no CTA leaves while its sums are read
}

// Joins the parts of every (sequence, group) that the split cut, where the whole cache is
// attended: one sequence may then have hundreds of them.  Grid (B H, head splits, D / COLS): a CTA
// takes heads blockIdx.y, + gridDim.y, ... and COLS value columns; its threads take parts side by
// side, each 4 columns.  Bound by latency: about 3 us behind the attention (one CTA over 16 heads of
// one long sequence: 344 us).
constexpr int kJoinThreads = 256;
template <int D, int COLS>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedDecode p) {
  constexpr int LANES = COLS / 4;                 // threads of a part
  constexpr int PARTS = kJoinThreads / LANES;     // parts at once
  __shared__ float s_w[kMaxCtas + 1], s_red[8], s_sum[8];
  __shared__ float4 s_acc[8][LANES];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.H, g = blockIdx.x - b * p.H;
  const int64_t head0 = ((int64_t)b * p.H + g) * p.G;
  const int col0 = blockIdx.z * COLS;
  griddep_wait();
  const int start = __ldcg(&p.starts[b]), end = __ldcg(&p.starts[b + 1]);
  const int total = __ldcg(&p.starts[p.B]), wh = __ldcg(&p.starts[p.B + 1]);
  if (start == end) return;  // an empty slot
  const int hg = wh == 4 ? g >> 2 : wh == 2 ? g >> 1 : g, HG = wh == 4 ? p.H >> 2 : wh == 2 ? p.H >> 1 : p.H;
  const int size = (end - start) / HG;
  const Parts parts(Cut(total, p.B * HG, p.ctas), start + hg * size, size - kOverhead);
  const int n = parts.n;
  if (n == 1) return;
  auto part_of = [&](int i) { return (parts.slot(i) * wh + (g - hg * wh)) * p.G; };
  for (int h = blockIdx.y; h < p.G; h += gridDim.y) {
    float top = -INFINITY;
    for (int i = tid; i < n; i += kJoinThreads) {
      const float x = __ldcg(&p.part_lse[part_of(i) + h]);
      s_w[i] = x;
      top = fmaxf(top, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s_red[warp] = top;
    __syncthreads();
    top = s_red[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) top = fmaxf(top, s_red[w]);
    float sum = 0.f;
    for (int i = tid; i < n; i += kJoinThreads) {
      const float x = weight(s_w[i], top);
      s_w[i] = x;
      sum += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) l += s_sum[w];
    const int col = col0 / 4 + tid % LANES;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = tid / LANES; i < n; i += PARTS) {
      const float4 y = __ldcg(reinterpret_cast<const float4*>(p.part_o + (part_of(i) + h) * D) + col);
      const float w = s_w[i];
      acc.x = fmaf(w, y.x, acc.x);
      acc.y = fmaf(w, y.y, acc.y);
      acc.z = fmaf(w, y.z, acc.z);
      acc.w = fmaf(w, y.w, acc.w);
    }
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {  // parts of the same columns within the warp
      acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
      acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
      acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
      acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
    }
    if (lane < LANES) s_acc[warp][lane] = acc;
    __syncthreads();
    if (tid < LANES) {
#pragma unroll
      for (int w = 1; w < 8; ++w) {
        const float4 y = s_acc[w][tid];
        acc.x += y.x;
        acc.y += y.y;
        acc.z += y.z;
        acc.w += y.w;
      }
      *reinterpret_cast<uint2*>(p.o + (head0 + h) * D + col0 + 4 * tid) =
          make_uint2(pack_bf16(acc.x / l, acc.y / l), pack_bf16(acc.z / l, acc.w / l));
      if (tid == 0 && col0 == 0) p.lse[head0 + h] = (top + log2f(l)) * 0.6931471805599453f;
    }
    __syncthreads();
  }
}

// Launches with programmatic stream serialization: the kernel may be scheduled while its
// predecessor drains, and waits for it (griddep_wait) before it touches what that wrote.
template <typename Kern, typename... More>
cudaError_t launch(Kern kern, dim3 grid, int threads, size_t smem, bool after, cudaStream_t stream,
                   const PagedDecode& p, const More&... more) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, p, more...);
}

// The dynamic shared memory of a kernel belongs to the function in a context: set again where that
// changes.  `done` is the kernel's own.
template <typename Kern>
cudaError_t allow_smem(Kern kern, int bytes, std::atomic<void*>& done) {
  void* ctx = current_context();
  if (ctx && done.load(std::memory_order_relaxed) == ctx) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.store(ctx, std::memory_order_relaxed);
  return e;
}

template <int D, int KIND, bool WIDE, bool SPARSE>
cudaError_t launch_attn(const PagedDecode& p, cudaStream_t stream) {
  using St = Stage<D, KIND, WIDE>;
  constexpr bool TOGETHER = St::F4 && !SPARSE;
  constexpr int smem = !TOGETHER ? St::SMEM : St::SMEM_TOGETHER > St::SMEM + 1024 ? St::SMEM_TOGETHER : St::SMEM + 1024;
  static_assert(Stage<D, KIND, WIDE>::COUNT * Stage<D, KIND, WIDE>::BYTES >= (WIDE ? 16 : 8) * (D + 4) * 4, "sums in the stages");
  static_assert(Stage<D, KIND, WIDE>::PER_SM == (WIDE && D == 128 ? 2 : 3), "ctas");
  static_assert(kMaxSelect * 128 / Stage<D, KIND, WIDE>::UNIT <= 64, "parts of selected blocks");
  auto* kern = paged_attn_kernel<D, KIND, WIDE, SPARSE>;
  static std::atomic<void*> done{nullptr};
  const cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  CodeMaps<TOGETHER> maps = {};
  if constexpr (TOGETHER) {
    if (p.together) {
      const uint64_t dims[3] = {128, (uint64_t)p.H * St::ROW / 128, (uint64_t)p.pages.num_pages * p.pages.page_size};
      const uint64_t strides[2] = {128, (uint64_t)p.H * St::ROW};
      const uint32_t box[3] = {128, 4 * St::ROW / 128, 16};
      if (!encode_tiled(&maps.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.k, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
          !encode_tiled(&maps.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.v, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    }
  }
  return launch(kern, dim3(p.ctas), kThreads, smem, SPARSE, stream, p, maps);
}

template <int D, int KIND>
cudaError_t launch_paged(const PagedDecode& p, bool wide, cudaStream_t stream) {
  const bool sparse = p.block_idx != nullptr;
  cudaError_t e;
  if (wide) e = sparse ? launch_attn<D, KIND, true, true>(p, stream) : launch_attn<D, KIND, true, false>(p, stream);
  else e = sparse ? launch_attn<D, KIND, false, true>(p, stream) : launch_attn<D, KIND, false, false>(p, stream);
  if (e != cudaSuccess) return e;
  if (sparse) return cudaSuccess;  // joined by the attention kernel
  // The join is a chain of loads, shorter the more CTAs share it, while all of them run together
  // (32 sequences, 4 groups of 4 heads, up to 22 parts: 22 us for the whole call with a CTA a
  // head, 30 us with four a head, 25 us with one a group; 8 x 64K, 16 heads a group: 321 us with
  // 9 a group, 344 us with one).
  const int64_t rows = (int64_t)p.B * p.H, together = 4 * 152;
  if (rows * p.G * (D / 32) <= together)
    return launch(paged_join_kernel<D, 32>, dim3((unsigned)rows, (unsigned)p.G, D / 32), kJoinThreads, 0, true,
                  stream, p);
  const int64_t split = together / rows < 1 ? 1 : together / rows < p.G ? together / rows : p.G;
  return launch(paged_join_kernel<D, D>, dim3((unsigned)rows, (unsigned)split), kJoinThreads, 0, true, stream, p);
}

template <int D, int KIND, bool WIDE, int DI>
cudaError_t launch_small(const PagedDecode& p, cudaStream_t stream) {
  constexpr int smem = Stage<D, KIND, WIDE>::SMEM;
  static_assert(smem >= 16 * D * 4, "a part");
  auto* kern = paged_small_kernel<D, KIND, WIDE, DI>;
  static std::atomic<void*> done{nullptr};
  const cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.H * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// The kernels of a kind of cache: the small form where p.cluster asks for it.
template <int D, int KIND>
cudaError_t launch_kind(const PagedDecode& p, int d_idx, cudaStream_t stream) {
  const bool wide = p.G > 8;
  if (!p.cluster) return launch_paged<D, KIND>(p, wide, stream);
  if (!p.block_idx) return wide ? launch_small<D, KIND, true, 0>(p, stream) : launch_small<D, KIND, false, 0>(p, stream);
  if (d_idx == 64) return wide ? launch_small<D, KIND, true, 64>(p, stream) : launch_small<D, KIND, false, 64>(p, stream);
  return wide ? launch_small<D, KIND, true, 32>(p, stream) : launch_small<D, KIND, false, 32>(p, stream);
}

}  // namespace

// decode_paged_e2m1.cu
cudaError_t launch_decode_e2m1(const PagedDecode& p, int d, int d_idx, cudaStream_t stream);

}  // namespace msa
