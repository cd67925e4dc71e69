// decode_paged.cu -- attention of one new token a sequence over a paged cache (see
// include/msa.h): over the whole cache (msa_decode_paged_dense), or over the blocks that the
// index branch selects (msa_decode_paged).
//
// For head h of group g, over the tokens T of the sequence (or of its selected blocks):
//   s_j = scale q_h . k_j,  o = sum_j e^(s_j - m) v_j / l,  l = sum_j e^(s_j - m),
//   lse = m + ln l,  m = max_j s_j,
// in one pass with a running m, l and o, and joined over the parts of a split by
//   lse = ln sum_i e^lse_i,  o = sum_i e^(lse_i - lse) o_i.
//
// The cache is read once and each byte meets 2 G multiply-adds, so HBM sets the pace and the
// products run on mma.sync with the group's heads as the 16 rows.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <atomic>

#include "decode_select.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace msa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// CTAs over which a call's units are spread: three on each of the 152 SMs.  Each leaves at
// most two partial results (its first and its last (sequence, group)), whatever the batch.
constexpr int kCtas = 152 * 3;
// Blocks a sequence up to which the attention kernel selects for itself, 8 scores a thread: every
// CTA of a (sequence, group) then repeats the counting, which is less than the launch it saves.
constexpr int kSelectPer = 8;

struct PagedDecode {
  PageView pages;
  const __nv_bfloat16* q;      // [B][H G][d]
  const __nv_bfloat16* q_idx;  // [B][H][d_idx]
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  const __nv_bfloat16* k_idx;
  const int32_t* lens;  // [B]
  int32_t* block_idx;   // [B][H][topk]; null: the whole cache
  float* pooled;        // [B][H][row]
  float* part_o;        // [2 kCtas][wh][G][d]
  float* part_lse;      // [2 kCtas][wh][G], in bits (log2)
  int* starts;          // [B + 2] first unit of each sequence, their total, wh: for the join
  int* arrive;          // [B][H] parts that are written (selected blocks; zeroed by the pooling)
  __nv_bfloat16* o;
  float* lse;
  int B, H, G, topk;
  int row;         // blocks of the table's length, rounded up to 4
  int cluster;     // CTAs of a (sequence, group) in the small form; 0: the other one
  int ctas;        // of the attention kernel
  int select;      // it selects the blocks itself
  int wh;          // heads (groups) that a CTA may serve side by side
  int keys_shift;  // log2 of a stage's keys
  float scale_log2;  // scale * log2 e: scores in bits
  int* status;
};

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
  // r cta / n by a float product: (x + 1/2) / n is 0.5 / n from an integer, and x < 2^18 moves
  // by at most 2^-5 / n in the roundings
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
  const bool sided = !SPARSE && p.wh > 1 && total1 >= kSideBySide * p.ctas;
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
//   by 16 bytes: the fragment loads then fall in distinct banks.
template <int D, bool F8, bool WIDE>
struct Stage {
  static constexpr int KEYS = F8 || D == 64 ? 32 : 16;
  static constexpr int ROW = F8 ? D : 2 * D;
  static constexpr int VROW = F8 ? D + 16 : 2 * D;
  static constexpr int V0 = KEYS * ROW;
  static constexpr int S0 = V0 + KEYS * VROW;  // [2][KEYS] scales
  static constexpr int BYTES = S0 + (F8 ? 2 * KEYS * 4 : 0);
  // CTAs of a SM.  More than 8 heads with d = 128 take more than the 168 registers a thread that
  // three CTAs leave: two with a third stage serve them better (8 x 128K, 16 heads a group, E4M3:
  // 423 -> 392 us), but not with d = 64 (E4M3 269 -> 321 us).
  static constexpr int PER_SM = WIDE && D == 128 ? 2 : 3;
  static constexpr int COUNT = PER_SM == 2 ? 3 : 2;
  static constexpr int UNIT = KEYS * kWarps;  // tokens of a unit of work
  static constexpr int PER = 128 / UNIT;      // units of a block
  static constexpr int HALVES = KEYS / 16;    // runs of 16 tokens, which never straddle a page
  __device__ __forceinline__ static uint32_t key_at(int r, int ch) {
    if constexpr (!F8) return swz<ROW>(r, ch);
    else return r * ROW + ((D == 128 ? ch ^ ((r & 1) << 2) : ch) << 4);
  }
  __device__ __forceinline__ static uint32_t value_at(int r, int ch) {
    if constexpr (!F8) return V0 + swz<ROW>(r, ch);
    else return V0 + r * VROW + (ch << 4);
  }
};

__device__ __forceinline__ float lg2_fast(float x) {  // relative to 1: about 2^-22; of subnormal x too
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kWeightBits = 15.f;  // E4M3: the largest weight of a code is 2^15

// One warp's running softmax over its keys.
//   S = Q K^T: rows are heads gq and gq + 8 (WIDE; else idle); columns are keys 8 t + 2 tq + e.
//   O^T = V^T P^T: rows are value columns, columns the heads 8 nt + 2 tq + e, so that the
//   accumulator of at most 8 heads has no idle rows; the fragments of S are those of P^T.
// (gq = lane / 4, tq = lane % 4.)
template <int D, bool F8, bool WIDE>
struct WarpState {
  using St = Stage<D, F8, WIDE>;
  static constexpr int R = WIDE ? 2 : 1;     // heads of a lane's rows of S
  static constexpr int MT = D / 16;          // tiles of 16 value columns
  static constexpr int KT = St::KEYS / 8;    // tiles of 8 keys
  static constexpr int QS = D / 16;
  uint32_t qa[QS][4];       // query fragments
  float o[MT][R][4];
  float m[R], mv[R], l[R];  // max, max with the value scale relative to it (E4M3), lane's part of the sum
  float fac[R];             // accumulator -> score in bits
  bool far;                 // E4M3: the queries are bf16, not fp16

  __device__ __forceinline__ void load_q(const PagedDecode& p, int64_t head0, int gq, int tq) {
    bool lost = false, huge[R] = {};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int h = gq + 8 * r;
      const bool ok = h < p.G;
      const __nv_bfloat16* row = p.q + (head0 + (ok ? h : 0)) * D;
      if constexpr (!F8) {
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
    far = F8 && __any_sync(0xffffffffu, lost);
    if constexpr (F8) {
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
    if constexpr (!F8) {
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
    float2 lv[F8 ? KT : 1];  // log2 of the value scales
    if constexpr (F8) {
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
        if constexpr (!F8) {
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
      if constexpr (F8) {
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
    // sc now holds P (E4M3: times the value scales)
    bool same = alpha[0] == 1.f;
    if constexpr (WIDE) same = same && alpha[R - 1] == 1.f;
    if (!__all_sync(0xffffffffu, same)) rescale(alpha, tq);
#pragma unroll
    for (int kp = 0; kp < KT / 2; ++kp) {  // 16 keys: one k step
      if constexpr (!F8) {
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
    return F8 ? (i >> 2) * 64 + 8 * gq + 2 * (i & 3) + (e >> 1) : 16 * i + gq + 8 * (e >> 1);
  }
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

// A warp's part of a span: units u0 .. u0 + n - 1 (n > 0) of group g of sequence b, in unit x the KEYS
// tokens from x unit + my_token on; or (SPARSE) in unit x of the selected blocks, of which lane i
// holds the i-th in blk.
template <int D, bool F8, bool WIDE, bool SPARSE>
__device__ __forceinline__ void attend(const PagedDecode& p, WarpState<D, F8, WIDE>& ws, uint8_t* ring, int b, int g,
                                       int len, int u0, int n, int blk, int my_token, int unit, bool side_by_side) {
  using St = Stage<D, F8, WIDE>;
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
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
  auto load = [&](int i) {
    if (i < n) {
      if (i > 0 && i % AHEAD == 0) {
        ids = ids_next;
        ids_next = page_ids(i + AHEAD);
      }
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
        if constexpr (F8) {  // lanes 0..15 the keys' scales, the others the values'
          const int r = lane & 15;
          const bool ok = good && r < have;
          const float* src = (lane < 16 ? p.k_scale : p.v_scale) + (ok ? (row0 + r) * p.H + g : 0);
          cp_async_4(st + St::S0 + ((lane < 16 ? 0 : St::KEYS) + 16 * hs + r) * 4, src, ok);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < St::COUNT - 1; ++i) load(i);
  ws.load_q(p, head0, gq, tq);
  for (int i = 0; i < n; ++i) {
    cp_async_wait<St::COUNT - 2>();
    // unit i has landed for all lanes, and all are done with unit i - 1; heads side by side
    // stay in step, so that what they load together lies together in memory
    if (side_by_side) __syncthreads(); else __syncwarp();
    load(i + St::COUNT - 1);
    const int have = len - first_token(i);
    if (have > 0) ws.step(ring + (i % St::COUNT) * St::BYTES, have, lane);
  }
  cp_async_wait<0>();
}

// What the warps of a CTA leave of a span: running sums in their own stages ([8 R][D + 4] floats),
// the rest here.
struct WarpSums {
  float m[kWarps][16], mv[kWarps][16], l[kWarps][16];
};
template <int D, bool F8, bool WIDE>
__device__ __forceinline__ void leave_sums(const WarpState<D, F8, WIDE>& ws, uint8_t* ring, WarpSums& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, tq = lane & 3;
  __syncwarp();  // the warp is done with its stages
  float* my_o = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int r = 0; r < ws.R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        my_o[(8 * r + 2 * tq + (e & 1)) * (D + 4) + ws.column(i, e, gq)] = ws.o[i][r][e];
#pragma unroll
  for (int r = 0; r < ws.R; ++r) {
    float l = ws.l[r];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (tq == 0) {
      s.m[warp][gq + 8 * r] = ws.m[r];
      if (F8) s.mv[warp][gq + 8 * r] = ws.mv[r] - kWeightBits;
      s.l[warp][gq + 8 * r] = l;
    }
  }
}

// Columns c .. c + 3 of head h, joined over the warps w0, w0 + wh, ... (subs of them), not yet
// divided by l; the maximum (in bits) and l.
template <int D, bool F8, bool WIDE>
__device__ __forceinline__ float4 join_warps(const uint8_t* smem, const WarpSums& s, int h, int c, int w0, int wh,
                                             int subs, float* top_out, float* l_out) {
  using St = Stage<D, F8, WIDE>;
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
    if constexpr (F8) {  // as its root twice: it underflows where value scales are subnormal
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
// (229 us, 5.0 TB/s) or 16 heads a group (392 us, 5.6 TB/s).
template <int D, bool F8, bool WIDE, bool SPARSE>
__global__ void __launch_bounds__(kThreads, Stage<D, F8, WIDE>::PER_SM) paged_attn_kernel(const PagedDecode p) {
  using St = Stage<D, F8, WIDE>;
  extern __shared__ __align__(128) uint8_t smem[];
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
  uint8_t* ring = smem + warp * St::COUNT * St::BYTES;
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
      WarpState<D, F8, WIDE> ws;
      attend<D, F8, WIDE, SPARSE>(p, ws, ring, b, g, len, u0, n, blk, my_token, unit, wh > 1);
      leave_sums(ws, ring, s_sums);
    }
    __syncthreads();
    const bool whole = n == units;
    const int64_t part = (int64_t)(2 * blockIdx.x + slot) * wh * p.G;
    const int64_t out0 = ((int64_t)b * p.H + hg * wh) * p.G;  // first of the wh G query heads
    for (int x = tid; x < wh * p.G * (D / 4); x += kThreads) {
      const int row = x / (D / 4), c = 4 * (x % (D / 4));
      const int w0 = wh == 1 ? 0 : row / p.G, h = row - w0 * p.G;
      float top, l;
      float4 acc = join_warps<D, F8, WIDE>(smem, s_sums, h, c, w0, wh, subs, &top, &l);
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

template <int D, bool F8, bool WIDE, int DI>  // DI = 0: the whole cache
__global__ void __launch_bounds__(kThreads, Stage<D, F8, WIDE>::PER_SM) paged_small_kernel(const PagedDecode p) {
  using St = Stage<D, F8, WIDE>;
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
  uint8_t* ring = smem + warp * St::COUNT * St::BYTES;
  float4 acc[ITEMS];
  if (n > 0) {
    {
      WarpState<D, F8, WIDE> ws;
      attend<D, F8, WIDE, SPARSE>(p, ws, ring, b, g, len, u0, n, blk, warp * St::KEYS, St::UNIT, false);
      leave_sums(ws, ring, s_sums);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int x = tid + k * kThreads, h = x / (D / 4), c = 4 * (x % (D / 4));
      if (h >= p.G) break;
      float top, l;
      acc[k] = join_warps<D, F8, WIDE>(smem, s_sums, h, c, 0, 1, kWarps, &top, &l);
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
  __shared__ float s_w[kCtas + 1], s_red[8], s_sum[8];
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

// pooled[b][g][c] = max over the 128 keys j of block c of q_idx[b, g] . k_idx[j], for every
// block wholly before the new token's.  The blocks of all sequences in order are dealt in turn to
// kPoolWarps warps a SM, which take 8 NT groups each.  A warp has two stages of half a block in
// shared memory: while it works on one half the next is on its way, and the page ids of the block
// after it.  Bound by HBM, so what counts are the bytes in flight: 192 KB a SM (8 x 128K, 134 MB:
// 23.6 us, 5.7 TB/s with the fill and drain; the halves in registers instead, 25.2 us; the warps of
// an SM next to one another in the deal, so that half of the SMs have no part in the last round,
// 24.1 us).
constexpr int kPoolCtas = 152, kPoolWarps = 12;
template <int DI>
constexpr int kPoolStage = 64 * DI * 2;  // bytes

template <int DI, int NT>
__global__ void __launch_bounds__(kPoolWarps * 32, 1) paged_pool_kernel(const PagedDecode p) {
  constexpr int NP = DI / 32;   // 32-wide d chunks: two k steps each
  constexpr int CH = DI / 8;    // 16-byte chunks of a key row
  constexpr int RPI = 32 / CH;  // rows of one copy instruction
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  const int warp = (threadIdx.x >> 5) * kPoolCtas + blockIdx.x;
  uint8_t* stages = smem + (threadIdx.x >> 5) * 2 * kPoolStage<DI>;
  if (blockIdx.y == 0)
    for (int64_t x = blockIdx.x * blockDim.x + threadIdx.x; x < (int64_t)p.B * p.H; x += gridDim.x * blockDim.x)
      p.arrive[x] = 0;
  // blocks before each lane's sequences
  const int per = (p.B + 31) / 32, b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
  int mine = 0;
  for (int i = b0; i < b1; ++i) mine += (max(1, seq_len(p, i)) - 1) / 128;
  int scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += x;
  }
  const int total = __shfl_sync(0xffffffffu, scan, 31);
  int u = warp;
  if (u >= total) return;
  // the sequence that holds block u, and the number `base` of its first block
  const int src = __ffs(__ballot_sync(0xffffffffu, u >= scan - mine && u < scan)) - 1;
  int b = __shfl_sync(0xffffffffu, b0, src), base = __shfl_sync(0xffffffffu, scan - mine, src);
  struct Place {
    int b, c;  // sequence and block
    int id;    // page id of tile lane % 8 of the block
  };
  const int tile_tok = (lane & 7) * 16;
  auto find = [&](int x) {  // of block x, which never decreases
    for (int n; n = (max(1, seq_len(p, b)) - 1) / 128, x >= base + n; base += n) ++b;
    const int c = x - base;
    return Place{b, c, __ldg(&p.pages.table[(int64_t)b * p.pages.table_stride + page_of(p.pages, c * 128 + tile_tok)])};
  };
  // half h of a block into stage h: 16-byte chunks, the 64-byte halves of odd rows swapped (d_idx 64)
  const int r0 = lane / CH, ch = lane % CH;
  auto load = [&](const Place& at, int h) {
    uint8_t* st = stages + h * kPoolStage<DI>;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int id = __shfl_sync(0xffffffffu, at.id, 4 * h + t);
      const int tok = at.c * 128 + (4 * h + t) * 16;
      const bool good = (unsigned)id < (unsigned)p.pages.num_pages;
      if (!good) set_status(p.status, MSA_ERR_ARG);
      const int64_t row = good ? (int64_t)id * p.pages.page_size + (tok - page_of(p.pages, tok) * p.pages.page_size) : 0;
      const __nv_bfloat16* k = p.k_idx + (row + r0) * DI + ch * 8;
#pragma unroll
      for (int i = 0; i < 16 / RPI; ++i) {
        const int r = r0 + i * RPI;
        const int put = DI == 64 ? ch ^ ((r & 1) << 2) : ch;
        if (good) cp_async_16(st + (t * 16 + r) * DI * 2 + put * 16, k + i * RPI * DI);
        else cp_async_16(st + (t * 16 + r) * DI * 2 + put * 16, p.k_idx, false);  // zero rows
      }
    }
    cp_async_commit();
  };
  uint4 bq[NT][NP];
  auto load_q = [&](int b) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int grp = blockIdx.y * 8 * NT + nt * 8 + gq;
      const uint4* qrow = reinterpret_cast<const uint4*>(p.q_idx + ((int64_t)b * p.H + grp) * DI);
#pragma unroll
      for (int j = 0; j < NP; ++j) bq[nt][j] = grp < p.H ? __ldg(&qrow[j * 4 + tq]) : make_uint4(0, 0, 0, 0);
    }
  };
  float mx[NT][2];
  // mma.sync A fragments from 16-byte chunks of rows gq and gq + 8, the k slots permuted alike in
  // the query fragments
  auto score = [&](int h) {
    const uint8_t* st = stages + h * kPoolStage<DI>;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint4 lo[NP], hi[NP];
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int get = DI == 64 ? (j * 4 + tq) ^ ((gq & 1) << 2) : tq;
        lo[j] = *reinterpret_cast<const uint4*>(st + (t * 16 + gq) * DI * 2 + get * 16);
        hi[j] = *reinterpret_cast<const uint4*>(st + (t * 16 + gq + 8) * DI * 2 + get * 16);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const uint32_t a0[4] = {lo[j].x, hi[j].x, lo[j].y, hi[j].y};
          const uint32_t a1[4] = {lo[j].z, hi[j].z, lo[j].w, hi[j].w};
          mma_bf16_16816(acc, a0, bq[nt][j].x, bq[nt][j].y);
          mma_bf16_16816(acc, a1, bq[nt][j].z, bq[nt][j].w);
        }
        mx[nt][0] = fmax3(mx[nt][0], acc[0], acc[2]);
        mx[nt][1] = fmax3(mx[nt][1], acc[1], acc[3]);
      }
    }
  };
  constexpr int STEP = kPoolCtas * kPoolWarps;
  Place now = find(u);
  load(now, 0);
  load(now, 1);
  load_q(now.b);
  Place next = u + STEP < total ? find(u + STEP) : now;
  while (true) {
    const bool more = u + STEP < total;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      cp_async_wait<1>();
      __syncwarp();  // half h has landed for all lanes
      score(h);
      __syncwarp();  // and all are done with its stage
      if (more) load(next, h);
      else cp_async_commit();
    }
    Place later = next;
    if (u + 2 * STEP < total) later = find(u + 2 * STEP);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = mx[nt][e];
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        const int grp = blockIdx.y * 8 * NT + nt * 8 + 2 * tq + e;
        if (gq == 0 && grp < p.H) p.pooled[((int64_t)now.b * p.H + grp) * p.row + now.c] = m;
      }
    if (!more) break;
    if (next.b != now.b) load_q(next.b);
    now = next;
    next = later;
    u += STEP;
  }
  cp_async_wait<0>();
}

// One CTA per (group, sequence): the new token's blocks, for caches of more blocks than the
// attention kernel selects from; none for an empty slot.
template <int KM>
__global__ void __launch_bounds__(256) paged_select_kernel(const PagedDecode p) {
  griddep_launch_dependents();
  const int64_t bg = (int64_t)blockIdx.y * p.H + blockIdx.x;
  const int len = seq_len(p, blockIdx.y);
  int32_t* dst = p.block_idx + bg * p.topk;
  griddep_wait();
  if (len == 0) {
    for (int s = threadIdx.x; s < p.topk; s += blockDim.x) dst[s] = -1;
    return;
  }
  const float* src = p.pooled + bg * p.row;
  const int c_own = (len - 1) / 128;
  // by rank while a thread's share of the blocks fits its registers, else by lists
  if (c_own <= 16 * 256) select_blocks_by_rank<16, 256>(src, c_own, p.topk, dst);
  else select_blocks<KM>(src, c_own, p.topk, dst);
}

// Launches with programmatic stream serialization: the kernel may be scheduled while its
// predecessor drains, and waits for it (griddep_wait) before it touches what that wrote.
template <typename Kern>
cudaError_t launch(Kern kern, dim3 grid, int threads, size_t smem, bool after, cudaStream_t stream,
                   const PagedDecode& p) {
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
  return cudaLaunchKernelEx(&cfg, kern, p);
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

template <int DI, int NT>
cudaError_t launch_pool(dim3 grid, const PagedDecode& p, cudaStream_t stream) {
  constexpr int smem = kPoolWarps * 2 * kPoolStage<DI>;
  static std::atomic<void*> done{nullptr};
  const cudaError_t e = allow_smem(paged_pool_kernel<DI, NT>, smem, done);
  return e != cudaSuccess ? e : launch(paged_pool_kernel<DI, NT>, grid, kPoolWarps * 32, smem, false, stream, p);
}

template <int D, bool F8, bool WIDE, bool SPARSE>
cudaError_t launch_attn(const PagedDecode& p, cudaStream_t stream) {
  constexpr int smem = kWarps * Stage<D, F8, WIDE>::COUNT * Stage<D, F8, WIDE>::BYTES;
  static_assert(Stage<D, F8, WIDE>::COUNT * Stage<D, F8, WIDE>::BYTES >= (WIDE ? 16 : 8) * (D + 4) * 4, "sums in the stages");
  static_assert(Stage<D, F8, WIDE>::PER_SM == (WIDE && D == 128 ? 2 : 3), "ctas");
  static_assert(kMaxSelect * 128 / Stage<D, F8, WIDE>::UNIT <= 64, "parts of selected blocks");
  auto* kern = paged_attn_kernel<D, F8, WIDE, SPARSE>;
  static std::atomic<void*> done{nullptr};
  const cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  return launch(kern, dim3(p.ctas), kThreads, smem, SPARSE, stream, p);
}

template <int D>
cudaError_t launch_paged(const PagedDecode& p, bool f8, bool wide, cudaStream_t stream) {
  const bool sparse = p.block_idx != nullptr;
  cudaError_t e;
  if (f8) {
    if (wide) e = sparse ? launch_attn<D, true, true, true>(p, stream) : launch_attn<D, true, true, false>(p, stream);
    else e = sparse ? launch_attn<D, true, false, true>(p, stream) : launch_attn<D, true, false, false>(p, stream);
  } else {
    if (wide) e = sparse ? launch_attn<D, false, true, true>(p, stream) : launch_attn<D, false, true, false>(p, stream);
    else e = sparse ? launch_attn<D, false, false, true>(p, stream) : launch_attn<D, false, false, false>(p, stream);
  }
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

template <int D, bool F8, bool WIDE, int DI>
cudaError_t launch_small(const PagedDecode& p, cudaStream_t stream) {
  constexpr int smem = kWarps * Stage<D, F8, WIDE>::COUNT * Stage<D, F8, WIDE>::BYTES;
  static_assert(smem >= 16 * D * 4, "a part");
  auto* kern = paged_small_kernel<D, F8, WIDE, DI>;
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

template <int D, int DI>
cudaError_t launch_small(const PagedDecode& p, bool f8, bool wide, cudaStream_t stream) {
  if (f8) return wide ? launch_small<D, true, true, DI>(p, stream) : launch_small<D, true, false, DI>(p, stream);
  return wide ? launch_small<D, false, true, DI>(p, stream) : launch_small<D, false, false, DI>(p, stream);
}

// CTAs of a cluster of the small form, or 0 for the other one: as many as let all pairs run
// together, if each then has at most kSmallUnits units, or twice that where the pairs alone fill
// the GPU and the cache is read whole.  Measured (GPU time of bf16, d 128, 8 groups of 4 heads,
// whole cache, small against other): 1 sequence of 512 tokens 6.2 / 9.1 us, of 4096 (8 units a
// CTA) 10.5 / 12.0, of 8192 15.4 / 12.9; 8 of 2048 (8 units) 11.1 / 15.5, 16 of ragged lengths to
// 4096 (32 units) 33.0 / 24.4; with 256 pairs, 32 of 1024 (16 units) 25.7 / 34.1 and of ragged
// lengths to 2048 (32 units) 36.3 / 32.9.  topk 16: 1 of 2048 11.9 / 25.5, 32 of 512 (8 units)
// 14.6 / 30.6, 64 of 1024 (16 units) 73.4 / 65.4.
constexpr int kSmallUnits = 8;
int small_cluster(int64_t pairs, int64_t cap, int topk, int unit, int ctas) {
  const int64_t nb = (cap + 127) / 128;
  if (topk > 0 && nb > kSmallBlocks) return 0;
  const int64_t units = topk > 0 ? (nb < topk ? nb : topk) * (128 / unit) : (cap + unit - 1) / unit;
  int c = 8;
  while (c > 1 && pairs * c > ctas) c >>= 1;
  return units <= (topk == 0 && c == 1 ? 2 : c) * kSmallUnits ? c : 0;
}

// Heads (groups) that a CTA serves side by side: all attend the same tokens when the whole cache
// is attended, and rows of one token are neighbours in a page; selected blocks differ by group.
int heads_side_by_side(int H, int topk) {
  if (topk > 0) return 1;
  return H % 4 == 0 ? 4 : H % 2 == 0 ? 2 : 1;
}

struct Layout {
  size_t part_o, part_lse, starts, arrive, pooled, bytes;
  int cluster, ctas, keys_shift;
};

// Sizes of a call; MSA_OK and the workspace's layout.  topk = 0: the whole cache.
int check_sizes(const msa_paged_cache_t* c, const msa_page_table_t* pt, int H_q, int topk, Layout* lay) {
  int rc = check_cache_sizes(c);
  if (rc) return rc;
  if (!pt) return MSA_ERR_ARG;
  if (pt->B < 0 || pt->max_pages < 0 || pt->stride < 0) return MSA_ERR_SHAPE;
  const int64_t cap = (int64_t)pt->max_pages * c->page_size;
  if (cap > 0x7fffffffLL) return MSA_ERR_UNSUPPORTED;
  if (H_q <= 0 || H_q % c->H_kv != 0) return MSA_ERR_SHAPE;
  const int G = H_q / c->H_kv;
  if (G > 16 || topk > kMaxSelect) return MSA_ERR_UNSUPPORTED;
  if ((int64_t)pt->B * c->H_kv > (1 << 24) || pt->B > 65535) return MSA_ERR_UNSUPPORTED;
  if (topk > 0 && c->d_idx == 0) return MSA_ERR_SHAPE;
  // the work of all pairs is counted in 32 bits
  const int64_t most = (cap >> (c->kind == MSA_CACHE_E4M3 || c->d == 64 ? 7 : 6)) + kOverhead + 4;
  if ((int64_t)pt->B * c->H_kv * most >= 1 << 30) return MSA_ERR_UNSUPPORTED;
  lay->keys_shift = c->kind == MSA_CACHE_E4M3 || c->d == 64 ? 5 : 4;
  lay->ctas = kCtas / 3 * (G > 8 && c->d == 128 ? 2 : 3);  // Stage::PER_SM
  lay->cluster = small_cluster((int64_t)pt->B * c->H_kv, cap, topk, kWarps << lay->keys_shift, lay->ctas);
  lay->bytes = 0;
  if (lay->cluster) return MSA_OK;
  lay->part_o = 0;
  const size_t parts = (size_t)2 * kCtas * heads_side_by_side(c->H_kv, topk) * G;
  lay->part_lse = align256(parts * c->d * 4);
  lay->starts = lay->part_lse + align256(parts * 4);
  lay->arrive = lay->starts + align256(((size_t)pt->B + 2) * 4);
  lay->pooled = lay->arrive + (topk > 0 ? align256((size_t)pt->B * c->H_kv * 4) : 0);
  lay->bytes = lay->pooled + (topk > 0 ? align256((size_t)pt->B * c->H_kv * (((cap + 127) / 128 + 3) & ~3) * 4) : 0);
  return MSA_OK;
}

int run_paged(const msa_paged_cache_t* c, const msa_page_table_t* pt, const int32_t* lens, int H_q,
              int topk, float scale, const void* q, const void* q_idx, int32_t* block_idx, void* o,
              float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  Layout lay;
  int rc = check_sizes(c, pt, H_q, topk, &lay);
  if (rc) return rc;
  if (!(scale > 0.f) || !isfinite(scale)) return MSA_ERR_ARG;
  PagedDecode p = {};
  if ((rc = check_cache(c))) return rc;
  if ((rc = check_pages(c, pt, &p.pages))) return rc;
  if (pt->B == 0) return MSA_OK;
  const void* ptrs[] = {q, o, lse, topk > 0 ? q_idx : q, topk > 0 ? (const void*)block_idx : q};
  for (const void* x : ptrs)
    if (!x || (reinterpret_cast<uintptr_t>(x) & 15) != 0) return MSA_ERR_ARG;
  if (!lens || (reinterpret_cast<uintptr_t>(lens) & 3)) return MSA_ERR_ARG;
  if (lay.bytes > 0 && (!workspace || workspace_bytes < lay.bytes)) return MSA_ERR_WORKSPACE;
  if (lay.bytes > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255) != 0) return MSA_ERR_ARG;
  Ctx cx;
  if ((rc = device_ctx(&cx))) return rc;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_idx = static_cast<const __nv_bfloat16*>(q_idx);
  // without pages every id is bad and every copy has no bytes: any address does for those
  const bool pages_exist = c->num_pages > 0;
  p.k = pages_exist ? c->k : q;
  p.v = pages_exist ? c->v : q;
  p.k_scale = pages_exist ? c->k_scale : static_cast<const float*>(q);
  p.v_scale = pages_exist ? c->v_scale : static_cast<const float*>(q);
  p.k_idx = static_cast<const __nv_bfloat16*>(pages_exist ? c->k_idx : q);
  p.lens = lens;
  p.block_idx = topk > 0 ? block_idx : nullptr;
  p.pooled = reinterpret_cast<float*>(w + lay.pooled);
  p.part_o = reinterpret_cast<float*>(w + lay.part_o);
  p.part_lse = reinterpret_cast<float*>(w + lay.part_lse);
  p.starts = reinterpret_cast<int*>(w + lay.starts);
  p.arrive = reinterpret_cast<int*>(w + lay.arrive);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.B = pt->B;
  p.H = c->H_kv;
  p.G = H_q / c->H_kv;
  p.topk = topk;
  const int nb = (int)(((int64_t)pt->max_pages * c->page_size + 127) / 128);
  p.row = (nb + 3) & ~3;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wh = heads_side_by_side(p.H, topk);
  p.ctas = lay.ctas;
  p.keys_shift = lay.keys_shift;
  p.cluster = lay.cluster;
  p.status = cx.status;
  cudaError_t e = cudaSuccess;
  const bool wide = p.G > 8, f8 = c->kind == MSA_CACHE_E4M3;
  if (p.cluster) {
    if (c->d == 128)
      e = topk == 0          ? launch_small<128, 0>(p, f8, wide, stream)
          : c->d_idx == 64 ? launch_small<128, 64>(p, f8, wide, stream)
                           : launch_small<128, 32>(p, f8, wide, stream);
    else
      e = topk == 0          ? launch_small<64, 0>(p, f8, wide, stream)
          : c->d_idx == 64 ? launch_small<64, 64>(p, f8, wide, stream)
                           : launch_small<64, 32>(p, f8, wide, stream);
    return finish(e);
  }
  if (topk > 0) {
    const int nt = p.H > 8 ? 2 : 1;
    const dim3 grid(kPoolCtas, (unsigned)((p.H + 8 * nt - 1) / (8 * nt)));
    if (nb > 0) {
      if (c->d_idx == 64) e = nt == 1 ? launch_pool<64, 1>(grid, p, stream) : launch_pool<64, 2>(grid, p, stream);
      else e = nt == 1 ? launch_pool<32, 1>(grid, p, stream) : launch_pool<32, 2>(grid, p, stream);
      if (e != cudaSuccess) return MSA_ERR_CUDA;
    }
    p.select = nb <= kSelectPer * kThreads;
    const dim3 gsel((unsigned)p.H, (unsigned)p.B);
    if (!p.select)
      e = topk <= 16 ? launch(paged_select_kernel<15>, gsel, 256, 0, true, stream, p)
                     : launch(paged_select_kernel<31>, gsel, 256, 0, true, stream, p);
    if (e != cudaSuccess) return MSA_ERR_CUDA;
  }
  e = c->d == 128 ? launch_paged<128>(p, f8, wide, stream) : launch_paged<64>(p, f8, wide, stream);
  return finish(e);
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

size_t msa_decode_paged_workspace_size(const msa_paged_cache_t* c, const msa_page_table_t* pages, int H_q,
                                       int topk) {
  Layout lay;
  return topk >= 0 && check_sizes(c, pages, H_q, topk, &lay) == MSA_OK ? lay.bytes : 0;
}

int msa_decode_paged(const msa_paged_cache_t* c, const msa_page_table_t* pages, const int32_t* lens,
                     int H_q, int topk, float scale, const void* q, const void* q_idx,
                     int32_t* block_idx, void* o, float* lse, void* workspace, size_t workspace_bytes,
                     cudaStream_t stream) {
  if (topk <= 0) return MSA_ERR_SHAPE;
  return run_paged(c, pages, lens, H_q, topk, scale, q, q_idx, block_idx, o, lse, workspace,
                   workspace_bytes, stream);
}

int msa_decode_paged_dense(const msa_paged_cache_t* c, const msa_page_table_t* pages,
                           const int32_t* lens, int H_q, float scale, const void* q, void* o, float* lse,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return run_paged(c, pages, lens, H_q, 0, scale, q, nullptr, nullptr, o, lse, workspace, workspace_bytes,
                   stream);
}

}  // extern "C"
