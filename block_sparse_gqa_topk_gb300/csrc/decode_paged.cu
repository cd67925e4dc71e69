// decode_paged.cu -- the calls of decode_paged.cuh: argument checks, the pooling of block scores, the
// selection, and the kernels of bf16 and E4M3 caches.
#include "decode_paged.cuh"

namespace msa {
namespace {

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

template <int DI, int NT>
cudaError_t launch_pool(dim3 grid, const PagedDecode& p, cudaStream_t stream) {
  constexpr int smem = kPoolWarps * 2 * kPoolStage<DI>;
  static std::atomic<void*> done{nullptr};
  const cudaError_t e = allow_smem(paged_pool_kernel<DI, NT>, smem, done);
  return e != cudaSuccess ? e : launch(paged_pool_kernel<DI, NT>, grid, kPoolWarps * 32, smem, false, stream, p);
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
  const bool coded = c->kind != MSA_CACHE_BF16;
  const int64_t most = (cap >> (coded || c->d == 64 ? 7 : 6)) + kOverhead + 4;
  if ((int64_t)pt->B * c->H_kv * most >= 1 << 30) return MSA_ERR_UNSUPPORTED;
  lay->keys_shift = coded || c->d == 64 ? 5 : 4;  // Stage::KEYS
  lay->ctas = kCtas / 3 * (G > 8 && c->d == 128 ? 2 : 3);  // Stage::PER_SM
  lay->cluster = small_cluster((int64_t)pt->B * c->H_kv, cap, topk, kWarps << lay->keys_shift, lay->ctas);
  if (c->kind == MSA_CACHE_E2M1 && topk == 0 && lay->ctas == kCtas) lay->ctas = kMaxCtas;  // Stage::DENSE_PER_SM
  lay->bytes = 0;
  if (lay->cluster) return MSA_OK;
  lay->part_o = 0;
  const size_t parts = (size_t)2 * (lay->ctas > kCtas ? lay->ctas : kCtas) * heads_side_by_side(c->H_kv, topk) * G;
  lay->part_lse = align256(parts * c->d * 4);
  lay->starts = lay->part_lse + align256(parts * 4);
  lay->arrive = lay->starts + align256(((size_t)pt->B + 2) * 4);
  lay->pooled = lay->arrive + (topk > 0 ? align256((size_t)pt->B * c->H_kv * 4) : 0);
  lay->bytes = lay->pooled + (topk > 0 ? align256((size_t)pt->B * c->H_kv * (((cap + 127) / 128 + 3) & ~3) * 4) : 0);
  return MSA_OK;
}

cudaError_t launch_attention(const msa_paged_cache_t* c, const PagedDecode& p, cudaStream_t stream) {
  if (c->kind == MSA_CACHE_E2M1) return launch_decode_e2m1(p, c->d, c->d_idx, stream);
  if (c->kind == MSA_CACHE_E4M3)
    return c->d == 128 ? launch_kind<128, MSA_CACHE_E4M3>(p, c->d_idx, stream)
                       : launch_kind<64, MSA_CACHE_E4M3>(p, c->d_idx, stream);
  return c->d == 128 ? launch_kind<128, MSA_CACHE_BF16>(p, c->d_idx, stream)
                     : launch_kind<64, MSA_CACHE_BF16>(p, c->d_idx, stream);
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
  p.k_scale = static_cast<const uint8_t*>(pages_exist ? c->k_scale : q);
  p.v_scale = static_cast<const uint8_t*>(pages_exist ? c->v_scale : q);
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
  // four groups of a 4-bit cache come together where a batch may be long enough for groups side by side
  const int64_t most = (int64_t)p.B * p.H * (((int64_t)pt->max_pages * c->page_size + 127) / 128 + kOverhead);
  p.together = c->kind == MSA_CACHE_E2M1 && p.wh == 4 && pages_exist && most >= (int64_t)kSideBySideTogether * p.ctas &&
               (int64_t)c->num_pages * c->page_size < (int64_t{1} << 31);
  p.withheld = cx.debug & MSA_DEBUG_WITHHOLD_LOAD ? 0 : -1;
  p.wait_ns = cx.wait_ns;
  p.status = cx.status;
  cudaError_t e = cudaSuccess;
  if (p.cluster) return finish(launch_attention(c, p, stream));
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
  return finish(launch_attention(c, p, stream));
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
