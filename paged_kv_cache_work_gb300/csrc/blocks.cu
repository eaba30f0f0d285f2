// Channel bounds of the pages' keys, scores of a sequence's pages from them, and the selection of
// the best pages.
//
// Bounds.  One CTA per (sequence, touched page, kv head): the least and largest value of each
// channel over the new rows, joined with the page's older bounds unless it is fresh.  Reading the
// rows bounds it: four rows of a thread are in flight at once (8 prompts, 33.6 MB that the append
// has just left in L2: 8.6 us; a step of 32 tokens 2.2 us, the launch).
//
// Score.  For a page with channel bounds lo, hi and a query row q no key k of the page (lo_d <=
// k_d <= hi_d) has <q, k> above sum_d max(q_d lo_d, q_d hi_d), and that is one dot product of
// length 2 D: sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d.  So the scores are a matrix product of
// the query rows with the pages' bounds, on mma.sync m16n8k16 with fp32 accumulation (products of
// 16-bit values are exact): 16 query rows by 8 pages.  What bounds it is the 4 D bytes of a (page,
// head), one contiguous piece; what it takes is enough of them in flight (about 100 KB an SM), which
// registers do not hold.  So each warp streams its pages on its own through a ring of shared-memory
// stages of 8 pages by 16-byte cp.async, a page a warp instruction at head dim 128, with the blocks
// of 32 pages looked up at a time (a lane each).  max(q, 0) and min(q, 0) stay in registers as A
// fragments.  With the contraction's order permuted alike on both sides (a lane's 8 channels of a
// 16-byte piece are 4 of one k-step and 4 of the next) a page's pieces are the B fragments as a lane
// reads them.
//   Measured on 32 contexts of 32,768 to 131,072 tokens in pages of 64 (168 MB, 25.1 us at the copy
// rate): 31.9 us with 12 warps an SM (8: 32.0, 16: 30.6, 48: 34.4), and 7.5 us on contexts of at
// most 4,096 in pages of 16, where 16 warps take 8.0 and 48 take 12.0.  Pages read straight into
// registers by 33, 12 and 8 warps an SM took 38, 41 and 56 us, a 512-byte bulk copy a page 50 us (the
// copy engine takes about 40 cycles for each, however short).
//
// A row tile holds whole query tokens where a group has 1, 2, 4 or 8 heads (16 / G tokens; a
// token's maximum is up to three shuffles away); other groups take ceil(G / 16) tiles a token.
//
// Select.  One CTA per row: scores become order-preserving 32-bit keys, the k-th largest is found,
// and one ordered pass writes the pages above it and the first of those equal to it.  What bounds
// it is the chain of block-wide steps of a row.  So the k-th key comes from one histogram: 256 bins
// of equal width between the row's least and greatest finite score spread the shared-memory atomics
// (a float's own upper bits fall into a few exponents: four passes of 8 bits took 14.3 us for 1,024
// rows of at most 2,048 pages, this takes 12.1), and the keys of the bin with the k-th are few enough
// to rank each against all of them.  Rows that leave more than 128 in the bin (ties, outliers) take
// the passes of 8 bits (1,024 rows of 2,048 equal scores: 18.8 us).  A warp keeps a run of a row's
// pages in registers where the row has at most 2,048.  Of the 12.1 us the reading of lengths and
// scores takes 5.4 (two waves of CTAs), the histogram 2.1, the bin's ranks 2.2, the ordered pass 2.5.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "append_block.cuh"

namespace pa {
namespace {

// Keys that row i of sequence b sees; -1 for lengths that break the rules.
__device__ __forceinline__ int keys_seen(const int32_t* ctx, const int32_t* qlens, int b, int i,
                                         int Sq, int maxb, int bs_shift, int causal) {
  const int n = __ldg(ctx + b), ql = __ldg(qlens + b);
  if (ql < 0 || ql > Sq || n < ql || (long long)n > ((long long)maxb << bs_shift)) return -1;
  if (i >= ql) return 0;
  return causal ? n - ql + i + 1 : n;
}
__device__ __forceinline__ int pages_of(int keys, int bs_shift) {
  return (int)(((long long)keys + (1 << bs_shift) - 1) >> bs_shift);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool page_size_ok(int bs) { return bs >= 16 && bs <= 1024 && (bs & (bs - 1)) == 0; }

// Launch with programmatic dependent launch: the kernels begin with grid_dependency_wait.
template <class P>
cudaError_t launch_pdl(void (*kernel)(P), const P& p, dim3 grid, int threads, size_t smem,
                       cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// ---- bounds ------------------------------------------------------------------------------
constexpr int kBoundsThreads = 128;

template <int QK, bool MAX>
__device__ __forceinline__ uint32_t extreme2(uint32_t x, uint32_t y) {  // NaN wins
  uint32_t r;
  if constexpr (QK == Q_BF16) {
    if constexpr (MAX)
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    else
      asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  } else {
    if constexpr (MAX)
      asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    else
      asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  }
  return r;
}
template <int QK, bool MAX>
__device__ __forceinline__ uint4 extreme8(const uint4& x, const uint4& y) {
  return make_uint4(extreme2<QK, MAX>(x.x, y.x), extreme2<QK, MAX>(x.y, y.y),
                    extreme2<QK, MAX>(x.z, y.z), extreme2<QK, MAX>(x.w, y.w));
}

struct BoundsParams {
  TouchParams t;
  const char* k_new;
  char* bounds;
};

template <int D, int QK>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const BoundsParams p) {
  constexpr int PPR = D / 8;                // 16-byte pieces of a row
  constexpr int RG = kBoundsThreads / PPR;  // rows taken at a time
  __shared__ uint4 s_lo[kBoundsThreads], s_hi[kBoundsThreads];
  const int tid = threadIdx.x, c = tid % PPR, rg = tid / PPR;
  const uint32_t bj = p.t.head_div.div(blockIdx.x);
  const int g = (int)(blockIdx.x - bj * p.t.Hkv);
  const int b = (int)p.t.page_div.div(bj), j = (int)p.t.page_div.mod(bj);
  grid_dependency_wait();
  grid_dependents_launch();
  TouchedPage t;
  if (!touched_page(p.t, b, j, tid == 0 && g == 0, &t)) return;
  const size_t row_stride = (size_t)p.t.Hkv * D;
  const uint4* src = reinterpret_cast<const uint4*>(
                         p.k_new + (((size_t)b * p.t.Sq + t.i0) * row_stride + (size_t)g * D) * 2) + c;
  // four rows of each thread at a time, all on their way at once
  uint4 lo, hi;
  if (rg < t.rows) {
    lo = hi = __ldg(src + (size_t)rg * (row_stride / 8));
    for (int r0 = rg; r0 < t.rows; r0 += 4 * RG) {
      uint4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[k] = __ldg(src + (size_t)min(r0 + k * RG, t.rows - 1) * (row_stride / 8));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        lo = extreme8<QK, false>(lo, x[k]);
        hi = extreme8<QK, true>(hi, x[k]);
      }
    }
    s_lo[tid] = lo;
    s_hi[tid] = hi;
  }
  const int blk = rg == 0 ? touched_block(p.t, b, t, tid == 0) : -1;
  __syncthreads();
  if (blk < 0) return;
  uint4* out = reinterpret_cast<uint4*>(p.bounds + ((size_t)blk * p.t.Hkv + g) * 2 * D * 2) + c;
  for (int k = 1; k < min(RG, t.rows); ++k) {
    lo = extreme8<QK, false>(lo, s_lo[k * PPR + c]);
    hi = extreme8<QK, true>(hi, s_hi[k * PPR + c]);
  }
  if (t.slot0 != 0) {
    lo = extreme8<QK, false>(lo, out[0]);
    hi = extreme8<QK, true>(hi, out[PPR]);
  }
  out[0] = lo;
  out[PPR] = hi;
}

// ---- score -------------------------------------------------------------------------------
constexpr int kScoreWarps = 4;
constexpr int kScoreWarpsPerSm = 12;
constexpr int kScoreMaxGroups = 32;

struct ScoreParams {
  const char* q;
  const char* bounds;
  const int32_t* bt;
  const int32_t* ctx;
  const int32_t* qlens;
  float* scores;
  int32_t* flags;
  int Sq, Hq, Hkv, G, bs_shift, maxb, nblocks, causal;
  int tpt;         // tokens of a warp's row tile (G 1, 2, 4 or 8), else 1
  int g_shift;     // log2(G) then, else -1
  int parts;       // row tiles per token
  int tok_groups;  // warps along the tokens
  int runs;        // warps along the pages
  int batch;
  int groups;      // groups of 8 pages of a warp
  float sm_scale;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int QK>
__device__ __forceinline__ void score_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if constexpr (QK == Q_FP16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

template <int D>
struct ScoreSmem {
  static constexpr int PAGE = 4 * D;       // bytes of a (page, head)
  static constexpr int STRIDE = PAGE + 64;  // so that two quads read distinct banks
  static constexpr int STAGE = 8 * STRIDE;
  static constexpr int NST = D == 64 ? 6 : 3;
  static constexpr int WARP = NST * STAGE;
  static constexpr int BYTES = kScoreWarps * WARP;
  static constexpr int CTAS_PER_SM = D == 256 ? 2 : 3;
  static_assert(CTAS_PER_SM * (BYTES + 1024) <= 228 * 1024, "shared memory");
};

template <int D, int QK>
__global__ void __launch_bounds__(kScoreWarps * 32, ScoreSmem<D>::CTAS_PER_SM)
    score_kernel(const ScoreParams p) {
  using M = ScoreSmem<D>;
  constexpr int NP = D / 32;  // 16-byte pieces a lane takes of each bound: two k-steps each
  extern __shared__ __align__(128) char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, qi = lane & 3;
  char* const ring = smem + warp * M::WARP;
  // the heads of a page are neighbours in memory and here
  const uint32_t w = blockIdx.x * (uint32_t)kScoreWarps + warp;
  const int tg = (int)(w % p.tok_groups), g = (int)(w / p.tok_groups % p.Hkv);
  const int run = (int)(w / p.tok_groups / p.Hkv);
  const int pg = run % p.runs, b = run / p.runs;
  const int tok0 = tg * p.tpt, toks = min(p.tpt, p.Sq - tok0);
  const int page0 = pg * 8 * p.groups, page_end = min(p.maxb, page0 + 8 * p.groups);
  grid_dependency_wait();
  grid_dependents_launch();
  if (b >= p.batch) return;

  const int n = __ldg(p.ctx + b), ql = __ldg(p.qlens + b);
  const bool bad = ql < 0 || ql > p.Sq || n < ql || (long long)n > ((long long)p.maxb << p.bs_shift);
  if (bad && lane == 0 && tg == 0 && g == 0 && pg == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_LENGTHS);
  // pages that token t of this warp sees; last: the end of those that any of its tokens sees
  auto pages_seen = [&](int t) {
    const int i = tok0 + t;
    return pages_of(bad || i >= ql ? 0 : p.causal ? n - ql + i + 1 : n, p.bs_shift);
  };
  const int last = min(page_end, bad || tok0 >= ql ? 0 : pages_seen(min(tok0 + toks, ql) - 1 - tok0));
  const int mine = last > page0 ? (last - page0 + 7) >> 3 : 0;  // groups of pages to score

  // group k's pages into stage st; lane l holds the block of page 32 (k / 4) + l.  A page outside the
  // pool or past the last is copied from block 0 and not used.
  int blk = 0;
  uint32_t ok = 0;  // pages of the 32 that count
  const char* const bounds = p.bounds + (size_t)g * M::PAGE;
  const size_t block_stride = (size_t)p.Hkv * M::PAGE;
  const uint32_t ring_addr = smem_addr(ring);
  auto issue = [&](int k, int st) -> uint32_t {  // returns the group's pages that count
    uint32_t in = 0;
    if (k < mine) {
      if ((k & 3) == 0) {
        const int page = page0 + 8 * k + lane;
        bool good = false;
        blk = 0;
        if (page < last) {
          blk = __ldg(p.bt + (size_t)b * p.maxb + page);
          good = blk >= 0 && blk < p.nblocks;
          if (!good) {
            blk = 0;
            if (p.flags) atomicOr(p.flags, PA_FLAG_BAD_BLOCK_ID);
          }
        }
        ok = __ballot_sync(kFull, good);
      }
      in = (ok >> (8 * (k & 3))) & 255;
      constexpr int LPP = M::PAGE / 16;  // 16-byte pieces of a page
#pragma unroll
      for (int e0 = 0; e0 < 8 * LPP; e0 += 32) {
        const int page = (e0 + lane) / LPP, piece = (e0 + lane) % LPP;
        const int bk = __shfl_sync(kFull, blk, 8 * (k & 3) + page);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         ring_addr + st * M::STAGE + page * M::STRIDE + piece * 16),
                     "l"(bounds + bk * block_stride + piece * 16)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return in;
  };
  uint32_t in_ring[M::NST - 1];  // of the groups on their way, the next one first
#pragma unroll
  for (int k = 0; k < M::NST - 1; ++k) in_ring[k] = issue(k, k);

  // A fragments of row tile `part` (rows quad, quad + 8): max(q, 0) and min(q, 0) of k-step 2 t + h;
  // rows past the group or the tokens are some real row, and their products are not used
  uint32_t up[NP][2][4], dn[NP][2][4];
  auto load_q = [&](int part) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = quad + 8 * h;
      const int t = p.g_shift >= 0 ? min(r >> p.g_shift, toks - 1) : 0;
      const int head = p.g_shift >= 0 ? r & (p.G - 1) : min(16 * part + r, p.G - 1);
      const uint4* row = reinterpret_cast<const uint4*>(
          p.q + ((((size_t)b * p.Sq + tok0 + t) * p.Hq + (size_t)g * p.G + head) * D) * 2) + qi;
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int s = 0; s < NP; ++s) {
        const uint4 x = __ldg(row + 4 * s);
        const uint4 u = extreme8<QK, true>(x, zero), d = extreme8<QK, false>(x, zero);
        up[s][0][h] = u.x;
        up[s][0][2 + h] = u.y;
        up[s][1][h] = u.z;
        up[s][1][2 + h] = u.w;
        dn[s][0][h] = d.x;
        dn[s][0][2 + h] = d.y;
        dn[s][1][h] = d.z;
        dn[s][1][2 + h] = d.w;
      }
    }
  };
  if (mine > 0) load_q(0);

  float* const out = p.scores + (((size_t)b * p.Sq + tok0) * p.Hkv + g) * p.maxb;
  const size_t tok_stride = (size_t)p.Hkv * p.maxb;
  int st = 0;
  for (int k = 0; k < mine; ++k) {
    asm volatile("cp.async.wait_group %0;" ::"n"(M::NST - 2) : "memory");
    __syncwarp();
    const uint32_t in = in_ring[0];
#pragma unroll
    for (int j = 0; j + 1 < M::NST - 1; ++j) in_ring[j] = in_ring[j + 1];
    in_ring[M::NST - 2] = issue(k + M::NST - 1, st == 0 ? M::NST - 1 : st - 1);
    const uint4* box = reinterpret_cast<const uint4*>(ring + st * M::STAGE + quad * M::STRIDE) + qi;
    const int pbase = page0 + 8 * k;
    // pages pbase + 2 qi, + 1 of token t score v0, v1
    auto put = [&](int t, float v0, float v1) {
      const int page = pbase + 2 * qi, seen = pages_seen(t);
      if (page < page_end) out[t * tok_stride + page] = page < seen && ((in >> (2 * qi)) & 1) ? v0 : -INFINITY;
      if (page + 1 < page_end)
        out[t * tok_stride + page + 1] = page + 1 < seen && ((in >> (2 * qi + 1)) & 1) ? v1 : -INFINITY;
    };
    float best[2] = {-INFINITY, -INFINITY};  // a token of several row tiles: over those so far
    for (int part = 0; part < p.parts; ++part) {
      if (p.parts > 1) load_q(part);
      float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < NP; ++t) {
        const uint4 lo = box[4 * t], hi = box[D / 8 + 4 * t];
        score_mma<QK>(c, up[t][0], hi.x, hi.y);
        score_mma<QK>(c2, dn[t][0], lo.x, lo.y);
        score_mma<QK>(c, up[t][1], hi.z, hi.w);
        score_mma<QK>(c2, dn[t][1], lo.z, lo.w);
      }
      // c: rows quad (c[0], c[1]) and quad + 8 of pages pbase + 2 qi, + 1
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = (c[e] + c2[e]) * p.sm_scale;
      if (p.g_shift >= 0) {
        const bool two = (8 >> p.g_shift) < toks;  // rows 8 and up hold tokens too
        for (int o = 4; o < 4 << p.g_shift; o <<= 1) {
          c[0] = max_nan(c[0], __shfl_xor_sync(kFull, c[0], o));
          c[1] = max_nan(c[1], __shfl_xor_sync(kFull, c[1], o));
          if (two) {
            c[2] = max_nan(c[2], __shfl_xor_sync(kFull, c[2], o));
            c[3] = max_nan(c[3], __shfl_xor_sync(kFull, c[3], o));
          }
        }
        const int t = quad >> p.g_shift, t8 = (quad + 8) >> p.g_shift;
        if ((quad & (p.G - 1)) == 0) {
          if (t < toks) put(t, c[0], c[1]);
          if (t8 < toks) put(t8, c[2], c[3]);
        }
      } else {
        if (16 * part + quad < p.G) {
          best[0] = max_nan(best[0], c[0]);
          best[1] = max_nan(best[1], c[1]);
        }
        if (16 * part + quad + 8 < p.G) {
          best[0] = max_nan(best[0], c[2]);
          best[1] = max_nan(best[1], c[3]);
        }
        if (part + 1 == p.parts) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            best[0] = max_nan(best[0], __shfl_xor_sync(kFull, best[0], o));
            best[1] = max_nan(best[1], __shfl_xor_sync(kFull, best[1], o));
          }
          if (quad == 0) put(0, best[0], best[1]);
        }
      }
    }
    if (++st == M::NST) st = 0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // pages that none of the tokens sees
  for (int t = 0; t < toks; ++t)
    for (int page = page0 + 8 * mine + lane; page < page_end; page += 32) out[t * tok_stride + page] = -INFINITY;
}

// ---- select ------------------------------------------------------------------------------
constexpr int kSelectRank = 128;      // keys of a bin that are ranked each against all
constexpr int kSelectKeys = 49152;  // keys that fit in shared memory

struct SelectParams {
  const float* scores;
  const int32_t* ctx;
  const int32_t* qlens;
  int32_t* selected;
  int32_t* num;
  int32_t* flags;
  int Sq, Hkv, bs_shift, maxb, causal, top_k, first, last;
};

// Larger score, larger key; NaN above every number, forced pages above all.
__device__ __forceinline__ uint32_t key_of(float x, bool forced) {
  if (forced) return 0xffffffffu;
  if (x != x) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 becomes +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
constexpr uint32_t kLeastFinite = 0x00800000u, kMostFinite = 0xff7fffffu;  // keys of -+FLT_MAX

// R > 0: keys in registers, R groups of 32 pages a warp; kKeysShared: in shared memory; kKeysAgain:
// made from the scores in each pass.
constexpr int kKeysShared = 0, kKeysAgain = -1;

template <int R, int THREADS>
__global__ void __launch_bounds__(THREADS) select_kernel(const SelectParams p) {
  constexpr int NW = THREADS / 32;
  extern __shared__ uint32_t s_key[];
  __shared__ __align__(16) uint32_t s_hist[256];
  __shared__ __align__(16) uint32_t s_cand[kSelectRank];
  __shared__ uint32_t s_prefix, s_left, s_num;
  __shared__ uint2 s_range[NW];
  __shared__ int2 s_cnt[NW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t row = blockIdx.x, tok = row / p.Hkv;
  const int i = (int)(tok % p.Sq), b = (int)(tok / p.Sq);
  for (int e = tid; e < 256; e += THREADS) s_hist[e] = 0;
  if (tid == 0) s_num = 0;
  grid_dependency_wait();
  grid_dependents_launch();
  int seen = keys_seen(p.ctx, p.qlens, b, i, p.Sq, p.maxb, p.bs_shift, p.causal);
  if (seen < 0) {
    if (tid == 0 && i == 0 && row % p.Hkv == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_LENGTHS);
    seen = 0;
  }
  const int N = pages_of(seen, p.bs_shift), k = min(p.top_k, N);
  int32_t* out = p.selected + (size_t)row * p.top_k;
  if (tid == 0) p.num[row] = k;
  for (int e = k + tid; e < p.top_k; e += THREADS) out[e] = -1;
  if (N <= p.top_k) {
    for (int e = tid; e < N; e += THREADS) out[e] = e;
    return;
  }
  const float* x = p.scores + (size_t)row * p.maxb;
  const int hi_first = N - p.last;
  auto make_key = [&](int e) { return key_of(__ldg(x + e), e < p.first || e >= hi_first); };
  const int per = round_up(ceil_div(N, NW), 32);  // a warp's run of pages
  const int e0 = min(warp * per, N), e1 = min(e0 + per, N);
  uint32_t keys[R > 0 ? R : 1];
  // f(page, its key) on the run's pages, 32 at a time: whole warps, key 0 (no score's) past its end
  auto each = [&](auto&& f) {
    if constexpr (R > 0) {
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (e0 + 32 * j < e1) f(e0 + 32 * j + lane, keys[j]);
    } else {
#pragma unroll 4
      for (int base = e0; base < e1; base += 32) {
        const int e = base + lane;
        uint32_t v = 0;
        if (e < e1) v = R == kKeysShared ? s_key[e] : make_key(e);
        f(e, v);
      }
    }
  };
  if constexpr (R > 0) {
#pragma unroll
    for (int j = 0; j < R; ++j) keys[j] = e0 + 32 * j + lane < e1 ? make_key(e0 + 32 * j + lane) : 0;
  } else if constexpr (R == kKeysShared) {
#pragma unroll 4
    for (int e = e0 + lane; e < e1; e += 32) s_key[e] = make_key(e);
    __syncwarp();
  }
  uint32_t least = ~0u, most = 0u;  // finite keys
  each([&](int, uint32_t v) {
    if (v >= kLeastFinite && v <= kMostFinite) {
      least = min(least, v);
      most = max(most, v);
    }
  });
  least = __reduce_min_sync(kFull, least);
  most = __reduce_max_sync(kFull, most);
  if (lane == 0) s_range[warp] = make_uint2(least, most);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    least = min(least, s_range[w].x);
    most = max(most, s_range[w].y);
  }

  // ---- the k-th largest key (prefix), and how many of those equal to it are in (left)
  uint32_t prefix = 0, left = (uint32_t)k;
  // the bin of 256 with the left-th key from the top: the same in every warp
  auto find_bin = [&]() -> uint32_t {
    uint32_t c[8], sum = 0;  // bins from the top, eight a lane
    const uint4 h1 = *reinterpret_cast<const uint4*>(s_hist + 252 - 8 * lane);
    const uint4 h0 = *reinterpret_cast<const uint4*>(s_hist + 248 - 8 * lane);
    c[0] = h1.w, c[1] = h1.z, c[2] = h1.y, c[3] = h1.x;
    c[4] = h0.w, c[5] = h0.z, c[6] = h0.y, c[7] = h0.x;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += c[j];
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += y;
    }
    uint32_t above = inc - sum, bin = 0, rest = 0;
    const int src = __ffs(__ballot_sync(kFull, above < left && left <= inc)) - 1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (above < left && left <= above + c[j]) {
        bin = 255 - (8 * lane + j);
        rest = left - above;
      }
      above += c[j];
    }
    left = __shfl_sync(kFull, rest, src);
    return __shfl_sync(kFull, bin, src);
  };
  // A monotone map: x - low, the product and the truncation are monotone each.  Where the range
  // overflows or vanishes, NaN and infinity still convert to bins that keep the order.
  const float low = least <= most ? score_of(least) : 0.f;
  const float width = least <= most ? score_of(most) - low : INFINITY;
  const float scale = 255.f / width;
  auto bin_of = [&](uint32_t v) -> uint32_t {
    if (v >= 0xfffffffeu) return 255u;
    return (uint32_t)min(max(__float2int_rz((score_of(v) - low) * scale), 0), 255);
  };
  each([&](int, uint32_t v) {
    if (v) atomicAdd(&s_hist[bin_of(v)], 1u);
  });
  __syncthreads();
  const uint32_t bin = find_bin();
  const int cand = (int)s_hist[bin];
  if (cand <= kSelectRank) {
    each([&](int, uint32_t v) {
      if (v && bin_of(v) == bin) s_cand[atomicAdd(&s_num, 1u)] = v;
    });
    __syncthreads();
    for (int c = tid; c < cand; c += THREADS) {  // rank each against all
      const uint32_t v = s_cand[c];
      uint32_t above = 0, equal = 0;
#pragma unroll 8
      for (int j = 0; j < cand; ++j) {
        const uint32_t y = s_cand[j];
        above += y > v;
        equal += y == v;
      }
      if (above < left && left <= above + equal) {  // equal keys write the same
        s_prefix = v;
        s_left = left - above;
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
  } else {  // its bytes from the top, among the keys that share those above
    left = (uint32_t)k;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      for (int e = tid; e < 256; e += THREADS) s_hist[e] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
      each([&](int, uint32_t v) {
        if (v && (v & mask) == prefix) atomicAdd(&s_hist[(v >> shift) & 255], 1u);
      });
      __syncthreads();
      prefix |= find_bin() << shift;
    }
  }

  // ---- ascending pages: those above the key, and the first `left` equal to it
  int above = 0, equal = 0;
  each([&](int, uint32_t v) {
    above += v > prefix;
    equal += v == prefix;
  });
  above = __reduce_add_sync(kFull, above);
  equal = __reduce_add_sync(kFull, equal);
  if (lane == 0) s_cnt[warp] = make_int2(above, equal);
  __syncthreads();
  int at = 0, eq = 0;  // pages above and equal before this warp's run
  for (int w = 0; w < warp; ++w) {
    at += s_cnt[w].x;
    eq += s_cnt[w].y;
  }
  const unsigned below = (1u << lane) - 1;
  each([&](int e, uint32_t v) {
    const unsigned gt = __ballot_sync(kFull, v > prefix);
    const unsigned same = __ballot_sync(kFull, v == prefix);
    const int rank = eq + __popc(same & below);
    const bool take = v > prefix || (v == prefix && rank < (int)left);
    if (take) out[at + __popc(gt & below) + min(rank, (int)left)] = e;
    at += __popc(gt);
    eq += __popc(same);
  });
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_update_bounds(const pa_config* cfg, const void* k_new,
                                      const int32_t* block_tables, const int32_t* context_lens,
                                      const int32_t* q_lens, void* k_bounds, int32_t* flags,
                                      pa_stream stream) {
  if (!cfg || !k_new || !block_tables || !context_lens || !q_lens || !k_bounds)
    return PA_ERR_INVALID_ARG;
  const pa_config& c = *cfg;
  if (c.batch < 1 || c.max_q_len < 1 || c.num_kv_heads < 1 || c.max_blocks_per_seq < 1 ||
      c.num_blocks < 1 || c.head_dim < 1 || c.block_size < 1)
    return PA_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(k_bounds, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(q_lens, 4) || !aligned(flags, 4))
    return PA_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (!page_size_ok(c.block_size)) return PA_ERR_UNSUPPORTED;
  if (c.q_dtype != PA_BF16 && c.q_dtype != PA_FP16) return PA_ERR_UNSUPPORTED;
  const double ctas = (double)c.batch * pages_touched(c) * c.num_kv_heads;
  if (ctas > INT32_MAX) return PA_ERR_UNSUPPORTED;
  BoundsParams p;
  p.t = touch_params(c, block_tables, context_lens, q_lens, flags);
  p.k_new = static_cast<const char*>(k_new);
  p.bounds = static_cast<char*>(k_bounds);
  const bool half = c.q_dtype == PA_FP16;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](void (*kernel)(BoundsParams)) {
    return launch_pdl(kernel, p, dim3((unsigned)ctas), kBoundsThreads, 0, s);
  };
  cudaError_t e;
  switch (c.head_dim) {
    case 64: e = go(half ? bounds_kernel<64, Q_FP16> : bounds_kernel<64, Q_BF16>); break;
    case 128: e = go(half ? bounds_kernel<128, Q_FP16> : bounds_kernel<128, Q_BF16>); break;
    default: e = go(half ? bounds_kernel<256, Q_FP16> : bounds_kernel<256, Q_BF16>); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status pa_score_blocks(const pa_config* cfg, const void* q, const void* k_bounds,
                                     const int32_t* block_tables, const int32_t* context_lens,
                                     const int32_t* q_lens, float* scores, int32_t* flags,
                                     pa_stream stream) {
  if (!cfg || !q || !k_bounds || !block_tables || !context_lens || !q_lens || !scores)
    return PA_ERR_INVALID_ARG;
  const pa_config& c = *cfg;
  if (c.batch < 1 || c.max_q_len < 1 || c.num_q_heads < 1 || c.num_kv_heads < 1 ||
      c.max_blocks_per_seq < 1 || c.num_blocks < 1 || c.head_dim < 1 || c.block_size < 1)
    return PA_ERR_INVALID_ARG;
  if ((c.causal != 0 && c.causal != 1) || !std::isfinite(c.sm_scale)) return PA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_bounds, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(q_lens, 4) || !aligned(scores, 4) || !aligned(flags, 4))
    return PA_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (!page_size_ok(c.block_size) || c.num_q_heads % c.num_kv_heads != 0) return PA_ERR_UNSUPPORTED;
  if (c.q_dtype != PA_BF16 && c.q_dtype != PA_FP16) return PA_ERR_UNSUPPORTED;
  const int G = c.num_q_heads / c.num_kv_heads;
  if ((long long)c.max_blocks_per_seq * c.block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;

  ScoreParams p;
  p.q = static_cast<const char*>(q);
  p.bounds = static_cast<const char*>(k_bounds);
  p.bt = block_tables;
  p.ctx = context_lens;
  p.qlens = q_lens;
  p.scores = scores;
  p.flags = flags;
  p.Sq = c.max_q_len;
  p.Hq = c.num_q_heads;
  p.Hkv = c.num_kv_heads;
  p.G = G;
  p.bs_shift = ilog2((uint32_t)c.block_size);
  p.maxb = c.max_blocks_per_seq;
  p.nblocks = c.num_blocks;
  p.causal = c.causal;
  p.sm_scale = c.sm_scale;
  const bool packed = G == 1 || G == 2 || G == 4 || G == 8;
  p.tpt = packed ? 16 / G : 1;
  p.g_shift = packed ? ilog2((uint32_t)G) : -1;
  p.parts = ceil_div(G, 16);
  if (p.tpt > c.max_q_len) p.tpt = c.max_q_len;
  p.tok_groups = ceil_div(c.max_q_len, p.tpt);
  if ((double)c.batch * c.num_kv_heads * p.tok_groups > INT32_MAX) return PA_ERR_UNSUPPORTED;
  // pages of a warp: as many as leave the GPU kScoreWarpsPerSm warps an SM, 256 at most
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  const int all = ceil_div(c.max_blocks_per_seq, 8);
  const double per = (double)c.batch * c.num_kv_heads * p.tok_groups * all / (kScoreWarpsPerSm * sms);
  p.groups = per < 1. ? 1 : per > kScoreMaxGroups ? kScoreMaxGroups : (int)per;
  p.runs = ceil_div(all, p.groups);
  p.batch = c.batch;
  const double warps = (double)c.batch * c.num_kv_heads * p.tok_groups * p.runs;
  if (warps > INT32_MAX) return PA_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(((long long)warps + kScoreWarps - 1) / kScoreWarps));
  static std::atomic<uint64_t> done[6];  // devices whose shared-memory limit is raised
  auto go = [&](void (*kernel)(ScoreParams), std::atomic<uint64_t>& d, int smem) {
    const cudaError_t e = set_smem_attr_once(d, reinterpret_cast<const void*>(kernel), smem);
    return e != cudaSuccess ? e
                            : launch_pdl(kernel, p, grid, kScoreWarps * 32, (size_t)smem,
                                         reinterpret_cast<cudaStream_t>(stream));
  };
  const bool half = c.q_dtype == PA_FP16;
  cudaError_t e;
  switch (c.head_dim) {
    case 64:
      e = half ? go(score_kernel<64, Q_FP16>, done[0], ScoreSmem<64>::BYTES)
               : go(score_kernel<64, Q_BF16>, done[1], ScoreSmem<64>::BYTES);
      break;
    case 128:
      e = half ? go(score_kernel<128, Q_FP16>, done[2], ScoreSmem<128>::BYTES)
               : go(score_kernel<128, Q_BF16>, done[3], ScoreSmem<128>::BYTES);
      break;
    default:
      e = half ? go(score_kernel<256, Q_FP16>, done[4], ScoreSmem<256>::BYTES)
               : go(score_kernel<256, Q_BF16>, done[5], ScoreSmem<256>::BYTES);
      break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status pa_select_blocks(const pa_config* cfg, const float* scores,
                                      const int32_t* context_lens, const int32_t* q_lens,
                                      int32_t top_k, int32_t num_first, int32_t num_last,
                                      int32_t* selected, int32_t* num_selected, int32_t* flags,
                                      pa_stream stream) {
  if (!cfg || !scores || !context_lens || !q_lens || !selected || !num_selected)
    return PA_ERR_INVALID_ARG;
  const pa_config& c = *cfg;
  if (c.batch < 1 || c.max_q_len < 1 || c.num_kv_heads < 1 || c.max_blocks_per_seq < 1 ||
      c.block_size < 1 || (c.causal != 0 && c.causal != 1))
    return PA_ERR_INVALID_ARG;
  if (top_k < 1 || num_first < 0 || num_last < 0 || (long long)num_first + num_last > top_k)
    return PA_ERR_INVALID_ARG;
  if (!aligned(scores, 4) || !aligned(context_lens, 4) || !aligned(q_lens, 4) ||
      !aligned(selected, 4) || !aligned(num_selected, 4) || !aligned(flags, 4))
    return PA_ERR_INVALID_ARG;
  if (!page_size_ok(c.block_size)) return PA_ERR_UNSUPPORTED;
  const double rows = (double)c.batch * c.max_q_len * c.num_kv_heads;
  if (rows > INT32_MAX || (long long)c.max_blocks_per_seq * c.block_size > INT32_MAX)
    return PA_ERR_UNSUPPORTED;
  SelectParams p;
  p.scores = scores;
  p.ctx = context_lens;
  p.qlens = q_lens;
  p.selected = selected;
  p.num = num_selected;
  p.flags = flags;
  p.Sq = c.max_q_len;
  p.Hkv = c.num_kv_heads;
  p.bs_shift = ilog2((uint32_t)c.block_size);
  p.maxb = c.max_blocks_per_seq;
  p.causal = c.causal;
  p.top_k = top_k;
  p.first = num_first;
  p.last = num_last;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](void (*kernel)(SelectParams), int threads, size_t smem) {
    return launch_pdl(kernel, p, dim3((unsigned)rows), threads, smem, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  };
  // Rows of 256 and 2,048 columns, 1,024 of them: 6.1 and 13.7 us with 2 and 8 groups of registers a
  // warp, 8.2 us for the first with 8, 15.3 us for the second from shared memory.  Longer rows
  // take 1,024 threads, 32 rows of 2,049 and 8,192 columns 6.5 and 9.9 us and 7.3 and 18.0 us with 256,
  // unless there are more rows than SMs: 1,024 rows 41 and 64 us, 16.4 and 42 us with 256 threads;
  // at 32,768 columns 251 us and 662 us.  Keys made again in each pass, 32 rows of 32,768: 33.9 us
  // for 25.6 us.
  if (c.max_blocks_per_seq <= 2 * 256) return go(select_kernel<2, 256>, 256, 0);
  if (c.max_blocks_per_seq <= 8 * 256) return go(select_kernel<8, 256>, 256, 0);
  if (c.max_blocks_per_seq > kSelectKeys) return go(select_kernel<kKeysAgain, 1024>, 1024, 0);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  const size_t smem = (size_t)c.max_blocks_per_seq * 4;
  if (c.max_blocks_per_seq <= 32 * 256 && rows > sms)  // (32 KB of keys at most: no raised limit)
    return go(select_kernel<kKeysShared, 256>, 256, smem);
  static std::atomic<uint64_t> done{0};  // devices whose shared-memory limit is raised
  void (*const kernel)(SelectParams) = select_kernel<kKeysShared, 1024>;
  if (set_smem_attr_once(done, reinterpret_cast<const void*>(kernel), kSelectKeys * 4) != cudaSuccess)
    return PA_ERR_CUDA;
  return go(kernel, 1024, smem);
}
