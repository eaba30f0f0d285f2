// Channel bounds of the pages' keys, scores of a sequence's pages from them, and the selection of
// the best pages.
//
// Bounds.  One CTA per (sequence, touched page, kv head): the least and largest value of each
// channel over the new rows, joined with the page's older bounds unless it is fresh.
//
// Score.  For a page with channel bounds lo, hi and a query row q no key k of the page (lo_d <=
// k_d <= hi_d) has <q, k> above sum_d max(q_d lo_d, q_d hi_d), and that is one dot product of
// length 2 D: sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d.  So the scores are a matrix product of
// the query rows with the pages' bounds, on mma.sync m16n8k16 with fp32 accumulation (products of
// 16-bit values are exact): 16 query rows by 8 pages.  A quad's four lanes read their page's
// bounds straight from global memory in 16-byte pieces; with the contraction's order permuted
// alike on both sides (a lane's 8 channels of a piece are 4 of one k-step and 4 of the next) the
// pieces are the B fragments as they land, so nothing is staged.  The query rows wait in shared
// memory in fragment order; a step's max(q, 0) and min(q, 0) are one instruction each.
// What bounds it is the 4 D bytes of a (page, head).
//
// Row tiles hold whole query tokens: 16 / G tokens of G heads for G <= 16 (the rows of a token
// are then reduced to their maximum through shared memory), or ceil(G / 16) tiles for one token.
//
// Select.  One CTA per row: scores become order-preserving 32-bit keys in shared memory, four
// passes over 8 bits each find the k-th largest key, and one ordered pass writes the pages above
// it and the first of those equal to it.
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
constexpr int kBoundsThreads = 256;

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
  TouchedPage t;
  if (!touched_page(p.t, b, j, tid == 0 && g == 0, &t)) return;
  const size_t row_stride = (size_t)p.t.Hkv * D;
  const uint4* src = reinterpret_cast<const uint4*>(
                         p.k_new + (((size_t)b * p.t.Sq + t.i0) * row_stride + (size_t)g * D) * 2) + c;
  uint4 lo, hi;
  if (rg < t.rows) {
    lo = hi = __ldg(src + (size_t)rg * (row_stride / 8));
#pragma unroll 4
    for (int r = rg + RG; r < t.rows; r += RG) {
      const uint4 x = __ldg(src + (size_t)r * (row_stride / 8));
      lo = extreme8<QK, false>(lo, x);
      hi = extreme8<QK, true>(hi, x);
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
constexpr int kScoreMaxTiles = 8;  // row tiles whose query rows fit one CTA

struct ScoreParams {
  const char* q;
  const char* bounds;
  const int32_t* bt;
  const int32_t* ctx;
  const int32_t* qlens;
  float* scores;
  int32_t* flags;
  int Sq, Hq, Hkv, G, bs_shift, maxb, nblocks, causal;
  int tpt;         // tokens per row tile (G <= 16), else 0
  int tiles_tok;   // row tiles per token (G > 16), else 1
  int toks_cta;    // tokens of one CTA
  int tok_groups;  // CTAs along the tokens
  int groups_cta;  // groups of 8 pages each warp takes
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

template <int D, int QK>
__global__ void __launch_bounds__(kScoreWarps * 32) score_kernel(const ScoreParams p) {
  constexpr int NP = D / 32;  // 16-byte pieces a lane holds of each bound: two k-steps each
  constexpr int KSTEPS = D / 16;
  // query rows in A fragment order: [tile][k-step][lane] (a0..a3)
  extern __shared__ uint4 s_q[];
  __shared__ float s_c[kScoreWarps][16][9];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, qi = lane & 3;
  const int g = blockIdx.y, b = blockIdx.z;
  const int tg = blockIdx.x % p.tok_groups, pg = blockIdx.x / p.tok_groups;
  const int tok0 = tg * p.toks_cta, toks = min(p.toks_cta, p.Sq - tok0);
  const int tiles = p.tpt ? ceil_div(toks, p.tpt) : toks * p.tiles_tok;
  grid_dependency_wait();
  grid_dependents_launch();

  const int page0 = pg * kScoreWarps * p.groups_cta * 8;  // this CTA's first page
  const int page_end = min(p.maxb, page0 + kScoreWarps * p.groups_cta * 8);
  // keys that any row of this CTA sees
  const int ql = __ldg(p.qlens + b);
  int most = keys_seen(p.ctx, p.qlens, b, 0, p.Sq, p.maxb, p.bs_shift, 0);
  const bool bad = most < 0;
  if (bad || tok0 >= ql) {
    if (bad && tid == 0 && blockIdx.x == 0 && g == 0 && p.flags)
      atomicOr(p.flags, PA_FLAG_BAD_LENGTHS);
    most = 0;
  } else if (p.causal) {
    most = most - ql + min(tok0 + toks, ql);
  }
  const int npages = pages_of(most, p.bs_shift);
  float* const out = p.scores + (((size_t)b * p.Sq + tok0) * p.Hkv + g) * p.maxb;
  const size_t tok_stride = (size_t)p.Hkv * p.maxb;

  if (page0 < npages) {
    // fragment (tile, k-step, lane): rows quad and quad + 8 of the tile, channels
    // 32 (k-step / 2) + 8 qi + 4 (k-step & 1) + {0, 1} and {2, 3}
    for (int e = tid; e < tiles * KSTEPS * 32; e += kScoreWarps * 32) {
      const int l = e & 31, ks = (e >> 5) % KSTEPS, tile = (e >> 5) / KSTEPS;
      uint32_t a[2][2] = {{0, 0}, {0, 0}};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = (l >> 2) + 8 * h;
        int t, head;
        bool real;
        if (p.tpt) {
          t = tile * p.tpt + r / p.G;
          head = r % p.G;
          real = r / p.G < p.tpt && t < toks;
        } else {
          t = tile / p.tiles_tok;
          head = (tile % p.tiles_tok) * 16 + r;
          real = head < p.G;
        }
        if (real) {
          const char* row = p.q + ((((size_t)b * p.Sq + tok0 + t) * p.Hq + (size_t)g * p.G + head) * D) * 2;
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(
              row + (32 * (ks >> 1) + 8 * (l & 3) + 4 * (ks & 1)) * 2));
          a[h][0] = v.x;
          a[h][1] = v.y;
        }
      }
      s_q[e] = make_uint4(a[0][0], a[1][0], a[0][1], a[1][1]);
    }
  }
  __syncthreads();

  for (int gi = 0; gi < p.groups_cta; ++gi) {
    const int pbase = page0 + (gi * kScoreWarps + warp) * 8;
    if (pbase >= page_end) break;
    const int page = pbase + quad;  // this lane's B column
    uint4 lo[NP], hi[NP];
    bool ok = false;
    if (page < npages) {
      const int blk = __ldg(p.bt + (size_t)b * p.maxb + page);
      ok = blk >= 0 && blk < p.nblocks;
      if (ok) {
        const uint4* box = reinterpret_cast<const uint4*>(p.bounds + ((size_t)blk * p.Hkv + g) * 2 * D * 2);
#pragma unroll
        for (int t = 0; t < NP; ++t) {
          lo[t] = __ldg(box + 4 * t + qi);
          hi[t] = __ldg(box + D / 8 + 4 * t + qi);
        }
      } else if (qi == 0 && p.flags) {
        atomicOr(p.flags, PA_FLAG_BAD_BLOCK_ID);
      }
    }
    if (!ok) {
#pragma unroll
      for (int t = 0; t < NP; ++t) lo[t] = hi[t] = make_uint4(0, 0, 0, 0);
    }
    const unsigned ok_mask = __ballot_sync(kFull, ok);  // bit 4 c: page c of the group
    float best[2] = {-INFINITY, -INFINITY};             // G > 16: over the token's tiles so far
    // whether row t of this CTA sees page pbase + col, and the score that goes out
    auto put = [&](int t, int col, float v) {
      const int seen = bad ? 0 : keys_seen(p.ctx, p.qlens, b, tok0 + t, p.Sq, p.maxb, p.bs_shift, p.causal);
      const bool in = pbase + col < pages_of(seen, p.bs_shift) && ((ok_mask >> (4 * col)) & 1);
      out[t * tok_stride + pbase + col] = in ? v : -INFINITY;
    };
    for (int tile = 0; tile < tiles; ++tile) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
      if (pbase < npages) {
#pragma unroll
        for (int t = 0; t < NP; ++t) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 a = s_q[(tile * KSTEPS + 2 * t + h) * 32 + lane];
            const uint32_t up[4] = {extreme2<QK, true>(a.x, 0u), extreme2<QK, true>(a.y, 0u),
                                    extreme2<QK, true>(a.z, 0u), extreme2<QK, true>(a.w, 0u)};
            const uint32_t dn[4] = {extreme2<QK, false>(a.x, 0u), extreme2<QK, false>(a.y, 0u),
                                    extreme2<QK, false>(a.z, 0u), extreme2<QK, false>(a.w, 0u)};
            score_mma<QK>(c, up, h ? hi[t].z : hi[t].x, h ? hi[t].w : hi[t].y);
            score_mma<QK>(c, dn, h ? lo[t].z : lo[t].x, h ? lo[t].w : lo[t].y);
          }
        }
      }
      // c: rows quad, quad + 8 of pages pbase + 2 qi, + 1
      if (p.tpt) {
        __syncwarp();
        s_c[warp][quad][2 * qi] = c[0] * p.sm_scale;
        s_c[warp][quad][2 * qi + 1] = c[1] * p.sm_scale;
        s_c[warp][quad + 8][2 * qi] = c[2] * p.sm_scale;
        s_c[warp][quad + 8][2 * qi + 1] = c[3] * p.sm_scale;
        __syncwarp();
        for (int e = lane; e < p.tpt * 8; e += 32) {
          const int tt = e >> 3, col = e & 7, t = tile * p.tpt + tt;
          if (t >= toks || pbase + col >= page_end) continue;
          float v = s_c[warp][tt * p.G][col];
          for (int h = 1; h < p.G; ++h) v = max_nan(v, s_c[warp][tt * p.G + h][col]);
          put(t, col, v);
        }
      } else {
        const int part = tile % p.tiles_tok;
        if (part == 0) best[0] = best[1] = -INFINITY;
        if (part * 16 + quad < p.G) {
          best[0] = max_nan(best[0], c[0] * p.sm_scale);
          best[1] = max_nan(best[1], c[1] * p.sm_scale);
        }
        if (part * 16 + quad + 8 < p.G) {
          best[0] = max_nan(best[0], c[2] * p.sm_scale);
          best[1] = max_nan(best[1], c[3] * p.sm_scale);
        }
        if (part + 1 == p.tiles_tok) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            best[0] = max_nan(best[0], __shfl_xor_sync(kFull, best[0], o));
            best[1] = max_nan(best[1], __shfl_xor_sync(kFull, best[1], o));
          }
          const int col = 2 * qi + quad;
          if (quad < 2 && pbase + col < page_end) put(tile / p.tiles_tok, col, quad ? best[1] : best[0]);
        }
      }
    }
  }
}

// ---- select ------------------------------------------------------------------------------
constexpr int kSelectThreads = 256;
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

template <bool CACHED>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectParams p) {
  constexpr int NW = kSelectThreads / 32;
  extern __shared__ uint32_t s_key[];
  __shared__ uint32_t s_hist[256];
  __shared__ uint32_t s_prefix, s_left;
  __shared__ int2 s_cnt[NW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t row = blockIdx.x;
  const int i = (int)((row / p.Hkv) % p.Sq), b = (int)(row / ((size_t)p.Hkv * p.Sq));
  grid_dependency_wait();
  grid_dependents_launch();
  int seen = keys_seen(p.ctx, p.qlens, b, i, p.Sq, p.maxb, p.bs_shift, p.causal);
  if (seen < 0) {
    if (tid == 0 && i == 0 && row % p.Hkv == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_LENGTHS);
    seen = 0;
  }
  const int N = pages_of(seen, p.bs_shift), k = min(p.top_k, N);
  int32_t* out = p.selected + row * p.top_k;
  if (tid == 0) p.num[row] = k;
  for (int e = k + tid; e < p.top_k; e += kSelectThreads) out[e] = -1;
  if (N <= p.top_k) {
    for (int e = tid; e < N; e += kSelectThreads) out[e] = e;
    return;
  }
  const float* x = p.scores + row * p.maxb;
  const int hi_first = N - p.last;
  auto key = [&](int e) -> uint32_t {
    if constexpr (CACHED) return s_key[e];
    return key_of(__ldg(x + e), e < p.first || e >= hi_first);
  };
  if constexpr (CACHED)
    for (int e = tid; e < N; e += kSelectThreads)
      s_key[e] = key_of(__ldg(x + e), e < p.first || e >= hi_first);

  // ---- the k-th largest key: its bytes from the top, among the keys that share those above
  uint32_t prefix = 0, left = (uint32_t)k;  // left: how many of the keys with `prefix` are in
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int e = tid; e < 256; e += kSelectThreads) s_hist[e] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
    for (int e = tid; e < N; e += kSelectThreads) {
      const uint32_t v = key(e);
      if ((v & mask) == prefix) atomicAdd(&s_hist[(v >> shift) & 255], 1u);
    }
    __syncthreads();
    if (warp == 0) {  // bins from the top, eight a lane
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += c[j] = s_hist[255 - (8 * lane + j)];
      uint32_t inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += y;
      }
      uint32_t above = inc - sum;
      if (above < left && left <= inc) {  // one lane
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (above < left && left <= above + c[j]) {
            s_prefix = prefix | (uint32_t)(255 - (8 * lane + j)) << shift;
            s_left = left - above;
          }
          above += c[j];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
  }

  // ---- ascending pages: those above the key, and the first `left` equal to it
  const int per = round_up(ceil_div(N, NW), 32);  // a warp's run of pages
  const int e0 = min(warp * per, N), e1 = min(e0 + per, N);
  int above = 0, equal = 0;
  for (int e = e0 + lane; e < e1; e += 32) {
    const uint32_t v = key(e);
    above += v > prefix;
    equal += v == prefix;
  }
  above = __reduce_add_sync(kFull, above);
  equal = __reduce_add_sync(kFull, equal);
  if (lane == 0) s_cnt[warp] = make_int2(above, equal);
  __syncthreads();
  int at = 0, eq = 0;  // pages above and equal before this warp's run
  for (int w = 0; w < warp; ++w) {
    at += s_cnt[w].x;
    eq += s_cnt[w].y;
  }
  for (int base = e0; base < e1; base += 32) {
    const int e = base + lane;
    const uint32_t v = e < e1 ? key(e) : 0u;
    const unsigned gt = __ballot_sync(kFull, e < e1 && v > prefix);
    const unsigned same = __ballot_sync(kFull, e < e1 && v == prefix);
    const unsigned below = (1u << lane) - 1;
    const int rank = eq + __popc(same & below);
    const bool take = ((gt >> lane) & 1) || (((same >> lane) & 1) && rank < (int)left);
    if (take) out[at + __popc(gt & below) + min(rank, (int)left)] = e;
    at += __popc(gt);
    eq += __popc(same);
  }
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
  if (c.batch > 65535 || c.num_kv_heads > 65535 || G > 16 * kScoreMaxTiles ||
      (long long)c.max_blocks_per_seq * c.block_size > INT32_MAX)
    return PA_ERR_UNSUPPORTED;

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
  p.tpt = G <= 16 ? 16 / G : 0;
  p.tiles_tok = G <= 16 ? 1 : ceil_div(G, 16);
  p.toks_cta = p.tpt ? kScoreMaxTiles * p.tpt : kScoreMaxTiles / p.tiles_tok;
  p.toks_cta = p.toks_cta < c.max_q_len ? p.toks_cta : c.max_q_len;
  p.tok_groups = ceil_div(c.max_q_len, p.toks_cta);
  p.groups_cta = 4;
  const long long gx = (long long)ceil_div(c.max_blocks_per_seq, kScoreWarps * 8 * p.groups_cta) * p.tok_groups;
  if (gx > INT32_MAX) return PA_ERR_UNSUPPORTED;
  const int tiles = p.tpt ? ceil_div(p.toks_cta, p.tpt) : p.toks_cta * p.tiles_tok;
  const dim3 grid((unsigned)gx, c.num_kv_heads, c.batch);
  const int tile_bytes = (c.head_dim / 16) * 32 * (int)sizeof(uint4);
  static std::atomic<uint64_t> done[6];  // devices whose shared-memory limit is raised
  auto go = [&](void (*kernel)(ScoreParams), std::atomic<uint64_t>& d) {
    const cudaError_t e = set_smem_attr_once(d, reinterpret_cast<const void*>(kernel), kScoreMaxTiles * tile_bytes);
    return e != cudaSuccess ? e
                            : launch_pdl(kernel, p, grid, kScoreWarps * 32, (size_t)tiles * tile_bytes,
                                         reinterpret_cast<cudaStream_t>(stream));
  };
  const bool half = c.q_dtype == PA_FP16;
  cudaError_t e;
  switch (c.head_dim) {
    case 64: e = half ? go(score_kernel<64, Q_FP16>, done[0]) : go(score_kernel<64, Q_BF16>, done[1]); break;
    case 128: e = half ? go(score_kernel<128, Q_FP16>, done[2]) : go(score_kernel<128, Q_BF16>, done[3]); break;
    default: e = half ? go(score_kernel<256, Q_FP16>, done[4]) : go(score_kernel<256, Q_BF16>, done[5]); break;
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
  const dim3 grid((unsigned)rows);
  if (c.max_blocks_per_seq > kSelectKeys)
    return launch_pdl(select_kernel<false>, p, grid, kSelectThreads, 0, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  static std::atomic<uint64_t> done{0};  // devices whose shared-memory limit is raised
  if (set_smem_attr_once(done, reinterpret_cast<const void*>(select_kernel<true>), kSelectKeys * 4) != cudaSuccess)
    return PA_ERR_CUDA;
  return launch_pdl(select_kernel<true>, p, grid, kSelectThreads, (size_t)c.max_blocks_per_seq * 4, s) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}
