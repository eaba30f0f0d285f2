// Attention of each row over a list of its pages (pa_decode_selected): one launch, no workspace.
//
// A unit of work is one new token of one sequence and one kv head with up to 16 of its query
// heads: they share the page list.  The list's 16-token chunks (a page holds a whole number of
// them) are dealt out in tiles to the warps of a thread-block cluster of S CTAs, S chosen from the
// sizes so that few units still spread over the GPU.  A warp looks up 32 chunks of its share at a
// time (a lane each: list entry, then block table) and streams them (page_stream.cuh).  At the end
// the warps' states are merged through shared memory, and the CTAs' through distributed shared
// memory, both in a fixed order.
//   Measured: 32 sequences with 8 kv heads of 128 and 64 pages of 16 tokens each (16-bit, 135 MB) 24.5
// us, 81 % of the copy rate, bound by the data of one wave of CTAs with its start and merge (256 units
// on 304 places: 104 SMs hold two of them, 48 one); 4 sequences with one kv head and 32 pages of 64
// (fp8, 2 MB) 7.6 us, a chain of list, block table, scales, first copies, two merges.
#pragma once

#include <cooperative_groups.h>

#include "page_stream.cuh"

namespace pa {

struct SelectedParams {
  CacheView cache;
  const char* q;
  const int32_t* bt;
  const int32_t* ctx;
  const int32_t* qlens;
  const int32_t* selected;
  const int32_t* num;
  void* out;
  float* lse;
  int32_t* flags;
  int Sq, Hq, Hkv, G, RB, maxb, nblocks, causal, top_k, split;
  float qk_scale;  // sm_scale * log2(e)
};

// CTAs of a unit's cluster: as many as leave all CTAs resident at once (`slots` at a time), each
// with 128 tokens or more.  A second wave costs its CTAs' start (four dependent loads before the
// first key arrives) more than a fuller first one gains: 64 units of 12,288 fp8 tokens took 46 us
// in clusters of 8 (1.7 waves).
constexpr int kSelMaxSplit = 8;
inline int selected_split(long long units, long long tokens, long long slots) {
  long long s = slots / units;
  if (s > tokens / 128) s = tokens / 128;
  return (int)(s < 1 ? 1 : s > kSelMaxSplit ? kSelMaxSplit : s);
}

// Shared memory: the warps' rings, then (after them) the warps' states and the merged one, in the
// same place; the states' maxima and sums, and the fp8 stages' chunks and barriers.
template <class T>
struct SelectedSmem {
  static constexpr int OFF_ML = round_up(cmax(T::RING, (T::NW + 1) * T::O_SLOT), 128);
  static constexpr int OFF_META = OFF_ML + (T::NW + 1) * T::ROWS * 8;
  static constexpr int OFF_BAR = OFF_META + T::NW * T::NST * T::META;
  static constexpr int BYTES = OFF_BAR + (T::FP8 ? T::NW * T::NST * 8 + 1024 : 0);  // + alignment
  static constexpr int CTAS_PER_SM = 2 * (BYTES + 1024) <= 228 * 1024 ? 2 : 1;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

template <class T>
__global__ void __launch_bounds__(T::NTHREADS, SelectedSmem<T>::CTAS_PER_SM)
    decode_selected_kernel(const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap, const SelectedParams p) {
  using M = SelectedSmem<T>;
  constexpr int SUB = T::SUB, ROWS = T::ROWS, D = T::D;
  extern __shared__ __align__(128) char smem_raw[];
  char* const smem = T::FP8 ? smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023) : smem_raw;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, qi = lane & 3;
  const int S = p.split, rank = blockIdx.x % S;
  int u = blockIdx.x / S;
  const int rb = u % p.RB;
  u /= p.RB;  // (b * Sq + i) * Hkv + g
  const int g = u % p.Hkv, bi = u / p.Hkv, i = bi % p.Sq, b = bi / p.Sq;
  char* const ring = smem + warp * T::NST * T::STAGE;
  const uint32_t ring_addr = smem_addr(ring);
  char* const meta = smem + M::OFF_META + warp * T::NST * T::META;
  uint64_t* const bar = reinterpret_cast<uint64_t*>(smem + M::OFF_BAR) + warp * T::NST;
  if constexpr (T::FP8) {  // (a warp's barriers are its own)
    if (lane == 0) {
      for (int s = 0; s < T::NST; ++s) mbar_init(&bar[s], kStreamArrivals<T>);
      fence_barrier_init();
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
    }
    __syncwarp();
  }
  grid_dependency_wait();
  grid_dependents_launch();

  // ---- what the row sees, and its list
  const int bs_shift = p.cache.bs_shift;
  const int n = __ldg(p.ctx + b), ql = __ldg(p.qlens + b), listed = __ldg(p.num + u);
  int L = 0, npages = 0;
  if (ql < 0 || ql > p.Sq || n < ql || (long long)n > ((long long)p.maxb << bs_shift)) {
    if (tid == 0 && rank == 0 && i == 0 && g == 0 && rb == 0 && p.flags)
      atomicOr(p.flags, PA_FLAG_BAD_LENGTHS);
  } else if (i < ql) {
    L = p.causal ? n - ql + i + 1 : n;
    npages = (int)(((long long)n + (1 << bs_shift) - 1) >> bs_shift);
  }
  int count = L > 0 ? listed : 0;
  if (count < 0 || count > p.top_k) {
    if (tid == 0 && rank == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_SELECTION);
    count = count < 0 ? 0 : p.top_k;
  }
  const int cshift = bs_shift - 4;  // a page's 16-token chunks
  const long long chunks = (long long)count << cshift;
  const long long tiles = (chunks + SUB - 1) / SUB;
  const long long tile0 = tiles * rank / S, tile1 = tiles * (rank + 1) / S;
  const int my = (int)max(0ll, (tile1 - tile0 - warp + T::NW - 1) / T::NW);  // this warp's tiles
  const int32_t* list = p.selected + (size_t)u * p.top_k;

  // lane l looks up chunk base + l of the warp's chunks (SUB a tile)
  int blk = -1, base = -32;
  Chunk ch{0, 0, 0.f, 0.f};
  auto look_up = [&](int x0) {
    base = x0;
    const int x = x0 + lane;
    const long long c = (tile0 + warp + (long long)T::NW * (x / SUB)) * SUB + x % SUB;
    blk = -1;
    ch = Chunk{0, 0, 0.f, 0.f};
    if (x / SUB < my && c < chunks) {
      const int page = __ldg(list + (int)(c >> cshift));
      if (page < 0 || page >= npages) {
        if (p.flags) atomicOr(p.flags, PA_FLAG_BAD_SELECTION);
      } else {
        ch.tok = (page << bs_shift) + (((int)c & ((1 << cshift) - 1)) << 4);
        blk = __ldg(p.bt + (size_t)b * p.maxb + page);
        if (blk < 0 || blk >= p.nblocks) {
          if (p.flags) atomicOr(p.flags, PA_FLAG_BAD_BLOCK_ID);
          blk = -1;
        } else {
          ch.rows = min(max(L - ch.tok, 0), 16);
          if constexpr (T::FP8 && !T::TOKS) {
            const size_t at = (size_t)(blk * p.cache.sc_block) + (size_t)g * p.cache.sc_head;
            ch.ks = p.cache.k_scale ? __ldg(p.cache.k_scale + at) : 1.f;
            ch.vs = p.cache.v_scale ? __ldg(p.cache.v_scale + at) : 1.f;
          }
        }
      }
    }
  };
  // tile j into a stage; the 16-bit path returns, a byte a chunk, how many tokens the row sees
  auto issue = [&](int j, int st) -> uint32_t {
    uint32_t valids = 0;
    if (j < my) {
      if (j * SUB >= base + 32) look_up(j * SUB);
      const int x0 = j * SUB - base;
      if constexpr (T::FP8) {
        stream_tma<T>(p.cache, &kmap, &vmap, g, ring + st * T::STAGE, meta + st * T::META, &bar[st], blk,
                      ch, x0, lane);
      } else {
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
          Chunk c;
          c.tok = __shfl_sync(kFull, ch.tok, x0 + s);
          c.rows = __shfl_sync(kFull, ch.rows, x0 + s);
          valids |= (uint32_t)c.rows << (8 * s);
          stream_copy<T>(p.cache, g, ring_addr + st * T::STAGE, s, __shfl_sync(kFull, blk, x0 + s), c, lane);
        }
      }
    }
    if constexpr (!T::FP8) cp_async_commit();
    return valids;
  };

  WarpAttention<T> att;
  att.clear();
  if (my > 0) look_up(0);
  __syncwarp();
  static_assert(T::NST == 3, "two tiles in flight");
  uint32_t v0 = issue(0, 0), v1 = issue(1, 1);
  att.load_q(
      [&](int h) -> const char* {
        const int head = rb * ROWS + quad + 8 * h;
        return head < p.G ? p.q + (((size_t)bi * p.Hq + (size_t)g * p.G + head) * D) * 2 : nullptr;
      },
      p.qk_scale, qi);
  int st = 0;
  uint32_t phase = 0;
  for (int j = 0; j < my; ++j) {
    if constexpr (T::FP8) {
      if (!stream_wait(&bar[st], phase)) {  // copies that never came: give up on the rest
        if (p.flags) atomicOr(p.flags, PA_FLAG_WAIT_TIMEOUT);
        if (j + 1 < my) mbar_wait_drain(&bar[st == 2 ? 0 : st + 1], st == 2 ? phase ^ 1 : phase);
        break;
      }
    } else {
      cp_async_wait_group<1>();
    }
    __syncwarp();
    const uint32_t v2 = issue(j + 2, st == 0 ? 2 : st - 1);
    const uint32_t stage = ring_addr + st * T::STAGE;
    if constexpr (T::FP8) {
      const Chunk* cs = reinterpret_cast<const Chunk*>(meta + st * T::META);
      const Chunk c0 = cs[0], c1 = cs[SUB - 1];
      const bool all = c0.rows == 16 && c1.rows == 16;
      if (!all) zero_rows<T>(ring + st * T::STAGE + T::TILE, c0.rows, c1.rows, lane);
      att.tile_fp8(stage, {c0.ks, c1.ks}, {c0.vs, c1.vs},
                   reinterpret_cast<const float*>(meta + st * T::META + 32), all,
                   [&](int s, int) { return s ? c1.rows : c0.rows; }, lane);
    } else {
      att.tile_16(stage, v0 == (SUB == 2 ? 0x1010u : 0x10u),
                  [&](int s, int) { return (int)((v0 >> (8 * s)) & 255); }, lane);
      v0 = v1;
      v1 = v2;
    }
    if (++st == T::NST) {
      st = 0;
      phase ^= 1;
    }
  }
  if constexpr (!T::FP8) cp_async_wait_all();

  // ---- merge the warps
  float* const obuf = reinterpret_cast<float*>(smem);              // [NW + 1][ROWS][OSTR]
  float2* const ml = reinterpret_cast<float2*>(smem + M::OFF_ML);  // [NW + 1][ROWS] (max, sum)
  __syncthreads();  // every warp is done with its stages
  att.stage_state(obuf, ml, warp, lane);
  __syncthreads();
  constexpr int D4 = D / 4, SLOT = ROWS * T::OSTR;
  const int rows = min(ROWS, p.G - rb * ROWS);
  auto finish = [&](int r, int d4, const float4& O, const float2& state) {
    const float inv = state.y == 0.f ? 0.f : 1.f / state.y;  // no key: zero (NaN stays NaN)
    const size_t row = (size_t)bi * p.Hq + (size_t)g * p.G + rb * ROWS + r;
    store_out4<T::QK>(p.out, row * D + 4 * d4, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
    if (d4 == 0 && p.lse) p.lse[row] = state.y == 0.f ? -INFINITY : (state.x + fast_log2(state.y)) * kLn2;
  };
  for (int e = tid; e < rows * D4; e += T::NTHREADS) {
    const int r = e / D4, d4 = e % D4;
    float4 O;
    const float2 state = merge_states(T::NW, [&](int s) { return ml + s * ROWS + r; },
                                      [&](int s) { return obuf + s * SLOT + r * T::OSTR + 4 * d4; }, O);
    if (S == 1) {
      finish(r, d4, O, state);
    } else {
      *reinterpret_cast<float4*>(obuf + T::NW * SLOT + r * T::OSTR + 4 * d4) = O;
      if (d4 == 0) ml[T::NW * ROWS + r] = state;
    }
  }
  if (S == 1) return;

  // ---- merge the cluster's CTAs: each finishes its share of the rows' pieces
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int e = rank * T::NTHREADS + tid; e < rows * D4; e += S * T::NTHREADS) {
    const int r = e / D4, d4 = e % D4;
    float4 O;
    const float2 state = merge_states(
        S, [&](int s) { return cluster.map_shared_rank(ml + T::NW * ROWS + r, s); },
        [&](int s) { return cluster.map_shared_rank(obuf + T::NW * SLOT + r * T::OSTR + 4 * d4, s); }, O);
    finish(r, d4, O, state);
  }
  cluster.sync();  // nobody leaves while its shared memory is read
}

template <class T>
cudaError_t launch_selected(SelectedParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                            long long units, long long tokens, int sms, cudaStream_t s) {
  using M = SelectedSmem<T>;
  p.split = selected_split(units, tokens, (long long)sms * M::CTAS_PER_SM);
  auto kern = decode_selected_kernel<T>;
  static std::atomic<uint64_t> attr_done{0};  // devices whose limit is raised
  const cudaError_t e = set_smem_attr_once(attr_done, reinterpret_cast<const void*>(kern), M::BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * p.split));
  cfg.blockDim = dim3(T::NTHREADS);
  cfg.dynamicSmemBytes = M::BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, kmap, vmap, p);
}

// What a call runs on: types, and whether each token has a scale.
struct SelectedKind {
  int kvk, qk;
  bool toks;
  long long units, tokens;  // units of work, and the most tokens of one
  int sms;
};

template <int D>
cudaError_t launch_selected_for_dim(SelectedParams& p, const SelectedKind& k,
                                    const CUtensorMap& kmap, const CUtensorMap& vmap,
                                    cudaStream_t s) {
#define PA_SELECTED(KVK_, QK_, TOKS_)                   \
  if (k.kvk == KVK_ && k.qk == QK_ && k.toks == TOKS_)  \
    return launch_selected<StreamTraits<D, KVK_, QK_, TOKS_>>(p, kmap, vmap, k.units, k.tokens, k.sms, s);
  PA_SELECTED(KV_BF16, Q_BF16, false)
  PA_SELECTED(KV_FP16, Q_FP16, false)
  PA_SELECTED(KV_FP8, Q_BF16, false)
  PA_SELECTED(KV_FP8, Q_BF16, true)
  PA_SELECTED(KV_FP8, Q_FP16, false)
  PA_SELECTED(KV_FP8, Q_FP16, true)
#undef PA_SELECTED
  return cudaErrorNotSupported;
}

cudaError_t launch_selected_d64(SelectedParams& p, const SelectedKind& k, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, cudaStream_t s);
cudaError_t launch_selected_d128(SelectedParams& p, const SelectedKind& k, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, cudaStream_t s);
cudaError_t launch_selected_d256(SelectedParams& p, const SelectedKind& k, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, cudaStream_t s);

}  // namespace pa
