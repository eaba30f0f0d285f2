// Persistent split-KV paged decode over an fp8 cache with one scale for each (page, kv head), for
// tiles of up to 16 query rows: the planner's work list, each item streamed by the warps of a CTA
// on their own (page_stream.cuh).
//
// A CTA takes its items one after the other.  An item's 16-token chunks go in tiles of one or two to
// the four warps in turn; a lane looks up one of the warp's next 32 chunks (block table, then the
// page's two scales).  When the item ends the warps' states are merged through the shared memory
// of their rings, and the rows go out whole or, for a piece of a split unit, as a normalised
// partial and its log2-sum-exp for the reducer, exactly as the other decode kernels leave them.
//
// The first item is derived from the lengths with the planner's own arithmetic, so that its copies
// and products start while the planner may still be running; nothing is written (flags included)
// and no other item is read before the planner has finished.
//   Measured, plan, decode and reduce: 64 sequences of 8,192 to 16,384 tokens (16 heads on one kv head
// of 128, 202 MB) 43.9 us, 32 of 512 to 4,096 with four new tokens each (32 heads on 8, 153 MB) 38.2
// us (43.9 and 41.8 when a tenth of the pages have a scale 1,000 times the others').  Pages stream at 6.2 TB/s once under way, bound by what two warps a scheduler issue (0.35 of a
// slot a cycle); about 10 us are the planner, the first copies, the last items' merge and the
// reducer.  The mma.sync kernel, whose CTAs pass tiles through one ring with barriers, takes 54.1 and
// 56.7 us.
#pragma once

#include "page_stream.cuh"

namespace pa {

template <class T>
struct DecodeStreamSmem {
  static constexpr int STATES = T::NW * T::O_SLOT;
  static constexpr int OFF_ML = round_up(cmax(T::RING, STATES), 128);
  static constexpr int OFF_META = OFF_ML + cmax(T::NW * T::ROWS * 8, 2 * T::ROWS * 4);
  static constexpr int OFF_BAR = OFF_META + T::NW * T::NST * T::META;
  static constexpr int BYTES = OFF_BAR + T::NW * T::NST * 8 + 16 + 1024;  // + pending merges, alignment
  static constexpr int CTAS_PER_SM = 2 * (BYTES + 1024) <= 228 * 1024 ? 2 : 1;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

template <class T>
__global__ void __launch_bounds__(T::NTHREADS, DecodeStreamSmem<T>::CTAS_PER_SM)
    decode_stream_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const KernelParams p,
                         const CacheView cache) {
  using M = DecodeStreamSmem<T>;
  constexpr int D = T::D, ROWS = T::ROWS, NW = T::NW, SUB = T::SUB;
  static_assert(T::FP8 && !T::TOKS && T::NST == 3, "fp8 tiles, two in flight");
  extern __shared__ char smem_raw[];
  char* const smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, qi = lane & 3;
  char* const ring = smem + warp * T::NST * T::STAGE;
  const uint32_t ring_addr = smem_addr(ring);
  char* const meta = smem + M::OFF_META + warp * T::NST * T::META;
  uint64_t* const bar = reinterpret_cast<uint64_t*>(smem + M::OFF_BAR) + warp * T::NST;
  int* const pend = reinterpret_cast<int*>(smem + M::OFF_BAR + NW * T::NST * 8);  // [4]
  float* const obuf = reinterpret_cast<float*>(smem);              // [NW][ROWS][OSTR]
  float2* const ml = reinterpret_cast<float2*>(smem + M::OFF_ML);  // [NW][ROWS] (max, sum)
  const bool planning = planner_runs(p);
  if (lane == 0) {  // (a warp's barriers are its own)
    for (int s = 0; s < T::NST; ++s) mbar_init(&bar[s], kStreamArrivals<T>);
    fence_barrier_init();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (!planning) grid_dependency_wait();
  __syncwarp();
  const int4 first = first_item_of(p, blockIdx.x, gridDim.x, lane);
  int it = 0, items = 1, list = 0;  // this CTA's items begin at p.items[list]
  int4 item_next = first;
  int bad = 0;  // flags this thread has yet to raise
  auto wait_planner = [&]() {
    grid_dependency_wait();
    grid_dependents_launch();
    list = p.item_off[blockIdx.x];
    items = max(p.item_off[blockIdx.x + 1] - list, 1);
    const int4 f = p.first_item[blockIdx.x];
    if (f.x != first.x || f.y != first.y || f.z != first.z || f.w != first.w) bad |= PA_FLAG_STALE_PLAN;
  };
  int2 pend_even = make_int2(-1, 0), pend_odd = make_int2(-1, 0);  // held by thread 0
  int st = 0;  // stage of the warp's next tile to read, and its barrier's phase
  uint32_t phase = 0;
  bool failed = false;  // copies that never came: this warp reads no more
  for (; it < items; ++it) {
    const int4 item = item_next;
    if (it > 0 && it + 1 < items) item_next = p.items[list + it + 1];
    const int u = item.x, t0 = item.y, t1 = item.z, slot = item.w;
    if (t1 <= t0) {
      if (it == 0) {
        wait_planner();
        if (items > 1) item_next = p.items[list + 1];
      }
      continue;
    }
    const int b = u / (p.Hkv * p.RB), g = (u / p.RB) % p.Hkv, rb = u % p.RB;
    const int n = __ldg(p.ctx + b), ql = __ldg(p.qlens + b);
    const int chunks = (t1 - t0 + 15) >> 4, tiles = (chunks + SUB - 1) / SUB;
    const int my = failed ? 0 : (tiles - warp + NW - 1) / NW;  // this warp's tiles

    // lane l looks up chunk base + l of the warp's chunks (SUB a tile)
    int blk = -1, base = -32;
    Chunk ch{0, 0, 0.f, 0.f};
    auto look_up = [&](int x0) {
      base = x0;
      const int x = x0 + lane, c = (warp + NW * (x / SUB)) * SUB + x % SUB;
      blk = -1;
      ch = Chunk{0, 0, 0.f, 0.f};
      if (x / SUB < my && c < chunks) {
        ch.tok = t0 + 16 * c;
        blk = __ldg(p.bt + (size_t)b * p.maxb + (ch.tok >> p.bs_shift));
        if (blk < 0 || blk >= p.nblocks) {
          bad |= PA_FLAG_BAD_BLOCK_ID;
        } else {
          ch.rows = min(t1 - ch.tok, 16);
          const size_t at = (size_t)blk * p.Hkv + g;
          ch.ks = __ldg(cache.k_scale + at);
          ch.vs = __ldg(cache.v_scale + at);
        }
      }
    };
    auto issue = [&](int j, int s) {
      if (j >= my) return;
      if (SUB * j >= base + 32) look_up(SUB * j);
      stream_tma<T>(cache, &kmap, &vmap, g, ring + s * T::STAGE, meta + s * T::META, &bar[s], blk, ch,
                    SUB * j - base, lane);
    };
    if (my > 0) look_up(0);
    __syncwarp();
    issue(0, st);
    issue(1, st == 2 ? 0 : st + 1);

    WarpAttention<T> att;
    att.clear();
    int lim[2], least = 0x7fffffff;  // keys that this thread's rows see, and the least of the tile's
    att.load_q(
        [&](int h) -> const char* {
          const int rg = rb * ROWS + quad + 8 * h;
          const bool real = rg < p.M;
          const int i = real ? rg / p.G : 0, head = g * p.G + (real ? rg % p.G : 0);
          lim[h] = real && i < ql ? (p.causal ? n - ql + i + 1 : n) : 0;
          if (real) least = min(least, lim[h]);
          return real ? reinterpret_cast<const char*>(p.q) + (((size_t)b * p.Sq + i) * p.Hq + head) * D * 2
                      : nullptr;
        },
        p.qk_scale, qi);
    least = __reduce_min_sync(kFull, least);

    for (int j = 0; j < my; ++j) {
      if (!stream_wait(&bar[st], phase)) {
        bad |= PA_FLAG_WAIT_TIMEOUT;
        if (j + 1 < my) mbar_wait_drain(&bar[st == 2 ? 0 : st + 1], st == 2 ? phase ^ 1 : phase);
        failed = true;
        break;
      }
      __syncwarp();
      issue(j + 2, st == 0 ? 2 : st - 1);
      const Chunk* cs = reinterpret_cast<const Chunk*>(meta + st * T::META);
      const Chunk c0 = cs[0], c1 = cs[SUB - 1];
      const bool whole = c0.rows == 16 && c1.rows == 16;
      if (!whole) zero_rows<T>(ring + st * T::STAGE + T::TILE, c0.rows, c1.rows, lane);
      att.tile_fp8(ring_addr + st * T::STAGE, {c0.ks, c1.ks}, {c0.vs, c1.vs}, nullptr,
                   whole && c1.tok + 16 <= least,
                   [&](int s, int h) { return s ? min(c1.rows, lim[h] - c1.tok) : min(c0.rows, lim[h] - c0.tok); },
                   lane);
      if (++st == T::NST) {
        st = 0;
        phase ^= 1;
      }
    }

    // ---- merge the warps, and write the rows (whole, or a piece's partial)
    __syncthreads();  // every warp is done with its stages
    att.stage_state(obuf, ml, warp, lane);
    if (it == 0) {
      wait_planner();
      if (items > 1) item_next = p.items[list + 1];
    }
    if (bad) atomicOr(p.flags, bad);
    bad = 0;
    __syncthreads();
    constexpr int D4 = D / 4, SLOT = ROWS * T::OSTR;
    for (int e = tid; e < ROWS * D4; e += T::NTHREADS) {
      const int r = e / D4, d4 = e % D4, rg = rb * ROWS + r;
      if (rg >= p.M) continue;
      float4 O;
      const float2 s = merge_states(NW, [&](int w) { return ml + w * ROWS + r; },
                                    [&](int w) { return obuf + w * SLOT + r * T::OSTR + 4 * d4; }, O);
      const float inv = s.y == 0.f ? 0.f : 1.f / s.y;  // no key: zero (NaN stays NaN)
      const float lse2 = s.y == 0.f ? -INFINITY : s.x + fast_log2(s.y);
      O = make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
      if (slot >= 0) {
        const size_t part = (size_t)slot * ROWS + r;
        *reinterpret_cast<float4*>(p.o_part + part * D + 4 * d4) = O;
        if (d4 == 0) p.lse_part[part] = lse2;
      } else {
        const size_t row = ((size_t)b * p.Sq + rg / p.G) * p.Hq + g * p.G + rg % p.G;
        store_out4<T::QK>(p.out, row * D + 4 * d4, O);
        if (d4 == 0 && p.lse) p.lse[row] = lse2 == -INFINITY ? lse2 : lse2 * kLn2;
      }
    }
    const bool in_dec = slot >= 0 && __ldg(&p.unit_info[u].y) <= p.ns_dec;
    if (in_dec) __threadfence();
    // the states lie where the next item's copies go
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    if (in_dec && tid == 0) publish_piece(p, u, slot, &pend_even, &pend_odd);
  }
  if (bad) atomicOr(p.flags, bad);
  if (tid == 0) {
    pend[0] = pend_even.x;
    pend[1] = pend_even.y;
    pend[2] = pend_odd.x;
    pend[3] = pend_odd.y;
  }
  __syncthreads();
  finish_pending<D, ROWS, T::QK, NW>(p, pend, obuf, T::RING / 4, reinterpret_cast<float*>(ml));
  zero_empty_units<D, ROWS, T::QK, T::NTHREADS>(p);
}

template <int D, int QK>
cudaError_t launch_stream_instance(const KernelParams& prm, const CUtensorMap& kmap,
                                   const CUtensorMap& vmap, int grid, cudaStream_t s) {
  using T = StreamTraits<D, KV_FP8, QK, false>;
  using M = DecodeStreamSmem<T>;
  auto kern = decode_stream_kernel<T>;
  static std::atomic<uint64_t> attr_done{0};  // devices whose limit is raised
  const cudaError_t e = set_smem_attr_once(attr_done, reinterpret_cast<const void*>(kern), M::BYTES);
  if (e != cudaSuccess) return e;
  CacheView cache{};
  cache.k_scale = prm.k_scale;
  cache.v_scale = prm.v_scale;
  cache.Hkv = prm.Hkv;
  cache.bs_shift = prm.bs_shift;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(T::NTHREADS);
  cfg.dynamicSmemBytes = M::BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, kmap, vmap, prm, cache);
}

}  // namespace pa
