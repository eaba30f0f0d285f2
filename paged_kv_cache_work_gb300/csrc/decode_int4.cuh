// Persistent split-KV paged decode over a 4-bit cache: the planner's work list, each item's 16-token
// chunks going to the warps of a CTA in turn, which attend on their own (int4_attention.cuh) and
// merge at the item's end, as in the streaming decode over fp8 pages.
#pragma once

#include "int4_attention.cuh"

namespace pa {

template <class T>
struct DecodeInt4Smem {
  static constexpr int NW = 4;
  static constexpr int NTHREADS = NW * 32;
  static constexpr int STATES = NW * T::O_SLOT;
  static constexpr int OFF_ML = round_up(STATES, 128);
  static constexpr int OFF_PEND = OFF_ML + cmax(NW * T::ROWS * 8, 2 * T::ROWS * 4);
  static constexpr int BYTES = OFF_PEND + 16;
  static constexpr int CTAS_PER_SM = T::D == 256 ? 2 : T::NT == 1 ? 4 : 3;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

template <class T>
__global__ void __launch_bounds__(DecodeInt4Smem<T>::NTHREADS, DecodeInt4Smem<T>::CTAS_PER_SM)
    decode_int4_kernel(const KernelParams p, const Int4View cache) {
  using M = DecodeInt4Smem<T>;
  constexpr int D = T::D, ROWS = T::ROWS, NW = M::NW, NT = T::NT;
  extern __shared__ __align__(16) char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, qi = lane & 3;
  int* const pend = reinterpret_cast<int*>(smem + M::OFF_PEND);    // [4]
  float* const obuf = reinterpret_cast<float*>(smem);              // [NW][ROWS][OSTR]
  float2* const ml = reinterpret_cast<float2*>(smem + M::OFF_ML);  // [NW][ROWS] (max, sum)
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
    const int chunks = (t1 - t0 + 15) >> 4;

    T att;
    att.clear();
    att.load_q(
        [&](int r) -> const char* {
          const int rg = rb * ROWS + r;
          if (rg >= p.M) return nullptr;
          return reinterpret_cast<const char*>(p.q) +
                 (((size_t)b * p.Sq + rg / p.G) * p.Hq + (size_t)g * p.G + rg % p.G) * D * 2;
        },
        p.qk_scale, lane);
    int2 lim[NT];  // keys that this thread's rows see, and the least of the tile's
    int least = 0x7fffffff;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      auto limit = [&](int r) {
        const int rg = rb * ROWS + r;
        if (rg >= p.M) return 0;
        const int i = rg / p.G, keys = i < ql ? (p.causal ? n - ql + i + 1 : n) : 0;
        least = min(least, keys);
        return keys;
      };
      lim[t] = make_int2(limit(8 * t + 2 * qi), limit(8 * t + 2 * qi + 1));
    }
    least = __reduce_min_sync(kFull, least);

    for (int c = warp; c < chunks; c += NW) {
      const int tok = t0 + 16 * c, rows = min(t1 - tok, 16);
      const int blk = __ldg(p.bt + (size_t)b * p.maxb + (tok >> p.bs_shift));
      if (blk < 0 || blk >= p.nblocks) {
        bad |= PA_FLAG_BAD_BLOCK_ID;
        continue;
      }
      const int at = tok & (p.bs - 1);
      const size_t row0 = (((size_t)blk << p.bs_shift) + at) * p.Hkv + g;
      const size_t pair0 = (((size_t)blk * p.Hkv + g) << p.bs_shift) + at;
      const size_t stride = (size_t)p.Hkv * T::ROW;
      float2 ks[1][2], vs[1][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool ok = quad + 8 * h < rows;  // (what lies behind the last token may hold anything)
        ks[0][h] = ok ? pair_values<T::QK>(__ldg(cache.k_pair + pair0 + quad + 8 * h)) : make_float2(0.f, 0.f);
        vs[0][h] = ok ? pair_values<T::QK>(__ldg(cache.v_pair + pair0 + quad + 8 * h)) : make_float2(0.f, 0.f);
      }
      auto kw = [&](int, int h, uint32_t (&w)[T::KW]) {
        const char* src = cache.k + row0 * T::ROW + (quad + 8 * h) * stride + qi * T::KW * 4;
#pragma unroll
        for (int i = 0; i < T::KW; i += 2) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + 4 * i));
          w[i] = v.x;
          w[i + 1] = v.y;
        }
      };
      auto vw = [&](int, int h, int e, uint32_t (&w)[T::VW]) {
        const int r = 2 * qi + 8 * h + (T::first_token(qi) ^ e);
        const char* src = cache.v + row0 * T::ROW + r * stride + quad * T::VW * 4;
#pragma unroll
        for (int i = 0; i < T::VW; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(src + 4 * i));
      };
      att.template tile<1>(
          kw, vw, ks, vs, rows == 16 && tok + 16 <= least,
          [&](int, int h, int t) {
            const int x = tok + quad + 8 * h;
            return make_uint2(x < min(lim[t].x, tok + rows), x < min(lim[t].y, tok + rows));
          },
          lane);
    }

    // ---- merge the warps, and write the rows (whole, or a piece's partial)
    att.stage_state(obuf, ml, warp, lane);
    if (it == 0) {
      wait_planner();
      if (items > 1) item_next = p.items[list + 1];
    }
    if (bad) atomicOr(p.flags, bad);
    bad = 0;
    __syncthreads();
    constexpr int D4 = D / 4, SLOT = ROWS * T::OSTR;
    for (int e = tid; e < ROWS * D4; e += M::NTHREADS) {
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
  finish_pending<D, ROWS, T::QK, NW>(p, pend, obuf, M::STATES / 4, reinterpret_cast<float*>(ml));
  zero_empty_units<D, ROWS, T::QK, M::NTHREADS>(p);
}

template <int D, int NT, int QK>
cudaError_t launch_int4_instance(const KernelParams& prm, const Int4View& cache, int grid,
                                 cudaStream_t s) {
  using T = Int4Attention<D, NT, QK>;
  using M = DecodeInt4Smem<T>;
  auto kern = decode_int4_kernel<T>;
  static std::atomic<uint64_t> attr_done{0};  // devices whose limit is raised
  const cudaError_t e = set_smem_attr_once(attr_done, reinterpret_cast<const void*>(kern), M::BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(M::NTHREADS);
  cfg.dynamicSmemBytes = M::BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, prm, cache);
}

// Both row tiles of a head dim.
template <int D>
cudaError_t launch_int4_dim(const KernelParams& prm, const Int4View& cache, int grid, int mp, int qk,
                            cudaStream_t s) {
  if (mp == 8)
    return qk == Q_BF16 ? launch_int4_instance<D, 1, Q_BF16>(prm, cache, grid, s)
                        : launch_int4_instance<D, 1, Q_FP16>(prm, cache, grid, s);
  return qk == Q_BF16 ? launch_int4_instance<D, 2, Q_BF16>(prm, cache, grid, s)
                      : launch_int4_instance<D, 2, Q_FP16>(prm, cache, grid, s);
}

}  // namespace pa
