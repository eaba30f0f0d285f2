// Persistent split-KV paged decode over a 4-bit cache: the planner's work list, each item's 16-token
// chunks going to the warps of a CTA in turn, which attend on their own (int4_attention.cuh) and
// merge at the item's end, as in the streaming decode over fp8 pages.
//
// A tile is one or two chunks: TMA boxes of up to 32 tokens of one page and kv head (K, V), and their
// pairs by a cp.async of a lane, into a ring of the warp's own, with no barrier between warps while data
// streams.
//
// Measured (plan, decode and reduce; replayed): 32 contexts of 512 to 4,096 tokens, 32 heads on 8 kv
// heads of 128, pages of 16 (81 MB) 32.5 us, with four new tokens each 45; 32 of 2,048 to 16,384, 16 heads
// of 256 (1.25 GB) 239 us, 5.2 TB/s; 4 of 32,768 to 131,072, 16 heads on one of 128 (45 MB) 28.7 us, of
// which plan, start, merge and reduce are about 10.  What bounds it is a warp's own chain: alone on its
// scheduler it takes 2,400 cycles a tile of 32 tokens (632 instructions; 320 are the widening of codes
// and the products), three together 3,200, so that a scheduler issues 0.55 instructions a cycle (head
// dim 128, 8 rows: 4.2 TB/s).  Head dim 256 has twice the codes for the same softmax.  Tried without
// gain: four neighbouring heads a unit (their rows as one box; four times the partials), one ring a CTA,
// tiles of 64 tokens, values a tile behind keys in one block of instructions, two accumulators a logit.
#pragma once

#include "int4_attention.cuh"

namespace pa {

template <class T>
struct DecodeInt4Smem {
  static constexpr int NW = 4;
  static constexpr int NTHREADS = NW * 32;
  static constexpr int TK = int4_tile_tokens(T::D, T::ROWS);  // tokens of a warp's tile
  static constexpr int SUB = TK / 16;                         // its chunks
  static constexpr int NST = 3;                               // stages of a warp's ring
  static constexpr int TILE = TK * T::ROW;                    // bytes of a K (or V) tile
  static constexpr int STAGE = 2 * TILE;                      // (a multiple of its swizzle's period)
  static constexpr int PAIRS = 2 * TK * 4;                    // a stage's pairs, K rows' before V rows'
  static constexpr int RING = NW * NST * STAGE;
  static constexpr int STATES = NW * T::O_SLOT;
  static constexpr int OFF_ML = round_up(cmax(RING, STATES), 128);
  static constexpr int OFF_QUERY = OFF_ML + round_up(cmax(NW * T::ROWS * 8, 2 * T::ROWS * 4), 128);
  static constexpr int OFF_FACTORS = OFF_QUERY + T::QUERY;
  static constexpr int OFF_PAIRS = OFF_FACTORS + NW * TK * 16;
  static constexpr int OFF_BAR = OFF_PAIRS + NW * NST * PAIRS;
  static constexpr int OFF_PEND = OFF_BAR + NW * NST * 8;
  static constexpr int BYTES = OFF_PEND + 16 + 1024;  // (alignment)
  // As many warps as fit without spilling the state of an unrolled tile.  Us a step with one CTA more
  // (or for head dim 64 one less): head dim 128, 8 rows (32 contexts of 8,192 to 16,384, 32 heads on 8)
  // 118 in place of 104; 16 rows (64 such contexts, one kv head) 60 in place of 48; 64, 16 rows 38.8 in
  // place of 36.3.
  static constexpr int CTAS_PER_SM =
      T::D == 256 ? 2 : T::D == 128 ? (T::NT == 1 ? 3 : 2) : (T::NT == 1 ? 4 : 3);
  static_assert(16 * T::ROW % 128 == 0 && STAGE % (8 * T::ROW) == 0 && STAGE % 128 == 0,
                "a tensor copy's destination");
  static_assert(CTAS_PER_SM * (BYTES + 1024) <= 228 * 1024, "shared memory");
};

template <class T>
__global__ void __launch_bounds__(DecodeInt4Smem<T>::NTHREADS, DecodeInt4Smem<T>::CTAS_PER_SM)
    decode_int4_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const KernelParams p) {
  using M = DecodeInt4Smem<T>;
  constexpr int D = T::D, ROWS = T::ROWS, NW = M::NW, SUB = M::SUB, NST = M::NST;
  static_assert(NST == 3, "two tiles in flight");
  extern __shared__ char smem_raw[];
  char* const smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, qi = lane & 3;
  char* const ring = smem + warp * NST * M::STAGE;
  char* const pairs = smem + M::OFF_PAIRS + warp * NST * M::PAIRS;
  uint64_t* const bar = reinterpret_cast<uint64_t*>(smem + M::OFF_BAR) + warp * NST;
  int* const pend = reinterpret_cast<int*>(smem + M::OFF_PEND);    // [4]
  float* const obuf = reinterpret_cast<float*>(smem);              // [NW][ROWS][OSTR]
  uint4* const query = reinterpret_cast<uint4*>(smem + M::OFF_QUERY);
  float4* const factors = reinterpret_cast<float4*>(smem + M::OFF_FACTORS) + warp * M::TK;
  float2* const ml = reinterpret_cast<float2*>(smem + M::OFF_ML);  // [NW][ROWS] (max, sum)
  const bool planning = planner_runs(p);
  if (lane == 0) {  // (a warp's barriers are its own)
    for (int s = 0; s < NST; ++s) mbar_init(&bar[s], SUB + 32);
    fence_barrier_init();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (!planning) grid_dependency_wait();
  __syncwarp();
  const int box = min(p.bs, M::TK);  // tokens of a box: a page's, or a tile's
  const int t = lane % M::TK;  // a lane's token
  const uint32_t box_bytes = 2u * (uint32_t)(box * T::ROW);
  // a lane's 16 bytes of pairs: K's or V's, chunk, four tokens
  const uint32_t* const pair_from =
      reinterpret_cast<const uint32_t*>(lane < 4 * SUB ? p.k_scale : p.v_scale) + 4 * (lane & 3);
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
    const int tiles = (t1 - t0 + M::TK - 1) / M::TK;
    const int my = failed ? 0 : (tiles - warp + NW - 1) / NW;  // this warp's tiles

    // lane l looks up the block of chunk base + l of the warp's chunks, SUB a tile (-1: none, or outside
    // the pool).  `held` says which of these are in the pool, `held_before` which of the 32 before them.
    int blk = -1, base = -32;
    uint32_t held = 0, held_before = 0;
    auto look_up = [&](int x0) {
      base = x0;
      const int x = x0 + lane, tok = t0 + ((warp + NW * (x / SUB)) * SUB + x % SUB) * 16;
      blk = -1;
      if (x / SUB < my && tok < t1) {
        blk = __ldg(p.bt + (size_t)b * p.maxb + (tok >> p.bs_shift));
        if (blk < 0 || blk >= p.nblocks) {
          bad |= PA_FLAG_BAD_BLOCK_ID;
          blk = -1;
        }
      }
      held_before = held;
      held = __ballot_sync(kFull, blk >= 0);
    };
    // The boxes of tile j into stage s: a lane a chunk, which arrives with what it copies (where a box
    // holds the tile, the first chunk's lane copies it).
    auto issue = [&](int j, int s) {
      if (j >= my) return;
      if (SUB * j >= base + 32) look_up(SUB * j);
      const int lane0 = SUB * j - base, c = lane - lane0, tok = t0 + (warp + NW * j) * M::TK;
      if (c >= 0 && c < SUB) {
        if (blk >= 0 && (16 * c & (box - 1)) == 0) {
          mbar_arrive_expect_tx(&bar[s], box_bytes);
          const int slot_in = (tok + 16 * c) & (p.bs - 1);
          char* const dst = ring + s * M::STAGE + c * 16 * T::ROW;
          tma_load_4d(dst, &kmap, &bar[s], 0, g, slot_in, blk);
          tma_load_4d(dst + M::TILE, &vmap, &bar[s], 0, g, slot_in, blk);
        } else {
          mbar_arrive(&bar[s]);
        }
      }
      __syncwarp();
      const int cp = (lane >> 2) % SUB, bk = __shfl_sync(kFull, blk, lane0 + cp);
      if (lane < 8 * SUB && bk >= 0)
        cp_async_16(pairs + s * M::PAIRS + lane * 16,
                    pair_from + ((((size_t)bk * p.Hkv + g) << p.bs_shift) + ((tok + 16 * cp) & (p.bs - 1))));
      cp_async_arrive_noinc(&bar[s]);
    };
    if (my > 0) look_up(0);
    __syncwarp();
    issue(0, st);
    issue(1, st == 2 ? 0 : st + 1);

    T att;
    att.clear();
    att.load_q(
        [&](int r) -> const char* {
          const int rg = rb * ROWS + r;
          if (rg >= p.M || rg / p.G >= ql) return nullptr;
          return reinterpret_cast<const char*>(p.q) +
                 (((size_t)b * p.Sq + rg / p.G) * p.Hq + (size_t)g * p.G + rg % p.G) * D * 2;
        },
        p.qk_scale, query, warp, lane);
    auto limit = [&](int r) {  // the keys that row r of the tile sees, -1 for one that is no row
      const int rg = rb * ROWS + r, i = rg / p.G;
      return rg >= p.M || i >= ql ? -1 : p.causal ? n - ql + i + 1 : n;
    };
    // (Rows behind the sequence's last keep no tile from the way without masks, since the merge clears
    // them: 32 contexts of 512 to 4,096 with one to four of four new tokens, 32 heads on 8 of 128, 44.3 us
    // a step; 59.6 when they were masked.)
    int least = limit(lane % ROWS);
    least = __reduce_min_sync(kFull, least < 0 ? 0x7fffffff : least);
    __syncthreads();  // the queries are there

    for (int j = 0; j < my; ++j) {
      if (!stream_wait(&bar[st], phase)) {
        bad |= PA_FLAG_WAIT_TIMEOUT;
        if (j + 1 < my) mbar_wait_drain(&bar[st == 2 ? 0 : st + 1], st == 2 ? phase ^ 1 : phase);
        failed = true;
        break;
      }
      __syncwarp();
      const int tok = t0 + (warp + NW * j) * M::TK;
      const uint32_t kt = smem_addr(ring + st * M::STAGE);
      // (before what decides how the tile goes on: the products are what its latencies hide behind)
      float s[SUB][T::NT][4];
      att.template keys<SUB>(kt, query, s, lane);
      issue(j + 2, st == 0 ? 2 : st - 1);
      const int x = SUB * j - base;  // (tile j + 2's look-up may have come in between)
      const uint32_t here = (x >= 0 ? held >> x : held_before >> (x + 32)) & ((1u << SUB) - 1);
      // a lane a token: its factors
      const uint32_t* const pair = reinterpret_cast<const uint32_t*>(pairs + st * M::PAIRS) + t;
      const float2 kp = pair_values<T::QK>(pair[0]), vp = pair_values<T::QK>(pair[M::TK]);
      float4 f = make_float4(kp.x, __fmaf_rn(8.f, kp.x, kp.y), vp.x, __fmaf_rn(8.f, vp.x, vp.y));
      const float unit = att.vref;
      const bool fits = fabsf(vp.x) <= unit && fabsf(vp.x) >= unit * kVRange;
      if (here == (1u << SUB) - 1 && tok + M::TK <= min(t1, least) && __all_sync(kFull, fits)) {
        f.z *= pow2_inverse(unit) * kPLift;
        factors[t] = f;
        __syncwarp();
        att.template whole_tile<SUB>(s, kt + M::TILE, factors, lane);
      } else {
        // (what lies behind the last token, or was not copied, may hold anything)
        const bool ok = (here >> (t >> 4) & 1) && tok + t < t1;
        factors[t] = ok ? f : make_float4(0.f, 0.f, 0.f, 0.f);
        __syncwarp();
        att.template any_tile<SUB>(
            s, kt + M::TILE, factors,
            [&](int c, int h, int i) {
              const int x = tok + 16 * c + 8 * h + quad, end = (here >> c & 1) ? t1 : 0;
              const int row = 8 * i + 2 * qi;
              return make_uint2(x < min(limit(row), end), x < min(limit(row + 1), end));
            },
            lane);
      }
      if (++st == NST) {
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
    for (int e = tid; e < ROWS * D4; e += M::NTHREADS) {
      const int r = e / D4, d4 = e % D4, rg = rb * ROWS + r;
      if (rg >= p.M) continue;
      float4 O;
      float2 s = merge_states(NW, [&](int w) { return ml + w * ROWS + r; },
                                    [&](int w) { return obuf + w * SLOT + r * T::OSTR + 4 * d4; }, O);
      if (rg / p.G >= ql) {
        O = make_float4(0.f, 0.f, 0.f, 0.f);
        s.y = 0.f;
      }
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
  finish_pending<D, ROWS, T::QK, NW>(p, pend, obuf, M::RING / 4, reinterpret_cast<float*>(ml));
  zero_empty_units<D, ROWS, T::QK, M::NTHREADS>(p);
}

template <int D, int NT, int QK>
cudaError_t launch_int4_instance(const KernelParams& prm, const CUtensorMap (&maps)[2], int grid,
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
  return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], prm);
}

// Both row tiles of a head dim.
template <int D>
cudaError_t launch_int4_dim(const KernelParams& prm, const CUtensorMap (&maps)[2], int grid, int mp,
                            int qk, cudaStream_t s) {
  if (mp == 8)
    return qk == Q_BF16 ? launch_int4_instance<D, 1, Q_BF16>(prm, maps, grid, s)
                        : launch_int4_instance<D, 1, Q_FP16>(prm, maps, grid, s);
  return qk == Q_BF16 ? launch_int4_instance<D, 2, Q_BF16>(prm, maps, grid, s)
                      : launch_int4_instance<D, 2, Q_FP16>(prm, maps, grid, s);
}

}  // namespace pa
