// The inner part of the decodes whose warps each stream pages on their own: a private ring of
// shared-memory stages, and the attention of up to 16 query rows over the tiles that pass through
// it.
//
// A tile is one or two chunks of 16 tokens, each inside one page.  No barrier joins the warps while
// data streams; their states (maximum m, sum l, accumulator o of each row) are merged at the end by
//     m = max_s m_s, w_s = 2^(m_s - m), l = sum_s w_s l_s, o = sum_s w_s o_s, out = o / l.
//
// 16-bit caches.  Copies are 16-byte cp.async; rows of a chunk that no key may be read from are
// zero-filled (so a masked row never holds NaN or infinity).  S = Q K^T and O += P V on mma.sync
// m16n8k16 (K by ldmatrix, V by ldmatrix.trans), an online softmax in log2 units on the
// accumulators whose running maximum moves only when a logit beats it by 2^8, P rounded to the
// operands' type (its sum is kept from the unrounded fp32 values).
//
// fp8 caches.  What bounds them is the instructions of the few warps that fit on an SM (one issues
// about every fifth cycle), so all is arranged for few of them.  Copies are TMA boxes of a chunk
// (K and V: two instructions of one lane).  Codes are widened to f16 on their way to the same MMA
// (exactly; one conversion for two codes.  mma.sync on E4M3 operands is no way out: on this GPU
// it runs as conversions and f16 MMAs, four instructions and more each, and the whole measured
// 66 us where widening by hand took 51).  A V tile is transposed by ldmatrix on bytes
// (m16n16.b8.trans), which hands a lane four rows of a channel, two f16 pairs for two conversions.
// Which tokens those are is up to the row addresses: tokens are assigned to the logits' columns
// (column n of 8-token block j of a chunk is token n, + 8 from n = 4 on, for j = 0 and n + 4 for
// j = 1) so that the weights a lane ends with are the ones it has to pass to the second product,
// and that the eight rows of every ldmatrix phase differ modulo 8, which the TMA swizzle needs to
// keep them in distinct banks.  A query row is scaled by a power of two into f16's range; a K
// scale multiplies the logit, a V scale (over the accumulator's own power of two, which follows the
// scales up and down) the weight.  A tile whose V scales lie more than 2^8 apart takes its weights
// and second product once for each unit that it needs; others, two comparisons more (64 sequences
// of 8,192 to 16,384 tokens, 16 heads on one kv head of 128: 43.7 us a step without, 44.1 with).
#pragma once

#include "decode_mma.cuh"

namespace pa {

// TOKS_: fp8 with a scale for each token (other scale modes: one for each chunk).
template <int D_, int KVK_, int QK_, bool TOKS_>
struct StreamTraits {
  static constexpr int D = D_;
  static constexpr int QK = QK_;
  static constexpr bool FP8 = KVK_ == KV_FP8;
  static constexpr bool TOKS = TOKS_;
  static constexpr int ROWS = 16;  // query rows of a tile
  static constexpr bool F16 = FP8 || QK == Q_FP16;  // operand type of the MMA
  static constexpr int BPE = FP8 ? 1 : 2;
  static constexpr int NW = 4;
  static constexpr int NTHREADS = NW * 32;
  static constexpr int ROW = D * BPE;                     // bytes of a row
  static constexpr int TK = ROW <= 128 ? 32 : 16;         // tokens of a warp's tile
  static constexpr int SUB = TK / 16;                     // 16-token chunks of a tile
  static constexpr int NST = 3;
  // fp8: a tile is SLABS column slabs of SLABW bytes a row, as the TMA boxes bring them
  static constexpr int SLABW = cmin(ROW, 128);
  static constexpr int SLABS = ROW / SLABW;
  static constexpr int TILE = TK * ROW;  // bytes of a K (or V) tile
  static constexpr int STAGE = 2 * TILE;
  static constexpr int RING = NW * NST * STAGE;
  // fp8: what a stage's chunks are (up to two Chunks), and its tokens' scales (K, then V)
  static constexpr int META = !FP8 ? 0 : 32 + (TOKS ? 2 * TK * 4 : 0);
  static constexpr int KSTEPS = D / 16;
  static constexpr int NB = D / 8;                // 8-channel blocks of the output
  static constexpr int OSTR = D + 4;              // floats between rows of a staged accumulator
  static constexpr int O_SLOT = ROWS * OSTR * 4;  // one staged state's accumulators
  static_assert(FP8 || !TOKS, "scales belong to fp8 caches");
};

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_4_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One or two 16x16 byte matrices transposed: register 2 j + r holds rows 4 qi .. + 3 of channel
// quad + 8 r of matrix j (lane 16 j + i gives the address of its row i).
__device__ __forceinline__ void ldsm_b8_t(uint32_t addr, uint32_t (&r)[2]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x1.trans.shared.b8 {%0, %1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_b8_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// 16-byte piece c of row r of a tile: eight rows that differ modulo 8 (64-byte rows: in (r / 2) % 4
// or r % 2) lie in distinct banks.  16-bit tiles are whole rows, fp8 tiles column slabs with the
// swizzle of their TMA boxes.
template <class T>
__device__ __forceinline__ uint32_t tile_piece(uint32_t base, int r, int c) {
  if constexpr (T::FP8) {
    constexpr int PPS = T::SLABW / 16;
    const int x = T::SLABW == 128 ? (r & 7) : ((r >> 1) & 3);
    return base + (c / PPS) * (T::TK * T::SLABW) + r * T::SLABW + (((c % PPS) ^ x) << 4);
  } else {
    return base + r * T::ROW + ((c ^ (r & 7)) << 4);
  }
}

// Where a cache's rows and scales lie.
struct CacheView {
  const char* k;
  const char* v;
  const float* k_scale;  // null when there is none
  const float* v_scale;
  long long sc_block;    // scale of (block, slot, head g): block * sc_block + slot * sc_slot +
  int sc_slot, sc_head;  // g * sc_head
  int Hkv, bs_shift;
};

// One chunk of a tile: the first `rows` of its 16 tokens, from token `tok` of the sequence on, are
// wanted (rows 0: nothing).  fp8 with one scale for the chunk: its K and V scales.
struct __align__(16) Chunk {
  int rows, tok;
  float ks, vs;
};

// 16-bit: copy chunk s of a tile, out of block blk, into the stage at `stage` (this warp's lanes
// together, no commit).
template <class T>
__device__ __forceinline__ void stream_copy(const CacheView& cv, int g, uint32_t stage, int s,
                                            int blk, const Chunk& ch, int lane) {
  constexpr int PPR = T::ROW / 16;
  const uint32_t kt = stage, vt = stage + T::TILE;
  const int slot = ch.tok & ((1 << cv.bs_shift) - 1);
  const size_t row0 = ch.rows > 0 ? (((size_t)blk << cv.bs_shift) + slot) * cv.Hkv + g : 0;
  const size_t rstr = (size_t)cv.Hkv * T::ROW;
  const char* ks = cv.k + row0 * T::ROW;
  const char* vs = cv.v + row0 * T::ROW;
#pragma unroll
  for (int e0 = 0; e0 < 16 * PPR; e0 += 32) {
    const int e = e0 + lane, r = e / PPR, c = e % PPR;
    const bool ok = r < ch.rows;
    const size_t off = ok ? r * rstr + c * 16 : 0;
    cp_async_16_zfill(tile_piece<T>(kt, s * 16 + r, c), ks + off, ok);
    cp_async_16_zfill(tile_piece<T>(vt, s * 16 + r, c), vs + off, ok);
  }
}

// fp8: the chunks of a tile into a stage of the warp's ring, completing on its barrier.  Lane
// lane0 + s holds chunk s (its block and Chunk); called by the whole warp.
template <class T>
__device__ __forceinline__ void stream_tma(const CacheView& cv, const CUtensorMap* kmap,
                                           const CUtensorMap* vmap, int g, char* stage, char* meta,
                                           uint64_t* bar, int blk, const Chunk& ch, int lane0,
                                           int lane) {
  const bool mine = lane / T::SUB == lane0 / T::SUB;
  const bool copies = mine && ch.rows > 0;
  const int s = lane % T::SUB;
  const uint32_t nv = __popc(__ballot_sync(kFull, copies));
  if (lane == 0) mbar_arrive_expect_tx(bar, nv * 2u * 16u * T::ROW);
  __syncwarp();
  const int slot = ch.tok & ((1 << cv.bs_shift) - 1);
  if (copies) {
#pragma unroll
    for (int h = 0; h < T::SLABS; ++h) {
      char* dst = stage + h * (T::TK * T::SLABW) + s * 16 * T::SLABW;
      tma_load_4d(dst, kmap, bar, h * T::SLABW, g, slot, blk);
      tma_load_4d(dst + T::TILE, vmap, bar, h * T::SLABW, g, slot, blk);
    }
  }
  if (mine) *reinterpret_cast<Chunk*>(meta + 16 * s) = ch;  // (its scales may still be on their way)
  if constexpr (T::TOKS) {  // a lane a token
    const int src = lane0 + (lane >> 4) % T::SUB, r = lane & 15;
    const int bk = __shfl_sync(kFull, blk, src), sl = __shfl_sync(kFull, slot, src);
    const bool ok = r < __shfl_sync(kFull, ch.rows, src);
    const size_t at = ok ? (size_t)(bk * cv.sc_block) + (size_t)((sl + r) * cv.sc_slot) +
                               (size_t)g * cv.sc_head
                         : 0;
    const uint32_t to = smem_addr(meta + 32) + lane % T::TK * 4;
    if (lane < T::TK) {
      cp_async_4_zfill(to, cv.k_scale + at, ok);
      cp_async_4_zfill(to + T::TK * 4, cv.v_scale + at, ok);
    }
    cp_async_arrive_noinc(bar);
  }
}
// Zeros in the rows of a V tile that hold no wanted token (they may hold anything, and a zero
// weight times NaN would not be zero): called by the whole warp before it reads the tile, and
// ordered before the copies that refill the stage.
template <class T>
__device__ __forceinline__ void zero_rows(char* vt, int rows0, int rows1, int lane) {
  constexpr int PPS = T::SLABW / 16;
  for (int e = lane; e < T::TK * T::SLABS * PPS; e += 32) {
    const int r = (e / PPS) % T::TK;
    if ((r & 15) >= (r < 16 ? rows0 : rows1)) *reinterpret_cast<uint4*>(vt + e * 16) = make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}
// Bounded wait for a stage's copies (the clock is read only when the first try fails).
__device__ __forceinline__ bool stream_wait(uint64_t* bar, uint32_t parity) {
  return mbar_try_wait(bar, parity) || mbar_wait_drain(bar, parity);
}
// Arrivals a stage's barrier expects.
template <class T>
constexpr int kStreamArrivals = T::TOKS ? 33 : 1;

// A warp's query rows and its softmax state.  Thread (quad, qi) = (lane / 4, lane % 4) holds rows
// quad and quad + 8.
template <class T>
struct WarpAttention {
  static constexpr int NB = T::NB, KSTEPS = T::KSTEPS;
  uint32_t qa[KSTEPS][4];
  float qk[2];     // logit scale (log2 units) of the rows
  float o[NB][4];  // fp8: in units of vref / kPLift
  float m[2], l[2];
  float vref, vtop;  // (see move_v_unit)

  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    vref = vtop = kPow2Least;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) o[nb][0] = o[nb][1] = o[nb][2] = o[nb][3] = 0.f;
  }

  // row_of(h): this thread's query row quad + 8 h, or null for a padding row.
  template <class F>
  __device__ __forceinline__ void load_q(F row_of, float qk_scale, int qi) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const char* row = row_of(h);
      qk[h] = qk_scale;
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
        uint32_t lo = 0, hi = 0;
        if (row) {
          if constexpr (T::FP8) {  // permuted k order: channels 16 kk + 4 qi + {0, 1}, {2, 3}
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + (16 * kk + 4 * qi) * 2));
            lo = v.x;
            hi = v.y;
          } else {
            lo = __ldg(reinterpret_cast<const uint32_t*>(row + (16 * kk + 2 * qi) * 2));
            hi = __ldg(reinterpret_cast<const uint32_t*>(row + (16 * kk + 8 + 2 * qi) * 2));
          }
        }
        qa[kk][h] = lo;
        qa[kk][2 + h] = hi;
      }
      if constexpr (T::FP8 && T::QK == Q_BF16) {
        // to f16, times the power of two that brings the largest element to [2^7, 2^8)
        float big = 0.f;
#pragma unroll
        for (int kk = 0; kk < KSTEPS; ++kk) {
          const float2 a = bf16x2_to_f2(qa[kk][h]), c = bf16x2_to_f2(qa[kk][2 + h]);
          big = fmaxf(big, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(c.x), fabsf(c.y))));
        }
        big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
        big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
        const float up = fmaxf(pow2_above(big), 0x1p-100f);  // (mul stays finite)
        const float mul = pow2_inverse(up) * 256.f;
        qk[h] = qk_scale * (up * (1.f / 256.f));
#pragma unroll
        for (int kk = 0; kk < KSTEPS; ++kk) {
          const float2 a = bf16x2_to_f2(qa[kk][h]), c = bf16x2_to_f2(qa[kk][2 + h]);
          qa[kk][h] = pack2<true>(a.x * mul, a.y * mul);
          qa[kk][2 + h] = pack2<true>(c.x * mul, c.y * mul);
        }
      }
    }
  }

  // The running maximum follows the tile's only when it is beaten by 2^8.
  __device__ __forceinline__ void follow(const float (&mx)[2]) {
    if (!__any_sync(kFull, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float mn = mx[h] > m[h] + 8.f ? mx[h] : m[h];
      const float alpha = mn == m[h] ? 1.f : fast_exp2(m[h] - mn);
      m[h] = mn;
      l[h] *= alpha;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        o[nb][2 * h] *= alpha;
        o[nb][2 * h + 1] *= alpha;
      }
    }
  }

  // One tile in the stage at shared address `stage`.  seen(s, h): how many of chunk s's 16 tokens
  // the row quad + 8 h sees; all: every row sees every token.
  template <class F>
  __device__ __forceinline__ void tile_16(uint32_t stage, bool all, F seen, int lane) {
    constexpr int SUB = T::SUB, NT8 = T::TK / 8;
    const uint32_t kt = stage, vt = stage + T::TILE;
    const int mat = lane >> 3, qi = lane & 3;
    float s[NT8][4];
#pragma unroll
    for (int nb = 0; nb < NT8; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
    for (int c = 0; c < SUB; ++c) {
      const int row = c * 16 + (lane & 7) + ((mat >> 1) << 3);
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
        uint32_t r0, r1, r2, r3;
        ldsm_x4(tile_piece<T>(kt, row, 2 * kk + (mat & 1)), r0, r1, r2, r3);
        mma16816<T::F16>(s[2 * c], qa[kk], r0, r1);
        mma16816<T::F16>(s[2 * c + 1], qa[kk], r2, r3);
      }
    }
    // s[nb]: tokens 8 nb + 2 qi + {0, 1} of rows quad, quad + 8
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nb = 0; nb < NT8; ++nb)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = s[nb][e] * qk[e >> 1];
        if (!all) x = (nb & 1) * 8 + 2 * qi + (e & 1) < seen(nb >> 1, e >> 1) ? x : -INFINITY;
        s[nb][e] = x;
        mx[e >> 1] = fmaxf(mx[e >> 1], x);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 2));
    }
    follow(mx);
    uint32_t pa[SUB][4];
#pragma unroll
    for (int nb = 0; nb < NT8; ++nb) {
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = s[nb][e];
        pr[e] = x != -INFINITY ? fast_exp2(x - m[e >> 1]) : 0.f;
        l[e >> 1] += pr[e];
      }
      pa[nb >> 1][2 * (nb & 1)] = pack2<T::F16>(pr[0], pr[1]);
      pa[nb >> 1][2 * (nb & 1) + 1] = pack2<T::F16>(pr[2], pr[3]);
    }
#pragma unroll
    for (int c = 0; c < SUB; ++c) {
      const int row = c * 16 + (lane & 7) + ((mat & 1) << 3);
#pragma unroll
      for (int nd = 0; nd < NB / 2; ++nd) {
        uint32_t r0, r1, r2, r3;
        ldsm_x4_t(tile_piece<T>(vt, row, 2 * nd + (mat >> 1)), r0, r1, r2, r3);
        mma16816<T::F16>(o[2 * nd], pa[c], r0, r1);
        mma16816<T::F16>(o[2 * nd + 1], pa[c], r2, r3);
      }
    }
  }

  // The same for an fp8 tile; ks, vs: its chunks' scales, or sc: its tokens' (K, then V).
  template <class F>
  __device__ __forceinline__ void tile_fp8(uint32_t stage, const float (&ks)[2], const float (&vs)[2],
                                           const float* sc, bool all, F seen, int lane) {
    constexpr int SUB = T::SUB, TK = T::TK, NT8 = 2 * SUB;
    const uint32_t kt = stage, vt = stage + T::TILE;
    const int mat = lane >> 3, qi = lane & 3, n = lane & 7;
    const int pair[2] = {2 * qi + 4 * (qi & 2), 2 * qi + 4};  // first of a block's two tokens
    // ---- logits: s[2 c + j] block j of chunk c
    float s[NT8][4];
#pragma unroll
    for (int nb = 0; nb < NT8; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
    const int krow = mat < 2 ? n + 2 * (n & 4) : n + 4;
#pragma unroll
    for (int kk = 0; kk < KSTEPS; kk += 2)
#pragma unroll
      for (int c = 0; c < SUB; ++c) {
        uint32_t r[4];  // block 0: k-steps kk, kk + 1; block 1
        ldsm_x4(tile_piece<T>(kt, 16 * c + krow, kk + (mat & 1)), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w = r[2 * j + h];
            mma16816<true>(s[2 * c + j], qa[kk + h], e4m3x2_to_f16x2(w), e4m3x2_to_f16x2(w >> 16));
          }
      }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int b = 0; b < NT8; ++b) {
      const int c = b >> 1, j = b & 1;
      float2 k2;
      if constexpr (T::TOKS)
        k2 = *reinterpret_cast<const float2*>(sc + 16 * c + pair[j]);
      else
        k2 = make_float2(ks[c], ks[c]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 x = fmul2(make_float2(s[b][2 * h], s[b][2 * h + 1]), make_float2(qk[h] * k2.x, qk[h] * k2.y));
        if (!all) {
          const int lim = seen(c, h);
          x.x = pair[j] < lim ? x.x : -INFINITY;
          x.y = pair[j] + 1 < lim ? x.y : -INFINITY;
        }
        s[b][2 * h] = x.x;
        s[b][2 * h + 1] = x.y;
        mx[h] = fmaxf(mx[h], fmaxf(x.x, x.y));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 2));
    }
    follow(mx);
    // the largest finite V scale (its magnitude) below `end`: warp-uniform
    auto largest = [&](float end) -> float {
      if constexpr (T::TOKS) {  // (magnitudes order as their bits do)
        const float a = fabsf(sc[TK + lane % TK]);
        return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(a < end ? a : 0.f)));
      } else {
        const float a = fabsf(vs[0]), c = fabsf(vs[SUB - 1]);
        return fmaxf(a < end ? a : 0.f, c < end ? c : 0.f);
      }
    };
    // the unit to the scale x, if need be; the least scale that it serves (0: any)
    auto serve = [&](float x) -> float {
      if (x > vref || (x > 0.f && x < vref * kVRange)) {
        const float f = move_v_unit(x, vref, vtop);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nb][e] *= f;
      }
      return x < vref * kVRange ? 0.f : vref * kVRange;
    };
    // weights (a masked logit, -inf, gives 0, also while the row has seen no key) and o += P V for
    // the V scales that `factor` does not make zero
    auto attend = [&](auto factor, bool first) {
      const float base[2] = {m[0] == -INFINITY ? 0.f : -m[0], m[1] == -INFINITY ? 0.f : -m[1]};
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t pa[SUB][4];
#pragma unroll
      for (int b = 0; b < NT8; ++b) {
        const int c = b >> 1, j = b & 1;
        float2 v2;
        if constexpr (T::TOKS) {
          v2 = *reinterpret_cast<const float2*>(sc + TK + 16 * c + pair[j]);
          v2 = make_float2(factor(v2.x), factor(v2.y));
        } else {
          const float f = factor(vs[c]);
          v2 = make_float2(f, f);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 e = fadd2(make_float2(s[b][2 * h], s[b][2 * h + 1]), make_float2(base[h], base[h]));
          e.x = fast_exp2(e.x);
          e.y = fast_exp2(e.y);
          sum[h] = fadd2(sum[h], e);
          e = fmul2(e, v2);
          pa[c][2 * j + h] = pack2<true>(e.x, e.y);
        }
      }
      if (first) {
        l[0] += sum[0].x + sum[0].y;
        l[1] += sum[1].x + sum[1].y;
      }
      // row i = 4 qi' + 2 j + e of a chunk's matrix is token e of block j of thread qi'
      const int i = lane & 15, iq = i >> 2;
      const int vrow = (SUB == 2 ? lane & 16 : 0) + ((i & 2) ? 2 * iq + 4 : 2 * iq + 4 * (iq & 2)) + (i & 1);
#pragma unroll
      for (int nd = 0; nd < NB / 2; ++nd) {
        uint32_t r[2 * SUB];  // chunk 0: channels quad, quad + 8 of the 16; chunk 1
        ldsm_b8_t(tile_piece<T>(vt, vrow, nd), r);
#pragma unroll
        for (int c = 0; c < SUB; ++c)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w = r[2 * c + j];
            mma16816<true>(o[2 * nd + j], pa[c], e4m3x2_to_f16x2(w), e4m3x2_to_f16x2(w >> 16));
          }
      }
    };
    bool served;  // the unit serves every scale of the tile, as a rule
    if constexpr (T::TOKS) {
      const float a = fabsf(sc[TK + lane % TK]);
      served = __all_sync(kFull, a <= vref && a >= vref * kVRange);
    } else {
      served = fmaxf(fabsf(vs[0]), fabsf(vs[SUB - 1])) <= vref &&
               fminf(fabsf(vs[0]), fabsf(vs[SUB - 1])) >= vref * kVRange;
    }
    constexpr bool ONE = !T::TOKS && SUB == 1;  // (one scale a tile)
    if (ONE && !served) serve(largest(INFINITY));
    if (ONE || served) {
      const float vinv = pow2_inverse(vref) * kPLift;
      attend([&](float v) { return v * vinv; }, true);
    } else {  // a pass for the scales that one unit serves after the other, from the largest on
      float done = __uint_as_float(0x7fc00000u);  // scales from here on are in o (NaN: none yet)
#pragma unroll 1
      for (float x = largest(INFINITY); x > 0.f || done != done;) {
        const float floor = serve(x), vinv = pow2_inverse(vref) * kPLift;
        // (NaN and infinity are in, in the first pass at least)
        attend([&](float v) { return fabsf(v) < floor || fabsf(v) >= done ? 0.f : v * vinv; }, done != done);
        done = floor;
        x = largest(floor);
      }
    }
  }

  // The state of this warp into slot `slot` of the staged ones (the quad's sums joined).
  __device__ __forceinline__ void stage_state(float* obuf, float2* ml, int slot, int lane) {
    const int quad = lane >> 2, qi = lane & 3;
    const float f = T::FP8 ? vref * (1.f / kPLift) : 1.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(kFull, l[h], 1);
      l[h] += __shfl_xor_sync(kFull, l[h], 2);
      float* row = obuf + (slot * T::ROWS + quad + 8 * h) * T::OSTR;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        *reinterpret_cast<float2*>(row + 8 * nb + 2 * qi) = make_float2(o[nb][2 * h] * f, o[nb][2 * h + 1] * f);
      if (qi == 0) ml[slot * T::ROWS + quad + 8 * h] = make_float2(m[h], l[h]);
    }
  }
};

// States s = 0 .. states - 1 of one row merged for four channels: (max, sum) at ml_of(s), the
// channels' accumulators at o_of(s).  Returns the sum's (max, sum).
template <class FM, class FO>
__device__ __forceinline__ float2 merge_states(int states, FM ml_of, FO o_of, float4& O) {
  float m = -INFINITY;
  for (int s = 0; s < states; ++s) m = fmaxf(m, ml_of(s)->x);
  float l = 0.f;
  O = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < states; ++s) {
    const float2 x = *ml_of(s);
    if (x.y == 0.f) continue;  // no key in this state
    const float w = fast_exp2(x.x - m);
    const float4 v = *reinterpret_cast<const float4*>(o_of(s));
    l = __fmaf_rn(w, x.y, l);
    O.x = __fmaf_rn(w, v.x, O.x);
    O.y = __fmaf_rn(w, v.y, O.y);
    O.z = __fmaf_rn(w, v.z, O.z);
    O.w = __fmaf_rn(w, v.w, O.w);
  }
  return make_float2(m, l);
}

}  // namespace pa
