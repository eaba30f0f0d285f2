// Attention of a warp's query rows over chunks of 16 tokens of a 4-bit cache.
//
// With codes c (taken as the integers c - 8, exact in f16), steps s, lows w and mid_j = w_j + 8 s_j,
//     logit_j = scale (s_j <q, c_j - 8> + mid_j sum(q)),
//     out = (sum_j p_j s_j (c_j - 8) + sum_j p_j mid_j) / sum_j p_j,
// so that neither product needs more than the codes and what belongs to a token enters its logit and
// its weight.  Both products run transposed on mma.sync m16n8k16, S^T = K Q^T and O^T = V^T P^T, with
// tokens (channels) along the MMA's 16 rows and query rows along its 8 columns: a tile of up to 8
// query rows then costs half of what one of 16 does, which is what widening the codes leaves to save.
// A word of codes is eight channels; two halves of it masked into the mantissa of 1024 (or 64; the
// conversion that int4.cuh cites), less 1032 (72), are two f16 operands.  The order of channels inside
// a k-step is the queries' own affair, so a K row's words are operands as they lie.  A V operand holds
// one channel of two tokens: one byte permute brings the halves of two tokens' words together.  P^T
// comes from S^T through movmatrix.
//
// What bounds it are the instructions of the few warps whose state fits the registers, so little is
// done twice: the queries' fragments lie in shared memory, one copy a CTA; a lane a token makes a
// token's factors from its pairs; of a K word's two masked halves one is taken as 64 + c, the 72 too
// much being in the logits' accumulators from the start (72 times the sum of those channels' queries);
// a tile that every row sees whole, with V steps that fit the accumulators' unit, passes no mask.
//
// Where bits are given up:
//   - A weight times its V step is rounded to f16, the operand's type, while the weights' sum is taken
// before it: 2^-12 of a weight at most.  An operand for the rest would double the second product, which is
// 91 of a chunk's 316 instructions.  A bf16 output hides it (relative error against 64 bits 0.00164 to
// 0.00168, 0.00164 to 0.00171 for fp32 arithmetic throughout); an fp16 output's is 2.3e-4 to 2.7e-4 where
// its own rounding is 2.0e-4 to 2.1e-4.
//   - A bf16 query goes into f16 times a power of two: elements below 2^-22 of its largest lose bits.  In
// two f16 terms the first product would take twice as long.
//   - 64 + c in place of c - 8 costs a logit up to three bits of fp32 (lse within 8e-7 relative; 2e-7
// for fp32 throughout), and a subtraction less for every other operand of K.
//
// Thread (quad, qi) = (lane / 4, lane % 4): tokens quad and quad + 8 of a chunk and query rows
// 8 t + 2 qi, + 1 of the logits; tokens 2 qi, 2 qi + 1 (+ 8) of V.
#pragma once

#include "int4.cuh"
#include "page_stream.cuh"

namespace pa {

// (c - 8) of nibbles 0 and 4 / 1 and 5 of a word's (its high half moved down: 2 and 6 / 3 and 7).
__device__ __forceinline__ uint32_t int4_even(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b32 t;\n lop3.b32 t, %1, 0x000f000f, %2, 0xea;\n sub.rn.f16x2 %0, t, %3;\n}"
      : "=r"(r)
      : "r"(w), "r"(0x64006400u), "r"(0x64086408u));
  return r;
}
__device__ __forceinline__ uint32_t int4_odd_64(uint32_t w) {  // 64 + c
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(r) : "r"(w), "r"(0x54005400u));
  return r;
}
__device__ __forceinline__ uint32_t int4_odd(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b32 t;\n lop3.b32 t, %1, 0x00f000f0, %2, 0xea;\n sub.rn.f16x2 %0, t, %3;\n}"
      : "=r"(r)
      : "r"(w), "r"(0x54005400u), "r"(0x54805480u));
  return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int D_, int NT_, int QK_>
struct Int4Attention {
  static constexpr int D = D_, NT = NT_, QK = QK_;
  static constexpr int ROWS = 8 * NT;      // query rows
  static constexpr int ROW = D / 2;        // bytes of a cached row
  static constexpr int KW = D / 32;        // words of a K row that a lane holds (two k-steps each)
  static constexpr int VW = D / 64;        // words of a V row that a lane holds (8 channels each)
  static constexpr int MB = D / 16;        // 16-channel blocks of the output
  static constexpr int OSTR = D + 4;       // floats between rows of a staged accumulator
  static constexpr int O_SLOT = ROWS * OSTR * 4;
  static constexpr int QUERY = KW * 32 * NT * 16;  // bytes of the queries' fragments

  // Rows of a tile in shared memory: as the TMA boxes bring them, 16-byte pieces swizzled over rows of
  // 64 bytes (by bits 1 and 2 of the row) and 128 (by its low three bits).  Which of the tokens
  // 2 qi, 2 qi + 1 a lane reads first is chosen so that a phase's lanes lie in distinct banks.
  static __device__ __forceinline__ int first_token(int qi) {
    return D == 128 ? qi & 1 : D == 64 ? qi >> 1 : 0;
  }
  // The lane's words of the K row of token quad + 8 h of chunk c: group j of GW.
  static constexpr int GW = cmin(KW, 4);
  static __device__ __forceinline__ void k_words(uint32_t tile, int c, int h, int j, int lane,
                                                 uint32_t (&w)[GW]) {
    const int quad = lane >> 2, qi = lane & 3;
    const uint32_t row = tile + (16 * c + 8 * h + quad) * ROW;
    if constexpr (D == 64) {
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(row + 8 * qi));
    } else {
      const int piece = D == 128 ? qi ^ (quad >> 1) : (2 * qi + j) ^ quad;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(row + (piece << 4)));
    }
  }
  // Its words of the V row of one of the tokens 2 qi, 2 qi + 1 (+ 8 h), the first one for e = 0.
  static __device__ __forceinline__ void v_words(uint32_t tile, int c, int h, int e, int lane,
                                                 uint32_t (&w)[VW]) {
    const int quad = lane >> 2, qi = lane & 3, r = 2 * qi + (first_token(qi) ^ e);
    const uint32_t row = tile + (16 * c + 8 * h + r) * ROW;
    if constexpr (D == 64)
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(row + 4 * quad));
    else if constexpr (D == 128)
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                   : "=r"(w[0]), "=r"(w[1])
                   : "r"(row + (((quad >> 1) ^ qi) << 4) + 8 * (quad & 1)));
    else
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(row + ((quad ^ r) << 4)));
  }

  // Of rows 8 t + 2 qi, + 1: the logit's factor (log2 units, >= 0), the sum of q (as scaled), -72 times
  // its sum over the channels that K words hold in odd nibbles, minus the running maximum in log2
  // units, and the sums of the weights and of the weights times low + 8 step.
  float2 scale[NT], qsum[NT], start[NT], base[NT], l[NT], low[NT];
  float o[MB][NT][4];  // channels 8 W + 2 j, + 1 of the two rows, in units of vref / kPLift
  float vref, vtop;

  __device__ __forceinline__ void clear() {
    vref = vtop = kPow2Least;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      base[t] = make_float2(INFINITY, INFINITY);
      l[t] = low[t] = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < MB; ++j) o[j][t][0] = o[j][t][1] = o[j][t][2] = o[j][t][3] = 0.f;
    }
  }

  // row_of(r): query row r of the tile, or null for a padding row.  The rows' fragments go to `query`
  // in shared memory: [KW][32 lanes][NT][4 words], of which warp `warp` of four writes its share.
  template <class F>
  __device__ __forceinline__ void load_q(F row_of, float qk_scale, uint4* query, int warp, int lane) {
    const int quad = lane >> 2, qi = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const char* row = row_of(8 * t + quad);
      uint32_t h[KW][4];  // word w of this lane: channels 8 W .. 8 W + 7 with W = qi KW + w
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const uint4 v = row ? __ldg(reinterpret_cast<const uint4*>(row) + qi * KW + w)
                            : make_uint4(0u, 0u, 0u, 0u);
        h[w][0] = v.x;
        h[w][1] = v.y;
        h[w][2] = v.z;
        h[w][3] = v.w;
      }
      float up = 1.f;
      if constexpr (QK == Q_BF16) {
        // to f16, times the power of two that brings the largest element to [2^7, 2^8)
        float big = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = bf16x2_to_f2(h[w][e]);
            big = fmaxf(big, fmaxf(fabsf(a.x), fabsf(a.y)));
          }
        big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
        big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
        up = fmaxf(pow2_above(big), 0x1p-100f);  // (mul stays finite)
        const float mul = pow2_inverse(up) * 256.f;
        up *= 1.f / 256.f;
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = bf16x2_to_f2(h[w][e]);
            h[w][e] = pack2<true>(a.x * mul, a.y * mul);
          }
      }
      if (qk_scale < 0.f) {  // the sign goes into the query: a row's largest logit is its largest product
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) h[w][e] ^= 0x80008000u;
      }
      float even = 0.f, odd = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = f16x2_to_f2(h[w][e]);
          even += a.x;
          odd += a.y;
        }
        // pairs of channels (0, 4), (1, 5), (2, 6), (3, 7), as a word's nibbles come
        if (warp == w % 4)
          query[(w * 32 + lane) * NT + t] =
              make_uint4(__byte_perm(h[w][0], h[w][2], 0x5410), __byte_perm(h[w][0], h[w][2], 0x7632),
                         __byte_perm(h[w][1], h[w][3], 0x5410), __byte_perm(h[w][1], h[w][3], 0x7632));
      }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        even += __shfl_xor_sync(kFull, even, d);
        odd += __shfl_xor_sync(kFull, odd, d);
      }
      // row r's sums and scale are with the lanes 4 r .. 4 r + 3
      const float sc = fabsf(qk_scale) * up, sum = even + odd, st = -72.f * odd;
      scale[t] = make_float2(__shfl_sync(kFull, sc, 8 * qi), __shfl_sync(kFull, sc, 8 * qi + 4));
      qsum[t] = make_float2(__shfl_sync(kFull, sum, 8 * qi), __shfl_sync(kFull, sum, 8 * qi + 4));
      start[t] = make_float2(__shfl_sync(kFull, st, 8 * qi), __shfl_sync(kFull, st, 8 * qi + 4));
    }
  }

  // The running maxima follow the raw logits mx only when one beats its row's by 2^8.  (A row that has
  // seen no key has base +inf, and a masked logit gives -inf or NaN, which beats nothing.)
  __device__ __forceinline__ void follow(const float2 (&mx)[NT]) {
    bool beaten = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      beaten |= __fmaf_rn(mx[t].x, scale[t].x, base[t].x) > 8.f ||
                __fmaf_rn(mx[t].y, scale[t].y, base[t].y) > 8.f;
    if (!__any_sync(kFull, beaten)) return;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float2 a = mx[t];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        a.x = fmaxf(a.x, __shfl_xor_sync(kFull, a.x, d));
        a.y = fmaxf(a.y, __shfl_xor_sync(kFull, a.y, d));
      }
      const bool up[2] = {__fmaf_rn(a.x, scale[t].x, base[t].x) > 8.f,
                          __fmaf_rn(a.y, scale[t].y, base[t].y) > 8.f};
      const float2 n = make_float2(up[0] ? -(a.x * scale[t].x) : base[t].x,
                                   up[1] ? -(a.y * scale[t].y) : base[t].y);
      const float2 f = make_float2(up[0] ? fast_exp2(n.x - base[t].x) : 1.f,
                                   up[1] ? fast_exp2(n.y - base[t].y) : 1.f);
      base[t] = n;
      l[t] = fmul2(l[t], f);
      low[t] = fmul2(low[t], f);
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        o[j][t][0] *= f.x;
        o[j][t][1] *= f.y;
        o[j][t][2] *= f.x;
        o[j][t][3] *= f.y;
      }
    }
  }

  // S^T = K Q^T of SUB chunks, their K rows at shared address kt and the queries' fragments at `query`,
  // into s.
  template <int SUB>
  __device__ __forceinline__ void keys(uint32_t kt, const uint4* query, float (&s)[SUB][NT][4], int lane) {
    uint32_t w[SUB][2][GW];
#pragma unroll
    for (int c = 0; c < SUB; ++c)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        s[c][t][0] = s[c][t][2] = start[t].x;
        s[c][t][1] = s[c][t][3] = start[t].y;
      }
#pragma unroll
    for (int i = 0; i < KW; ++i) {
      if (i % GW == 0) {
#pragma unroll
        for (int c = 0; c < SUB; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) k_words(kt, c, h, i / GW, lane, w[c][h]);
      }
      uint4 q[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) q[t] = query[(i * 32 + lane) * NT + t];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int c = 0; c < SUB; ++c) {
          const uint32_t u0 = k ? w[c][0][i % GW] >> 8 : w[c][0][i % GW];
          const uint32_t u1 = k ? w[c][1][i % GW] >> 8 : w[c][1][i % GW];
          const uint32_t a[4] = {int4_even(u0), int4_even(u1), int4_odd_64(u0), int4_odd_64(u1)};
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma16816<true>(s[c][t], a, k ? q[t].z : q[t].x, k ? q[t].w : q[t].y);
        }
    }
  }

  // O^T += V^T P^T of SUB chunks, V rows at vt, weights (times their V steps) in pb.
  template <int SUB>
  __device__ __forceinline__ void values(uint32_t vt, const uint32_t (&pb)[SUB][NT][2], int lane) {
    const uint32_t sel = first_token(lane & 3) ? 0x1054u : 0x5410u;  // low halves of tokens 2 qi, 2 qi + 1
#pragma unroll
    for (int c = 0; c < SUB; ++c) {
      uint32_t w[2][2][VW];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v_words(vt, c, h, 0, lane, w[h][0]);
        v_words(vt, c, h, 1, lane, w[h][1]);
      }
#pragma unroll
      for (int i = 0; i < VW; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // channels 0 .. 3, 4 .. 7 of the word
          uint32_t z[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) z[h] = __byte_perm(w[h][0][i], w[h][1][i], sel + (k ? 0x2222u : 0u));
          const uint32_t y[2] = {z[0] >> 8, z[1] >> 8};
          const uint32_t a[4] = {int4_even(z[0]), int4_odd(z[0]), int4_even(z[1]), int4_odd(z[1])};
          const uint32_t b[4] = {int4_even(y[0]), int4_odd(y[0]), int4_even(y[1]), int4_odd(y[1])};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma16816<true>(o[4 * i + 2 * k][t], a, pb[c][t][0], pb[c][t][1]);
            mma16816<true>(o[4 * i + 2 * k + 1][t], b, pb[c][t][0], pb[c][t][1]);
          }
        }
    }
  }

  // The raw logits of a tile in place of the products s, with the tokens' factors: (K step, K low + 8
  // step, V factor, V low + 8 step), zeros where no row may see the token; the running maxima follow.
  // vf: the V factors of tokens quad + 8 h, in x the one for the weight, in y low + 8 step.
  // HOT: every row sees every token; otherwise sees(c, h, t) says which of the rows 8 t + 2 qi, + 1 see
  // token quad + 8 h of chunk c.
  template <int SUB, bool HOT, class FS>
  __device__ __forceinline__ void logits(float (&s)[SUB][NT][4], const float4* factors,
                                         float2 (&vf)[SUB][2], FS sees, int lane) {
    const int quad = lane >> 2;
    float2 mx[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) mx[t] = make_float2(-INFINITY, -INFINITY);
#pragma unroll
    for (int c = 0; c < SUB; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 f = factors[16 * c + 8 * h + quad];
        vf[c][h] = make_float2(f.z, f.w);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float x0 = __fmaf_rn(s[c][t][2 * h], f.x, f.y * qsum[t].x);
          float x1 = __fmaf_rn(s[c][t][2 * h + 1], f.x, f.y * qsum[t].y);
          if (!HOT) {
            const uint2 ok = sees(c, h, t);
            x0 = ok.x ? x0 : -INFINITY;
            x1 = ok.y ? x1 : -INFINITY;
          }
          mx[t].x = fmaxf(mx[t].x, x0);
          mx[t].y = fmaxf(mx[t].y, x1);
          s[c][t][2 * h] = x0;
          s[c][t][2 * h + 1] = x1;
        }
      }
    follow(mx);
  }

  // Weights exp2(scale x - maximum), summed alone and times low + 8 step, then times `factor` of their V
  // factor as operands; a masked logit (-inf) gives 0.
  template <int SUB, bool HOT, class FF>
  __device__ __forceinline__ void weigh(const float (&s)[SUB][NT][4], const float2 (&vf)[SUB][2],
                                        FF factor, bool sums, uint32_t (&pb)[SUB][NT][2]) {
#pragma unroll
    for (int c = 0; c < SUB; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float f = factor(vf[c][h].x), mid = vf[c][h].y;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float x0 = s[c][t][2 * h], x1 = s[c][t][2 * h + 1];
          float2 e = make_float2(fast_exp2(__fmaf_rn(x0, scale[t].x, base[t].x)),
                                 fast_exp2(__fmaf_rn(x1, scale[t].y, base[t].y)));
          float2 m = make_float2(mid, mid), g = make_float2(f, f);
          if (!HOT) {  // (nothing of a token that its row does not see, whatever its V pair holds)
            if (x0 == -INFINITY) e.x = m.x = g.x = 0.f;
            if (x1 == -INFINITY) e.y = m.y = g.y = 0.f;
          }
          if (sums) {
            l[t] = fadd2(l[t], e);
            low[t].x = __fmaf_rn(e.x, m.x, low[t].x);
            low[t].y = __fmaf_rn(e.y, m.y, low[t].y);
          }
          pb[c][t][h] = transpose8(pack2<true>(e.x * g.x, e.y * g.y));
        }
      }
  }

  // What follows a tile's products s where every row sees every token and the V factors are the V steps
  // over the accumulators' unit times kPLift.
  template <int SUB>
  __device__ __forceinline__ void whole_tile(float (&s)[SUB][NT][4], uint32_t vt, const float4* factors,
                                             int lane) {
    uint32_t pb[SUB][NT][2];
    float2 vf[SUB][2];
    logits<SUB, true>(s, factors, vf, [](int, int, int) { return make_uint2(1, 1); }, lane);
    weigh<SUB, true>(s, vf, [](float v) { return v; }, true, pb);
    values<SUB>(vt, pb, lane);
  }

  // The same whatever its rows see and its V steps are (the V factors are the steps).
  template <int SUB, class FS>
  __device__ __forceinline__ void any_tile(float (&s)[SUB][NT][4], uint32_t vt, const float4* factors,
                                           FS sees, int lane) {
    uint32_t pb[SUB][NT][2];
    float2 vf[SUB][2];
    logits<SUB, false>(s, factors, vf, sees, lane);
    // the largest finite V step (its magnitude) below `end`: warp-uniform
    auto largest = [&](float end) -> float {
      float a = 0.f;
#pragma unroll
      for (int c = 0; c < SUB; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float v = fabsf(vf[c][h].x);
          a = fmaxf(a, v < end ? v : 0.f);
        }
      return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(a)));
    };
    // a pass for the steps that one unit serves after the other, from the largest on
    float done = __uint_as_float(0x7fc00000u);  // steps from here on are in o (NaN: none yet)
#pragma unroll 1
    for (float v = largest(INFINITY); v > 0.f || done != done;) {
      if (v > vref || (v > 0.f && v < vref * kVRange)) {  // the unit to the step v
        const float f = move_v_unit(v, vref, vtop);
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][t][e] *= f;
      }
      // the least step that it serves (0: any); NaN and infinity are in, in the first pass at least
      const float floor = v < vref * kVRange ? 0.f : vref * kVRange;
      const float vinv = pow2_inverse(vref) * kPLift;
      weigh<SUB, false>(s, vf, [&](float a) { return fabsf(a) < floor || fabsf(a) >= done ? 0.f : a * vinv; },
                        done != done, pb);
      values<SUB>(vt, pb, lane);
      done = floor;
      v = largest(floor);
    }
  }

  // The state of this warp into slot `slot` of the staged ones.
  __device__ __forceinline__ void stage_state(float* obuf, float2* ml, int slot, int lane) {
    const int quad = lane >> 2, qi = lane & 3;
    const float f = vref * (1.f / kPLift);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l[t].x += __shfl_xor_sync(kFull, l[t].x, d);
        l[t].y += __shfl_xor_sync(kFull, l[t].y, d);
        low[t].x += __shfl_xor_sync(kFull, low[t].x, d);
        low[t].y += __shfl_xor_sync(kFull, low[t].y, d);
      }
      const int r = slot * ROWS + 8 * t + 2 * qi;
      float* row0 = obuf + r * OSTR + 8 * VW * quad;
      float* row1 = row0 + OSTR;
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        *reinterpret_cast<float2*>(row0 + 2 * j) =
            make_float2(__fmaf_rn(o[j][t][0], f, low[t].x), __fmaf_rn(o[j][t][2], f, low[t].x));
        *reinterpret_cast<float2*>(row1 + 2 * j) =
            make_float2(__fmaf_rn(o[j][t][1], f, low[t].y), __fmaf_rn(o[j][t][3], f, low[t].y));
      }
      if (quad == 0) {
        ml[r] = make_float2(-base[t].x, l[t].x);
        ml[r + 1] = make_float2(-base[t].y, l[t].y);
      }
    }
  }
};

}  // namespace pa
