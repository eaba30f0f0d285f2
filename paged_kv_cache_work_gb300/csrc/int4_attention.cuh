// Attention of a warp's query rows over chunks of 16 tokens of a 4-bit cache.
//
// With codes c (taken as the integers c - 8, exact in f16), steps s, lows w and mid_j = w_j + 8 s_j,
//     logit_j = scale (s_j <q, c_j - 8> + mid_j sum(q)),
//     out = (sum_j p_j s_j (c_j - 8) + sum_j p_j mid_j) / sum_j p_j,
// so that neither product needs more than the codes and what belongs to a token enters its logit and
// its weight.  Both products run transposed on mma.sync m16n8k16, S^T = K Q^T and O^T = V^T P^T, with
// tokens (channels) along the MMA's 16 rows and query rows along its 8 columns: a tile of up to 8
// query rows then costs half of what one of 16 does, which is what widening the codes leaves to save.
// A word of codes is eight channels; two halves of it masked into the mantissa of 1024 (or 64), less
// 1032 (72), are two f16 operands.  The order of channels inside a k-step is the queries' own affair,
// so a K row's words are operands as they lie.  A V operand holds one channel of two tokens: one byte
// permute brings the halves of two tokens' words together.  P^T comes from S^T through movmatrix.
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
  static constexpr int KSTEPS = D / 16;
  static constexpr int MB = D / 16;        // 16-channel blocks of the output
  static constexpr int OSTR = D + 4;       // floats between rows of a staged accumulator
  static constexpr int O_SLOT = ROWS * OSTR * 4;

  // Rows of a tile in shared memory: as the TMA boxes bring them, 16-byte pieces swizzled over rows of
  // 64 bytes (by bits 1 and 2 of the row) and 128 (by its low three bits).  Which of the tokens
  // 2 qi, 2 qi + 1 a lane reads first is chosen so that a phase's lanes lie in distinct banks.
  static __device__ __forceinline__ int first_token(int qi) {
    return D == 128 ? qi & 1 : D == 64 ? qi >> 1 : 0;
  }
  // The lane's words of the K row of token quad + 8 h of chunk c.
  static __device__ __forceinline__ void k_words(uint32_t tile, int c, int h, int lane, uint32_t (&w)[KW]) {
    const int quad = lane >> 2, qi = lane & 3;
    const uint32_t row = tile + (16 * c + 8 * h + quad) * ROW;
    if constexpr (D == 64) {
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(row + 8 * qi));
    } else {
#pragma unroll
      for (int j = 0; j < KW / 4; ++j) {
        const int piece = D == 128 ? qi ^ (quad >> 1) : (2 * qi + j) ^ quad;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * j]), "=r"(w[4 * j + 1]), "=r"(w[4 * j + 2]), "=r"(w[4 * j + 3])
                     : "r"(row + (piece << 4)));
      }
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

  uint32_t qb[KSTEPS][NT][2];
  float2 scale[NT], qsum[NT];  // of rows 8 t + 2 qi, + 1: logit scale (log2 units), sum of q (as scaled)
  float2 m[NT], l[NT], low[NT];
  float o[MB][NT][4];  // channels 8 W + 2 j, + 1 of the two rows, in units of vref / kPLift
  float vref, vtop;

  __device__ __forceinline__ void clear() {
    vref = vtop = kPow2Least;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t] = make_float2(-INFINITY, -INFINITY);
      l[t] = low[t] = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < MB; ++j) o[j][t][0] = o[j][t][1] = o[j][t][2] = o[j][t][3] = 0.f;
    }
  }

  // row_of(r): query row r of the tile, or null for a padding row.
  template <class F>
  __device__ __forceinline__ void load_q(F row_of, float qk_scale, int lane) {
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
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = f16x2_to_f2(h[w][e]);
          sum += a.x + a.y;
        }
        // pairs of channels (0, 4), (1, 5), (2, 6), (3, 7), as a word's nibbles come
        qb[2 * w][t][0] = __byte_perm(h[w][0], h[w][2], 0x5410);
        qb[2 * w][t][1] = __byte_perm(h[w][0], h[w][2], 0x7632);
        qb[2 * w + 1][t][0] = __byte_perm(h[w][1], h[w][3], 0x5410);
        qb[2 * w + 1][t][1] = __byte_perm(h[w][1], h[w][3], 0x7632);
      }
      sum += __shfl_xor_sync(kFull, sum, 1);
      sum += __shfl_xor_sync(kFull, sum, 2);
      // row r's sum and scale are with the lanes 4 r .. 4 r + 3
      const float sc = qk_scale * up;
      scale[t] = make_float2(__shfl_sync(kFull, sc, 8 * qi), __shfl_sync(kFull, sc, 8 * qi + 4));
      qsum[t] = make_float2(__shfl_sync(kFull, sum, 8 * qi), __shfl_sync(kFull, sum, 8 * qi + 4));
    }
  }

  // The running maxima follow the logits x only when one beats its row's by 2^8.
  __device__ __forceinline__ void follow(const float2 (&mx)[NT]) {
    bool beaten = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) beaten |= mx[t].x > m[t].x + 8.f || mx[t].y > m[t].y + 8.f;
    if (!__any_sync(kFull, beaten)) return;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float2 a = mx[t];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        a.x = fmaxf(a.x, __shfl_xor_sync(kFull, a.x, d));
        a.y = fmaxf(a.y, __shfl_xor_sync(kFull, a.y, d));
      }
      const float2 n = make_float2(a.x > m[t].x + 8.f ? a.x : m[t].x, a.y > m[t].y + 8.f ? a.y : m[t].y);
      const float2 f = make_float2(n.x == m[t].x ? 1.f : fast_exp2(m[t].x - n.x),
                                   n.y == m[t].y ? 1.f : fast_exp2(m[t].y - n.y));
      m[t] = n;
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

  // SUB chunks of 16 tokens, their K rows at shared address kt and V rows at vt.
  // ks, vs [c][h]: (step, low) of token quad + 8 h, zero where no row may see the token;
  // sees(c, h, t): which of the rows 8 t + 2 qi, + 1 see token quad + 8 h of chunk c; all: every row
  // sees every token.
  template <int SUB, class FS>
  __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, const float2 (&ks)[SUB][2],
                                       const float2 (&vs)[SUB][2], bool all, FS sees, int lane) {
    const int qi = lane & 3;
    float2 x[SUB][2][NT];  // logits of token quad + 8 h
#pragma unroll
    for (int c = 0; c < SUB; ++c) {
      float s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
      uint32_t w[2][KW];
      k_words(kt, c, 0, lane, w[0]);
      k_words(kt, c, 1, lane, w[1]);
#pragma unroll
      for (int i = 0; i < KW; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t u0 = k ? w[0][i] >> 8 : w[0][i], u1 = k ? w[1][i] >> 8 : w[1][i];
          const uint32_t a[4] = {int4_even(u0), int4_even(u1), int4_odd(u0), int4_odd(u1)};
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816<true>(s[t], a, qb[2 * i + k][t][0], qb[2 * i + k][t][1]);
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float step = ks[c][h].x, mid = __fmaf_rn(8.f, step, ks[c][h].y);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float2 v = fmul2(make_float2(mid, mid), qsum[t]);
          v = ffma2(make_float2(s[t][2 * h], s[t][2 * h + 1]), make_float2(step, step), v);
          v = fmul2(v, scale[t]);
          if (!all) {
            const uint2 ok = sees(c, h, t);
            v.x = ok.x ? v.x : -INFINITY;
            v.y = ok.y ? v.y : -INFINITY;
          }
          x[c][h][t] = v;
        }
      }
    }
    float2 mx[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      mx[t] = x[0][0][t];
#pragma unroll
      for (int c = 0; c < SUB; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[t].x = fmaxf(mx[t].x, x[c][h][t].x);
          mx[t].y = fmaxf(mx[t].y, x[c][h][t].y);
        }
    }
    follow(mx);
    // the largest finite V step (its magnitude) below `end`: warp-uniform
    auto largest = [&](float end) -> float {
      float a = 0.f;
#pragma unroll
      for (int c = 0; c < SUB; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float v = fabsf(vs[c][h].x);
          a = fmaxf(a, v < end ? v : 0.f);
        }
      return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(a)));
    };
    // the unit to the step v, if need be; the least step that it serves (0: any)
    auto serve = [&](float v) -> float {
      if (v > vref || (v > 0.f && v < vref * kVRange)) {
        const float f = move_v_unit(v, vref, vtop);
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][t][e] *= f;
      }
      return v < vref * kVRange ? 0.f : vref * kVRange;
    };
    // weights (a masked logit, -inf, gives 0, also while the row has seen no key) and O^T += V^T P^T
    // for the V steps that `factor` does not make zero
    auto attend = [&](auto factor, bool first) {
      uint32_t pb[SUB][NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float2 base = make_float2(m[t].x == -INFINITY ? 0.f : -m[t].x,
                                        m[t].y == -INFINITY ? 0.f : -m[t].y);
#pragma unroll
        for (int c = 0; c < SUB; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float step = vs[c][h].x, f = factor(step);
            float2 p = fadd2(x[c][h][t], base);
            p.x = fast_exp2(p.x);
            p.y = fast_exp2(p.y);
            if (first) {
              const float mid = __fmaf_rn(8.f, step, vs[c][h].y);
              l[t] = fadd2(l[t], p);
              low[t] = ffma2(p, make_float2(mid, mid), low[t]);
            }
            p = fmul2(p, make_float2(f, f));
            pb[c][t][h] = transpose8(pack2<true>(p.x, p.y));
          }
      }
      const uint32_t sel = first_token(qi) ? 0x1054u : 0x5410u;  // low halves of tokens 2 qi, 2 qi + 1
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
    };
    bool mine = true;
#pragma unroll
    for (int c = 0; c < SUB; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a = fabsf(vs[c][h].x);
        mine &= a <= vref && (a >= vref * kVRange || a == 0.f);
      }
    if (__all_sync(kFull, mine)) {  // the unit serves every step of the tile, as a rule
      const float vinv = pow2_inverse(vref) * kPLift;
      attend([&](float v) { return v * vinv; }, true);
    } else {  // a pass for the steps that one unit serves after the other, from the largest on
      float done = __uint_as_float(0x7fc00000u);  // steps from here on are in o (NaN: none yet)
#pragma unroll 1
      for (float v = largest(INFINITY); v > 0.f || done != done;) {
        const float floor = serve(v), vinv = pow2_inverse(vref) * kPLift;
        // (NaN and infinity are in, in the first pass at least)
        attend([&](float a) { return fabsf(a) < floor || fabsf(a) >= done ? 0.f : a * vinv; }, done != done);
        done = floor;
        v = largest(floor);
      }
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
        ml[r] = make_float2(m[t].x, l[t].x);
        ml[r + 1] = make_float2(m[t].y, l[t].y);
      }
    }
  }
};

}  // namespace pa
