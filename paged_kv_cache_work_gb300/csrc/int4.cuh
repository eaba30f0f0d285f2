// Rows of a 4-bit cache: codes c in 0 .. 15, two a byte, and a pair (step, low) of the queries' type
// for each token and kv head; a value is low + step c.
//
// D / 8 lanes quantise a row, eight consecutive elements each.  low is the row's least
// element rounded down to the pair's type (an element itself when the row has that type), step the
// least number of the type that is not below (max - low) / 15, so that every quotient lies in
// [0, 15] and none is clipped.  One row of pairs for a page and kv head lies together: the decode
// copies a tile's pairs as one run.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_internal.cuh"

namespace pa {
#if defined(__CUDACC__)

// (step, low) of a pair's four bytes as fp32.
template <int QK>
__device__ __forceinline__ float2 pair_values(uint32_t w) {
  if constexpr (QK == Q_BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// The eight codes of a word as fp32: two at a time masked into the mantissas of 1024 (64) in f16 (Kim,
// Henry, Fahmy and Hassan Awadalla, "Who says elephants can't run: bringing large scale MoE models into
// cloud scale production", 2022).
__device__ __forceinline__ void code_values(uint32_t w, float (&c)[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t even, odd;
    asm("{\n .reg .b32 t;\n lop3.b32 t, %1, 0x000f000f, %2, 0xea;\n sub.rn.f16x2 %0, t, %2;\n}"
        : "=r"(even)
        : "r"(w), "r"(0x64006400u));
    asm("{\n .reg .b32 t;\n lop3.b32 t, %1, 0x00f000f0, %2, 0xea;\n sub.rn.f16x2 %0, t, %2;\n}"
        : "=r"(odd)
        : "r"(w), "r"(0x54005400u));
    const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&even));
    const float2 o = __half22float2(*reinterpret_cast<const __half2*>(&odd));
    c[2 * k] = e.x;
    c[2 * k + 4] = e.y;
    c[2 * k + 1] = o.x;
    c[2 * k + 5] = o.y;
    w >>= 8;
  }
}

// The largest number of the pair's type that is <= x / the least that is >= x (bits).
template <int QK>
__device__ __forceinline__ uint16_t round_down(float x) {
  if constexpr (QK == Q_BF16) {
    const uint32_t u = __float_as_uint(x);  // a negative number's magnitude grows
    return (uint16_t)(((u >> 31) ? u + 0xffffu : u) >> 16);
  } else {
    return __half_as_ushort(__float2half_rd(x));
  }
}
template <int QK>
__device__ __forceinline__ uint16_t round_up_nonneg(float x) {
  if constexpr (QK == Q_BF16)
    return (uint16_t)((__float_as_uint(x) + 0xffffu) >> 16);
  else
    return __half_as_ushort(__float2half_ru(x));
}

// y / s correctly rounded for y = 0 or y in [2^-70, 2^70] and s in [2^-60, 2^60]: with the
// reciprocal r correctly rounded, one step of Markstein's ("Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990): q = y r, q + (y - q s) r, as q - (q s - y) r, which
// leaves a zero its sign.
__device__ __forceinline__ float quotient(float y, float s, float r) {
  const float q = __fmul_rn(y, r);
  return __fmaf_rn(-__fmaf_rn(q, s, -y), r, q);
}

// A row over L lanes (of a warp that is here as a whole), eight elements a lane: the lane's codes (its
// first element's in the lowest four bits) and the row's pair.
template <int QK, int L>
__device__ __forceinline__ uint32_t quantise_row(const float (&x)[8], uint32_t* pair) {
  float lo = x[0], hi = x[0], zero = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    lo = fminf(lo, x[k]);
    hi = fmaxf(hi, x[k]);
    zero = __fmaf_rn(x[k], 0.f, zero);
  }
  lo = zero == 0.f ? lo : -INFINITY;  // (NaN or infinity: no finite range)
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
  }
  const uint32_t low_bits = round_down<QK>(lo);
  const float low = pair_values<QK>(low_bits << 16).y;
  const float range = hi - low;
  if (!(range < INFINITY)) {
    *pair = 0x7fffu | low_bits << 16;  // step NaN (in both types)
    return 0;
  }
  const uint32_t step_bits = round_up_nonneg<QK>(__fdiv_rn(range, 15.f));
  const float step = pair_values<QK>(step_bits).x;
  const bool fits = step < INFINITY;  // (an fp32 row's step may pass fp16)
  *pair = (fits ? step_bits : 0x7fffu) | low_bits << 16;
  if (step == 0.f || !fits) return 0;
  uint32_t codes = 0;
  const bool plain = step >= 0x1p-60f && step <= 0x1p60f;
  const float inv = __fdiv_rn(1.f, step);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float y = x[k] - low;
    // (a y below 2^-70 gives a quotient below a half by either way of dividing)
    const float q = plain ? quotient(y, step, inv) : __fdiv_rn(y, step);
    // the integer nearest to q in [0, 15] in the low bits of 2^23 + q (ties to even)
    codes |= (__float_as_uint(q + 8388608.f) & 15u) << (4 * k);
  }
  return codes;
}

#endif  // __CUDACC__
}  // namespace pa
