// One K or V row of a token and kv head into its place in the cache, as pa_append_kv and
// pa_append_rotated write it: a warp a row, E = D / 32 consecutive elements a lane.
#pragma once

#include "append_block.cuh"
#include "int4.cuh"

namespace pa {

// What a cache holds of a row.
enum StoreKind { STORE_16 = 0, STORE_FP8 = 1, STORE_INT4 = 2 };

inline int store_kind(const pa_config& c) {
  return c.kv_dtype == PA_INT4 ? STORE_INT4 : c.kv_dtype == PA_FP8_E4M3 ? STORE_FP8 : STORE_16;
}

#if defined(__CUDACC__)

// Elements of E 16-bit numbers at `src` (a multiple of 2 E bytes).
template <int E>
__device__ __forceinline__ void load_row16(const char* src, uint32_t (&w)[E / 2]) {
  if constexpr (E == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if constexpr (E == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(src);
  }
}
template <int E>
__device__ __forceinline__ void store_row16(char* dst, const uint32_t (&w)[E / 2]) {
  if constexpr (E == 8)
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (E == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = w[0];
}
template <int QK, int E>
__device__ __forceinline__ void widen_row(const uint32_t (&w)[E / 2], float (&x)[E]) {
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    const float2 f = pair_values<QK>(w[k]);
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
}
template <int QK, int E>
__device__ __forceinline__ void narrow_row(const float (&x)[E], uint32_t (&w)[E / 2]) {
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    if constexpr (QK == Q_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}

// Where a row goes: the cache (whole), its scales (or pairs), the block and the slot in it, and
// the kv head.
struct RowPlace {
  int blk, slot, head;
};

// The fp8 row x in one of the scale modes of a token, a tensor or none.
template <int D>
__device__ __forceinline__ void put_fp8(const float (&x)[D / 32], char* cache, float* scale,
                                        size_t row, int scale_mode, int lane) {
  constexpr int E = D / 32;
  float s = 1.f;
  if (scale_mode == PA_SCALE_PER_TOKEN) {
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < E; ++k) amax = fmaxf(amax, fabsf(x[k]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    s = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    if (lane == 0) scale[row] = s;
  } else if (scale_mode == PA_SCALE_PER_TENSOR) {
    s = __ldg(scale);
  }
  uint32_t c[E / 2];
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    const float a = scale_mode == PA_SCALE_NONE ? x[2 * k] : __fdiv_rn(x[2 * k], s);
    const float b = scale_mode == PA_SCALE_NONE ? x[2 * k + 1] : __fdiv_rn(x[2 * k + 1], s);
    c[k] = e4m3x2_rn_sat(a, b);
  }
  char* d = cache + row * D + (size_t)lane * E;
  if constexpr (E == 8)
    *reinterpret_cast<uint2*>(d) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  else if constexpr (E == 4)
    *reinterpret_cast<uint32_t*>(d) = c[0] | (c[1] << 16);
  else
    *reinterpret_cast<uint16_t*>(d) = (uint16_t)c[0];
}

// The 4-bit row x.
template <int D, int QK>
__device__ __forceinline__ void put_int4(const float (&x)[D / 32], char* cache, void* pairs,
                                         size_t row, const RowPlace& at, int Hkv, int bs, int lane) {
  constexpr int E = D / 32;
  uint32_t pair;
  const uint32_t codes = quantise_row<QK, E>(x, &pair);
  char* d = cache + row * (D / 2) + (size_t)lane * (E / 2);
  if constexpr (E == 8)
    *reinterpret_cast<uint32_t*>(d) = codes;
  else if constexpr (E == 4)
    *reinterpret_cast<uint16_t*>(d) = (uint16_t)codes;
  else
    *reinterpret_cast<uint8_t*>(d) = (uint8_t)codes;
  if (lane == 0)
    reinterpret_cast<uint32_t*>(pairs)[((size_t)at.blk * Hkv + at.head) * bs + at.slot] = pair;
}

#endif  // __CUDACC__

}  // namespace pa
