// The fp8 append with one scale per (page, kv head), and the E4M3 conversions both appends use.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pa_internal.cuh"

namespace pa {

// Arguments already checked (head_dim, block_size, types, pointers).
pa_status append_block(const pa_config& c, const void* k_new, const void* v_new,
                       const int32_t* block_tables, const int32_t* context_lens,
                       const int32_t* q_lens, void* k_cache, void* v_cache, float* k_scale,
                       float* v_scale, int32_t* flags, cudaStream_t s);

#if defined(__CUDACC__)

// Two fp32 values to two E4M3 codes (lo -> low byte): round to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2_rn_sat(float lo, float hi) {
  uint16_t r;
  asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n mov.b16 %0, t;\n}"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// Four codes under scale `from` as codes under scale `to`.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float from, float to) {
  uint32_t out = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w >> (16 * h)) & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
    out |= e4m3x2_rn_sat(__fdiv_rn(__fmul_rn(f.x, from), to), __fdiv_rn(__fmul_rn(f.y, from), to))
           << (16 * h);
  }
  return out;
}

#endif  // __CUDACC__

}  // namespace pa
