// The fp8 append with one scale per (page, kv head), what it shares with the update of the pages'
// key bounds (the walk over the pages that a step's new rows go to), and the E4M3 conversions that
// both appends use.
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

struct TouchParams {
  const int32_t* bt;
  const int32_t* ctx;
  const int32_t* qlens;
  int32_t* flags;
  int Sq, Hkv, bs, bs_shift, maxb, nblocks;
  FastDiv head_div, page_div;  // by Hkv and by the pages a sequence can touch
};

// The pages a sequence can touch with Sq new rows: they start anywhere in a page.
inline long long pages_touched(const pa_config& c) {
  return ((long long)c.max_q_len + c.block_size - 2) / c.block_size + 1;
}

inline TouchParams touch_params(const pa_config& c, const int32_t* block_tables,
                                const int32_t* context_lens, const int32_t* q_lens,
                                int32_t* flags) {
  TouchParams p{};
  p.bt = block_tables;
  p.ctx = context_lens;
  p.qlens = q_lens;
  p.flags = flags;
  p.Sq = c.max_q_len;
  p.Hkv = c.num_kv_heads;
  p.bs = c.block_size;
  p.bs_shift = ilog2((uint32_t)c.block_size);
  p.maxb = c.max_blocks_per_seq;
  p.nblocks = c.num_blocks;
  p.head_div = FastDiv((uint32_t)c.num_kv_heads);
  p.page_div = FastDiv((uint32_t)pages_touched(c));
  return p;
}

#if defined(__CUDACC__)

// A touched page: the new rows [i0, i0 + rows) of sequence b go to slots [slot0, slot0 + rows) of
// its logical page `page`.  False when there is none (or the lengths are flagged).
struct TouchedPage {
  int i0, rows, slot0, page;
};
__device__ __forceinline__ bool touched_page(const TouchParams& p, int b, int j, bool reports,
                                             TouchedPage* t) {
  const int n = __ldg(p.ctx + b), ql = __ldg(p.qlens + b);
  const long long cap = (long long)p.maxb << p.bs_shift;
  if (ql < 0 || ql > p.Sq || n < ql || (long long)n > cap) {
    if (reports && j == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_LENGTHS);
    return false;
  }
  const int first = n - ql;
  t->page = (first >> p.bs_shift) + j;
  const long long start = (long long)t->page << p.bs_shift;
  if (ql == 0 || start >= n) return false;
  const int lo = max((int)start, first), hi = (int)min(start + p.bs, (long long)n);
  t->i0 = lo - first;
  t->rows = hi - lo;
  t->slot0 = lo - (int)start;
  return true;
}
// Its block, -1 (and flagged) for one outside the pool.
__device__ __forceinline__ int touched_block(const TouchParams& p, int b, const TouchedPage& t,
                                             bool reports) {
  const int blk = __ldg(p.bt + (size_t)b * p.maxb + t.page);
  if (blk >= 0 && blk < p.nblocks) return blk;
  if (reports && p.flags) atomicOr(p.flags, PA_FLAG_BAD_BLOCK_ID);
  return -1;
}

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
