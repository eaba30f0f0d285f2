// A step's new K/V rows into an fp8 cache with one scale for each (page, kv head).
//
// Quantise-on-write.  A page's codes share one scale s, so a new row with a larger magnitude
// raises it: with a the largest finite magnitude of the call's new rows in the page, w = a / 448,
//     fresh page (its slot 0 is new):  s = w (1 for a = 0)
//     else                             s = max(s_old, w); for w > s_old the older codes c become
//                                      E4M3(c s_old / s), for w <= s_old they stay
// and the new codes are E4M3(x / s).  An infinite element does not set the scale (it saturates to
// 448 s), so it cannot wipe out its neighbours.  All of a page's new rows of one call are taken
// together: the order of rows does not enter.
//
// The quotient.  x / s is the correctly rounded one, by Markstein's correction (P. Markstein, IBM
// J. Res. Dev. 34, 1990): with r = RN(1 / s) and q = RN(x r), q + r (x - q s), the remainder and
// the sum each one fused multiply-add, is RN(x / s) while the remainder is exact, which it is for
// every q that E4M3 does not round to zero when s >= 2^-90.  Three packed instructions for two
// elements.  Pages with a smaller scale or with infinities or NaN among their new rows divide.
//
// One CTA per (sequence, touched page, kv head, K or V): nobody else writes that page's codes of
// that head or its scale, so there is nothing to join.  A thread keeps up to kKeep 16-byte pieces
// of the new rows in registers between the pass for a and the pass for the codes; only pages
// with more new rows than that are read twice (the second time from L2).  A thread keeps its column,
// so its rows are one stride apart.  Most of the grid may be pages that nobody touches (the host
// does not know the lengths), so CTAs are small.  Eight prompts of 1 to 4,096 rows, 8 heads of 128:
// 20.7 us (100 MB, 14.7 us at the copy rate), 27.2 with the bounds' update behind it.  The two
// calls took 32.3 us with 256 threads (4 pieces kept), 29.2 with 4 pieces kept, 30.4 with registers cut
// to 64 for eight CTAs an SM; earlier forms 27.6 us with 128 threads, 52.7 with 512, 32.7 with 64,
// and 36.9 as a persistent grid that walks over the pages.  What bounds it: instructions, about
// ten for two values, at 0.6 a cycle and scheduler, while a CTA's loads come in once.  These are
// calls that raise no scale.  One that does divides for every older code of the page: raising that
// of every page that holds any adds 11.7 us to the prompts' two calls (a few CTAs with up to 63 rows
// to re-encode, after the others have ended) and 2.8 us to those of 32 single tokens (3.7 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "append_block.cuh"

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kKeep = 8;  // 16-byte pieces of new rows a thread keeps in registers
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

struct AppendBlockParams {
  TouchParams t;
  const char* k_new;
  const char* v_new;
  char* k_cache;
  char* v_cache;
  float* k_scale;
  float* v_scale;
};

template <int QK>
__device__ __forceinline__ float2 pair_to_f2(uint32_t w) {
  if constexpr (QK == Q_BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<__half2*>(&w));
}

__device__ __forceinline__ float finite_amax(float a, float x) {
  const float m = fabsf(x);
  return m <= 3.402823466e38f ? fmaxf(a, m) : a;  // false for inf and NaN
}

// The larger magnitude of each half under some sign (NaN wins).
template <int QK>
__device__ __forceinline__ uint32_t amax2(uint32_t a, uint32_t w) {
  uint32_t r;
  if constexpr (QK == Q_BF16)
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(w));
  else
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(w));
  return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}

template <int D, int QK>
__global__ void __launch_bounds__(kThreads) append_block_kernel(const AppendBlockParams p) {
  constexpr int PPR = D / 8;  // 16-byte pieces (8 elements) of a new row
  constexpr int NW = kThreads / 32;
  constexpr int RG = kThreads / PPR;  // rows taken at a time: a thread keeps its column
  __shared__ uint32_t s_max[NW];
  const int tid = threadIdx.x;
  const bool is_v = blockIdx.x & 1;
  const uint32_t u = blockIdx.x >> 1, bj = p.t.head_div.div(u);
  const int g = (int)(u - bj * p.t.Hkv);
  const int b = (int)p.t.page_div.div(bj), j = (int)p.t.page_div.mod(bj);
  grid_dependency_wait();
  TouchedPage t;
  if (!touched_page(p.t, b, j, tid == 0 && !is_v && g == 0, &t)) return;
  // the new rows are on their way while the block table and the old scale are looked up
  const size_t row_stride = (size_t)p.t.Hkv * D;  // elements between a head's rows (new and cached)
  const uint4* src = reinterpret_cast<const uint4*>(
      (is_v ? p.v_new : p.k_new) + (((size_t)b * p.t.Sq + t.i0) * row_stride + (size_t)g * D) * 2);
  const int c = tid % PPR, r0 = tid / PPR;
  const size_t step = RG * (row_stride / 8);
  src += (size_t)r0 * (row_stride / 8) + c;
  auto piece = [&](int k) { return __ldg(src + (size_t)k * step); };  // of row r0 + k RG
  const int count = (t.rows - r0 + RG - 1) / RG;                       // this thread's pieces
  uint4 keep[kKeep];
#pragma unroll
  for (int k = 0; k < kKeep; ++k) keep[k] = k < count ? piece(k) : make_uint4(0, 0, 0, 0);
  const int blk = touched_block(p.t, b, t, tid == 0 && !is_v);
  if (blk < 0) return;
  float* scale = (is_v ? p.v_scale : p.k_scale) + (size_t)blk * p.t.Hkv + g;
  const bool fresh = t.slot0 == 0;
  const float s_old = fresh ? 0.f : *scale;

  // ---- largest finite magnitude of the page's new rows
  uint32_t big = 0;
  auto amax_of = [&](const uint4& v) {
    big = amax2<QK>(amax2<QK>(amax2<QK>(amax2<QK>(big, v.x), v.y), v.z), v.w);
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k) amax_of(keep[k]);
  for (int k = kKeep; k < count; ++k) amax_of(piece(k));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) big = amax2<QK>(big, __shfl_xor_sync(kFull, big, o));
  if ((tid & 31) == 0) s_max[tid >> 5] = big;
  __syncthreads();
#pragma unroll
  for (int x = 0; x < NW; ++x) big = amax2<QK>(big, s_max[x]);
  const float2 big2 = pair_to_f2<QK>(big & 0x7fff7fffu);
  float a = fmaxf(big2.x, big2.y);
  const bool finite = fabsf(big2.x) <= 3.402823466e38f && fabsf(big2.y) <= 3.402823466e38f;
  if (!finite) {  // the same for the whole CTA: look again, past infinities and NaN
    a = 0.f;
    for (int k = 0; k < count; ++k) {
      const uint4 v = piece(k);
      const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = pair_to_f2<QK>(h[k]);
        a = finite_amax(finite_amax(a, f.x), f.y);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kFull, a, o));
    __syncthreads();
    if ((tid & 31) == 0) s_max[tid >> 5] = __float_as_uint(a);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NW; ++x) a = fmaxf(a, __uint_as_float(s_max[x]));
  }

  const float w = a > 0.f ? fmaxf(__fdiv_rn(a, 448.f), kMinScale) : 0.f;
  const bool grown = !fresh && w > s_old;
  const float s = fresh ? (w > 0.f ? w : 1.f) : (grown ? w : s_old);
  if (tid == 0 && (fresh || grown)) *scale = s;  // every thread has read s_old

  // ---- the older codes under the larger scale
  char* cache = (is_v ? p.v_cache : p.k_cache) +
                ((size_t)blk * p.t.bs) * row_stride + (size_t)g * D;  // slot 0, this head
  if (grown) {
    char* at = cache + (size_t)r0 * row_stride + c * 8;
    for (int row = r0; row < t.slot0; row += RG, at += RG * row_stride) {
      uint2 x = *reinterpret_cast<uint2*>(at);
      x.x = rescale4(x.x, s_old, s);
      x.y = rescale4(x.y, s_old, s);
      *reinterpret_cast<uint2*>(at) = x;
    }
  }
  // ---- the new codes
  const float r = __frcp_rn(s);
  const float2 r2 = make_float2(r, r), neg_s2 = make_float2(-s, -s);
  const bool fast = finite && s >= 0x1p-90f;  // the same for the whole CTA
  char* const dst = cache + (size_t)(t.slot0 + r0) * row_stride + c * 8;
  auto put = [&](int k, const uint4& v) {
    const uint32_t h[4] = {v.x, v.y, v.z, v.w};
    uint32_t e[4];
    if (fast) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = pair_to_f2<QK>(h[j]);
        float2 q = mul2(x, r2);
        q = ffma2(ffma2(q, neg_s2, x), r2, q);
        e[j] = e4m3x2_rn_sat(q.x, q.y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = pair_to_f2<QK>(h[j]);
        e[j] = e4m3x2_rn_sat(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s));
      }
    }
    *reinterpret_cast<uint2*>(dst + (size_t)k * RG * row_stride) =
        make_uint2(__byte_perm(e[0], e[1], 0x5410), __byte_perm(e[2], e[3], 0x5410));
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (k < count) put(k, keep[k]);
  for (int k = kKeep; k < count; ++k) put(k, piece(k));
}

template <class K>
cudaError_t launch(K kernel, const AppendBlockParams& p, uint32_t grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

pa_status append_block(const pa_config& c, const void* k_new, const void* v_new,
                       const int32_t* block_tables, const int32_t* context_lens,
                       const int32_t* q_lens, void* k_cache, void* v_cache, float* k_scale,
                       float* v_scale, int32_t* flags, cudaStream_t s) {
  const double ctas = 2.0 * c.batch * (double)pages_touched(c) * c.num_kv_heads;
  if (ctas > INT32_MAX) return PA_ERR_UNSUPPORTED;
  AppendBlockParams p{};
  p.t = touch_params(c, block_tables, context_lens, q_lens, flags);
  p.k_new = static_cast<const char*>(k_new);
  p.v_new = static_cast<const char*>(v_new);
  p.k_cache = static_cast<char*>(k_cache);
  p.v_cache = static_cast<char*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  const bool half = c.q_dtype == PA_FP16;
  const uint32_t grid = (uint32_t)ctas;
  cudaError_t e;
  switch (c.head_dim) {
    case 64: e = launch(half ? append_block_kernel<64, Q_FP16> : append_block_kernel<64, Q_BF16>, p, grid, s); break;
    case 128: e = launch(half ? append_block_kernel<128, Q_FP16> : append_block_kernel<128, Q_BF16>, p, grid, s); break;
    default: e = launch(half ? append_block_kernel<256, Q_FP16> : append_block_kernel<256, Q_BF16>, p, grid, s); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
