// pa_dequant_kv: a batch's rows of an fp8 or 4-bit cache read back as 16-bit values into contiguous
// buffers, as pa_gather_kv lays out its copies.
//
// A CTA a page (of a sequence): eight values a thread at a time, one 16-byte store each.
#include "append_row.cuh"

namespace pa {
namespace {

constexpr int kDequantThreads = 256;
constexpr int kDequantMaxBatch = 8192;

struct DequantParams {
  const char* k_cache;
  const char* v_cache;
  const void* k_scale;
  const void* v_scale;
  char* k_out;
  char* v_out;
  const int32_t* bt;
  const int32_t* ctx;
  int32_t* row_offsets;
  int32_t* flags;
  long long max_rows;
  int batch, Hkv, bs, bs_shift, maxb, nblocks, scale_mode;
};

template <int D, int QK, int KIND>
__global__ void __launch_bounds__(kDequantThreads) dequant_kernel(const DequantParams p) {
  __shared__ long long sums[2][kDequantThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const long long cap = (long long)p.maxb << p.bs_shift;
  const bool reports = blockIdx.x == 0 && blockIdx.y == 0;
  grid_dependency_wait();
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    // rows before this sequence's, and of all
    long long before = 0, all = 0;
    bool bad = false;
    for (int j = tid; j < p.batch; j += kDequantThreads) {
      int n = __ldg(p.ctx + j);
      if (n < 0 || (long long)n > cap) {
        bad = true;
        n = 0;
      }
      all += n;
      if (j < b) before += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      before += __shfl_xor_sync(kFull, before, o);
      all += __shfl_xor_sync(kFull, all, o);
    }
    __syncthreads();
    if (lane == 0) {
      sums[0][tid >> 5] = before;
      sums[1][tid >> 5] = all;
    }
    bad = __syncthreads_or(bad);
    before = all = 0;
    for (int w = 0; w < kDequantThreads / 32; ++w) {
      before += sums[0][w];
      all += sums[1][w];
    }
    const bool overflow = all > p.max_rows;
    if (reports && b == 0 && tid == 0 && p.flags && (bad || overflow))
      atomicOr(p.flags, PA_FLAG_BAD_LENGTHS);
    if (blockIdx.x == 0 && tid == 0 && p.row_offsets) {
      p.row_offsets[b] = (int32_t)before;
      if (b == p.batch - 1) p.row_offsets[p.batch] = (int32_t)all;
    }
    if (overflow) continue;
    int n = __ldg(p.ctx + b);
    if (n < 0 || (long long)n > cap) n = 0;
    for (int page = blockIdx.x; ((long long)page << p.bs_shift) < n; page += gridDim.x) {
      const int blk = __ldg(p.bt + (size_t)b * p.maxb + page);
      if (blk < 0 || blk >= p.nblocks) {
        if (tid == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_BLOCK_ID);
        continue;
      }
      const int rows = min(p.bs, n - (page << p.bs_shift));
      constexpr int G8 = D / 8;  // groups of eight values in a row
      const int groups = rows * p.Hkv * G8;
      for (int t = 0; t < 2; ++t) {
        const char* cache = t ? p.v_cache : p.k_cache;
        const void* scale = t ? p.v_scale : p.k_scale;
        char* out = (t ? p.v_out : p.k_out) + (size_t)(before + ((long long)page << p.bs_shift)) * p.Hkv * D * 2;
        for (int e = tid; e < groups; e += kDequantThreads) {
          const int r = e / G8, slot = r / p.Hkv, g = r % p.Hkv;
          const size_t at = (size_t)blk * p.bs * p.Hkv * G8 + e;  // the group among the cache's
          float x[8];
          if constexpr (KIND == STORE_INT4) {
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(cache) + at);
            const float2 f = pair_values<QK>(
                __ldg(static_cast<const uint32_t*>(scale) + ((size_t)blk * p.Hkv + g) * p.bs + slot));
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = __fmaf_rn((float)((w >> (4 * k)) & 15u), f.x, f.y);
          } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(cache) + at);
            float s = 1.f;
            if (p.scale_mode == PA_SCALE_PER_TENSOR)
              s = __ldg(static_cast<const float*>(scale));
            else if (p.scale_mode == PA_SCALE_PER_TOKEN)
              s = __ldg(static_cast<const float*>(scale) + ((size_t)blk * p.bs + slot) * p.Hkv + g);
            else if (p.scale_mode == PA_SCALE_PER_BLOCK)
              s = __ldg(static_cast<const float*>(scale) + (size_t)blk * p.Hkv + g);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t c = ((k < 2 ? w.x : w.y) >> (16 * (k & 1))) & 0xffffu;
              const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3);
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
              x[2 * k] = f.x * s;
              x[2 * k + 1] = f.y * s;
            }
          }
          uint32_t o[4];
          narrow_row<QK, 8>(x, o);
          *reinterpret_cast<uint4*>(out + (size_t)e * 16) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }
  grid_dependents_launch();
}

template <int D>
cudaError_t launch_dequant_d(const DequantParams& p, int qk, int kind, dim3 grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kDequantThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (kind == STORE_INT4)
    return qk == Q_BF16 ? cudaLaunchKernelEx(&cfg, dequant_kernel<D, Q_BF16, STORE_INT4>, p)
                        : cudaLaunchKernelEx(&cfg, dequant_kernel<D, Q_FP16, STORE_INT4>, p);
  return qk == Q_BF16 ? cudaLaunchKernelEx(&cfg, dequant_kernel<D, Q_BF16, STORE_FP8>, p)
                      : cudaLaunchKernelEx(&cfg, dequant_kernel<D, Q_FP16, STORE_FP8>, p);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_dequant_kv(const pa_config* cfg, const void* k_cache, const void* v_cache,
                                   const void* k_scale, const void* v_scale,
                                   const int32_t* block_tables, const int32_t* context_lens,
                                   void* k_out, void* v_out, int64_t max_rows,
                                   int32_t* row_offsets, int32_t* flags, pa_stream stream) {
  if (!cfg || !k_cache || !v_cache || !block_tables || !context_lens || !k_out || !v_out)
    return PA_ERR_INVALID_ARG;
  const pa_config& c = *cfg;
  if (c.batch < 1 || c.num_kv_heads < 1 || c.max_blocks_per_seq < 1 || c.num_blocks < 1 ||
      c.head_dim < 1 || c.block_size < 1 || max_rows < 0)
    return PA_ERR_INVALID_ARG;
  if (c.q_dtype < PA_BF16 || c.q_dtype > PA_INT4 || c.kv_dtype < PA_BF16 || c.kv_dtype > PA_INT4 ||
      !scale_mode_known(c))
    return PA_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (c.block_size < 16 || c.block_size > 1024 || (c.block_size & (c.block_size - 1)))
    return PA_ERR_UNSUPPORTED;
  if (c.q_dtype != PA_BF16 && c.q_dtype != PA_FP16) return PA_ERR_UNSUPPORTED;
  if (!kv_kind_taken(c) || store_kind(c) == STORE_16) return PA_ERR_UNSUPPORTED;
  if (c.batch > kDequantMaxBatch) return PA_ERR_UNSUPPORTED;
  if (c.kv_scale_mode != PA_SCALE_NONE && (!k_scale || !v_scale)) return PA_ERR_INVALID_ARG;
  auto aligned = [](const void* ptr, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) % a) == 0;
  };
  const uintptr_t scale_align = c.kv_dtype == PA_INT4 ? 16 : 4;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
      !aligned(k_scale, scale_align) || !aligned(v_scale, scale_align) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(row_offsets, 4) ||
      !aligned(flags, 4))
    return PA_ERR_INVALID_ARG;
  // a page's groups and the row offsets are int32
  if ((long long)c.num_kv_heads * c.head_dim > (1 << 19) ||
      (long long)c.batch * c.max_blocks_per_seq * c.block_size > INT32_MAX)
    return PA_ERR_UNSUPPORTED;
  DequantParams p{};
  p.k_cache = static_cast<const char*>(k_cache);
  p.v_cache = static_cast<const char*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_out = static_cast<char*>(k_out);
  p.v_out = static_cast<char*>(v_out);
  p.bt = block_tables;
  p.ctx = context_lens;
  p.row_offsets = row_offsets;
  p.flags = flags;
  p.max_rows = max_rows;
  p.batch = c.batch;
  p.Hkv = c.num_kv_heads;
  p.bs = c.block_size;
  p.bs_shift = ilog2((uint32_t)c.block_size);
  p.maxb = c.max_blocks_per_seq;
  p.nblocks = c.num_blocks;
  p.scale_mode = c.kv_scale_mode;
  const dim3 grid(c.max_blocks_per_seq < 65535 ? c.max_blocks_per_seq : 65535, c.batch);
  const int qk = c.q_dtype == PA_FP16 ? Q_FP16 : Q_BF16, kind = store_kind(c);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (c.head_dim) {
    case 64: e = launch_dequant_d<64>(p, qk, kind, grid, s); break;
    case 128: e = launch_dequant_d<128>(p, qk, kind, grid, s); break;
    default: e = launch_dequant_d<256>(p, qk, kind, grid, s); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
