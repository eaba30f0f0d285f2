// pa_dequant_kv: a batch's rows of an fp8 or 4-bit cache read back as 16-bit values into contiguous
// buffers, as pa_gather_kv lays out its copies.
//
// Every CTA sums the lengths for itself and takes an equal run of the batch's rows.  A thread takes
// eight values at a time (8 or 4 bytes in, 16 out), several such groups of its CTA's rows at once: for
// each it looks up the page and the scale, so that pages of any size stream alike.
#include "append_row.cuh"

namespace pa {
namespace {

constexpr int kDequantThreads = 256;
constexpr int kDequantMaxBatch = 8192;
// CTAs of an SM and groups of K (and as many of V) that a thread has in flight.  Us a pass over 64
// contexts of 8,192 to 16,384 tokens of an fp8 cache with a scale a token (one kv head of 128), 8 of
// 2,048 to 16,384 of a 4-bit cache (16 heads of 256), and a 4-bit step (append too): 4 CTAs of 4 groups
// 118, 267 and 9.6; 6 of 2 103, 267 and 10.1; 6 of 1 103, 281 and 12.8; 8 of 1 110, 265 and 13.5; 2 of
// 8 153, 267 and 11.7.  The same over other shapes: 4 of 4 against 6 of 2, fp8 (a scale a token, a tensor
// or a page differ by 1 us), 64 long contexts of one head of 64 62.2 and 55.0, 32 of 512 to 4,096, 8 heads
// of 64 46 and 42, 8 heads of 128 85.5 and 78.6, 16 heads of 256 353 and 321, short ones (8 of up to 1,000;
// one of 4,000) 6.1 and 6.7, 5.5 and 6.0; 4 bits, in the same order, 49.3 and 49.2, 38.8 and 37.9, 72 and
// 71.6, 292 and 294, 6.0 and 6.7, 5.4 and 6.2.
constexpr int dequant_ctas(int kind) { return kind == STORE_INT4 ? 4 : 6; }
constexpr int dequant_groups(int kind) { return kind == STORE_INT4 ? 4 : 2; }

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
  FastDiv head_div;  // by Hkv
};

template <int D, int QK, int KIND>
__global__ void __launch_bounds__(kDequantThreads, dequant_ctas(KIND)) dequant_kernel(const DequantParams p) {
  constexpr int G8 = D / 8;                        // groups of eight values in a row
  constexpr int U = dequant_groups(KIND);
  extern __shared__ int32_t off[];                 // [batch + 1] rows before each sequence
  __shared__ int sums[kDequantThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long cap = (long long)p.maxb << p.bs_shift;
  grid_dependency_wait();
  int run = 0;
  bool bad = false;
  for (int b0 = 0; b0 < p.batch; b0 += kDequantThreads) {
    const int b = b0 + tid;
    int n = b < p.batch ? __ldg(p.ctx + b) : 0;
    if (n < 0 || (long long)n > cap) {
      bad = true;
      n = 0;
    }
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int before = run;
#pragma unroll
    for (int w = 0; w < kDequantThreads / 32; ++w) {
      before += w < warp ? sums[w] : 0;
      run += sums[w];
    }
    if (b < p.batch) off[b] = before + x - n;
  }
  if (tid == 0) off[p.batch] = run;
  bad = __syncthreads_or(bad);
  const bool overflow = run > p.max_rows;
  if (blockIdx.x == 0) {
    if (tid == 0 && p.flags && (bad || overflow)) atomicOr(p.flags, PA_FLAG_BAD_LENGTHS);
    if (p.row_offsets)
      for (int b = tid; b <= p.batch; b += kDequantThreads) p.row_offsets[b] = off[b];
  }
  if (overflow) return;
  // this CTA's rows (a row: a token's heads), sequence by sequence
  const int r0 = (int)((long long)run * blockIdx.x / gridDim.x);
  const int r1 = (int)((long long)run * (blockIdx.x + 1) / gridDim.x);
  if (r0 >= r1) return;
  int seq = 0;  // the last sequence that starts at or before r0 (empty ones share their successor's start)
  for (int step = 1 << (31 - __clz(p.batch)); step > 0; step >>= 1)
    if (seq + step < p.batch && off[seq + step] <= r0) seq += step;
  float tensor_scale[2] = {1.f, 1.f};
  if (KIND == STORE_FP8 && p.scale_mode == PA_SCALE_PER_TENSOR) {
    tensor_scale[0] = __ldg(static_cast<const float*>(p.k_scale));
    tensor_scale[1] = __ldg(static_cast<const float*>(p.v_scale));
  }
  bool bad_block = false;
  // a thread's group of its row is always the same, its rows kDequantThreads / G8 apart
  constexpr int S = kDequantThreads / G8;
  const uint32_t group = tid % G8;
  const int most_rows = INT32_MAX / 2 / p.Hkv;  // (row-heads are counted in 32 bits)
  for (int at = r0; at < r1;) {
    while (off[seq + 1] <= at) ++seq;
    const int t0 = at - off[seq], rows = min(min(off[seq + 1], r1) - at, most_rows);
    const int32_t* const table = p.bt + (size_t)seq * p.maxb;
    const int heads = rows * p.Hkv;
    uint4* const ko = reinterpret_cast<uint4*>(p.k_out) + (size_t)at * p.Hkv * G8 + group;
    uint4* const vo = reinterpret_cast<uint4*>(p.v_out) + (size_t)at * p.Hkv * G8 + group;
    for (int h0 = tid / G8; h0 < heads; h0 += U * S) {
      uint2 raw[U][2];
      uint32_t pair[U][2];
      float sc[U][2];
      bool ok[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int rh = h0 + u * S;
        ok[u] = rh < heads;
        if (!ok[u]) continue;
        const int r = (int)p.head_div.div((uint32_t)rh), g = rh - r * p.Hkv;
        const int tok = t0 + r, slot = tok & (p.bs - 1);
        const int blk = __ldg(table + (tok >> p.bs_shift));
        if (blk < 0 || blk >= p.nblocks) {
          bad_block = true;
          ok[u] = false;
          continue;
        }
        const size_t row = ((size_t)blk * p.bs + slot) * p.Hkv + g, from = row * G8 + group;
        if constexpr (KIND == STORE_INT4) {
          raw[u][0].x = __ldg(reinterpret_cast<const uint32_t*>(p.k_cache) + from);
          raw[u][1].x = __ldg(reinterpret_cast<const uint32_t*>(p.v_cache) + from);
          const size_t i = ((size_t)blk * p.Hkv + g) * p.bs + slot;
          pair[u][0] = __ldg(static_cast<const uint32_t*>(p.k_scale) + i);
          pair[u][1] = __ldg(static_cast<const uint32_t*>(p.v_scale) + i);
        } else {
          raw[u][0] = __ldg(reinterpret_cast<const uint2*>(p.k_cache) + from);
          raw[u][1] = __ldg(reinterpret_cast<const uint2*>(p.v_cache) + from);
          sc[u][0] = tensor_scale[0];
          sc[u][1] = tensor_scale[1];
          if (p.scale_mode >= PA_SCALE_PER_TOKEN) {
            const size_t i = p.scale_mode == PA_SCALE_PER_TOKEN ? row : (size_t)blk * p.Hkv + g;
            sc[u][0] = __ldg(static_cast<const float*>(p.k_scale) + i);
            sc[u][1] = __ldg(static_cast<const float*>(p.v_scale) + i);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!ok[u]) continue;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float x[8];
          if constexpr (KIND == STORE_INT4) {
            const float2 f = pair_values<QK>(pair[u][t]);
            code_values(raw[u][t].x, x);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = __fmaf_rn(x[k], f.x, f.y);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t c = ((k < 2 ? raw[u][t].x : raw[u][t].y) >> (16 * (k & 1))) & 0xffffu;
              const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3);
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
              x[2 * k] = f.x * sc[u][t];
              x[2 * k + 1] = f.y * sc[u][t];
            }
          }
          __stcs((t ? vo : ko) + (size_t)(h0 + u * S) * G8, narrow_row<QK>(x));
        }
      }
    }
    at += rows;
  }
  if (bad_block && p.flags) atomicOr(p.flags, PA_FLAG_BAD_BLOCK_ID);
  grid_dependents_launch();
}

template <int D>
cudaError_t launch_dequant_d(const DequantParams& p, int qk, int kind, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.dynamicSmemBytes = (size_t)(p.batch + 1) * 4;
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
  // the row offsets are int32
  if ((long long)c.num_kv_heads * c.head_dim > (1 << 24) ||
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
  p.head_div = FastDiv((uint32_t)c.num_kv_heads);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  // a CTA for every few thousand values that there may be, as many as fit at once
  const double most = (double)c.batch * c.max_blocks_per_seq * c.block_size * c.num_kv_heads * c.head_dim;
  const double ctas = most / (8.0 * kDequantThreads) + 1;
  const int most_ctas = sms * dequant_ctas(store_kind(c));
  const int grid = ctas < most_ctas ? (int)ctas : most_ctas;
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
