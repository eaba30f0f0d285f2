// pa_append_rotated: a step's queries and keys normalised for each head and rotated by their
// positions, and its K/V rows written into their pages, in one pass.
//
//     y = x / sqrt(mean(x^2) + eps) * weight,  (z_a, z_b) = (y_a cos - y_b sin, y_b cos + y_a sin)
//
// A warp a row (a token's q, k or v head): E = D / 32 consecutive elements a lane, the mean square a
// shuffle sum, a pair's other channel in the same lane (interleaved) or rotary_dim / 2 / E lanes away.
// All in fp32; one rounding to q_dtype at the end, or the cache's own quantisation (append_row.cuh).
#include "append_row.cuh"

namespace pa {
namespace {

constexpr int kRotateWarps = 8;

struct RotateParams {
  const char* q;
  const char* k_new;
  const char* v_new;
  const char* q_weight;
  const char* k_weight;
  const float* cos_sin;
  const int32_t* positions;
  const int32_t* bt;
  const int32_t* ctx;
  const int32_t* qlens;
  char* q_out;
  char* k_out;
  char* k_cache;
  char* v_cache;
  void* k_scale;
  void* v_scale;
  int32_t* flags;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  long long rows;                          // tokens * heads
  int heads;                               // Hq + Hkv, and Hkv more where values are stored
  int tokens;                              // B * Sq
  int Sq, Hq, Hkv, bs, bs_shift, maxb, nblocks, scale_mode;
  int half, interleaved, table_rows, axes, axis1, axis2;  // pairs from axis1 (axis2) on: next axis
  float eps;
};


template <int D, int QK, int KIND>
__global__ void __launch_bounds__(kRotateWarps * 32) rotate_kernel(const RotateParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * kRotateWarps;
  grid_dependency_wait();
  for (long long row = (long long)blockIdx.x * kRotateWarps + (threadIdx.x >> 5); row < p.rows;
       row += warps) {
    const int head = (int)(row % p.heads), token = (int)(row / p.heads);
    const int b = token / p.Sq, i = token % p.Sq;
    const int n = __ldg(p.ctx + b), ql = __ldg(p.qlens + b);
    const long long cap = (long long)p.maxb << p.bs_shift;
    if (ql < 0 || ql > p.Sq || n < ql || (long long)n > cap) {
      if (lane == 0 && i == 0 && head == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_LENGTHS);
      continue;
    }
    if (i >= ql) continue;
    const int pos = n - ql + i;
    int at[3] = {pos, pos, pos};
    if (p.half > 0) {
      bool bad = false;
      for (int a = 0; a < p.axes; ++a) {
        if (p.positions) at[a] = __ldg(p.positions + (size_t)a * p.tokens + token);
        bad |= at[a] < 0 || at[a] >= p.table_rows;
      }
      if (bad) {
        if (lane == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_POSITION);
        continue;
      }
    }
    const bool is_q = head < p.Hq, is_v = head >= p.Hq + p.Hkv;
    const int g = is_q ? head : is_v ? head - p.Hq - p.Hkv : head - p.Hq;
    const char* src = is_q ? p.q + ((size_t)token * p.q_stride + (size_t)g * D) * 2
                      : is_v ? p.v_new + ((size_t)token * p.v_stride + (size_t)g * D) * 2
                             : p.k_new + ((size_t)token * p.k_stride + (size_t)g * D) * 2;
    uint32_t w[E / 2];
    load_row16<E>(src + (size_t)lane * E * 2, w);
    float x[E];
    widen_row<QK, E>(w, x);
    if (!is_v) {
      const char* weight = is_q ? p.q_weight : p.k_weight;
      if (weight) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) sum = __fmaf_rn(x[e], x[e], sum);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        const float inv = 1.f / sqrtf(sum * (1.f / D) + p.eps);
        uint32_t ww[E / 2];
        float f[E];
        load_row16<E>(weight + (size_t)lane * E * 2, ww);
        widen_row<QK, E>(ww, f);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = x[e] * inv * f[e];
      }
      if (p.half > 0) {
        const int c0 = lane * E;  // the lane's first channel
        const bool turns = c0 < 2 * p.half;
        auto angle = [&](int pair, float* c, float* s) {
          const int a = p.axes == 1 ? at[0] : pair < p.axis1 ? at[0] : pair < p.axis2 ? at[1] : at[2];
          const float* t = p.cos_sin + (size_t)a * (2 * p.half) + pair;
          *c = __ldg(t);
          *s = __ldg(t + p.half);
        };
        if (p.interleaved) {
          if (turns) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              float c, s;
              angle((c0 + e) / 2, &c, &s);
              const float u = x[e], v = x[e + 1];
              x[e] = u * c - v * s;
              x[e + 1] = v * c + u * s;
            }
          }
        } else {
          const int away = p.half / E;  // lanes to the pair's other channel (half is a multiple of 8)
          const bool second = c0 >= p.half;
          const int from = turns ? (second ? lane - away : lane + away) : lane;
          float y[E];
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] = __shfl_sync(kFull, x[e], from);
          if (turns) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              float c, s;
              angle(c0 + e - (second ? p.half : 0), &c, &s);
              x[e] = second ? x[e] * c + y[e] * s : x[e] * c - y[e] * s;
            }
          }
        }
      }
      char* dense = is_q ? p.q_out : p.k_out;
      if (dense || KIND == STORE_16) narrow_row<QK, E>(x, w);
      if (dense)
        store_row16<E>(dense + (((size_t)token * (is_q ? p.Hq : p.Hkv) + g) * D + (size_t)lane * E) * 2, w);
    }
    if (is_q || !p.k_cache) continue;
    const int blk = __ldg(p.bt + (size_t)b * p.maxb + (pos >> p.bs_shift));
    if (blk < 0 || blk >= p.nblocks) {
      if (lane == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_BLOCK_ID);
      continue;
    }
    const RowPlace place{blk, pos & (p.bs - 1), g};
    const size_t crow = ((size_t)blk * p.bs + place.slot) * p.Hkv + g;
    char* cache = is_v ? p.v_cache : p.k_cache;
    void* scale = is_v ? p.v_scale : p.k_scale;
    if constexpr (KIND == STORE_16)
      store_row16<E>(cache + (crow * D + (size_t)lane * E) * 2, w);
    else if constexpr (KIND == STORE_FP8)
      put_fp8<D>(x, cache, static_cast<float*>(scale), crow, p.scale_mode, lane);
    else
      put_int4<D, QK>(x, cache, scale, crow, place, p.Hkv, p.bs, lane);
  }
  grid_dependents_launch();
}

template <int D>
cudaError_t launch_rotate_d(const RotateParams& p, int qk, int kind, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kRotateWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
#define PA_ROTATE(KIND_)                                                                \
  if (kind == KIND_)                                                                    \
    return qk == Q_BF16 ? cudaLaunchKernelEx(&cfg, rotate_kernel<D, Q_BF16, KIND_>, p)  \
                        : cudaLaunchKernelEx(&cfg, rotate_kernel<D, Q_FP16, KIND_>, p);
  PA_ROTATE(STORE_16)
  PA_ROTATE(STORE_FP8)
  PA_ROTATE(STORE_INT4)
#undef PA_ROTATE
  return cudaErrorNotSupported;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_append_rotated(const pa_config* cfg, const pa_rotary* rotary, const void* q,
                                       const void* k_new, const void* v_new,
                                       const int32_t* block_tables, const int32_t* context_lens,
                                       const int32_t* q_lens, void* q_out, void* k_out,
                                       void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                                       int32_t* flags, pa_stream stream) {
  if (!cfg || !rotary || !q || !k_new || !context_lens || !q_lens || !q_out)
    return PA_ERR_INVALID_ARG;
  const pa_config& c = *cfg;
  const pa_rotary& r = *rotary;
  if (c.batch < 1 || c.max_q_len < 1 || c.num_q_heads < 1 || c.num_kv_heads < 1 ||
      c.max_blocks_per_seq < 1 || c.num_blocks < 1 || c.head_dim < 1 || c.block_size < 1)
    return PA_ERR_INVALID_ARG;
  if (c.q_dtype < PA_BF16 || c.q_dtype > PA_INT4 || c.kv_dtype < PA_BF16 || c.kv_dtype > PA_INT4 ||
      !scale_mode_known(c))
    return PA_ERR_INVALID_ARG;
  const bool stores = k_cache || v_cache;
  if (stores ? !k_cache || !v_cache || !v_new || !block_tables : !k_out) return PA_ERR_INVALID_ARG;
  if (!(r.eps >= 0.f && r.eps <= 3e38f) || r.rotary_dim < 0 ||
      (r.interleaved != 0 && r.interleaved != 1) || r.q_stride < 0 || r.k_stride < 0 ||
      r.v_stride < 0)
    return PA_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (c.block_size < 16 || c.block_size > 1024 || (c.block_size & (c.block_size - 1)))
    return PA_ERR_UNSUPPORTED;
  if (c.q_dtype != PA_BF16 && c.q_dtype != PA_FP16) return PA_ERR_UNSUPPORTED;
  if (c.num_q_heads % c.num_kv_heads != 0) return PA_ERR_UNSUPPORTED;
  if (stores && (!kv_kind_taken(c) || c.kv_scale_mode == PA_SCALE_PER_BLOCK))
    return PA_ERR_UNSUPPORTED;
  if (stores && c.kv_scale_mode != PA_SCALE_NONE && (!k_scale || !v_scale)) return PA_ERR_INVALID_ARG;
  if (r.rotary_dim > c.head_dim || r.rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
  const int half = r.rotary_dim / 2;
  if (half > 0) {
    if (!r.cos_sin || r.table_rows < 1 || r.num_axes < 1 || r.num_axes > 3) return PA_ERR_INVALID_ARG;
    long long sum = 0;
    for (int a = 0; a < r.num_axes; ++a) {
      if (r.axis_pairs[a] < 0) return PA_ERR_INVALID_ARG;
      sum += r.axis_pairs[a];
    }
    if (sum != half) return PA_ERR_INVALID_ARG;
  }
  // a token's rows, dense or apart
  const long long q_row = (long long)c.num_q_heads * c.head_dim;
  const long long k_row = (long long)c.num_kv_heads * c.head_dim;
  const long long qs = r.q_stride ? r.q_stride : q_row, ks = r.k_stride ? r.k_stride : k_row;
  const long long vs = r.v_stride ? r.v_stride : k_row;
  if (qs < q_row || ks < k_row || vs < k_row || qs % 8 || ks % 8 || vs % 8) return PA_ERR_INVALID_ARG;
  if ((q_out == q && qs != q_row) || (k_out == k_new && ks != k_row)) return PA_ERR_INVALID_ARG;
  auto aligned = [](const void* ptr, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) % a) == 0;
  };
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q_out, 16) ||
      !aligned(k_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(r.q_weight, 16) || !aligned(r.k_weight, 16) || !aligned(r.cos_sin, 16))
    return PA_ERR_INVALID_ARG;
  const uintptr_t scale_align = c.kv_dtype == PA_INT4 ? 16 : 4;
  if (!aligned(k_scale, scale_align) || !aligned(v_scale, scale_align) || !aligned(flags, 4) ||
      !aligned(r.positions, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
      !aligned(q_lens, 4))
    return PA_ERR_INVALID_ARG;
  const long long tokens = (long long)c.batch * c.max_q_len;
  if (tokens > INT32_MAX || (long long)c.max_blocks_per_seq * c.block_size > INT32_MAX ||
      (long long)c.num_q_heads + 2LL * c.num_kv_heads > INT32_MAX)
    return PA_ERR_UNSUPPORTED;
  RotateParams p{};
  p.q = static_cast<const char*>(q);
  p.k_new = static_cast<const char*>(k_new);
  p.v_new = static_cast<const char*>(v_new);
  p.q_weight = static_cast<const char*>(r.q_weight);
  p.k_weight = static_cast<const char*>(r.k_weight);
  p.cos_sin = r.cos_sin;
  p.positions = r.positions;
  p.bt = block_tables;
  p.ctx = context_lens;
  p.qlens = q_lens;
  p.q_out = static_cast<char*>(q_out);
  p.k_out = static_cast<char*>(k_out);
  p.k_cache = static_cast<char*>(k_cache);
  p.v_cache = static_cast<char*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.flags = flags;
  p.q_stride = qs;
  p.k_stride = ks;
  p.v_stride = vs;
  p.heads = c.num_q_heads + c.num_kv_heads * (stores ? 2 : 1);
  p.tokens = (int)tokens;
  p.rows = tokens * p.heads;
  p.Sq = c.max_q_len;
  p.Hq = c.num_q_heads;
  p.Hkv = c.num_kv_heads;
  p.bs = c.block_size;
  p.bs_shift = ilog2((uint32_t)c.block_size);
  p.maxb = c.max_blocks_per_seq;
  p.nblocks = c.num_blocks;
  p.scale_mode = c.kv_scale_mode;
  p.half = half;
  p.interleaved = r.interleaved;
  p.table_rows = r.table_rows;
  p.axes = half ? r.num_axes : 0;
  p.axis1 = half ? r.axis_pairs[0] : 0;
  p.axis2 = half && r.num_axes > 1 ? p.axis1 + r.axis_pairs[1] : half;
  p.eps = r.eps;
  const long long ctas = (p.rows + kRotateWarps - 1) / kRotateWarps;
  const int grid = (int)(ctas < 65535 ? ctas : 65535);
  const int qk = c.q_dtype == PA_FP16 ? Q_FP16 : Q_BF16, kind = stores ? store_kind(c) : STORE_16;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (c.head_dim) {
    case 64: e = launch_rotate_d<64>(p, qk, kind, grid, s); break;
    case 128: e = launch_rotate_d<128>(p, qk, kind, grid, s); break;
    default: e = launch_rotate_d<256>(p, qk, kind, grid, s); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
