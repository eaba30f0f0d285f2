// pa_append_rotated: a step's queries and keys normalised for each head and rotated by their
// positions, and its K/V rows written into their pages, in one pass.
//
//     y = x / sqrt(mean(x^2) + eps) * weight,  (z_a, z_b) = (y_a cos - y_b sin, y_b cos + y_a sin)
//
// The kernel is the append's (append_row.cuh): D / 8 lanes a row and eight consecutive elements a
// lane, the mean square a shuffle sum, a pair's other channel in the same lane (interleaved) or
// rotary_dim / 16 lanes away.  A warp takes up to 24 steps of one token's rows, for which it reads
// the lengths, positions and angles once.  All in fp32; one rounding to q_dtype at the end, or the
// cache's own quantisation.
#include "append_row.cuh"

namespace pa {

cudaError_t launch_rotate(const AppendParams& p, int head_dim, int qk, int kind, cudaStream_t s) {
  switch (head_dim) {
    case 64: return launch_append_d<64, true>(p, qk, kind, s);
    case 128: return launch_append_d<128, true>(p, qk, kind, s);
    default: return launch_append_d<256, true>(p, qk, kind, s);
  }
}

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
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  AppendParams p{};
  p.q = static_cast<const char*>(q);
  p.k_new = static_cast<const char*>(k_new);
  p.v_new = static_cast<const char*>(v_new);
  p.r.q_weight = static_cast<const char*>(r.q_weight);
  p.r.k_weight = static_cast<const char*>(r.k_weight);
  p.r.cos_sin = r.cos_sin;
  p.r.positions = r.positions;
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
  p.tokens = (int)tokens;
  p.Sq = c.max_q_len;
  p.Hq = c.num_q_heads;
  p.Hkv = c.num_kv_heads;
  p.bs = c.block_size;
  p.bs_shift = ilog2((uint32_t)c.block_size);
  p.maxb = c.max_blocks_per_seq;
  p.nblocks = c.num_blocks;
  p.scale_mode = c.kv_scale_mode;
  p.r.half = half;
  p.r.interleaved = r.interleaved;
  p.r.table_rows = r.table_rows;
  p.r.axes = half ? r.num_axes : 0;
  p.r.axis1 = half ? r.axis_pairs[0] : 0;
  p.r.axis2 = half && r.num_axes > 1 ? r.axis_pairs[0] + r.axis_pairs[1] : half;
  p.r.eps = r.eps;
  split_rows(p, c.head_dim, sms, stores);
  const int qk = c.q_dtype == PA_FP16 ? Q_FP16 : Q_BF16, kind = stores ? store_kind(c) : STORE_16;
  return launch_rotate(p, c.head_dim, qk, kind, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}
