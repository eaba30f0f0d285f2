// pa_append_kv: a decode step's new K/V rows written into the paged cache, with fp8
// quantise-on-write.
//
// New row i < q_lens[b] of sequence b is cache position pos = context_lens[b] - q_lens[b] + i
// (the new tokens are the last q_lens[b] of the context_lens[b] cached tokens, as the decode
// reads them), i.e. slot pos % block_size of physical block block_tables[b][pos / block_size]
// ("HSTU Paged Attention", RecSDK issue 1281, background: K/V live in a paged cache reached
// through per-sequence page lists).  A 16-bit cache receives the row unchanged.  An fp8 cache
// receives OCP E4M3 codes of the row over its scale, in one of the scale modes of "Optimize
// paged-attention metadata decode" (FlyDSL PR #910, Breaking Changes: per_token_kv):
// per-token, the row's scale is amax / 448 (1 for an all-zero row) and is written beside the
// codes; per-tensor, the caller's one scale is read; with no scale the values are encoded as
// they are.  (One scale for each page and kv head: append_block.cu.)  The scale and every quotient
// are IEEE fp32 operations (correctly rounded division), and the code is the E4M3 value nearest to
// the quotient, ties to even, magnitudes past 448 saturating to 448.  A 4-bit cache receives codes of
// the row between its least and largest element and their step and low (int4.cuh).
//
// D / 8 lanes a row and one to four rows a warp's step, 16 bytes of input a lane, a token's K and V rows
// over as many warps as fill the GPU (append_row.cuh).  The work is a few bytes per new token, a
// latency-bound kernel on the path before pa_plan / pa_decode.
#include <cstdint>

#include "append_row.cuh"

namespace pa {

cudaError_t launch_append(const AppendParams& p, int head_dim, int qk, int kind, cudaStream_t s) {
  switch (head_dim) {
    case 64: return launch_append_d<64, false>(p, qk, kind, s);
    case 128: return launch_append_d<128, false>(p, qk, kind, s);
    default: return launch_append_d<256, false>(p, qk, kind, s);
  }
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_append_kv(const pa_config* cfg, const void* k_new, const void* v_new,
                                  const int32_t* block_tables, const int32_t* context_lens,
                                  const int32_t* q_lens, void* k_cache, void* v_cache,
                                  void* k_scale, void* v_scale, int32_t* flags,
                                  pa_stream stream) {
  if (!cfg || !k_new || !v_new || !block_tables || !context_lens || !q_lens || !k_cache ||
      !v_cache)
    return PA_ERR_INVALID_ARG;
  const pa_config& c = *cfg;
  if (c.batch < 1 || c.max_q_len < 1 || c.num_kv_heads < 1 || c.max_blocks_per_seq < 1 ||
      c.num_blocks < 1 || c.head_dim < 1 || c.block_size < 1)
    return PA_ERR_INVALID_ARG;
  if (!scale_mode_known(c))
    return PA_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (c.block_size < 16 || c.block_size > 1024 || (c.block_size & (c.block_size - 1)))
    return PA_ERR_UNSUPPORTED;
  if (c.q_dtype != PA_BF16 && c.q_dtype != PA_FP16) return PA_ERR_UNSUPPORTED;
  const bool fp8 = c.kv_dtype == PA_FP8_E4M3;
  if (!kv_kind_taken(c)) return PA_ERR_UNSUPPORTED;
  if (c.kv_scale_mode != PA_SCALE_NONE && (!k_scale || !v_scale)) return PA_ERR_INVALID_ARG;
  auto aligned = [](const void* ptr, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) % a) == 0;
  };
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return PA_ERR_INVALID_ARG;
  const uintptr_t scale_align = c.kv_dtype == PA_INT4 ? 16 : 4;
  if (!aligned(k_scale, scale_align) || !aligned(v_scale, scale_align) || !aligned(flags, 4))
    return PA_ERR_INVALID_ARG;
  if (fp8 && c.kv_scale_mode == PA_SCALE_PER_BLOCK)
    return append_block(c, k_new, v_new, block_tables, context_lens, q_lens, k_cache, v_cache,
                        static_cast<float*>(k_scale), static_cast<float*>(v_scale), flags,
                        reinterpret_cast<cudaStream_t>(stream));
  const long long tokens = (long long)c.batch * c.max_q_len;
  if (tokens > INT32_MAX || (long long)c.num_kv_heads > INT32_MAX / 2) return PA_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  AppendParams p{};
  p.k_new = static_cast<const char*>(k_new);
  p.v_new = static_cast<const char*>(v_new);
  p.bt = block_tables;
  p.ctx = context_lens;
  p.qlens = q_lens;
  p.k_cache = static_cast<char*>(k_cache);
  p.v_cache = static_cast<char*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.flags = flags;
  p.k_stride = p.v_stride = (long long)c.num_kv_heads * c.head_dim;
  p.tokens = (int)tokens;
  p.Sq = c.max_q_len;
  p.Hkv = c.num_kv_heads;
  p.bs = c.block_size;
  p.bs_shift = ilog2((uint32_t)c.block_size);
  p.maxb = c.max_blocks_per_seq;
  p.nblocks = c.num_blocks;
  p.scale_mode = c.kv_scale_mode;
  split_rows(p, c.head_dim, sms, true);
  const int qk = c.q_dtype == PA_FP16 ? Q_FP16 : Q_BF16;
  return launch_append(p, c.head_dim, qk, store_kind(c), reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}
