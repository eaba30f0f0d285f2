// The C ABI declared in include/pa.h: host-side validation, the kernel variant for a
// configuration, the TMA descriptors of the two caches, and the stream-ordered launches.
// Nothing here allocates, synchronises (except pa_read_flags) or aborts.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstring>
#include <mutex>

#include "decode_selected.cuh"

using namespace pa;

namespace {

bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Shape and type checks that need no device.  Unsupported-but-well-formed configurations
// (head dim, page size, dtype combination, head grouping) map to PA_ERR_UNSUPPORTED, as the
// block-size and dtype rejection cases of "Optimize paged-attention metadata decode"
// (FlyDSL PR #910, validation coverage) do; malformed values to PA_ERR_INVALID_ARG.
pa_status validate(const pa_config* c) {
  if (!c) return PA_ERR_INVALID_ARG;
  if (c->batch < 1 || c->max_q_len < 1 || c->num_q_heads < 1 || c->num_kv_heads < 1 ||
      c->max_blocks_per_seq < 1 || c->num_blocks < 1 || c->head_dim < 1 || c->block_size < 1)
    return PA_ERR_INVALID_ARG;
  if (c->q_dtype < PA_BF16 || c->q_dtype > PA_INT4 || c->kv_dtype < PA_BF16 ||
      c->kv_dtype > PA_INT4)
    return PA_ERR_INVALID_ARG;
  if (!scale_mode_known(*c))
    return PA_ERR_INVALID_ARG;
  if (c->causal != 0 && c->causal != 1) return PA_ERR_INVALID_ARG;
  if (!std::isfinite(c->sm_scale)) return PA_ERR_INVALID_ARG;
  if (c->num_ctas < 0 || c->grid_mult < 0) return PA_ERR_INVALID_ARG;
  if (c->split_merge < PA_MERGE_AUTO || c->split_merge > PA_MERGE_IN_REDUCE)
    return PA_ERR_INVALID_ARG;
  if (c->num_q_heads % c->num_kv_heads != 0) return PA_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (!is_pow2(c->block_size) || c->block_size < 16 || c->block_size > 1024)
    return PA_ERR_UNSUPPORTED;
  if (c->q_dtype != PA_BF16 && c->q_dtype != PA_FP16) return PA_ERR_UNSUPPORTED;
  if (!kv_kind_taken(*c)) return PA_ERR_UNSUPPORTED;
  const long long rows = (long long)(c->num_q_heads / c->num_kv_heads) * c->max_q_len;
  if (rows > (1 << 20)) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// Persistent grid: num_ctas if given, else (SMs x grid_mult) x the decode CTAs that fit
// on one SM: one resident wave at multiplier 1; with a larger one the later CTAs start as
// earlier ones finish.
pa_status resolve_ctas(const pa_config& c, Variant* v) {
  if (c.num_ctas > 0) {
    v->ctas = c.num_ctas > 65535 ? 65535 : c.num_ctas;
    return PA_OK;
  }
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  v->sms = sms;
  const int mult = c.grid_mult > 0 ? c.grid_mult : 1;
  long long n = (long long)sms * mult * v->ctas_per_sm;
  v->ctas = (int)(n > 65535 ? 65535 : n);
  return PA_OK;
}

pa_status prepare(const pa_config* cfg, Variant* v, WsLayout* L) {
  pa_status st = validate(cfg);
  if (st != PA_OK) return st;
  *v = make_variant(*cfg);
  st = resolve_ctas(*cfg, v);
  if (st != PA_OK) return st;
  // The planner's concatenated token space is indexed with int32.
  const long long per_unit =
      (long long)cfg->max_blocks_per_seq * cfg->block_size + v->tt + v->item_cost;
  constexpr long long most = 1ll << 30;
  const long long heads = (long long)cfg->batch * cfg->num_kv_heads;
  if (heads >= most || heads * v->rb >= most || per_unit >= most || heads * v->rb * per_unit >= most)
    return PA_ERR_UNSUPPORTED;
  *L = ws_layout(*cfg, *v);
  return PA_OK;
}

pa_status check_ws(const void* ws, size_t ws_bytes, const WsLayout& L) {
  if (!ws || !aligned(ws, 256)) return PA_ERR_INVALID_ARG;
  if (ws_bytes < L.total) return PA_ERR_WORKSPACE;
  return PA_OK;
}

ProblemArgs problem_args(const pa_config& c, const int32_t* bt, const int32_t* ctx,
                         const int32_t* ql) {
  ProblemArgs a;
  a.block_tables = bt;
  a.context_lens = ctx;
  a.q_lens = ql;
  a.batch = c.batch;
  a.max_q_len = c.max_q_len;
  a.num_q_heads = c.num_q_heads;
  a.num_kv_heads = c.num_kv_heads;
  a.head_dim = c.head_dim;
  a.block_size = c.block_size;
  a.max_blocks = c.max_blocks_per_seq;
  a.num_blocks = c.num_blocks;
  a.causal = c.causal;
  return a;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point, so the library does not
// link libcuda directly.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Descriptor of a cache [num_blocks, block_size, Hkv, D] seen as a 4-D tensor (D innermost)
// with a box of one head's rows of one page.  CUDA-core kernel: {D, 1, rows, 1}, no swizzle.
// Tensor-core kernels: {128 bytes of D, 1, rows, 1} with the 128-byte swizzle, one box per
// 128-byte column slab (64-byte rows: the whole row, with the 64-byte swizzle; 32-byte rows: as it
// lies).
bool kv_tensor_map(CUtensorMap* m, const void* base, const pa_config& c, int box_rows, bool slabs) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const int bpe = c.kv_dtype == PA_FP8_E4M3 || c.kv_dtype == PA_INT4 ? 1 : 2;
  CUtensorMapDataType dt = bpe == 1                ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                           : c.kv_dtype == PA_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int width = c.kv_dtype == PA_INT4 ? c.head_dim / 2 : c.head_dim;  // elements of a row
  cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)c.num_kv_heads, (cuuint64_t)c.block_size,
                        (cuuint64_t)c.num_blocks};
  cuuint64_t strides[3] = {(cuuint64_t)width * bpe, (cuuint64_t)c.num_kv_heads * width * bpe,
                           (cuuint64_t)c.block_size * c.num_kv_heads * width * bpe};
  const int row = width * bpe;
  const bool narrow = row < 128;  // 64- or 32-byte rows: one slab of them
  const cuuint32_t inner = slabs && !narrow ? (cuuint32_t)(128 / bpe) : (cuuint32_t)width;
  cuuint32_t box[4] = {inner, 1, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  // L2 fetches no more than a head's row at a time: past it lies the next head's, which another CTA
  // reads at another time (128-byte rows, 8 kv heads, 150 MB of cache: 172 MB read and 39.9 us a
  // step with 256 bytes, 36.9 us with 128; one kv head: 43.4 us either way)
  const auto promotion = row >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                         : row >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                         : row >= 64  ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                      : CU_TENSOR_MAP_L2_PROMOTION_NONE;
  std::memset(m, 0, sizeof(*m));
  CUresult r = enc(m, dt, 4, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE,
                   !slabs || row < 64 ? CU_TENSOR_MAP_SWIZZLE_NONE
                   : narrow           ? CU_TENSOR_MAP_SWIZZLE_64B
                                      : CU_TENSOR_MAP_SWIZZLE_128B,
                   promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

pa_status pa_workspace_size(const pa_config* cfg, size_t* bytes) {
  if (!cfg || !bytes) return PA_ERR_INVALID_ARG;
  Variant v;
  WsLayout L;
  pa_status st = prepare(cfg, &v, &L);
  if (st != PA_OK) return st;
  *bytes = L.total;
  return PA_OK;
}

pa_status pa_plan(const pa_config* cfg, const int32_t* block_tables, const int32_t* context_lens,
                  const int32_t* q_lens, void* ws, size_t ws_bytes, pa_stream stream) {
  Variant v;
  WsLayout L;
  pa_status st = prepare(cfg, &v, &L);
  if (st != PA_OK) return st;
  if (!block_tables || !context_lens || !q_lens) return PA_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, L)) != PA_OK) return st;
  const ProblemArgs a = problem_args(*cfg, block_tables, context_lens, q_lens);
  if (launch_plan(a, v, L, static_cast<char*>(ws), reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

pa_status pa_decode(const pa_config* cfg, const void* q, const void* k_cache, const void* v_cache,
                    const void* k_scale, const void* v_scale, const int32_t* block_tables,
                    const int32_t* context_lens, const int32_t* q_lens, void* out, float* lse,
                    void* ws, size_t ws_bytes, pa_stream stream) {
  Variant v;
  WsLayout L;
  pa_status st = prepare(cfg, &v, &L);
  if (st != PA_OK) return st;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !q_lens || !out)
    return PA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
    return PA_ERR_INVALID_ARG;
  if (lse && !aligned(lse, 4)) return PA_ERR_INVALID_ARG;
  if (cfg->kv_scale_mode != PA_SCALE_NONE) {
    const uintptr_t to = cfg->kv_dtype == PA_INT4 ? 16 : 4;
    if (!k_scale || !v_scale || !aligned(k_scale, to) || !aligned(v_scale, to))
      return PA_ERR_INVALID_ARG;
  }
  if ((st = check_ws(ws, ws_bytes, L)) != PA_OK) return st;

  const int tile_rows = v.path == 4 ? int4_tile_tokens(cfg->head_dim, v.mp) : v.tt;
  const int box_rows = v.path == 3 ? 16 : cfg->block_size < tile_rows ? cfg->block_size : tile_rows;
  CUtensorMap maps[2];
  if (!kv_tensor_map(&maps[0], k_cache, *cfg, box_rows, v.path >= 1) ||
      !kv_tensor_map(&maps[1], v_cache, *cfg, box_rows, v.path >= 1))
    return PA_ERR_CUDA;
  DecodeArgs a;
  a.p = problem_args(*cfg, block_tables, context_lens, q_lens);
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.scale_mode = cfg->kv_scale_mode;
  a.qk_scale = cfg->sm_scale * kLog2e;
  a.out = out;
  a.lse = lse;
  a.ws = static_cast<char*>(ws);
  a.L = L;
  a.v = v;
  a.q_kind = cfg->q_dtype == PA_FP16 ? Q_FP16 : Q_BF16;
  a.kv_kind = cfg->kv_dtype == PA_INT4       ? KV_INT4
              : cfg->kv_dtype == PA_FP8_E4M3 ? KV_FP8
              : cfg->kv_dtype == PA_FP16     ? KV_FP16
                                             : KV_BF16;
  cudaError_t e = launch_decode(a, maps, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return PA_ERR_UNSUPPORTED;
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_reduce(const pa_config* cfg, void* out, float* lse, void* ws, size_t ws_bytes,
                    pa_stream stream) {
  Variant v;
  WsLayout L;
  pa_status st = prepare(cfg, &v, &L);
  if (st != PA_OK) return st;
  if (!out || !aligned(out, 16)) return PA_ERR_INVALID_ARG;
  if (lse && !aligned(lse, 4)) return PA_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, L)) != PA_OK) return st;
  if (cfg->split_merge == PA_MERGE_IN_DECODE) return PA_OK;  // pa_decode finished the step
  DecodeArgs a{};
  a.p = problem_args(*cfg, nullptr, nullptr, nullptr);
  a.out = out;
  a.lse = lse;
  a.ws = static_cast<char*>(ws);
  a.L = L;
  a.v = v;
  a.q_kind = cfg->q_dtype == PA_FP16 ? Q_FP16 : Q_BF16;
  return launch_reduce(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK
                                                                                : PA_ERR_CUDA;
}

pa_status pa_decode_selected(const pa_config* cfg, const void* q, const void* k_cache,
                             const void* v_cache, const float* k_scale, const float* v_scale,
                             const int32_t* block_tables, const int32_t* context_lens,
                             const int32_t* q_lens, const int32_t* selected,
                             const int32_t* num_selected, int32_t top_k, void* out, float* lse,
                             int32_t* flags, pa_stream stream) {
  const pa_status st = validate(cfg);
  if (st != PA_OK) return st;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !q_lens || !selected ||
      !num_selected || !out || top_k < 1)
    return PA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(q_lens, 4) ||
      !aligned(selected, 4) || !aligned(num_selected, 4) || !aligned(lse, 4) || !aligned(flags, 4))
    return PA_ERR_INVALID_ARG;
  const pa_config& c = *cfg;
  if (c.kv_dtype == PA_INT4) return PA_ERR_UNSUPPORTED;
  const int mode = c.kv_scale_mode;
  if (mode != PA_SCALE_NONE &&
      (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)))
    return PA_ERR_INVALID_ARG;
  SelectedParams p;
  const int scales = staged_scales(mode);
  p.cache.k = static_cast<const char*>(k_cache);
  p.cache.v = static_cast<const char*>(v_cache);
  p.cache.k_scale = mode == PA_SCALE_NONE ? nullptr : k_scale;
  p.cache.v_scale = mode == PA_SCALE_NONE ? nullptr : v_scale;
  p.cache.sc_head = scales != SC_NONE ? 1 : 0;
  p.cache.sc_slot = scales == SC_TOKEN ? c.num_kv_heads : 0;
  p.cache.sc_block = scales == SC_TOKEN   ? (long long)c.block_size * c.num_kv_heads
                     : scales == SC_BLOCK ? c.num_kv_heads
                                          : 0;
  p.cache.Hkv = c.num_kv_heads;
  p.cache.bs_shift = ilog2((uint32_t)c.block_size);
  p.q = static_cast<const char*>(q);
  p.bt = block_tables;
  p.ctx = context_lens;
  p.qlens = q_lens;
  p.selected = selected;
  p.num = num_selected;
  p.out = out;
  p.lse = lse;
  p.flags = flags;
  p.Sq = c.max_q_len;
  p.Hq = c.num_q_heads;
  p.Hkv = c.num_kv_heads;
  p.G = c.num_q_heads / c.num_kv_heads;
  p.RB = ceil_div(p.G, 16);
  p.maxb = c.max_blocks_per_seq;
  p.nblocks = c.num_blocks;
  p.causal = c.causal;
  p.top_k = top_k;
  p.qk_scale = c.sm_scale * kLog2e;
  const double units_d = (double)c.batch * c.max_q_len * c.num_kv_heads * p.RB;
  if (units_d * kSelMaxSplit > INT32_MAX ||
      (long long)c.max_blocks_per_seq * c.block_size > INT32_MAX ||
      (long long)top_k * c.block_size > INT32_MAX)
    return PA_ERR_UNSUPPORTED;
  SelectedKind k;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&k.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  const int pages = top_k < c.max_blocks_per_seq ? top_k : c.max_blocks_per_seq;
  k.units = (long long)units_d;
  k.tokens = (long long)pages * c.block_size;
  k.kvk = c.kv_dtype == PA_FP8_E4M3 ? KV_FP8 : c.kv_dtype == PA_FP16 ? KV_FP16 : KV_BF16;
  k.qk = c.q_dtype == PA_FP16 ? Q_FP16 : Q_BF16;
  k.toks = scales == SC_TOKEN;
  CUtensorMap kmap{}, vmap{};
  if (k.kvk == KV_FP8 && (!kv_tensor_map(&kmap, k_cache, c, 16, true) ||
                          !kv_tensor_map(&vmap, v_cache, c, 16, true)))
    return PA_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (c.head_dim) {
    case 64: e = launch_selected_d64(p, k, kmap, vmap, s); break;
    case 128: e = launch_selected_d128(p, k, kmap, vmap, s); break;
    default: e = launch_selected_d256(p, k, kmap, vmap, s); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_read_flags(const void* ws, size_t ws_bytes, int32_t* flags, pa_stream stream) {
  if (!ws || !flags || !aligned(ws, 256) || ws_bytes < 64 * sizeof(int32_t))
    return PA_ERR_INVALID_ARG;
  int32_t host = 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(&host, static_cast<const char*>(ws) + HDR_FLAGS * sizeof(int32_t),
                      sizeof(int32_t), cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return PA_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return PA_ERR_CUDA;
  *flags = host;
  return host ? PA_ERR_DEVICE : PA_OK;
}

const char* pa_status_string(pa_status status) {
  switch (status) {
    case PA_OK: return "ok";
    case PA_ERR_INVALID_ARG: return "invalid argument";
    case PA_ERR_UNSUPPORTED: return "unsupported configuration";
    case PA_ERR_WORKSPACE: return "workspace too small";
    case PA_ERR_CUDA: return "CUDA error";
    case PA_ERR_DEVICE: return "device-side input problem (see flags)";
    default: return "unknown status";
  }
}

}  // extern "C"
