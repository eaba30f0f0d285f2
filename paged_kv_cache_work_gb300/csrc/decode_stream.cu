// Instances of the streaming decode over fp8 caches with one scale for each (page, kv head).
#include "decode_stream.cuh"

namespace pa {

cudaError_t launch_stream(const KernelParams& prm, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          int grid, int head_dim, int qk, cudaStream_t s) {
#define PA_STREAM(D_)                                                             \
  if (head_dim == D_)                                                             \
    return qk == Q_BF16 ? launch_stream_instance<D_, Q_BF16>(prm, kmap, vmap, grid, s) \
                        : launch_stream_instance<D_, Q_FP16>(prm, kmap, vmap, grid, s);
  PA_STREAM(64)
  PA_STREAM(128)
  PA_STREAM(256)
#undef PA_STREAM
  return cudaErrorNotSupported;
}

int stream_ctas_per_sm(int head_dim) {
  switch (head_dim) {
    case 64: return DecodeStreamSmem<StreamTraits<64, KV_FP8, Q_BF16, false>>::CTAS_PER_SM;
    case 128: return DecodeStreamSmem<StreamTraits<128, KV_FP8, Q_BF16, false>>::CTAS_PER_SM;
    default: return DecodeStreamSmem<StreamTraits<256, KV_FP8, Q_BF16, false>>::CTAS_PER_SM;
  }
}

}  // namespace pa
