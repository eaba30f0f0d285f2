// pa_decode_selected's kernel instances for head dim 128.
#include "decode_selected.cuh"

namespace pa {

cudaError_t launch_selected_d128(SelectedParams& p, const SelectedKind& k, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, cudaStream_t s) {
  return launch_selected_for_dim<128>(p, k, kmap, vmap, s);
}

}  // namespace pa
