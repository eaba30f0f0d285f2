// pa_decode_selected's kernel instances for head dim 256.
#include "decode_selected.cuh"

namespace pa {

cudaError_t launch_selected_d256(SelectedParams& p, const SelectedKind& k, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, cudaStream_t s) {
  return launch_selected_for_dim<256>(p, k, kmap, vmap, s);
}

}  // namespace pa
