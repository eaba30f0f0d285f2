// pa_decode_selected's kernel instances for head dim 64.
#include "decode_selected.cuh"

namespace pa {

cudaError_t launch_selected_d64(SelectedParams& p, const SelectedKind& k, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, cudaStream_t s) {
  return launch_selected_for_dim<64>(p, k, kmap, vmap, s);
}

}  // namespace pa
