// pa_decode_selected's kernel instances for head dim 64.
#include "decode_selected.cuh"

namespace pa {

cudaError_t launch_selected_d64(const SelectedParams& p, int kvk, int qk, long long units,
                                cudaStream_t s) {
  return launch_selected_for_dim<64>(p, kvk, qk, units, s);
}

}  // namespace pa
