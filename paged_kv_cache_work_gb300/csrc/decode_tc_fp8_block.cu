// tcgen05 decode kernel instances for fp8 (E4M3) caches with one scale for each (page, kv head):
// head dim 128, query tiles of 64 or 128 rows.
#include "decode_tc.cuh"

namespace pa {

#define PA_TC_FP8_BLOCK(X) \
  X(64, Q_BF16) X(64, Q_FP16) X(128, Q_BF16) X(128, Q_FP16)

cudaError_t launch_tc_fp8_block_d128(const KernelParams& prm, const CUtensorMap& kmap,
                                     const CUtensorMap& vmap, int grid, int mp, int qk,
                                     cudaStream_t s) {
#define PA_TC_CASE(MP_, QK_)  \
  if (mp == MP_ && qk == QK_) \
    return launch_tc_instance<128, MP_, KV_FP8, QK_, SC_BLOCK>(prm, kmap, vmap, grid, s);
  PA_TC_FP8_BLOCK(PA_TC_CASE)
#undef PA_TC_CASE
  return cudaErrorNotSupported;
}

}  // namespace pa
