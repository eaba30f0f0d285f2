// Instances of the decode over 4-bit caches for head dim 64.
#include "decode_int4.cuh"

namespace pa {

cudaError_t launch_int4_d64(const KernelParams& prm, const CUtensorMap (&maps)[2], int grid, int mp,
                           int qk, cudaStream_t s) {
  return launch_int4_dim<64>(prm, maps, grid, mp, qk, s);
}
int int4_ctas_per_sm_d64(int mp) {
  return mp == 8 ? DecodeInt4Smem<Int4Attention<64, 1, Q_BF16>>::CTAS_PER_SM
                 : DecodeInt4Smem<Int4Attention<64, 2, Q_BF16>>::CTAS_PER_SM;
}

}  // namespace pa
