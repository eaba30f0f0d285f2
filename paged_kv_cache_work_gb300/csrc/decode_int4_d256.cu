// Instances of the decode over 4-bit caches for head dim 256.
#include "decode_int4.cuh"

namespace pa {

cudaError_t launch_int4_d256(const KernelParams& prm, const CUtensorMap (&maps)[2], int grid, int mp,
                            int qk, cudaStream_t s) {
  return launch_int4_dim<256>(prm, maps, grid, mp, qk, s);
}
int int4_ctas_per_sm_d256(int mp) {
  return mp == 8 ? DecodeInt4Smem<Int4Attention<256, 1, Q_BF16>>::CTAS_PER_SM
                 : DecodeInt4Smem<Int4Attention<256, 2, Q_BF16>>::CTAS_PER_SM;
}

}  // namespace pa
