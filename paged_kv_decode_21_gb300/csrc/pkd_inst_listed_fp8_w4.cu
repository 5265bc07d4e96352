// Instantiations of the tensor-core decode kernel over block lists, E4M3 caches,
// at four CTAs per SM.
#include "pkd_mma_launch.cuh"
#include "pkd_src_launch.h"

namespace pkd {
cudaError_t launch_decode_listed_fp8_w4(int D, int BS, int G, const DecodeParams& p, long long grid,
                                        cudaStream_t stream) {
  return mma_host::launch_all<mma_host::SingleQuery, 1, 4, kListed>(D, BS, G, p, grid, stream);
}
}  // namespace pkd
