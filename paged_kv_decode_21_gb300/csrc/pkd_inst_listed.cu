// Instantiations of the tensor-core decode kernel over block lists, fp16 caches.
#include "pkd_mma_launch.cuh"
#include "pkd_src_launch.h"

namespace pkd {
cudaError_t launch_decode_listed(int D, int BS, int G, const DecodeParams& p, long long grid, cudaStream_t stream) {
  return mma_host::launch_all<mma_host::SingleQuery, 2, 0, kListed>(D, BS, G, p, grid, stream);
}
}  // namespace pkd
