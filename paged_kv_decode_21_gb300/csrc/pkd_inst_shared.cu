// Instantiations of the tensor-core decode kernel over a group's shared
// context, fp16 caches.
#include "pkd_mma_launch.cuh"
#include "pkd_src_launch.h"

namespace pkd {
cudaError_t launch_decode_shared(int D, int BS, int G, const DecodeParams& p, long long grid, cudaStream_t stream) {
  return mma_host::launch_all<mma_host::MultiQuery, 2, 0, kShared>(D, BS, G, p, grid, stream);
}
}  // namespace pkd
