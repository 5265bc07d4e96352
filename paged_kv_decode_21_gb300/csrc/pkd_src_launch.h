// pkd_src_launch.h -- host entries of the mma.sync decode kernel's builds
// whose keys are a block list or a group's shared context (KeySource).
#pragma once
#include <cuda_runtime.h>
#include "pkd_decode.cuh"

namespace pkd {

// p.block_lists, p.list_lens and p.max_listed set; one query token per sequence.
cudaError_t launch_decode_listed(int D, int BS, int G, const DecodeParams& p, long long grid, cudaStream_t stream);
cudaError_t launch_decode_listed_fp8(int D, int BS, int G, const DecodeParams& p, long long grid,
                                     cudaStream_t stream);
// The same at four CTAs per SM.
cudaError_t launch_decode_listed_fp8_w4(int D, int BS, int G, const DecodeParams& p, long long grid,
                                        cudaStream_t stream);
// p.group_starts and p.num_groups set, p.mode 1; p.q_chunks chunks of
// mma_query_chunk(G) query tokens cover every group.
cudaError_t launch_decode_shared(int D, int BS, int G, const DecodeParams& p, long long grid, cudaStream_t stream);
cudaError_t launch_decode_shared_fp8(int D, int BS, int G, const DecodeParams& p, long long grid,
                                     cudaStream_t stream);

}  // namespace pkd
