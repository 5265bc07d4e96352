// pkd_int4_launch.h -- host entry of the decode kernel over 4-bit caches.
#pragma once
#include <cuda_runtime.h>
#include "pkd_decode.cuh"

namespace pkd {

// Query tokens per CTA for q_len of them and groups of G heads: what fits eight
// rows where all do, else sixteen.
inline int int4_query_chunk(int q_len, int G) { return q_len * G <= 8 ? q_len : (q_len < 16 / G ? q_len : 16 / G); }
// Resident CTAs per SM.
constexpr int kInt4CtasPerSm = 3;
// p.q_chunks chunks of int4_query_chunk(p.q_len, G) tokens; partials unless a sequence has one partition.
cudaError_t launch_decode_int4(int D, int BS, int G, const DecodeParams& p, long long grid, cudaStream_t stream);

}  // namespace pkd
