// pkd_int4_launch.h -- host entry of the decode kernel over 4-bit caches.
#pragma once
#include <cuda_runtime.h>
#include "pkd_decode.cuh"

namespace pkd {

// Query rows (tokens times the group's heads) of a CTA, for q_len tokens and
// groups of G heads: 8, 16 or 32, the fewest that hold all, else 32.
inline int int4_rows(int q_len, int G) {
  const long long all = (long long)q_len * G;
  return all <= 8 ? 8 : (all <= 16 ? 16 : 32);
}
// Query tokens of a CTA.
inline int int4_query_chunk(int q_len, int G) {
  const int most = int4_rows(q_len, G) / G;
  return q_len < most ? q_len : most;
}
// Resident CTAs per SM.
constexpr int kInt4CtasPerSm = 4;
inline int int4_ctas_per_sm(int rows) { return rows == 8 ? kInt4CtasPerSm : (rows == 16 ? 3 : 2); }
// p.q_chunks chunks of int4_query_chunk(p.q_len, G) tokens; partials unless a sequence has one partition.
cudaError_t launch_decode_int4(int D, int BS, int G, const DecodeParams& p, long long grid, cudaStream_t stream);

}  // namespace pkd
