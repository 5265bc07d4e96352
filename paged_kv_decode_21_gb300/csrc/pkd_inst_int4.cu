// Instantiations of the decode kernel over 4-bit caches.
#include "pkd_int4.cuh"
#include "pkd_int4_launch.h"

namespace pkd {
namespace {

template <int D, int BS, int NT>
cudaError_t launch(const Int4Params& p, long long grid, cudaStream_t stream) {
  using T = Int4Traits<D, BS, NT>;
  static_assert(T::MIN_BLOCKS == kInt4CtasPerSm, "the split counts on these");
  auto* fn = paged_decode_int4_kernel<D, BS, NT>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM_BYTES);
  if (failed(e)) return e;
  fn<<<(unsigned)grid, T::THREADS, T::SMEM_BYTES, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int BS>
cudaError_t launch_rows(const Int4Params& p, long long grid, cudaStream_t stream) {
  return p.group * p.q_chunk <= 8 ? launch<D, BS, 1>(p, grid, stream) : launch<D, BS, 2>(p, grid, stream);
}

}  // namespace

cudaError_t launch_decode_int4(int D, int BS, int G, const DecodeParams& p, long long grid, cudaStream_t stream) {
  const Int4Params ip{p, G, int4_query_chunk(p.q_len, G)};
  if (D == 128 && BS == 16) return launch_rows<128, 16>(ip, grid, stream);
  if (D == 128 && BS == 32) return launch_rows<128, 32>(ip, grid, stream);
  if (D == 64 && BS == 16) return launch_rows<64, 16>(ip, grid, stream);
  if (D == 64 && BS == 32) return launch_rows<64, 32>(ip, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkd
