// Instantiations of the decode kernel over 4-bit caches.
#include <algorithm>
#include <cmath>

#include "pkd_int4.cuh"
#include "pkd_int4_launch.h"

namespace pkd {
namespace {

template <int D, int BS, int NT>
cudaError_t launch(const Int4Params& p, long long grid, cudaStream_t stream) {
  using T = Int4Traits<D, BS, NT>;
  auto* fn = paged_decode_int4_kernel<D, BS, NT>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM_BYTES);
  if (failed(e)) return e;
  if (!p.d.piece_order) {
    fn<<<(unsigned)grid, T::THREADS, T::SMEM_BYTES, stream>>>(p);
    return cudaGetLastError();
  }
  // a programmatic dependent of the order kernel
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(T::THREADS);
  cfg.dynamicSmemBytes = T::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

template <int D, int BS>
cudaError_t launch_rows(const Int4Params& p, long long grid, cudaStream_t stream) {
  switch (int4_rows(p.d.q_len, p.group)) {
    case 8: return launch<D, BS, 1>(p, grid, stream);
    case 16: return launch<D, BS, 2>(p, grid, stream);
    default: return launch<D, BS, 4>(p, grid, stream);
  }
}

}  // namespace

cudaError_t launch_decode_int4(int D, int BS, int G, const DecodeParams& p, long long grid, cudaStream_t stream) {
  Int4Params ip{p, G, int4_query_chunk(p.q_len, G), p.scale_log2 < 0.f ? 0x80008000u : 0u, kInt4Bases};
  // (a scale of 0, equal weights: one too small to tell, so that -inf times it stays -inf)
  ip.d.scale_log2 = std::max(std::fabs(p.scale_log2), 1e-30f);
  if (D == 128 && BS == 16) return launch_rows<128, 16>(ip, grid, stream);
  if (D == 128 && BS == 32) return launch_rows<128, 32>(ip, grid, stream);
  if (D == 64 && BS == 16) return launch_rows<64, 16>(ip, grid, stream);
  if (D == 64 && BS == 32) return launch_rows<64, 32>(ip, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkd
