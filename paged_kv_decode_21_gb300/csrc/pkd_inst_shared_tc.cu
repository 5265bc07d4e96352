// Instantiations and launch of the shared-context tcgen05 kernel
// (pkd_shared_tc.cuh): fp16 caches at head_dim 64 or 128, E4M3 caches at
// head_dim 128, block sizes 16 and 32.
#include "pkd_mma_launch.cuh"
#include "pkd_shared_tc.cuh"
#include "pkd_tc_launch.h"

namespace pkd {
static_assert(kSharedRows == kSharedRowsPerCta, "rows per CTA of the kernel and of its host entry");

namespace {

// A CTA holds all 512 columns of its SM's tensor memory, so it and a CTA of the
// tcgen05 decode kernel, which may run beside it, must not share an SM: one
// would wait for the other's columns.  Their shared memory rules it out.
template <int KVB, int HD>
constexpr bool apart() {
  return SharedTcTraits<16, KVB, HD>::SMEM_BYTES + TcTraits<16, KVB, HD>::SMEM_BYTES > 226 * 1024;
}
static_assert(apart<2, 128>() && apart<2, 64>() && apart<1, 128>(), "never on one SM");

template <int BS, int KVB, int HD>
cudaError_t launch_bs(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeParams& p, long long grid,
                      cudaStream_t stream) {
  using T = SharedTcTraits<BS, KVB, HD>;
  auto* fn = paged_shared_tc_kernel<BS, KVB, HD>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM_BYTES);
  if (failed(e)) return e;
  fn<<<(unsigned)grid, T::THREADS, T::SMEM_BYTES, stream>>>(mk, mv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_shared_tc(int D, int BS, const DecodeParams& p, long long grid, cudaStream_t stream, int kvb) {
  if ((D != 128 && !(D == 64 && kvb == 2)) || (BS != 16 && BS != 32) || (kvb != 1 && kvb != 2))
    return cudaErrorInvalidValue;
  CUtensorMap mk, mv;
  const cudaError_t e = mma_host::make_maps(p, D, BS, kvb, &mk, &mv);
  if (failed(e)) return e;
  if (kvb == 1) return BS == 16 ? launch_bs<16, 1, 128>(mk, mv, p, grid, stream) : launch_bs<32, 1, 128>(mk, mv, p, grid, stream);
  if (D == 64) return BS == 16 ? launch_bs<16, 2, 64>(mk, mv, p, grid, stream) : launch_bs<32, 2, 64>(mk, mv, p, grid, stream);
  return BS == 16 ? launch_bs<16, 2, 128>(mk, mv, p, grid, stream) : launch_bs<32, 2, 128>(mk, mv, p, grid, stream);
}

}  // namespace pkd
