// pkd_split.h -- how a context of any 32-bit length is cut into partitions.
// Plain arithmetic for the kernels and the host, without a step that could pass
// 32 bits: lengths come from device memory, where a corrupt one may be as large
// as INT_MAX, and a block-table row may hold as many tokens.
#pragma once
#ifdef __CUDACC__
#define PKD_SPLIT_FN __host__ __device__ __forceinline__
#else
#define PKD_SPLIT_FN inline
#endif

namespace pkd {

// Partitions of `part` tokens that hold L tokens, np at most; none for L <= 0.
PKD_SPLIT_FN int partitions_of(int L, int part, int np) {
  const unsigned n = ((unsigned)(L > 0 ? L : 0) + (unsigned)part - 1u) / (unsigned)part;
  return n < (unsigned)np ? (int)n : np;
}

// Half of L tokens (L >= 0), rounded up.
PKD_SPLIT_FN int half_up(int L) { return L / 2 + L % 2; }

// The partition of a sequence of L tokens that is split in two: half of it,
// rounded up to whole 64-token tiles (so a sequence of at most 64 tokens stays whole).
PKD_SPLIT_FN int tail_half_partition(int L) { return (half_up(L) + 63) / 64 * 64; }

}  // namespace pkd
