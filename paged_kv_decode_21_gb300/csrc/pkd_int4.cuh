// pkd_int4.cuh -- 4-bit caches: how a tile lies in memory, how codes become
// fp16 operands, the decode kernel and the read-back of rows.
//
// value = (u - 8) * s * cache scale, u a code of 4 bits, s the E4M3 scale of
// its 16 dims.  A (block, kv head) tile is one run of bytes: codes
// [D / 32][BS][16], two dims a byte, then scales [BS][D / 16].
#pragma once
#include <cstdint>
#include <cuda_fp16.h>
#include "pkd_decode.cuh"
#include "pkd_decode_mma.cuh"
#include "pkd_int4_launch.h"
#include "pkd_ptx.cuh"

namespace pkd {

__host__ __device__ constexpr int int4_tile_bytes(int D, int BS) { return BS * D * 9 / 16; }

// ---------------------------------------------------------------- codes -> fp16
// A code's bits dropped into an fp16 mantissa give 1024 + u (bits 0..3 under
// the exponent of 1024) or 64 + u (bits 4..7 under that of 64), so one fused
// multiply-add per pair makes (u - 8) s of it: (1024 + u) s - 1032 s and
// (64 + u) s - 72 s.  All exact: s = s8 * 2^-8 below has four significant bits,
// 1032 s eleven (129 * 15 < 2048), u - 8 four; the smallest product, 2^-17, is a
// multiple of fp16's 2^-24 and the largest, 8 * 1.75, and 1032 * 1.75 are far
// from its largest.  Eight codes take a shift, four logical operations and four
// multiply-adds; converting E2M1 codes by cvt takes as many, and more where
// codes of two tokens have to meet in a pair first.
//
// Scale bytes: E4M3 bits shifted to fp16's exponent and mantissa are s * 2^-8
// exactly, subnormals too (the sign bit is 0); the 2^8 goes into the softmax
// scale for K and into the result for V.
constexpr float kInt4Unscale = 256.f;

__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hadd2_u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

constexpr uint32_t kHalf1032 = 0xE408E408u;  // -1032 twice
constexpr uint32_t kHalf72 = 0xD480D480u;    // -72 twice

// (x & MASK) | base, one instruction where base is a register the compiler
// cannot see through: with both constants known it takes two.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t masked_or(uint32_t x, uint32_t base) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "n"(MASK), "r"(base));
  return d;
}
// 1024 and 64 in both halves, from the kernel's arguments.
struct Int4Bases {
  uint32_t b1024, b64;
};
constexpr Int4Bases kInt4Bases{0x64006400u, 0x54005400u};

// The scales of two words, or of a word's two halves, with the addends they need.
struct Int4Scale {
  uint32_t s, a1, a2;
};
__device__ __forceinline__ Int4Scale int4_scale(uint32_t s) { return {s, hmul2_u(s, kHalf1032), hmul2_u(s, kHalf72)}; }

// Half h of x in both halves (a multiply-add takes it without an instruction of its own).
__device__ __forceinline__ uint32_t both_halves(uint32_t x, int h) {
  uint32_t d;
  if (h)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(d) : "r"(x));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ Int4Scale both_halves(const Int4Scale& x, int h) {
  return {both_halves(x.s, h), both_halves(x.a1, h), both_halves(x.a2, h)};
}

// Codes j and j + 4 of a word (j = 0..3) as the halves of d[j], times the
// scales in the halves of s.
__device__ __forceinline__ void int4_words(uint32_t x, const Int4Scale& s, const Int4Bases& base, uint32_t (&d)[4]) {
  const uint32_t y = x >> 8;
  d[0] = hfma2_u(masked_or<0x000F000Fu>(x, base.b1024), s.s, s.a1);
  d[1] = hfma2_u(masked_or<0x00F000F0u>(x, base.b64), s.s, s.a2);
  d[2] = hfma2_u(masked_or<0x000F000Fu>(y, base.b1024), s.s, s.a1);
  d[3] = hfma2_u(masked_or<0x00F000F0u>(y, base.b64), s.s, s.a2);
}

// Two scale bytes as an fp16 pair of s * 2^-8: byte i of a and byte j - 4 of b
// for sel = int4_scale_sel(i, j).  The selectors' sign mode fills the bytes
// between with the (clear) sign bit, so that a permutation and a shift do.
__device__ __forceinline__ uint32_t int4_scale_sel(uint32_t i, uint32_t j) {
  return (i | (j << 8)) * 0x11u + 0x8080u;
}
__device__ __forceinline__ uint32_t int4_scale_pair(uint32_t a, uint32_t b, uint32_t sel) {
  return prmt(a, b, sel) * 128u;
}

// ---------------------------------------------------------------- instructions
// d = (zero ? 0 : d) + A . B for one m16n8k16 tile; `zero` known when compiled.
__device__ __forceinline__ void mma_16816_from(float (&d)[4], bool zero, uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  if (zero) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  } else {
    const uint32_t a[4] = {a0, a1, a2, a3};
    mma_16816(d, a, b0, b1);
  }
}

// An arrival that announces `bytes`, and a copy that completes on the barrier (shared addresses).
__device__ __forceinline__ void int4_expect(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\t"
      "mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void int4_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// An 8 x 8 matrix of 16-bit elements, lane (r, c) holding row r's columns 2c and 2c + 1, transposed.
__device__ __forceinline__ uint32_t transposed_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// ---------------------------------------------------------------- decode
// The split of the work, the online softmax, the merge of the warps and the
// meaning of rows are those of paged_decode_mma_kernel; here a warp's ring
// holds whole (block, kv head) tiles, brought by two plain bulk copies.
//
// Both products have the cache as their A operand (16 rows: tokens, or dims) and
// the queries as their B operand (8 columns): S^T = K Q^T, O^T = V^T P^T, so that
// eight query rows and less waste no half of a tile.  (With Q as A, of 16 rows,
// single queries took twice the products for S, and moves that put zeros into
// the operands' registers: 386 instructions per 16 tokens instead of 356.)
// Fragments (c = lane % 4, r = lane / 4), for a slab of 32 dims:
//   K  an ldmatrix of 8 tokens x 16 bytes gives lane (r, c) the codes of dims 8c
//      .. 8c + 7 of token r: two k-steps' A operands, dims (8c + j, 8c + j + 4)
//      in the halves.  Q's B fragments follow that order of dims.
//   S^T  lane (r, c) receives tokens r and r + 8 of query rows 2c and 2c + 1;
//      packed in pairs of rows and transposed in 8 x 8 matrices (movmatrix),
//      the weights are P^T's B fragments.
//   V  the transposed ldmatrix gives lane (r, c) dims 4r .. 4r + 3 of tokens 2c
//      and 2c + 1, one token a half: rows r and r + 8 of two m-tiles of V^T.
// Query rows are the group's heads times up to `q_chunk` query tokens, NT tiles
// of 8 of them: 1, 2 or 4.  With 4 the Q fragments stay in shared memory.
//
// Bound by its instructions' dependencies and pipes.  Of a 16-token subtile's 356
// (one row tile) half are the codes' way into fp16 pairs, 16 the products.  They
// fill 0.59 of a scheduler's cycles, HBM at half its rate: the registers leave 3.9
// warps a scheduler, and of the 6.5 cycles from one instruction of a warp to its
// next 1.3 wait for the one before, 1.1 for another warp's turn, 1.0 for a pipe
// (ALU 50%, fp16 31%, tensor 23% busy), 0.8 for loads, 0.6 for the dispatch.
// 128 x 32/8 heads, 512-4096 tokens, 83 us; 32 x 40/8, 16K-32K, 180; the bytes
// alone 50 and 135.  Four row tiles (48 x 4 tokens x 28/4): 714 instructions, 0.38 a
// cycle of the 1.8 warps a scheduler that their accumulators leave room for, 1.6 of
// 4.7 cycles waiting for the instruction before, 0.5 for loads.  Three or five CTAs an SM for one row tile: 207 and 216 against 193 us at 16K-32K;
// chunks of two row tiles for 28 rows: +6%; the next scores beside a subtile's
// P V: no change; K scales spread by permutations, or shifts as multiplications: +5%.
struct Int4Params {
  DecodeParams d;
  int group, q_chunk;
  uint32_t q_sign;  // flips Q where the softmax scale is negative: d.scale_log2 is positive
  Int4Bases bases;
};

template <int D, int BS, int NT>
struct Int4Traits {
  static constexpr int NW = 4;
  static constexpr int THREADS = NW * 32;
  static constexpr int MIN_BLOCKS = NT == 1 ? kInt4CtasPerSm : (NT == 2 ? 3 : 2);
  static constexpr int TILE = int4_tile_bytes(D, BS);
  // a ring slot, one barrier: 32 tokens, K's tiles, then V's
  static constexpr int UNIT = 32, TILES = UNIT / BS;
  static constexpr int SLOT = 2 * TILES * TILE;
  static constexpr int SUBS = NT == 4 ? 1 : 2;  // 16-token subtiles per softmax step
  static constexpr int SLABS = D / 32;
  static constexpr int SCALE_OFF = BS * D / 2;
  static constexpr int SB = D / 16;  // scale bytes a token
  static constexpr int RING_KIB = MIN_BLOCKS >= 4 ? 54 : 72;
  static constexpr int SW_RAW = RING_KIB * 1024 / (NW * SLOT);
  static constexpr int SW = SW_RAW > 8 ? 8 : SW_RAW;
  static constexpr int RING_BYTES = NW * SW * SLOT;
  static constexpr int ROWS = 8 * NT;
  // the warps' maxima and sums; per row their factors, its sum and its place; their O's, rows of PITCH floats
  static constexpr int MRG_C_OFF = 2 * NW * ROWS, MRG_Z_OFF = MRG_C_OFF + NW * ROWS, MRG_ACC_OFF = MRG_Z_OFF + 2 * ROWS;
  static constexpr int PITCH = D + 4;  // (four query rows and two quads of dims at a time meet no bank twice)
  static constexpr int MERGE_BYTES = (MRG_ACC_OFF + NW * ROWS * PITCH) * 4;
  static constexpr int Q_BYTES = NT == 4 ? 2 * (D / 16) * 32 * 16 : 0;  // B fragments of four 8-row tiles
  static constexpr int MAIN_BYTES = RING_BYTES + Q_BYTES > MERGE_BYTES ? RING_BYTES + Q_BYTES : MERGE_BYTES;
  static constexpr int SMEM_BYTES = MAIN_BYTES + NW * SW * 8;
  static_assert(SW >= 2 && TILE % 16 == 0 && MAIN_BYTES % 16 == 0, "ring");
};

template <int D, int BS, int NT>
__global__ void __launch_bounds__(Int4Traits<D, BS, NT>::THREADS, Int4Traits<D, BS, NT>::MIN_BLOCKS)
    paged_decode_int4_kernel(const __grid_constant__ Int4Params IP) {
  using T = Int4Traits<D, BS, NT>;
  constexpr int NW = T::NW, SW = T::SW, SLABS = T::SLABS, ROWS = T::ROWS;
  const DecodeParams& P = IP.d;
  const Int4Bases bases = IP.bases;
  extern __shared__ __align__(128) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::MAIN_BYTES);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int np_grid = P.max_partitions, G = IP.group, QC = IP.q_chunk;
  const int qc = blockIdx.x % P.q_chunks;
  const int rest = blockIdx.x / P.q_chunks;
  int j, b, g;
  if (P.piece_order) {  // longest first, written by the grid this one is the programmatic dependent of
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int piece = P.piece_order[rest / P.num_kv_heads];
    g = rest % P.num_kv_heads;
    b = piece / np_grid;
    j = piece % np_grid;
  } else {
    j = rest % np_grid;
    g = rest / np_grid % P.num_kv_heads;
    b = rest / np_grid / P.num_kv_heads;
  }
  const int jq0 = qc * QC, QL = P.q_len, tok0 = b * QL;
  const int L = row_clamped_len<BS>(P, b);
  const int nq = min(QC, QL - jq0), rows = G * nq;
  const int PS = P.partition_size;
  const int np_b = L > 0 ? min((L - 1) / PS + 1, np_grid) : 0;
  const bool final_out = np_b <= 1;
  const int h0 = g * G, Hq = P.num_q_heads;
  auto out_row = [&](int rr) { return ((size_t)tok0 + jq0 + rr / G) * Hq + h0 + rr % G; };
  if (L <= 0) {
    if (j == 0)
      for (int i = threadIdx.x; i < rows * D; i += T::THREADS)
        P.out[out_row(i / D) * D + i % D] = __float2half_rn(0.f);
    return;
  }
  if (j >= np_b) return;
  const int t0 = j * PS;
  const int t1 = min(min(t0 + PS, L), L - QL + jq0 + nq);  // nothing past the chunk's last query is read
  const int units = t1 > t0 ? (t1 - t0 + T::UNIT - 1) / T::UNIT : 0;
  const int nblk = t1 > t0 ? (t1 - t0 + BS - 1) / BS : 0;
  const int32_t* bt = P.block_tables + (size_t)b * P.max_blocks_per_seq + t0 / BS;
  const uint64_t block_stride = (uint64_t)P.num_kv_heads * T::TILE;
  const char* kbase = reinterpret_cast<const char*>(P.k_cache) + (size_t)g * T::TILE;
  const char* vbase = reinterpret_cast<const char*>(P.v_cache) + (size_t)g * T::TILE;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int r = lane / 4, c = lane % 4;

  uint64_t* full = bars + warp * SW;
  unsigned char* ring = smem + (size_t)warp * SW * T::SLOT;
  if (lane == 0) {
    for (int s = 0; s < SW; ++s) mbar_init(&full[s], 1);
    fence_mbarrier_init();
  }
  __syncwarp();
  const int mine = units > warp ? (units - warp + NW - 1) / NW : 0;  // the warp's units: warp, warp + NW, ...
  // block ids of 32 / TILES of the warp's units at a time, the next ones requested ahead
  constexpr int TILES = T::TILES, IDS = 32 / TILES;
  auto ids_at = [&](int first) {
    const int n = first + lane / TILES, k = (warp + NW * n) * TILES + lane % TILES;
    return n < mine && k < nblk ? bt[k] : -1;
  };
  int ids = ids_at(0), ids_next = ids_at(IDS);
  uint32_t bad_slots = 0;  // TILES bits a slot: tiles that are not there
  uint32_t in_slot = 0;    // the next copies'
  const uint32_t ring_at = smem_u32(ring), full_at = smem_u32(full);
  auto issue = [&](int n) {  // copies of the warp's n-th unit, n ascending
    if (n > 0 && n % IDS == 0) {
      ids = ids_next;
      ids_next = ids_at(n + IDS);
    }
    const uint32_t slot = in_slot;
    in_slot = in_slot + 1 == SW ? 0 : in_slot + 1;
    // lanes 0 .. 2 TILES - 1 each copy a tile: K's, then V's
    const int pb = __shfl_sync(0xffffffffu, ids, (n % IDS) * TILES + lane % TILES);
    const bool good = (uint32_t)pb < (uint32_t)P.num_blocks;
    const uint32_t there = __ballot_sync(0xffffffffu, good) & ((1u << TILES) - 1);
    const uint32_t bar = full_at + slot * 8;
    if (there != (1u << TILES) - 1) {
      bad_slots |= (~there & ((1u << TILES) - 1)) << (slot * TILES);
      // (past the last block of the partition there is none)
      if (lane < TILES && !good && (warp + NW * n) * TILES + lane < nblk) record_error(P.error_word, kErrBadBlock);
    }
    if (lane == 0) int4_expect(bar, __popc(there) * 2 * T::TILE);
    if (lane < 2 * TILES && good)
      int4_copy(ring_at + slot * T::SLOT + lane * T::TILE,
                (lane < TILES ? kbase : vbase) + (uint64_t)(uint32_t)pb * block_stride, T::TILE, bar);
  };
  int issued = 0;
  for (; issued < SW && issued < mine; ++issued) issue(issued);

  // tokens at or past it are masked for query row rr (the first row sees the fewest)
  auto limit = [&](int rr) { return rr < rows ? min(t1, L - QL + jq0 + rr / G + 1) : t1; };
  const int lim_min = limit(0);

  // Q as B fragments: k-step 2s + e of slab s has slots (2c, 2c + 1) = dims 8c
  // + 2e and 8c + 2e + 4 of the slab, slots (8 + 2c, 9 + 2c) = the dims behind
  auto q_word = [&](int rr, int s) {
    if (rr >= rows) return make_uint4(0u, 0u, 0u, 0u);
    uint4 u = *reinterpret_cast<const uint4*>(P.q + out_row(rr) * D + 32 * s + 8 * c);
    u.x ^= IP.q_sign;
    u.y ^= IP.q_sign;
    u.z ^= IP.q_sign;
    u.w ^= IP.q_sign;
    return u;
  };
  uint32_t qb[NT < 4 ? 2 * SLABS : 1][NT][2];
  uint4* qs = reinterpret_cast<uint4*>(smem + T::RING_BYTES);  // [k-step][tile pair][lane]
  if constexpr (NT < 4) {
#pragma unroll
    for (int hf = 0; hf < NT; ++hf)
#pragma unroll
      for (int s = 0; s < SLABS; ++s) {
        const uint4 u = q_word(r + 8 * hf, s);
        qb[2 * s][hf][0] = prmt(u.x, u.z, 0x5410);
        qb[2 * s][hf][1] = prmt(u.x, u.z, 0x7632);
        qb[2 * s + 1][hf][0] = prmt(u.y, u.w, 0x5410);
        qb[2 * s + 1][hf][1] = prmt(u.y, u.w, 0x7632);
      }
  } else {
    for (int i = warp; i < 2 * SLABS; i += NW) {
      const int pair = i / SLABS, s = i % SLABS;
      const uint4 u = q_word(16 * pair + r, s), w = q_word(16 * pair + r + 8, s);
      qs[(2 * s * 2 + pair) * 32 + lane] = make_uint4(prmt(u.x, u.z, 0x5410), prmt(u.x, u.z, 0x7632),
                                                      prmt(w.x, w.z, 0x5410), prmt(w.x, w.z, 0x7632));
      qs[((2 * s + 1) * 2 + pair) * 32 + lane] = make_uint4(prmt(u.y, u.w, 0x5410), prmt(u.y, u.w, 0x7632),
                                                            prmt(w.y, w.w, 0x5410), prmt(w.y, w.w, 0x7632));
    }
    __syncthreads();
  }
  // O^T: tile 2s + e holds dims 32s + 4r + 2e (rows r) and the dims behind (rows r + 8)
  float o[2 * SLABS][NT][4];
#pragma unroll
  for (int k = 0; k < 2 * SLABS; ++k)
#pragma unroll
    for (int hf = 0; hf < NT; ++hf) o[k][hf][0] = o[k][hf][1] = o[k][hf][2] = o[k][hf][3] = 0.f;
  // per row 8 hf + 2c + x: the shift (within 2^tau of the maximum, and as good as
  // that in a partial), and the lane's own sum
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int hf = 0; hf < NT; ++hf)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      m[hf][x] = -INFINITY;
      l[hf][x] = 0.f;
    }

  // matrix loads: lane l addresses row l % 8 of matrix l / 8, matrices in the
  // order (slab, tokens 0-7), (slab, tokens 8-15), then the next slab's
  const uint32_t lm = (((lane >> 4) * BS) + (lane & 7) + 8 * ((lane >> 3) & 1)) * 16;
  // scale bytes 4i .. 4i + 3 of a token are those of slabs 2i and 2i + 1, two
  // halves each: a lane's K dims are in half c / 2, its V dims in half r / 4
  const uint32_t ksel = int4_scale_sel(c >> 1, 2 + (c >> 1));  // of one token: slab 2i, slab 2i + 1
  const uint32_t vsel = int4_scale_sel(r >> 2, 4 + (r >> 2));  // of two tokens; slab 2i + 1: 0x2222 on
  constexpr int SUBS = T::SUBS, SBW = T::SB / 4;
  auto lds_words = [](uint32_t at, uint32_t (&w)[SBW]) {
    if constexpr (SBW == 2)
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    else
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
  };

  uint32_t slot = 0, parity = 0;
  for (int u = 0; u < mine; ++u) {
    if (!mbar_wait_bounded(&full[slot], parity, P.timeout_ns)) {
      if (lane == 0) record_error(P.error_word, kErrTimeout);
      for (int v = u + 1; v < issued; ++v) mbar_wait_bounded(&full[v % SW], (v / SW) & 1, P.timeout_ns);
      break;
    }
    const uint32_t at = ring_at + slot * T::SLOT;
    const int base = t0 + (warp + NW * u) * T::UNIT;  // the unit's first token
    const uint32_t missing = bad_slots >> (slot * TILES) & ((1u << TILES) - 1);
    const bool whole = missing == 0 && base + T::UNIT <= t1;
    if (!whole) {
      // Rows that were not copied, or may never have been written: their V
      // scales are zeroed, so that a weight of 0 times them is 0; their scores
      // become -inf below, whatever K holds.
      if (base + lane >= t1 || (missing >> (lane / BS)) & 1) {
        unsigned char* row = ring + slot * T::SLOT + (TILES + lane / BS) * T::TILE + T::SCALE_OFF + lane % BS * T::SB;
        *reinterpret_cast<uint32_t*>(row) = 0u;
        if (SBW == 2) *reinterpret_cast<uint32_t*>(row + 4) = 0u;
      }
      fence_proxy_async_smem();  // ordered before the next copy into this slot
      __syncwarp();
    }
#pragma unroll
    for (int step = 0; step < 2 / SUBS; ++step) {
      if (SUBS == 1 && base + 16 * step >= t1) break;
      // ---- S^T = K Q^T: st[.][hf][2 y + x] is token r + 8 y, row 8 hf + 2c + x
      float st[SUBS][NT][4];  // (the first product of each starts from zero)
#pragma unroll
      for (int sub = 0; sub < SUBS; ++sub) {
        const int row0 = 16 * (step * SUBS + sub) % BS;
        const uint32_t ks = at + 16 * (step * SUBS + sub) / BS * T::TILE;
        uint32_t w0[SBW], w1[SBW];  // scales of tokens r and 8 + r
        lds_words(ks + T::SCALE_OFF + (row0 + r) * T::SB, w0);
        lds_words(ks + T::SCALE_OFF + (row0 + 8 + r) * T::SB, w1);
#pragma unroll
        for (int i = 0; i < SLABS / 2; ++i) {
          uint32_t kb[4];
          ldsm_x4(ks + lm + (uint32_t)(2 * i * BS + row0) * 16, kb);
          const Int4Scale s0 = int4_scale(int4_scale_pair(w0[i], w0[i], ksel));
          const Int4Scale s1 = int4_scale(int4_scale_pair(w1[i], w1[i], ksel));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t d0[4], d1[4];
            int4_words(kb[2 * h], both_halves(s0, h), bases, d0);
            int4_words(kb[2 * h + 1], both_halves(s1, h), bases, d1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = 4 * i + 2 * h + e;
              if constexpr (NT < 4) {
#pragma unroll
                for (int hf = 0; hf < NT; ++hf)
                  mma_16816_from(st[sub][hf], k == 0, d0[2 * e], d1[2 * e], d0[2 * e + 1], d1[2 * e + 1], qb[k][hf][0],
                                 qb[k][hf][1]);
              } else {
#pragma unroll
                for (int pair = 0; pair < 2; ++pair) {
                  const uint4 w = qs[(k * 2 + pair) * 32 + lane];
                  mma_16816_from(st[sub][2 * pair], k == 0, d0[2 * e], d1[2 * e], d0[2 * e + 1], d1[2 * e + 1], w.x,
                                 w.y);
                  mma_16816_from(st[sub][2 * pair + 1], k == 0, d0[2 * e], d1[2 * e], d0[2 * e + 1], d1[2 * e + 1], w.z,
                                 w.w);
                }
              }
            }
          }
        }
      }
      // ---- online softmax
      if (!whole || base + T::UNIT > lim_min) {
#pragma unroll
        for (int sub = 0; sub < SUBS; ++sub) {
          const int first = 16 * (step * SUBS + sub);  // the subtile's first token in the unit
          const bool none = (missing >> (first / BS)) & 1;
#pragma unroll
          for (int hf = 0; hf < NT; ++hf)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int lt = none ? 0 : limit(8 * hf + 2 * c + x) - base - first;
              if (r >= lt) st[sub][hf][x] = -INFINITY;
              if (r + 8 >= lt) st[sub][hf][2 + x] = -INFINITY;
            }
        }
      }
      float lmax[NT][2];  // (scale_log2 > 0: the largest product is the largest score)
      bool need = false;
#pragma unroll
      for (int hf = 0; hf < NT; ++hf)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          lmax[hf][x] = fmaxf(st[0][hf][x], st[0][hf][2 + x]);
          if constexpr (SUBS == 2)
            lmax[hf][x] = fmaxf(lmax[hf][x], fmaxf(st[SUBS - 1][hf][x], st[SUBS - 1][hf][2 + x]));
          lmax[hf][x] *= P.scale_log2;
          need |= lmax[hf][x] > m[hf][x] + kLazyTau;
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int hf = 0; hf < NT; ++hf)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float mx = lmax[hf][x];
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
            const float mn = fmaxf(m[hf][x], mx);
            const float alpha = (mn == -INFINITY) ? 1.f : ex2_approx(m[hf][x] - mn);
            l[hf][x] *= alpha;
            m[hf][x] = mn;
#pragma unroll
            for (int k = 0; k < 2 * SLABS; ++k) {  // O^T's columns are the same rows
              o[k][hf][x] *= alpha;
              o[k][hf][2 + x] *= alpha;
            }
          }
      }
      uint32_t pb[NT][SUBS][2];
#pragma unroll
      for (int hf = 0; hf < NT; ++hf) {
        // (a row that has seen no token yet: shift 0)
        const float mu0 = m[hf][0] == -INFINITY ? 0.f : -m[hf][0], mu1 = m[hf][1] == -INFINITY ? 0.f : -m[hf][1];
#pragma unroll
        for (int sub = 0; sub < SUBS; ++sub) {
          const float p0 = ex2_approx(fmaf(st[sub][hf][0], P.scale_log2, mu0));
          const float p1 = ex2_approx(fmaf(st[sub][hf][1], P.scale_log2, mu1));
          const float p2 = ex2_approx(fmaf(st[sub][hf][2], P.scale_log2, mu0));
          const float p3 = ex2_approx(fmaf(st[sub][hf][3], P.scale_log2, mu1));
          l[hf][0] += p0 + p2;
          l[hf][1] += p1 + p3;
          pb[hf][sub][0] = transposed_8x8(pack_half2(p0, p1));
          pb[hf][sub][1] = transposed_8x8(pack_half2(p2, p3));
        }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int sub = 0; sub < SUBS; ++sub) {
        const int row0 = 16 * (step * SUBS + sub) % BS;
        const uint32_t vs = at + (TILES + 16 * (step * SUBS + sub) / BS) * T::TILE;
        uint32_t w[4][SBW];  // scales of tokens 2c, 2c + 1, 8 + 2c, 9 + 2c
#pragma unroll
        for (int k = 0; k < 4; ++k)
          lds_words(vs + T::SCALE_OFF + (row0 + 2 * c + (k >> 1) * 8 + (k & 1)) * T::SB, w[k]);
#pragma unroll
        for (int i = 0; i < SLABS / 2; ++i) {
          uint32_t vb[4];
          ldsm_x4_trans(vs + lm + (uint32_t)(2 * i * BS + row0) * 16, vb);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sel = vsel + 0x2222u * h;
            uint32_t dl[4], dh[4];
            int4_words(vb[2 * h], int4_scale(int4_scale_pair(w[0][i], w[1][i], sel)), bases, dl);
            int4_words(vb[2 * h + 1], int4_scale(int4_scale_pair(w[2][i], w[3][i], sel)), bases, dh);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t va[4] = {dl[2 * e], dl[2 * e + 1], dh[2 * e], dh[2 * e + 1]};
#pragma unroll
              for (int hf = 0; hf < NT; ++hf)
                mma_16816(o[2 * (2 * i + h) + e][hf], va, pb[hf][sub][0], pb[hf][sub][1]);
            }
          }
        }
      }
    }
    __syncwarp();
    bad_slots &= ~(((1u << TILES) - 1) << (slot * TILES));
    if (++slot == SW) {
      slot = 0;
      parity ^= 1;
    }
    if (issued < mine) {
      fence_proxy_async_smem();  // our reads of the slot precede the next copies into it
      issue(issued);
      ++issued;
    }
  }

  // ------------------------------------------------------------------ merge
  __syncthreads();
  float* mrg = reinterpret_cast<float*>(smem);
  float* mrg_m = mrg;
  float* mrg_l = mrg + NW * ROWS;
  float* mrg_acc = mrg + T::MRG_ACC_OFF;
#pragma unroll
  for (int hf = 0; hf < NT; ++hf) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float lv = l[hf][x];
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) lv += __shfl_xor_sync(0xffffffffu, lv, k);
      if (r == 0) {
        mrg_m[warp * ROWS + 8 * hf + 2 * c + x] = m[hf][x];
        mrg_l[warp * ROWS + 8 * hf + 2 * c + x] = lv;
      }
    }
    float* acc = mrg_acc + (warp * ROWS + 8 * hf + 2 * c) * T::PITCH + 4 * r;
#pragma unroll
    for (int k = 0; k < SLABS; ++k) {  // dims 32k + 4r ..
      const float(&lo)[4] = o[2 * k][hf];
      const float(&hi)[4] = o[2 * k + 1][hf];
      *reinterpret_cast<float4*>(acc + 32 * k) = make_float4(lo[0], lo[2], hi[0], hi[2]);
      *reinterpret_cast<float4*>(acc + T::PITCH + 32 * k) = make_float4(lo[1], lo[3], hi[1], hi[3]);
    }
  }
  __syncthreads();
  static_assert(NW == 4 && ROWS <= T::THREADS, "a factor a warp, a thread a row");
  float4* mrg_c = reinterpret_cast<float4*>(mrg + T::MRG_C_OFF);
  float* mrg_z = mrg + T::MRG_Z_OFF;
  int* mrg_row = reinterpret_cast<int*>(mrg_z + ROWS);
  if (threadIdx.x < rows) {
    const int rr = threadIdx.x;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, mrg_m[w * ROWS + rr]);
    float Z = 0.f, f[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = mrg_m[w * ROWS + rr];
      f[w] = (mw == -INFINITY) ? 0.f : ex2_approx(mw - M);
      Z = fmaf(f[w], mrg_l[w * ROWS + rr], Z);
    }
    const size_t row = out_row(rr);  // (rows of all sequences stay in 31 bits)
    mrg_c[rr] = make_float4(f[0], f[1], f[2], f[3]);
    mrg_z[rr] = Z;
    mrg_row[rr] = (int)row;
    if (!final_out) {
      P.max_logits[row * P.max_partitions + j] = M * 0.69314718055994530942f;
      P.exp_sums[row * P.max_partitions + j] = Z;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += T::THREADS) {
    const int rr = i / (D / 4), d = i % (D / 4) * 4;
    const float4 fc = mrg_c[rr];
    const float f[NW] = {fc.x, fc.y, fc.z, fc.w};
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float4 a = *reinterpret_cast<const float4*>(mrg_acc + (w * ROWS + rr) * T::PITCH + d);
      O.x = fmaf(f[w], a.x, O.x);
      O.y = fmaf(f[w], a.y, O.y);
      O.z = fmaf(f[w], a.z, O.z);
      O.w = fmaf(f[w], a.w, O.w);
    }
    O.x *= P.v_scale;
    O.y *= P.v_scale;
    O.z *= P.v_scale;
    O.w *= P.v_scale;
    const size_t row = mrg_row[rr];
    if (final_out) {
      const float Z = mrg_z[rr];
      const bool any = Z != 0.f;  // Z = 0: the query saw no token; a query that is not a number has a result that is none
      *reinterpret_cast<uint2*>(P.out + row * D + d) =
          make_uint2(any ? pack_half2(O.x / Z, O.y / Z) : 0u, any ? pack_half2(O.z / Z, O.w / Z) : 0u);
    } else {
      *reinterpret_cast<float4*>(P.tmp_out + (row * P.max_partitions + j) * D + d) = O;
    }
  }
}

// ---------------------------------------------------------------- rows back to fp16
struct Int4ReadParams {
  const uint8_t *k_cache, *v_cache;
  const int32_t *block_tables, *start_lens, *token_starts;
  __half *k_out, *v_out;
  long long k_stride, v_stride;
  int num_tokens, num_seqs, num_kv_heads, num_blocks, max_blocks_per_seq;
  float k_scale, v_scale;
  Int4Bases bases;
  int* error_word;
};

// A warp per token; a lane takes 8 dims at a time, a word of codes, and writes 16 bytes
// behind its neighbour's, eight words in flight (16 dims and 32 bytes a lane, so that
// every store met half of each sector: 35 us).  28842 tokens of 8
// heads: 26.6 us, 5.7 TB/s, mostly writing.
constexpr int kInt4ReadWarps = 8;
template <int D, int BS>
__global__ void __launch_bounds__(32 * kInt4ReadWarps) paged_kv_read_int4_kernel(const Int4ReadParams P) {
  constexpr int GROUPS = D / 16, TILE = int4_tile_bytes(D, BS);
  const int lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * kInt4ReadWarps + (threadIdx.x >> 5);
  if (t >= P.num_tokens) return;
  int b, j;
  if (P.token_starts) {
    b = find_segment(P.token_starts, P.num_seqs, (int)t);
    if (b >= P.num_seqs) return;
    j = (int)t - P.token_starts[b];
    if (j < 0) return;
  } else {
    const int per = P.num_tokens / P.num_seqs;
    b = (int)t / per;
    j = (int)t - b * per;
  }
  const int L = P.start_lens[b];
  const long long at = (long long)L + j, lb = at / BS;
  int block = -1;
  if (L >= 0 && lb < P.max_blocks_per_seq) block = P.block_tables[(size_t)b * P.max_blocks_per_seq + lb];
  if (block < 0 || block >= P.num_blocks) {
    if (lane == 0) record_error(P.error_word, kErrBadBlock);
    return;
  }
  const int row = (int)(at - lb * BS);
  const size_t tile0 = (size_t)block * P.num_kv_heads * TILE;
  constexpr int U = 8;  // words in flight a lane
  constexpr int WORDS = D / 8;
  const int items = 2 * P.num_kv_heads * WORDS;
  for (int i0 = lane; i0 < items; i0 += 32 * U) {
    uint32_t x[U], sb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 32 * u;
      if (i >= items) break;
      const int word = i % WORDS, hv = i / WORDS;
      const bool is_v = hv >= P.num_kv_heads;
      const uint8_t* tile = (is_v ? P.v_cache : P.k_cache) + tile0 + (size_t)(hv - (is_v ? P.num_kv_heads : 0)) * TILE;
      x[u] = *reinterpret_cast<const uint32_t*>(tile + ((word / 4) * BS + row) * 16 + (word % 4) * 4);
      sb[u] = tile[BS * D / 2 + row * GROUPS + word / 2];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 32 * u;
      if (i >= items) break;
      const int word = i % WORDS, hv = i / WORDS;
      const bool is_v = hv >= P.num_kv_heads;
      const float step = __half2float(__ushort_as_half((unsigned short)((sb[u] & 0x7Fu) << 7))) * kInt4Unscale *
                         (is_v ? P.v_scale : P.k_scale);
      // u - 8 of dims j and j + 4, exact in fp16; their values in fp32, rounded once
      const uint32_t y = x[u] >> 8;
      const uint32_t c[4] = {hadd2_u(masked_or<0x000F000Fu>(x[u], P.bases.b1024), kHalf1032),
                             hadd2_u(masked_or<0x00F000F0u>(x[u], P.bases.b64), kHalf72),
                             hadd2_u(masked_or<0x000F000Fu>(y, P.bases.b1024), kHalf1032),
                             hadd2_u(masked_or<0x00F000F0u>(y, P.bases.b64), kHalf72)};
      float2 f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = __half22float2(*reinterpret_cast<const __half2*>(&c[k]));
      __half* dst = (is_v ? P.v_out + t * P.v_stride : P.k_out + t * P.k_stride) +
                    (size_t)(hv - (is_v ? P.num_kv_heads : 0)) * D + 8 * word;
      *reinterpret_cast<uint4*>(dst) =
          make_uint4(pack_half2(f[0].x * step, f[1].x * step), pack_half2(f[2].x * step, f[3].x * step),
                     pack_half2(f[0].y * step, f[1].y * step), pack_half2(f[2].y * step, f[3].y * step));
    }
  }
}

}  // namespace pkd
