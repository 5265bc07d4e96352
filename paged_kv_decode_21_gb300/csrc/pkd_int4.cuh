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
// scale for K and into the result for V.  No byte gives an infinity or a NaN, so
// rows that were never written cannot poison a product with a weight of 0.
constexpr float kInt4Unscale = 256.f;

__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
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

// Codes j and j + 4 of a word (j = 0..3) as the halves of d[j], times the
// scales in the halves of s.
__device__ __forceinline__ void int4_words(uint32_t x, uint32_t s, uint32_t (&d)[4]) {
  const uint32_t y = x >> 8;
  const uint32_t a1 = hmul2_u(s, kHalf1032), a2 = hmul2_u(s, kHalf72);
  d[0] = hfma2_u((x & 0x000F000Fu) | 0x64006400u, s, a1);
  d[1] = hfma2_u((x & 0x00F000F0u) | 0x54005400u, s, a2);
  d[2] = hfma2_u((y & 0x000F000Fu) | 0x64006400u, s, a1);
  d[3] = hfma2_u((y & 0x00F000F0u) | 0x54005400u, s, a2);
}

// Scale bytes 0 and 2 (LO), or 1 and 3, of x as an fp16 pair of s * 2^-8.
template <bool LO>
__device__ __forceinline__ uint32_t int4_scale_pair(uint32_t x) {
  return LO ? (x & 0x007F007Fu) << 7 : (x & 0x7F007F00u) >> 1;
}

// ---------------------------------------------------------------- decode
// The split of the work, the online softmax, the merge of the warps and the
// meaning of rows are those of paged_decode_mma_kernel; here a warp's ring
// holds whole (block, kv head) tiles, brought by two plain bulk copies.
//
// Fragments (c = lane % 4, r = lane / 4), for a slab of 32 dims:
//   K  an ldmatrix of 8 tokens x 16 bytes gives lane (r, c) the codes of dims 8c
//      .. 8c + 7 of token r: two k-steps' B operands, dims (8c + j, 8c + j + 4)
//      in the halves.  Q's A fragments follow that order of dims.
//   V  the transposed ldmatrix gives lane (r, c) dims 4r .. 4r + 3 of tokens 2c
//      and 2c + 1, one token a half: rows r and r + 8 of two m-tiles of V^T.
// Q rows are the group's heads times up to `q_chunk` query tokens; NT = 1 where
// they fit 8 rows, else 2.
struct Int4Params {
  DecodeParams d;
  int group, q_chunk;
};

template <int D, int BS, int NT>
struct Int4Traits {
  static constexpr int NW = 4;
  static constexpr int THREADS = NW * 32;
  static constexpr int MIN_BLOCKS = 3;
  static constexpr int TILE = int4_tile_bytes(D, BS);
  static constexpr int SLOT = 2 * TILE;  // K, then V
  static constexpr int SLABS = D / 32;
  static constexpr int SCALE_OFF = BS * D / 2;
  static constexpr int SB = D / 16;  // scale bytes a token
  static constexpr int SW_RAW = 72 * 1024 / (NW * SLOT);
  static constexpr int SW = SW_RAW > 8 ? 8 : SW_RAW;
  static constexpr int RING_BYTES = NW * SW * SLOT;
  static constexpr int ROWS = 8 * NT;
  static constexpr int MRG_ACC_OFF = 3 * NW * 16;
  static constexpr int MERGE_BYTES = (MRG_ACC_OFF + NW * ROWS * D) * 4;
  static constexpr int MAIN_BYTES = RING_BYTES > MERGE_BYTES ? RING_BYTES : MERGE_BYTES;
  static constexpr int SMEM_BYTES = MAIN_BYTES + NW * SW * 8;
  static_assert(SW >= 2 && TILE % 16 == 0 && MAIN_BYTES % 16 == 0, "ring");
};

template <int D, int BS, int NT>
__global__ void __launch_bounds__(Int4Traits<D, BS, NT>::THREADS, Int4Traits<D, BS, NT>::MIN_BLOCKS)
    paged_decode_int4_kernel(const __grid_constant__ Int4Params IP) {
  using T = Int4Traits<D, BS, NT>;
  constexpr int NW = T::NW, SW = T::SW, SLABS = T::SLABS, ROWS = T::ROWS;
  const DecodeParams& P = IP.d;
  extern __shared__ __align__(128) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::MAIN_BYTES);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int np_grid = P.max_partitions, G = IP.group, QC = IP.q_chunk;
  const int qc = blockIdx.x % P.q_chunks;
  const int rest = blockIdx.x / P.q_chunks;
  const int j = rest % np_grid, bg = rest / np_grid;
  const int g = bg % P.num_kv_heads, b = bg / P.num_kv_heads;
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
  const int nblk = t1 > t0 ? (t1 - t0 + BS - 1) / BS : 0;
  const int32_t* bt = P.block_tables + (size_t)b * P.max_blocks_per_seq + t0 / BS;
  const size_t block_stride = (size_t)P.num_kv_heads * T::TILE;
  const char* kbase = reinterpret_cast<const char*>(P.k_cache) + (size_t)g * T::TILE;
  const char* vbase = reinterpret_cast<const char*>(P.v_cache) + (size_t)g * T::TILE;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int r = lane / 4, c = lane % 4;
  int lim[NT];  // tokens at or past it are masked for the lane's rows r + 8 hf
#pragma unroll
  for (int hf = 0; hf < NT; ++hf) {
    const int rr = r + 8 * hf;
    lim[hf] = rr < rows ? min(t1, L - QL + jq0 + rr / G + 1) : t1;
  }
  const int lim_min = NT == 2 ? min(lim[0], lim[NT - 1]) : lim[0];

  // Q as A fragments: k-step 2s + e of slab s has slots (2c, 2c + 1) = dims 8c
  // + 2e and 8c + 2e + 4 of the slab, slots (8 + 2c, 9 + 2c) = the dims behind
  uint32_t qa[2 * SLABS][2 * NT];
#pragma unroll
  for (int hf = 0; hf < NT; ++hf) {
    const int rr = r + 8 * hf;
    const __half* qr = P.q + (rr < rows ? out_row(rr) * D : 0);
#pragma unroll
    for (int s = 0; s < SLABS; ++s) {
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      if (rr < rows) u = *reinterpret_cast<const uint4*>(qr + 32 * s + 8 * c);
      qa[2 * s][hf] = prmt(u.x, u.z, 0x5410);
      qa[2 * s][NT + hf] = prmt(u.x, u.z, 0x7632);
      qa[2 * s + 1][hf] = prmt(u.y, u.w, 0x5410);
      qa[2 * s + 1][NT + hf] = prmt(u.y, u.w, 0x7632);
    }
  }
  // O^T: tile 2s + e holds dims 32s + 4r + 2e (rows r) and the dims behind (rows r + 8)
  float o[2 * SLABS][NT][4];
#pragma unroll
  for (int k = 0; k < 2 * SLABS; ++k)
#pragma unroll
    for (int hf = 0; hf < NT; ++hf) o[k][hf][0] = o[k][hf][1] = o[k][hf][2] = o[k][hf][3] = 0.f;
  float m[NT], mt[NT], l[NT];
#pragma unroll
  for (int hf = 0; hf < NT; ++hf) {
    m[hf] = mt[hf] = -INFINITY;
    l[hf] = 0.f;
  }

  uint64_t* full = bars + warp * SW;
  unsigned char* ring = smem + (size_t)warp * SW * T::SLOT;
  if (lane == 0) {
    for (int s = 0; s < SW; ++s) mbar_init(&full[s], 1);
    fence_mbarrier_init();
  }
  __syncwarp();
  const int mine = nblk > warp ? (nblk - warp + NW - 1) / NW : 0;  // the warp's blocks: warp, warp + NW, ...
  // block ids, 32 of the warp's at a time, the next 32 requested ahead
  auto ids_at = [&](int first) { return first + lane < mine ? bt[warp + NW * (first + lane)] : -1; };
  int ids = ids_at(0), ids_next = ids_at(32);
  uint32_t bad_slots = 0;
  auto issue = [&](int n) {  // copies of the warp's n-th block, n ascending
    if (n > 0 && n % 32 == 0) {
      ids = ids_next;
      ids_next = ids_at(n + 32);
    }
    const int slot = n % SW;
    const int pb = __shfl_sync(0xffffffffu, ids, n % 32);
    const bool bad = pb < 0 || pb >= P.num_blocks;
    bad_slots = bad ? (bad_slots | (1u << slot)) : (bad_slots & ~(1u << slot));
    if (lane == 0) {
      if (bad) {
        record_error(P.error_word, kErrBadBlock);
        mbar_arrive(&full[slot]);
      } else {
        unsigned char* dst = ring + (size_t)slot * T::SLOT;
        mbar_arrive_expect_tx(&full[slot], T::SLOT);
        bulk_copy_g2s(dst, kbase + (size_t)pb * block_stride, T::TILE, &full[slot]);
        bulk_copy_g2s(dst + T::TILE, vbase + (size_t)pb * block_stride, T::TILE, &full[slot]);
      }
    }
  };
  int issued = 0;
  for (; issued < SW && issued < mine; ++issued) issue(issued);

  // matrix loads: lane l addresses row l % 8 of matrix l / 8, matrices in the
  // order (slab, tokens 0-7), (slab, tokens 8-15), then the next slab's
  const uint32_t lm = (((lane >> 4) * BS) + (lane & 7) + 8 * ((lane >> 3) & 1)) * 16;
  const int kh = c >> 1;  // K: the lane's dims are in this half of the slab's two groups
  const int vh = r >> 2;  // V: the same
  const uint32_t ksel = (uint32_t)(kh | ((kh + 2) << 4)) * 0x101u + 0x4400u;  // bytes (a.h, a.h+2, b.h, b.h+2)
  const uint32_t vsel = (uint32_t)(vh | ((vh + 2) << 4)) * 0x101u + 0x4400u;

  for (int u = 0; u < mine; ++u) {
    const int slot = u % SW;
    const bool bad = (bad_slots >> slot) & 1u;
    if (!mbar_wait_bounded(&full[slot], (u / SW) & 1, P.timeout_ns)) {
      if (lane == 0) record_error(P.error_word, kErrTimeout);
      for (int v = u + 1; v < issued; ++v) mbar_wait_bounded(&full[v % SW], (v / SW) & 1, P.timeout_ns);
      break;
    }
    if (!bad) {
      const uint32_t ks = smem_u32(ring + (size_t)slot * T::SLOT);
      const uint32_t vs = ks + T::TILE;
      const int base0 = t0 + (warp + NW * u) * BS;
#pragma unroll
      for (int rg = 0; rg < BS / 16; ++rg) {
        const int base = base0 + 16 * rg;
        if (BS > 16 && base >= t1) break;
        // ---- S = Q K^T over tokens 0..7 (sa) and 8..15 (sb)
        float sa[2][4], sb[2][4];
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
          for (int e = 0; e < 4; ++e) sa[ch][e] = sb[ch][e] = 0.f;
        auto qk = [&](int k, uint32_t b00, uint32_t b01, uint32_t b10, uint32_t b11) {
          if constexpr (NT == 1) {
            mma_16816_top(sa[k % 2], qa[k][0], qa[k][1], b00, b01);
            mma_16816_top(sb[k % 2], qa[k][0], qa[k][1], b10, b11);
          } else {
            mma_16816(sa[k % 2], qa[k], b00, b01);
            mma_16816(sb[k % 2], qa[k], b10, b11);
          }
        };
        const uint32_t ksc = ks + T::SCALE_OFF + (16 * rg + r) * T::SB;
#pragma unroll
        for (int i = 0; i < SLABS / 2; ++i) {
          uint32_t kb[4];
          ldsm_x4(ks + lm + (uint32_t)(2 * i * BS + 16 * rg) * 16, kb);
          // scales of tokens r and 8 + r, slabs 2i and 2i + 1: bytes (slab 2i, slab 2i + 1) of each
          uint32_t w0, w1;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w0) : "r"(ksc + 4 * i));
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w1) : "r"(ksc + 8 * T::SB + 4 * i));
          const uint32_t w = prmt(w0, w1, ksel);
          const uint32_t se = int4_scale_pair<true>(w), so = int4_scale_pair<false>(w);  // slab 2i, slab 2i + 1
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sc = h ? so : se;
            uint32_t d0[4], d1[4];
            int4_words(kb[2 * h], prmt(sc, sc, 0x1010), d0);
            int4_words(kb[2 * h + 1], prmt(sc, sc, 0x3232), d1);
            qk(4 * i + 2 * h, d0[0], d0[1], d1[0], d1[1]);
            qk(4 * i + 2 * h + 1, d0[2], d0[3], d1[2], d1[3]);
          }
        }
        // ---- online softmax of rows r + 8hf over tokens 2c, 2c+1, 8+2c, 9+2c
        float sc[NT][4];
#pragma unroll
        for (int hf = 0; hf < NT; ++hf) {
          sc[hf][0] = (sa[0][2 * hf] + sa[1][2 * hf]) * P.scale_log2;
          sc[hf][1] = (sa[0][2 * hf + 1] + sa[1][2 * hf + 1]) * P.scale_log2;
          sc[hf][2] = (sb[0][2 * hf] + sb[1][2 * hf]) * P.scale_log2;
          sc[hf][3] = (sb[0][2 * hf + 1] + sb[1][2 * hf + 1]) * P.scale_log2;
        }
        if (base + 16 > lim_min) {
#pragma unroll
          for (int hf = 0; hf < NT; ++hf) {
            const int lt = lim[hf] - base;
            if (2 * c >= lt) sc[hf][0] = -INFINITY;
            if (2 * c + 1 >= lt) sc[hf][1] = -INFINITY;
            if (8 + 2 * c >= lt) sc[hf][2] = -INFINITY;
            if (9 + 2 * c >= lt) sc[hf][3] = -INFINITY;
          }
        }
        float lmax[NT];
        bool need = false;
#pragma unroll
        for (int hf = 0; hf < NT; ++hf) {
          lmax[hf] = fmaxf(fmaxf(sc[hf][0], sc[hf][1]), fmaxf(sc[hf][2], sc[hf][3]));
          mt[hf] = fmaxf(mt[hf], lmax[hf]);
          need |= lmax[hf] > m[hf] + kLazyTau;
        }
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
          for (int hf = 0; hf < NT; ++hf) {
            float mx = fmaxf(lmax[hf], __shfl_xor_sync(0xffffffffu, lmax[hf], 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[hf], mx);
            const float alpha = (mn == -INFINITY) ? 1.f : ex2_approx(m[hf] - mn);
            l[hf] *= alpha;
            m[hf] = mn;
            const float a_lo = __shfl_sync(0xffffffffu, alpha, 8 * c);
            const float a_hi = __shfl_sync(0xffffffffu, alpha, 8 * c + 4);
#pragma unroll
            for (int k = 0; k < 2 * SLABS; ++k) {
              o[k][hf][0] *= a_lo;
              o[k][hf][1] *= a_hi;
              o[k][hf][2] *= a_lo;
              o[k][hf][3] *= a_hi;
            }
          }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int hf = 0; hf < NT; ++hf) {
          const float mu = m[hf] == -INFINITY ? 0.f : m[hf];  // a row that has seen no token yet
          const float p0 = ex2_approx(sc[hf][0] - mu), p1 = ex2_approx(sc[hf][1] - mu);
          const float p2 = ex2_approx(sc[hf][2] - mu), p3 = ex2_approx(sc[hf][3] - mu);
          l[hf] += (p0 + p1) + (p2 + p3);
          pb[hf][0] = pack_half2(p0, p1);
          pb[hf][1] = pack_half2(p2, p3);
        }
        // ---- O^T += V^T P^T
        const uint32_t vsc = vs + T::SCALE_OFF + (16 * rg + 2 * c) * T::SB;
#pragma unroll
        for (int i = 0; i < SLABS / 2; ++i) {
          uint32_t vb[4];
          ldsm_x4_trans(vs + lm + (uint32_t)(2 * i * BS + 16 * rg) * 16, vb);
          // scales of token pairs (2c, 2c + 1) and (8 + 2c, 9 + 2c)
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            asm volatile("ld.shared.b32 %0, [%1];"
                         : "=r"(w[k])
                         : "r"(vsc + ((k >> 1) * 8 + (k & 1)) * T::SB + 4 * i));
          const uint32_t wl = prmt(w[0], w[1], vsel), wh = prmt(w[2], w[3], vsel);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t dl[4], dh[4];
            int4_words(vb[2 * h], h ? int4_scale_pair<false>(wl) : int4_scale_pair<true>(wl), dl);
            int4_words(vb[2 * h + 1], h ? int4_scale_pair<false>(wh) : int4_scale_pair<true>(wh), dh);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t va[4] = {dl[2 * e], dl[2 * e + 1], dh[2 * e], dh[2 * e + 1]};
#pragma unroll
              for (int hf = 0; hf < NT; ++hf) mma_16816(o[2 * (2 * i + h) + e][hf], va, pb[hf][0], pb[hf][1]);
            }
          }
        }
      }
    }
    __syncwarp();
    if (issued < mine) {
      if (lane == 0) fence_proxy_async_smem();  // our reads of the slot precede the next copy into it
      issue(issued);
      ++issued;
    }
  }

  // ------------------------------------------------------------------ merge
  __syncthreads();
  float* mrg = reinterpret_cast<float*>(smem);
  float* mrg_m = mrg;
  float* mrg_mt = mrg + NW * 16;
  float* mrg_l = mrg + 2 * NW * 16;
  float* mrg_acc = mrg + T::MRG_ACC_OFF;
#pragma unroll
  for (int hf = 0; hf < NT; ++hf) {
    float lv = l[hf] + __shfl_xor_sync(0xffffffffu, l[hf], 1);
    lv += __shfl_xor_sync(0xffffffffu, lv, 2);
    float mx = fmaxf(mt[hf], __shfl_xor_sync(0xffffffffu, mt[hf], 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (c == 0) {
      mrg_m[warp * 16 + 8 * hf + r] = m[hf];
      mrg_mt[warp * 16 + 8 * hf + r] = mx;
      mrg_l[warp * 16 + 8 * hf + r] = lv;
    }
    float* acc = mrg_acc + (warp * ROWS + 8 * hf + 2 * c) * D;
#pragma unroll
    for (int k = 0; k < 2 * SLABS; ++k) {
      const int d = 32 * (k / 2) + 4 * r + 2 * (k % 2);
      *reinterpret_cast<float2*>(acc + d) = make_float2(o[k][hf][0], o[k][hf][2]);
      *reinterpret_cast<float2*>(acc + D + d) = make_float2(o[k][hf][1], o[k][hf][3]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * D; i += T::THREADS) {
    const int rr = i / D, d = i % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, mrg_mt[w * 16 + rr]);
    float Z = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = mrg_m[w * 16 + rr];
      const float cw = (mw == -INFINITY) ? 0.f : ex2_approx(mw - M);
      Z = fmaf(cw, mrg_l[w * 16 + rr], Z);
      O = fmaf(cw, mrg_acc[(w * ROWS + rr) * D + d], O);
    }
    O *= P.v_scale;
    const size_t row = out_row(rr);
    if (final_out) {
      P.out[row * D + d] = __float2half_rn(Z > 0.f ? O / Z : 0.f);
    } else {
      const size_t pidx = row * P.max_partitions + j;
      P.tmp_out[pidx * D + d] = O;
      if (d == 0) {
        P.max_logits[pidx] = M * 0.69314718055994530942f;
        P.exp_sums[pidx] = Z;
      }
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
  int* error_word;
};

// A warp per token; a lane takes the 16 dims of a group, 8 bytes of codes and
// one of scale, and writes 32 bytes.
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
  for (int i = lane; i < 2 * P.num_kv_heads * GROUPS; i += 32) {
    const int d16 = i % GROUPS, hv = i / GROUPS;
    const bool is_v = hv >= P.num_kv_heads;
    const int g = is_v ? hv - P.num_kv_heads : hv;
    const uint8_t* tile = (is_v ? P.v_cache : P.k_cache) + tile0 + (size_t)g * TILE;
    const uint2 x = *reinterpret_cast<const uint2*>(tile + ((d16 / 2) * BS + row) * 16 + (d16 % 2) * 8);
    const uint32_t sb = tile[BS * D / 2 + row * GROUPS + d16] & 0x7Fu;
    const float step = __half2float(__ushort_as_half((unsigned short)(sb << 7))) * kInt4Unscale *
                       (is_v ? P.v_scale : P.k_scale);
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t by = ((k < 4 ? x.x : x.y) >> (8 * (k % 4))) & 0xFFu;
      w[k] = pack_half2((float)((int)(by & 15u) - 8) * step, (float)((int)(by >> 4) - 8) * step);
    }
    uint4* dst = reinterpret_cast<uint4*>((is_v ? P.v_out + t * P.v_stride : P.k_out + t * P.k_stride) +
                                          (size_t)g * D + 16 * d16);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

}  // namespace pkd
