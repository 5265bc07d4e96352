// pkd_evict.cuh -- what keeps a cache from growing: the softmax weights that
// queries give to cached tokens, the choice of the tokens to keep by them, and
// the copy of the kept rows into blocks of their own.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>
#include "pkd_decode_mma.cuh"
#include "pkd_int4.cuh"

namespace pkd {

// What a cache holds (the values of pkd_kv_type).
enum KvType : int { kKvFp16 = 0, kKvE4m3 = 1, kKvInt4 = 2 };

// ---------------------------------------------------------------------------
// Attention weights.  w_t = sum over rows (query token, head) of
// exp(s_rt - M_r) / Z_r needs every row's maximum and sum before the first
// weight, so two grids: the first reads K, and leaves each row's maximum and
// sum over every partition of the tokens; the second merges those to
// log2(Z_r) + M_r, which is all a weight needs, 2^(s - that), and adds up the
// weights.  Where rows are few, the first also leaves the scores, 4 bytes a row
// and token, and the second reads those; where they are many it reads K again
// and multiplies again, since a score written and read takes 8 bytes and a key
// 2D and less.
//
// S = Q K^T by mma.m16n8k16: 16 rows times 8 tokens.  Lane (r, c) holds the dims
// of token r that come as its 16-byte loads, as B fragments, and Q's A fragments
// (registers for up to 16 rows, shared memory for more) follow that order of
// dims (below).  Few rows: bound by K's read, so K comes by bulk copies of whole
// (block, kv head) tiles into a ring of every warp's own, 32 tokens a slot.  Many
// rows: bound by the products, so keys go from global memory straight into the
// fragments, 16 tokens a warp and step over fp16 caches, 32 over the others, the
// next step's requested before this one's products.
//
// One query row of 4 (64 x 32/8 heads, 512-4096 tokens, fp16): 54 us for the
// first grid, 5.7 TB/s, and 13 for the second, latencies of its merge and scores
// (HBM at 22%).  112 rows (8 x 16 tokens x 28/4, 4000-16384 tokens, E4M3): 48 and
// 47 us, 89 one behind the other, the products at 43% of mma.sync's peak, 70%
// while an SM has three CTAs; Q's fragments are 3 of a CTA's 35 us (7 when every
// thread wrote words where they went).  For that case:
// two columns of keys a step, 4 to 6 CTAs an SM, or chunks of 2 or 4 row tiles: 109
// to 401 against 97 us for both; tcgen05 products with the scores in tensor memory,
// one softmax thread a row: 91 to 110 (fp16 142 against 104), better only from
// 128 rows and many sequences on.
struct WeightsParams {
  const __half* q;
  const void* k_cache;
  const int32_t *block_tables, *context_lens, *start_lens;
  float* weights;
  float *row_max, *row_sum;  // [B * Hkv][np][R], log2 units
  float* scores;             // [B * Hkv][R][score_stride], log2 units, or null
  long long score_stride;
  int num_seqs, q_len, num_q_heads, num_kv_heads, block_size, num_blocks, max_blocks_per_seq;
  int rows;       // R = q_len * group
  int part, np;   // tokens per partition (a multiple of 128), partitions
  int row_chunks; // first grid: chunks of 16 RT rows
  int q_tiles;    // second grid, keys again: row tiles of Q in shared memory at a time
  float scale_log2, decay;  // scale_log2 > 0
  uint32_t q_sign;          // flips Q where the scale is negative
  int* error_word;
  Int4Bases bases;
};

constexpr int kWeightsWarps = 4;
constexpr int kWeightsFinishThreads = 256;
constexpr int kManyRowsCtas = 3;  // an SM

// 8-token columns of a warp's step.
constexpr __host__ __device__ int key_tiles(int KV) { return KV == kKvFp16 ? 2 : 4; }

// The order of dims: k-step s has in slot pair h (0: slots 2c, 2c + 1; 1: slots
// 8 + 2c, 9 + 2c), half e, of lane c the dim
//   fp16   32 (s / 2) + 8c + 4 (s % 2) + 2h + e
//   E4M3   64 (s / 4) + 16c + 4 (s % 4) + 2h + e
//   4 bits (D / 4) c + 8 (s / 2) + 2 (s % 2) + h + 4e     (words of eight codes, halves four dims apart)

// Raw keys of 8 tokens, one of them (and a quarter of its dims) a lane's.
template <int KV, int D>
struct KeyRow {
  static constexpr int N = KV == kKvFp16 ? D / 32 : (KV == kKvE4m3 ? D / 64 : 1);
  uint4 u[N];
  uint32_t s;  // kKvInt4: the lane's scale bytes

  // Row `row` of the tile of block pb and head g, with the tile's index in the cache.
  __device__ __forceinline__ void load(const void* cache, size_t tile, int BS, int row, int c) {
    if constexpr (KV == kKvInt4) {
      const uint8_t* t = static_cast<const uint8_t*>(cache) + tile * ((size_t)BS * D * 9 / 16);
      if constexpr (D == 128) {
        u[0] = *reinterpret_cast<const uint4*>(t + (c * BS + row) * 16);
        s = *reinterpret_cast<const unsigned short*>(t + BS * (D / 2) + row * (D / 16) + 2 * c);
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(t + ((c / 2) * BS + row) * 16 + 8 * (c % 2));
        u[0] = make_uint4(x.x, x.y, 0u, 0u);
        s = t[BS * (D / 2) + row * (D / 16) + c];
      }
    } else {
      constexpr int E = KV == kKvFp16 ? 2 : 1;
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(cache) +
                                                      (tile * BS + row) * ((size_t)D * E)) + c;
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] = p[4 * i];
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = make_uint4(0u, 0u, 0u, 0u);
    s = 0;
  }

  // B fragments of all k-steps: b[2 s], b[2 s + 1].
  __device__ __forceinline__ void fragments(uint32_t (&b)[D / 8], const Int4Bases& bases) const {
    if constexpr (KV == kKvFp16) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        b[4 * i] = u[i].x;
        b[4 * i + 1] = u[i].y;
        b[4 * i + 2] = u[i].z;
        b[4 * i + 3] = u[i].w;
      }
    } else if constexpr (KV == kKvE4m3) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        e4m3x4_to_f16x2x2(u[i].x, b[8 * i], b[8 * i + 1]);
        e4m3x4_to_f16x2x2(u[i].y, b[8 * i + 2], b[8 * i + 3]);
        e4m3x4_to_f16x2x2(u[i].z, b[8 * i + 4], b[8 * i + 5]);
        e4m3x4_to_f16x2x2(u[i].w, b[8 * i + 6], b[8 * i + 7]);
      }
    } else {
      const uint32_t lo = (s & 0x7Fu) * 0x00800080u;  // the first group's scale twice, as fp16
      const uint32_t hi = D == 128 ? ((s >> 8) & 0x7Fu) * 0x00800080u : lo;
      const Int4Scale first = int4_scale(lo), second = int4_scale(hi);
      const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t d[4];
        int4_words(w[i], i < 2 ? first : second, bases, d);
#pragma unroll
        for (int k = 0; k < 4; ++k) b[4 * i + k] = d[k];
      }
    }
  }
};

// Row `row` of Q for (b, g): query token row / G, head row % G of the group.
template <int D>
__device__ __forceinline__ const __half* query_row(const WeightsParams& P, int b, int g, int row) {
  const int G = P.rows / P.q_len;
  return P.q + (((size_t)b * P.q_len + row / G) * P.num_q_heads + (size_t)g * G + row % G) * D;
}
// Eight dims of Q, 8 ch on, as the halves that two neighbouring k-steps take:
// w[2 p + h] is slot pair h of step s + p for lane c (the order above, the other way round).
struct QueryWords {
  int s, c;
  uint32_t w[4];
};
template <int KV, int D>
__device__ __forceinline__ QueryWords query_words(const uint4 u, int ch, uint32_t sign) {
  QueryWords q;
  if constexpr (KV == kKvInt4) {
    q.c = ch / (D / 32);
    q.s = 2 * (ch % (D / 32));
    q.w[0] = prmt(u.x, u.z, 0x5410);
    q.w[1] = prmt(u.x, u.z, 0x7632);
    q.w[2] = prmt(u.y, u.w, 0x5410);
    q.w[3] = prmt(u.y, u.w, 0x7632);
  } else {
    q.c = KV == kKvFp16 ? ch % 4 : ch / 2 % 4;
    q.s = KV == kKvFp16 ? 2 * (ch / 4) : 4 * (ch / 8) + 2 * (ch % 2);
    q.w[0] = u.x;
    q.w[1] = u.y;
    q.w[2] = u.z;
    q.w[3] = u.w;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) q.w[k] ^= sign;
  return q;
}
// The i-th of the D / 32 such eights that lane c takes.
template <int KV, int D>
__device__ __forceinline__ int query_eight(int i, int c) {
  return KV == kKvFp16 ? 4 * i + c : (KV == kKvE4m3 ? 8 * (i / 2) + 2 * c + i % 2 : (D / 32) * c + i);
}

// Q's rows 16 rt .. of tiles [first, first + n) as A fragments in shared memory: [tile][k-step][lane] uint4.
// A warp a tile, a lane its own fragments, two tiles in flight.
template <int KV, int D>
__device__ __forceinline__ void load_query_tiles(const WeightsParams& P, uint4* qs, int b, int g, int first, int n) {
  constexpr int U = 2, EIGHTS = D / 32, KS = D / 16;
  const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
  for (int k0 = threadIdx.x / 32; k0 < n; k0 += U * kWeightsWarps) {
    uint4 u[U][2][EIGHTS];
#pragma unroll
    for (int x = 0; x < U; ++x)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int k = k0 + x * kWeightsWarps, row = (first + k) * 16 + r + 8 * hf;
        const __half* q = k < n && row < P.rows ? query_row<D>(P, b, g, row) : nullptr;
#pragma unroll
        for (int i = 0; i < EIGHTS; ++i)
          u[x][hf][i] = q ? *reinterpret_cast<const uint4*>(q + 8 * query_eight<KV, D>(i, c)) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const int k = k0 + x * kWeightsWarps;
      if (k >= n) break;
#pragma unroll
      for (int i = 0; i < EIGHTS; ++i) {
        const int ch = query_eight<KV, D>(i, c);
        const QueryWords lo = query_words<KV, D>(u[x][0][i], ch, P.q_sign);
        const QueryWords hi = query_words<KV, D>(u[x][1][i], ch, P.q_sign);
        qs[(k * KS + lo.s) * 32 + lane] = make_uint4(lo.w[0], hi.w[0], lo.w[1], hi.w[1]);
        qs[(k * KS + lo.s + 1) * 32 + lane] = make_uint4(lo.w[2], hi.w[2], lo.w[3], hi.w[3]);
      }
    }
  }
}

// A warp's steps over tokens [t0, t1): step n has tokens t0 + STEP (warp + NW n) ..; keys a step ahead, block ids
// further.
template <int KV, int D>
struct KeyStream {
  static constexpr int TILES = key_tiles(KV), STEP = 8 * TILES, HALVES = STEP / 16;
  static constexpr int IDS = 32 / HALVES;  // steps whose block ids the lanes hold
  KeyRow<KV, D> next[TILES];
  int ids;                   // lane: half lane % HALVES of step lane / HALVES of this run of IDS
  int block[HALVES];         // of the next step's halves; negative where there is none
  int t0, t1, warp;

  __device__ __forceinline__ int token(int n) const { return t0 + STEP * (warp + kWeightsWarps * n); }
  __device__ __forceinline__ void fetch_ids(const WeightsParams& P, int b, int n) {
    const int lane = threadIdx.x & 31, t = token(n + lane / HALVES) + 16 * (lane % HALVES);
    ids = t < t1 ? P.block_tables[(size_t)b * P.max_blocks_per_seq + t / P.block_size] : -1;
    if (t < t1 && (ids < 0 || ids >= P.num_blocks)) {
      record_error(P.error_word, kErrBadBlock);
      ids = -1;
    }
  }
  __device__ __forceinline__ void start(const WeightsParams& P, int b, int g, int first, int end) {
    t0 = first;
    t1 = end;
    warp = threadIdx.x / 32;
    request(P, b, g, 0);
  }
  __device__ __forceinline__ void request(const WeightsParams& P, int b, int g, int n) {
    if (n % IDS == 0) fetch_ids(P, b, n);
    const int lane = threadIdx.x & 31, r = lane / 4, c = lane % 4, t = token(n);
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      block[h] = __shfl_sync(0xffffffffu, ids, n % IDS * HALVES + h);
      const size_t tile = (size_t)max(block[h], 0) * P.num_kv_heads + g;
#pragma unroll
      for (int nt = 2 * h; nt < 2 * h + 2; ++nt) {
        // rows past the length may hold anything; nothing of them is used
        if (block[h] >= 0 && t + 8 * nt + r < t1)
          next[nt].load(P.k_cache, tile, P.block_size, (t + 16 * h) % P.block_size + 8 * (nt % 2) + r, c);
        else
          next[nt].clear();
      }
    }
  }
};

__device__ __forceinline__ int clamped_len(const int32_t* lens, int b, int block_size, int max_blocks, int* error_word) {
  const int L = lens[b];
  if (L > 0 && (L - 1) / block_size >= max_blocks) {
    record_error(error_word, kErrBadBlock);
    return max_blocks * block_size;
  }
  return L;
}

// Scores outside [0, lim) of a step's tokens, and of halves without a block, become -inf; sc[nt][e]: row r + 8 (e /
// 2), token 8 nt + 2c + e % 2.
template <int TILES>
__device__ __forceinline__ void mask_scores(float (&sc)[TILES][4], const int (&lim)[2], const int* block) {
  const int c = threadIdx.x & 3;
#pragma unroll
  for (int nt = 0; nt < TILES; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (block[nt / 2] < 0 || 8 * nt + 2 * c + e % 2 >= lim[e / 2]) sc[nt][e] = -INFINITY;
}

// A row's maximum and sum over its four lanes, then over the warps, into partition j's place.
template <int NR, int HF>
__device__ __forceinline__ void store_rows(const WeightsParams& P, float (&m)[NR][HF], float (&l)[NR][HF], float* red,
                                           int bg, int j, int first) {
  constexpr int NW = kWeightsWarps, N = 16 * NR;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
#pragma unroll
  for (int k = 0; k < NR; ++k)
#pragma unroll
    for (int hf = 0; hf < HF; ++hf) {
      float mx = fmaxf(m[k][hf], __shfl_xor_sync(0xffffffffu, m[k][hf], 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      float z = mx == -INFINITY ? 0.f : l[k][hf] * ex2_approx(m[k][hf] - mx);
      z += __shfl_xor_sync(0xffffffffu, z, 1);
      z += __shfl_xor_sync(0xffffffffu, z, 2);
      if (c == 0) {
        red[warp * N + 16 * k + 8 * hf + r] = mx;
        red[(NW + warp) * N + 16 * k + 8 * hf + r] = z;
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < (HF == 1 ? 8 : N); i += 32 * NW) {
    const int row = first + i;
    if (row >= P.rows) break;
    float mx = -INFINITY, z = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) mx = fmaxf(mx, red[w * N + i]);
    if (mx != -INFINITY)
#pragma unroll
      for (int w = 0; w < NW; ++w) z = fmaf(red[(NW + w) * N + i], ex2_approx(red[w * N + i] - mx), z);
    const size_t at = ((size_t)bg * P.np + j) * P.rows + row;
    P.row_max[at] = mx;
    P.row_sum[at] = z;
  }
}

// First grid, few rows (HF * 8 of them at most): CTA (partition, b, g).
template <int KV, int D>
struct WeightsRing {
  static constexpr int UNIT = 32;  // tokens of a slot
  static constexpr int SLOT = KV == kKvInt4 ? UNIT * D * 9 / 16 : UNIT * D * (KV == kKvFp16 ? 2 : 1);
  static constexpr int SW = KV == kKvFp16 ? (D == 128 ? 3 : 4) : 4;  // slots a warp
  static constexpr int SMEM = kWeightsWarps * SW * (SLOT + 8);
};
template <int KV, int D, int HF>
__global__ void __launch_bounds__(32 * kWeightsWarps, KV == kKvFp16 && D == 128 ? 2 : 3)
    paged_weights_few_kernel(const WeightsParams P, unsigned long long timeout_ns) {
  using T = WeightsRing<KV, D>;
  constexpr int NW = kWeightsWarps, TILES = T::UNIT / 8, KS = D / 16, SW = T::SW;
  extern __shared__ __align__(128) unsigned char weights_smem[];
  __shared__ float red[2 * NW * 16];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int j = blockIdx.x % P.np, bg = blockIdx.x / P.np;
  const int g = bg % P.num_kv_heads, b = bg / P.num_kv_heads;
  const int L = clamped_len(P.context_lens, b, P.block_size, P.max_blocks_per_seq, P.error_word);
  const int t0 = j * P.part, t1 = min(L, t0 + P.part);
  if (t0 >= L) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
  const int BS = P.block_size, per = T::UNIT / BS;  // tiles a slot: 1 or 2
  const uint32_t tile_bytes = T::SLOT / per;
  unsigned char* ring = weights_smem + warp * SW * T::SLOT;
  uint64_t* full = reinterpret_cast<uint64_t*>(weights_smem + NW * SW * T::SLOT) + warp * SW;
  if (lane == 0) {
    for (int s = 0; s < SW; ++s) mbar_init(&full[s], 1);
    fence_mbarrier_init();
  }
  __syncwarp();
  const int units = (t1 - t0 + T::UNIT - 1) / T::UNIT, nblk = (t1 - t0 + BS - 1) / BS;
  const int mine = units > warp ? (units - warp + NW - 1) / NW : 0;
  const int32_t* bt = P.block_tables + (size_t)b * P.max_blocks_per_seq + t0 / BS;
  // block ids: two places a unit, 16 units at a time, the next ones requested ahead
  auto ids_at = [&](int first) {
    const int n = first + lane / 2, k = (warp + NW * n) * per + lane % 2;
    return n < mine && lane % 2 < per && k < nblk ? bt[k] : -1;
  };
  int ids = ids_at(0), ids_next = ids_at(16);
  uint32_t bad_slots = 0;  // two bits a slot: tiles that are not there
  const uint32_t ring_at = smem_u32(ring), full_at = smem_u32(full);
  const char* kbase = static_cast<const char*>(P.k_cache) + (size_t)g * tile_bytes;
  const uint64_t block_stride = (uint64_t)P.num_kv_heads * tile_bytes;
  auto issue = [&](int n) {
    if (n > 0 && n % 16 == 0) {
      ids = ids_next;
      ids_next = ids_at(n + 16);
    }
    const uint32_t slot = (uint32_t)n % SW, bar = full_at + slot * 8;
    const int pb = __shfl_sync(0xffffffffu, ids, n % 16 * 2 + lane % 2);
    const bool good = (uint32_t)pb < (uint32_t)P.num_blocks;
    const uint32_t there = __ballot_sync(0xffffffffu, good) & (per == 2 ? 3u : 1u);
    bad_slots |= (~there & 3u) << (2 * slot);
    if (lane < per && !good && (warp + NW * n) * per + lane < nblk) record_error(P.error_word, kErrBadBlock);
    if (lane == 0) int4_expect(bar, __popc(there) * tile_bytes);
    if (lane < per && good)
      int4_copy(ring_at + slot * T::SLOT + lane * tile_bytes, kbase + (uint64_t)(uint32_t)pb * block_stride, tile_bytes, bar);
  };
  int issued = 0;
  for (; issued < SW && issued < mine; ++issued) issue(issued);
  uint32_t qa[KS][2 * HF];
#pragma unroll
  for (int hf = 0; hf < HF; ++hf) {
    const int row = r + 8 * hf;
    const __half* q = query_row<D>(P, b, g, min(row, P.rows - 1));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      if (row < P.rows) u = *reinterpret_cast<const uint4*>(q + 8 * query_eight<KV, D>(i, c));
      const QueryWords w = query_words<KV, D>(u, query_eight<KV, D>(i, c), P.q_sign);
      // (steps by position: the i-th eight of a lane is steps 2i and 2i + 1)
#pragma unroll
      for (int x = 0; x < 4; ++x) qa[2 * i + x / 2][HF * (x % 2) + hf] = w.w[x];
    }
  }
  const int G = P.rows / P.q_len;
  const int all_see = min(t1, L - P.q_len + 1);
  int see[2] = {0, 0};
#pragma unroll
  for (int hf = 0; hf < HF; ++hf)
    if (r + 8 * hf < P.rows) see[hf] = min(L - P.q_len + (r + 8 * hf) / G + 1, t1);
  float m[1][HF], l[1][HF];
#pragma unroll
  for (int hf = 0; hf < HF; ++hf) {
    m[0][hf] = -INFINITY;
    l[0][hf] = 0.f;
  }
  float* scores[HF];
#pragma unroll
  for (int hf = 0; hf < HF; ++hf)
    scores[hf] = P.scores + ((size_t)bg * P.rows + min(r + 8 * hf, P.rows - 1)) * P.score_stride + 2 * c;
  for (int n = 0; n < mine; ++n) {
    const uint32_t slot = (uint32_t)n % SW;
    if (!mbar_wait_bounded(&full[slot], ((uint32_t)n / SW) & 1, timeout_ns)) {
      if (lane == 0) record_error(P.error_word, kErrTimeout);
      for (int v = n + 1; v < issued; ++v) mbar_wait_bounded(&full[v % SW], (v / SW) & 1, timeout_ns);
      break;
    }
    const unsigned char* at = ring + slot * T::SLOT;
    const int t = t0 + (warp + NW * n) * T::UNIT;
    const uint32_t missing = bad_slots >> (2 * slot) & (per == 2 ? 3u : 1u);
    bad_slots &= ~(3u << (2 * slot));
    float sc[TILES][4];
#pragma unroll
    for (int nt = 0; nt < TILES; ++nt) {
      KeyRow<KV, D> key;
      const int row = 8 * nt + r;  // of the slot's tiles, one behind the other
      key.load(at, row / BS, BS, row % BS, c);
      uint32_t kb[D / 8];
      key.fragments(kb, P.bases);
#pragma unroll
      for (int s = 0; s < KS; ++s)
        mma_16816_from(sc[nt], s == 0, qa[s][0], HF == 2 ? qa[s][1] : 0u, qa[s][HF], HF == 2 ? qa[s][2 * HF - 1] : 0u,
                       kb[2 * s], kb[2 * s + 1]);
    }
    __syncwarp();
    if (issued < mine) {
      fence_proxy_async_smem();  // our reads of the slot precede the next copies into it
      issue(issued);
      ++issued;
    }
    if (missing != 0 || t + T::UNIT > all_see) {
      const int lim[2] = {see[0] - t, see[1] - t};
      const int block[2] = {missing & 1 ? -1 : 0, (per == 2 ? missing & 2 : missing & 1) ? -1 : 0};
      mask_scores<TILES>(sc, lim, block);
    }
#pragma unroll
    for (int hf = 0; hf < HF; ++hf) {
      float x[2 * TILES], mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2 * TILES; ++i) {
        x[i] = sc[i / 2][2 * hf + i % 2] * P.scale_log2;
        mx = fmaxf(mx, x[i]);
      }
      if (r + 8 * hf < P.rows) {
#pragma unroll
        for (int nt = 0; nt < TILES; ++nt)
          *reinterpret_cast<float2*>(scores[hf] + t + 8 * nt) = make_float2(x[2 * nt], x[2 * nt + 1]);
      }
      const float mn = fmaxf(m[0][hf], mx);
      const float mu = mn == -INFINITY ? 0.f : mn;  // nothing seen so far
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * TILES; ++i) sum += ex2_approx(x[i] - mu);
      l[0][hf] = fmaf(l[0][hf], ex2_approx(m[0][hf] - mu), sum);
      m[0][hf] = mn;
    }
  }
  store_rows<1, HF>(P, m, l, red, bg, j, 0);
}

// First grid, many rows: CTA (chunk of 16 RT rows, partition, b, g).
template <int KV, int D, int RT>
__global__ void __launch_bounds__(32 * kWeightsWarps, kManyRowsCtas) paged_weights_rows_kernel(const WeightsParams P) {
  constexpr int NW = kWeightsWarps, TILES = key_tiles(KV), KS = D / 16, CHUNK = 16 * RT;
  extern __shared__ __align__(128) unsigned char weights_smem[];
  uint4* qs = reinterpret_cast<uint4*>(weights_smem);
  __shared__ float red[2 * NW * CHUNK];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rc = blockIdx.x % P.row_chunks;
  const int rest = blockIdx.x / P.row_chunks;
  const int j = rest % P.np, bg = rest / P.np;
  const int g = bg % P.num_kv_heads, b = bg / P.num_kv_heads;
  const int L = clamped_len(P.context_lens, b, P.block_size, P.max_blocks_per_seq, P.error_word);
  const int t0 = j * P.part, t1 = min(L, t0 + P.part);
  if (t0 >= L) return;
  const int lane = threadIdx.x % 32, r = lane / 4;
  KeyStream<KV, D> keys;
  keys.start(P, b, g, t0, t1);
  const int tiles = min(RT, (P.rows - rc * CHUNK + 15) / 16);
  load_query_tiles<KV, D>(P, qs, b, g, rc * RT, tiles);
  __syncthreads();
  const int G = P.rows / P.q_len;
  const int all_see = min(t1, L - P.q_len + 1);  // tokens that every row sees
  auto sees = [&](int k, int hf) {
    const int row = (rc * RT + k) * 16 + r + 8 * hf;
    return row < P.rows ? min(L - P.q_len + row / G + 1, t1) : 0;
  };
  float m[RT][2], l[RT][2];
#pragma unroll
  for (int k = 0; k < RT; ++k)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      m[k][hf] = -INFINITY;
      l[k][hf] = 0.f;
    }
  for (int n = 0; keys.token(n) < t1; ++n) {
    const int t = keys.token(n);
    uint32_t kb[TILES][D / 8];
    int block[TILES / 2];
    bool whole = t + 8 * TILES <= all_see;
#pragma unroll
    for (int nt = 0; nt < TILES; ++nt) keys.next[nt].fragments(kb[nt], P.bases);
#pragma unroll
    for (int h = 0; h < TILES / 2; ++h) {
      block[h] = keys.block[h];
      whole &= block[h] >= 0;
    }
    keys.request(P, b, g, n + 1);
#pragma unroll
    for (int k = 0; k < RT; ++k) {
      if (k >= tiles) break;
      float sc[TILES][4];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint4 w = qs[(k * KS + s) * 32 + lane];
#pragma unroll
        for (int nt = 0; nt < TILES; ++nt)
          mma_16816_from(sc[nt], s == 0, w.x, w.y, w.z, w.w, kb[nt][2 * s], kb[nt][2 * s + 1]);
      }
      if (!whole) {
        const int lim[2] = {sees(k, 0) - t, sees(k, 1) - t};
        mask_scores<TILES>(sc, lim, block);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float mx = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < TILES; ++nt) mx = fmaxf(mx, fmaxf(sc[nt][2 * hf], sc[nt][2 * hf + 1]));
        const float mn = fmaxf(m[k][hf], mx * P.scale_log2);
        const float mu = mn == -INFINITY ? 0.f : mn;  // nothing seen so far
        float sum = 0.f;
#pragma unroll
        for (int nt = 0; nt < TILES; ++nt)
          sum += ex2_approx(fmaf(sc[nt][2 * hf], P.scale_log2, -mu)) +
                 ex2_approx(fmaf(sc[nt][2 * hf + 1], P.scale_log2, -mu));
        l[k][hf] = fmaf(l[k][hf], ex2_approx(m[k][hf] - mu), sum);
        m[k][hf] = mn;
      }
    }
  }
  store_rows<RT, 2>(P, m, l, red, bg, j, rc * CHUNK);
}

// Rows first .. first + n - 1 of (b, g): M + log2(Z) over the partitions written (+inf where nothing is seen).
__device__ __forceinline__ void merge_rows(const WeightsParams& P, int bg, int L, int first, int n, float* out,
                                           int threads) {
  const int np = min(P.np, (L - 1) / P.part + 1);
  constexpr int U = 8;  // partitions in flight
  for (int i = threadIdx.x; i < n; i += threads) {
    const size_t at = (size_t)bg * P.np * P.rows + first + i;
    float mx = -INFINITY, z = 0.f;
    for (int j0 = 0; j0 < np; j0 += U) {
      float m[U], l[U], top = mx;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        m[u] = j0 + u < np ? P.row_max[at + (size_t)(j0 + u) * P.rows] : -INFINITY;
        l[u] = j0 + u < np ? P.row_sum[at + (size_t)(j0 + u) * P.rows] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, m[u]);
      if (top == -INFINITY) continue;
      z *= ex2_approx(mx - top);
#pragma unroll
      for (int u = 0; u < U; ++u) z = fmaf(l[u], ex2_approx(m[u] - top), z);
      mx = top;
    }
    out[i] = z > 0.f ? mx + __log2f(z) : INFINITY;
  }
}

// Second grid, few rows: CTA (1024 tokens, b, g); a thread takes four neighbouring tokens.
constexpr int kFinishMaxRows = 16;
__global__ void __launch_bounds__(kWeightsFinishThreads) paged_weights_scores_kernel(const WeightsParams P, int chunks);

// Second grid, many rows: CTA (partition, b, g) multiplies again.
template <int KV, int D>
__global__ void __launch_bounds__(32 * kWeightsWarps, kManyRowsCtas) paged_weights_keys_kernel(const WeightsParams P) {
  constexpr int NW = kWeightsWarps, TILES = key_tiles(KV), KS = D / 16;
  extern __shared__ __align__(16) unsigned char weights_smem[];
  uint4* qs = reinterpret_cast<uint4*>(weights_smem);
  float* row_off = reinterpret_cast<float*>(qs + P.q_tiles * KS * 32);
  const int j = blockIdx.x % P.np, bg = blockIdx.x / P.np;
  const int g = bg % P.num_kv_heads, b = bg / P.num_kv_heads;
  const int L = clamped_len(P.context_lens, b, P.block_size, P.max_blocks_per_seq, nullptr);
  const int t0 = j * P.part, t1 = min(L, t0 + P.part);
  if (t0 >= L) return;
  const int start = P.start_lens ? P.start_lens[b] : L;
  const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
  const int G = P.rows / P.q_len;
  const int all_see = min(t1, L - P.q_len + 1);
  for (int first = 0; first < P.rows; first += 16 * P.q_tiles) {
    const int tiles = min(P.q_tiles, (P.rows - first + 15) / 16);
    KeyStream<KV, D> keys;
    keys.start(P, b, g, t0, t1);
    __syncthreads();  // the rows before are done with
    load_query_tiles<KV, D>(P, qs, b, g, first / 16, tiles);
    if (first == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    merge_rows(P, bg, L, first, min(16 * tiles, P.rows - first), row_off, 32 * NW);
    for (int i = P.rows - first + threadIdx.x; i < 16 * tiles; i += 32 * NW) row_off[i] = INFINITY;
    __syncthreads();
    for (int n = 0; keys.token(n) < t1; ++n) {
      const int t = keys.token(n);
      uint32_t kb[TILES][D / 8];
      int block[TILES / 2];
      bool whole = t + 8 * TILES <= all_see;
#pragma unroll
      for (int nt = 0; nt < TILES; ++nt) keys.next[nt].fragments(kb[nt], P.bases);
#pragma unroll
      for (int h = 0; h < TILES / 2; ++h) {
        block[h] = keys.block[h];
        whole &= block[h] >= 0;
      }
      keys.request(P, b, g, n + 1);
      float sum[TILES][2];  // tokens 8 nt + 2c + e over the lane's rows
#pragma unroll
      for (int nt = 0; nt < TILES; ++nt) sum[nt][0] = sum[nt][1] = 0.f;
      for (int k = 0; k < tiles; ++k) {
        const float off[2] = {row_off[16 * k + r], row_off[16 * k + 8 + r]};
        float sc[TILES][4];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint4 w = qs[(k * KS + s) * 32 + lane];
#pragma unroll
          for (int nt = 0; nt < TILES; ++nt)
            mma_16816_from(sc[nt], s == 0, w.x, w.y, w.z, w.w, kb[nt][2 * s], kb[nt][2 * s + 1]);
        }
        if (!whole) {
          int lim[2];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int row = first + 16 * k + r + 8 * hf;
            lim[hf] = (row < P.rows ? min(L - P.q_len + row / G + 1, t1) : 0) - t;
          }
          mask_scores<TILES>(sc, lim, block);
        }
#pragma unroll
        for (int nt = 0; nt < TILES; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[nt][e % 2] += ex2_approx(fmaf(sc[nt][e], P.scale_log2, -off[e / 2]));
      }
#pragma unroll
      for (int nt = 0; nt < TILES; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], k);
      // lane (r, c) writes token 8 (r / 2) + 2c + r % 2
      float w = 0.f;
      int pb = -1;
#pragma unroll
      for (int x = 0; x < 2 * TILES; ++x)
        if (r == x) {
          w = sum[x / 2][x % 2];
          pb = block[x / 4];
        }
      const int tok = t + 8 * (r / 2) + 2 * c + r % 2;
      if (pb >= 0 && tok < t1) {
        float* o = P.weights + ((size_t)pb * P.num_kv_heads + g) * P.block_size + tok % P.block_size;
        if (first > 0)
          *o += w;
        else
          *o = tok < start && P.decay != 0.f ? fmaf(P.decay, *o, w) : w;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Choice of tokens: CTA (b, g).  Weights as ordered 32-bit keys (equal values
// equal keys, larger ones larger, not a number the largest, no block the
// smallest), kept in shared memory; the need-th largest key of the candidates by
// at most three passes of 2048 bins, the first as the keys come; then every warp
// votes on its own stretch, counts and writes the chosen tokens, ascending.  A
// thread loads four neighbouring tokens at a time, eight such loads in flight.
//
// Bound by latencies and instructions, not by its bytes: of a CTA's 19 us for 28,000
// tokens 7.5 are the tables and weights coming in with the first counts, 3.3-4.9
// the passes over the bits, 2.3 the votes, 1.7 the writing.  48 x 8 rows of
// 8000-32768 tokens 44 us (58 with the first pass apart and ranks by token), 32 x
// 8 rows of 1150 7.8.  One CTA of 1024 threads an SM, as the keys fill its shared
// memory; 512 threads took 58, two CTAs of 512 with 22,000 keys each 126, as the
// longer rows are read again.
struct TokenSelectParams {
  const float* weights;
  const int32_t *block_tables, *context_lens;
  int32_t *kept, *kept_lens;
  int num_seqs, num_kv_heads, block_size, num_blocks, max_blocks_per_seq, max_kept, sink, recent;
  int cached;  // keys held in shared memory, a multiple of 4
  int block_shift;  // log2(block_size) where that is a power of two from 4 on and quads of weights are aligned, else -1
  int* error_word;
};

__device__ __forceinline__ uint32_t ordered_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// ---------------------------------------------------------------------------
// Copy of kept rows: a warp takes a few dozen new rows of one (b, g).  Its lanes look
// up where the rows come from and go to, a row a lane, then copy 16-byte pieces,
// K's and V's, four in flight a lane; warps do not wait for one another, so one's
// look-ups (three dependent loads) run beside the others' copies.
// Bound by HBM, by 128- and 256-byte pieces in no order: 48 x 8 x 2048 rows of E4M3
// 71 us, 5.8 TB/s, 32 x 8 x 1024 of fp16 47 us, 5.8 TB/s.  4-bit rows lie in pieces of
// 16 bytes, half a sector each, one of 8: 48 x 8 x 2048 of them 122 us, 1.9 TB/s of
// their bytes (256 threads that look up
// together first, eight pieces in flight: 78 and 48; 10 or 12 CTAs an SM: 72 and 76;
// six pieces in flight: 73).
struct CompactParams {
  uint8_t *k_cache, *v_cache;
  float* weights;
  const int32_t *block_tables, *context_lens, *kept, *kept_lens, *new_tables;
  int num_seqs, num_kv_heads, num_blocks, block_size, max_blocks_per_seq, max_kept, max_new_blocks, chunks;
  int* error_word;
};

constexpr int kCompactThreads = 128;
constexpr int kCompactCtas = 9;  // an SM
// New rows of a warp: a dozen to two dozen 16-byte pieces a lane.
__host__ __device__ constexpr int compact_rows(int KV, int D) {
  return KV == kKvFp16 && D == 128 ? 16 : 32;
}

template <int KV, int D>
__global__ void __launch_bounds__(kCompactThreads, kCompactCtas) paged_kv_compact_kernel(const CompactParams P) {
  // pieces of a row in one cache: 16 bytes each; 4-bit rows: D / 32 of codes, and the scales
  constexpr int PIECES = KV == kKvFp16 ? D / 8 : (KV == kKvE4m3 ? D / 16 : D / 32 + 1);
  constexpr int ROWS = compact_rows(KV, D), WARPS = kCompactThreads / 32;
  static_assert(ROWS <= 32, "a lane looks up a row");
  const int lane = threadIdx.x % 32;
  const int chunk = blockIdx.x % P.chunks, bg = blockIdx.x / P.chunks;
  const int g = bg % P.num_kv_heads, b = bg / P.num_kv_heads;
  const int i0 = (chunk * WARPS + (int)threadIdx.x / 32) * ROWS;
  const int room = min(P.max_kept, (int)min((long long)P.max_new_blocks * P.block_size, 0x7fffffffLL));
  const int kept = P.kept_lens[b];
  if (chunk == 0 && g == 0 && threadIdx.x == 0 && (kept < 0 || kept > room)) record_error(P.error_word, kErrBadBlock);
  const int rows = min(min(kept, room) - i0, ROWS);
  if (rows <= 0) return;
  const int BS = P.block_size;
  const size_t TILE = KV == kKvInt4 ? (size_t)BS * D * 9 / 16 : (size_t)BS * PIECES * 16;
  size_t src = 0, dst = 0;  // the tiles' first bytes
  int src_row = -1;         // -1: nothing to copy
  if (lane < rows) {
    const int i = i0 + lane;
    const int t = P.kept[(size_t)bg * P.max_kept + i];
    const int to = P.new_tables[(size_t)b * P.max_new_blocks + i / BS];
    int from = -1;
    if (t >= 0 && t < P.context_lens[b] && t / BS < P.max_blocks_per_seq)
      from = P.block_tables[(size_t)b * P.max_blocks_per_seq + t / BS];
    if (from < 0 || from >= P.num_blocks || to < 0 || to >= P.num_blocks) {
      record_error(P.error_word, kErrBadBlock);
    } else {
      const size_t from_tile = (size_t)from * P.num_kv_heads + g, to_tile = (size_t)to * P.num_kv_heads + g;
      src = from_tile * TILE;
      dst = to_tile * TILE;
      src_row = t % BS;
      if (P.weights) P.weights[to_tile * BS + i % BS] = P.weights[from_tile * BS + src_row];
    }
  }
  constexpr int U = 4;
  constexpr int ITEMS = ROWS * 2 * PIECES;
  static_assert(ITEMS % 32 == 0, "whole warps look at every row");
  const int items = rows * 2 * PIECES;
  for (int at = 0; at < items; at += 32 * U) {
    uint4 x[U];
    uint8_t* to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int it = at + u * 32 + lane;
      const int piece = it % PIECES, kv = it / PIECES % 2, i = it / (2 * PIECES);
      const int from_row = __shfl_sync(0xffffffffu, src_row, i);
      const size_t from = __shfl_sync(0xffffffffu, src, i), into = __shfl_sync(0xffffffffu, dst, i);
      to[u] = nullptr;
      if (it >= items || from_row < 0) continue;
      const uint8_t* s = (kv ? P.v_cache : P.k_cache) + from;
      uint8_t* o = (kv ? P.v_cache : P.k_cache) + into;
      const int to_row = (i0 + i) % BS;
      if constexpr (KV == kKvInt4) {
        if (piece < D / 32) {
          x[u] = *reinterpret_cast<const uint4*>(s + (piece * BS + from_row) * 16);
          to[u] = o + (piece * BS + to_row) * 16;
        } else {
          s += BS * (D / 2) + from_row * (D / 16);
          o += BS * (D / 2) + to_row * (D / 16);
          if constexpr (D == 128)
            *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(s);
          else
            *reinterpret_cast<uint32_t*>(o) = *reinterpret_cast<const uint32_t*>(s);
        }
      } else {
        x[u] = *reinterpret_cast<const uint4*>(s + (from_row * PIECES + piece) * 16);
        to[u] = o + (to_row * PIECES + piece) * 16;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u]) *reinterpret_cast<uint4*>(to[u]) = x[u];
  }
}

}  // namespace pkd
