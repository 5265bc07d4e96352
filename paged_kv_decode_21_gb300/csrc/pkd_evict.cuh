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
// sum over every partition of the tokens; the second merges those and adds up
// the weights.  Where rows are few, the first also leaves the scores, 4 bytes a
// row and token, and the second reads those; where they are many it reads K
// again and multiplies again, since a score written and read takes 8 bytes and a
// key 2D and less.
//
// S = Q K^T by mma.m16n8k16: 16 rows times 8 tokens, keys going from global
// memory straight into B fragments: lane (r, c) holds the dims of token r that
// come as its 16-byte loads, and Q's A fragments, kept in shared memory, follow
// that order of dims (key_dim).  The next 16 tokens' loads are requested before
// this tile's products.
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
  int part, np;   // tokens per partition (a multiple of 64), partitions
  int row_chunks; // first grid: chunks of 16 RT rows
  int q_tiles;    // second grid, keys again: row tiles of Q in shared memory at a time
  float scale_log2, decay;
  int* error_word;
  Int4Bases bases;
};

constexpr int kWeightsWarps = 4;
constexpr int kWeightsFinishThreads = 256;

// The dim that k-step s has in slot pair h (0: slots 2c, 2c + 1; 1: slots 8 +
// 2c, 9 + 2c), half e, of lane c.
template <int KV, int D>
__device__ __forceinline__ int key_dim(int s, int c, int h, int e) {
  if (KV == kKvFp16) return 32 * (s / 2) + 8 * c + 4 * (s % 2) + 2 * h + e;
  if (KV == kKvE4m3) return 64 * (s / 4) + 16 * c + 4 * (s % 4) + 2 * h + e;
  // words of eight codes, halves four dims apart; a lane has D / 4 neighbouring dims
  return (D / 4) * c + 8 * (s / 2) + 2 * (s % 2) + h + 4 * e;
}

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

// Q's rows 16 rt .. of tiles [first, first + n) as A fragments in shared memory: [tile][k-step][lane] uint4.
template <int KV, int D>
__device__ __forceinline__ void load_query_tiles(const WeightsParams& P, uint4* qs, int b, int g, int first, int n) {
  const int G = P.rows / P.q_len;
  uint32_t* w = reinterpret_cast<uint32_t*>(qs);
  for (int i = threadIdx.x; i < n * (D / 16) * 128; i += blockDim.x) {
    const int reg = i % 4, lane = (i / 4) % 32, s = (i / 128) % (D / 16), rt = i / 128 / (D / 16);
    const int row = (first + rt) * 16 + lane / 4 + 8 * (reg & 1);
    uint32_t x = 0;
    if (row < P.rows) {
      const unsigned short* q = reinterpret_cast<const unsigned short*>(P.q) +
                                (((size_t)b * P.q_len + row / G) * P.num_q_heads + (size_t)g * G + row % G) * D;
      x = q[key_dim<KV, D>(s, lane % 4, reg >> 1, 0)] | ((uint32_t)q[key_dim<KV, D>(s, lane % 4, reg >> 1, 1)] << 16);
    }
    w[i] = x;
  }
}

// Scores (log2 units, masked) of one row tile over 16 tokens: sc[nt][e] of row
// r + 8 (e / 2), token 8 nt + 2c + e % 2.  lim: tokens that the rows r, r + 8 see from the tile's first on.
template <int D>
__device__ __forceinline__ void tile_scores(const uint4* qs, const uint32_t (&b0)[D / 8], const uint32_t (&b1)[D / 8],
                                            float scale_log2, const int (&lim)[2], float (&sc)[2][4]) {
  const int lane = threadIdx.x & 31, c = lane % 4;
#pragma unroll
  for (int e = 0; e < 4; ++e) sc[0][e] = sc[1][e] = 0.f;
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    const uint4 u = qs[s * 32 + lane];
    const uint32_t a[4] = {u.x, u.y, u.z, u.w};
    mma_16816(sc[0], a, b0[2 * s], b0[2 * s + 1]);
    mma_16816(sc[1], a, b1[2 * s], b1[2 * s + 1]);
  }
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      sc[nt][e] = 8 * nt + 2 * c + e % 2 < lim[e / 2] ? sc[nt][e] * scale_log2 : -INFINITY;
}

// The keys of a warp's tiles of 16 tokens, a tile requested ahead.
template <int KV, int D>
struct KeyStream {
  KeyRow<KV, D> next[2];
  bool next_ok;
  __device__ __forceinline__ void request(const WeightsParams& P, int b, int g, int t, int t1) {
    const int lane = threadIdx.x & 31, r = lane / 4, c = lane % 4;
    next_ok = false;
    if (t < t1) {
      const int pb = P.block_tables[(size_t)b * P.max_blocks_per_seq + t / P.block_size];
      next_ok = pb >= 0 && pb < P.num_blocks;
      if (!next_ok && lane == 0) record_error(P.error_word, kErrBadBlock);
      const size_t tile = (size_t)(next_ok ? pb : 0) * P.num_kv_heads + g;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        // rows past the length may hold anything; nothing of them is used
        if (next_ok && t + 8 * nt + r < t1)
          next[nt].load(P.k_cache, tile, P.block_size, t % P.block_size + 8 * nt + r, c);
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

// First grid: CTA (row chunk, partition, b, g).
template <int KV, int D, int RT>
__global__ void __launch_bounds__(32 * kWeightsWarps) paged_weights_rows_kernel(const WeightsParams P) {
  constexpr int NW = kWeightsWarps;
  __shared__ uint4 qs[RT * (D / 16) * 32];
  __shared__ float red[2][NW][16 * RT];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rc = blockIdx.x % P.row_chunks;
  const int rest = blockIdx.x / P.row_chunks;
  const int j = rest % P.np, bg = rest / P.np;
  const int g = bg % P.num_kv_heads, b = bg / P.num_kv_heads;
  const int L = clamped_len(P.context_lens, b, P.block_size, P.max_blocks_per_seq, P.error_word);
  const int t0 = j * P.part, t1 = min(L, t0 + P.part);
  if (t0 >= L) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
  KeyStream<KV, D> keys;
  keys.request(P, b, g, t0 + 16 * warp, t1);
  const int tiles = min(RT, (P.rows - rc * 16 * RT + 15) / 16);
  load_query_tiles<KV, D>(P, qs, b, g, rc * RT, tiles);
  __syncthreads();
  const int G = P.rows / P.q_len;
  int see[RT][2];  // tokens that the lane's rows see
  float m[RT][2], l[RT][2];
#pragma unroll
  for (int k = 0; k < RT; ++k)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int row = (rc * RT + k) * 16 + r + 8 * hf;
      see[k][hf] = row < P.rows ? L - P.q_len + row / G + 1 : 0;
      m[k][hf] = -INFINITY;
      l[k][hf] = 0.f;
    }
  for (int t = t0 + 16 * warp; t < t1; t += 16 * NW) {
    uint32_t b0[D / 8], b1[D / 8];
    keys.next[0].fragments(b0, P.bases);
    keys.next[1].fragments(b1, P.bases);
    const bool ok = keys.next_ok;
    keys.request(P, b, g, t + 16 * NW, t1);
#pragma unroll
    for (int k = 0; k < RT; ++k) {
      if (k >= tiles) break;
      const int lim[2] = {ok ? min(see[k][0], t1) - t : 0, ok ? min(see[k][1], t1) - t : 0};
      float sc[2][4];
      tile_scores<D>(qs + k * (D / 16) * 32, b0, b1, P.scale_log2, lim, sc);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float s0 = sc[0][2 * hf], s1 = sc[0][2 * hf + 1], s2 = sc[1][2 * hf], s3 = sc[1][2 * hf + 1];
        const float mn = fmaxf(m[k][hf], fmaxf(fmaxf(s0, s1), fmaxf(s2, s3)));
        const float mu = mn == -INFINITY ? 0.f : mn;  // nothing seen so far
        l[k][hf] = l[k][hf] * ex2_approx(m[k][hf] - mu) + (ex2_approx(s0 - mu) + ex2_approx(s1 - mu)) +
                   (ex2_approx(s2 - mu) + ex2_approx(s3 - mu));
        m[k][hf] = mn;
        const int row = (rc * RT + k) * 16 + r + 8 * hf;
        if (P.scores && row < P.rows) {
          float* o = P.scores + ((size_t)bg * P.rows + row) * P.score_stride + t + 2 * c;
          *reinterpret_cast<float2*>(o) = make_float2(s0, s1);
          *reinterpret_cast<float2*>(o + 8) = make_float2(s2, s3);
        }
      }
    }
  }
  // a row's statistics over its four lanes, then over the warps
#pragma unroll
  for (int k = 0; k < RT; ++k)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float mx = fmaxf(m[k][hf], __shfl_xor_sync(0xffffffffu, m[k][hf], 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      float z = mx == -INFINITY ? 0.f : l[k][hf] * ex2_approx(m[k][hf] - mx);
      z += __shfl_xor_sync(0xffffffffu, z, 1);
      z += __shfl_xor_sync(0xffffffffu, z, 2);
      if (c == 0) {
        red[0][warp][16 * k + 8 * hf + r] = mx;
        red[1][warp][16 * k + 8 * hf + r] = z;
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * RT; i += 32 * NW) {
    const int row = rc * 16 * RT + i;
    if (row >= P.rows) break;
    float mx = -INFINITY, z = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) mx = fmaxf(mx, red[0][w][i]);
    if (mx != -INFINITY)
#pragma unroll
      for (int w = 0; w < NW; ++w) z = fmaf(red[1][w][i], ex2_approx(red[0][w][i] - mx), z);
    const size_t at = ((size_t)bg * P.np + j) * P.rows + row;
    P.row_max[at] = mx;
    P.row_sum[at] = z;
  }
}

// Rows first .. first + n - 1 of (b, g): maximum and 1 / sum over the partitions written (0 where nothing is seen).
__device__ __forceinline__ void merge_rows(const WeightsParams& P, int bg, int L, int first, int n, float* mx_out,
                                           float* inv_out) {
  const int np = min(P.np, (L - 1) / P.part + 1);
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const size_t at = (size_t)bg * P.np * P.rows + first + i;
    float mx = -INFINITY, z = 0.f;
    for (int j = 0; j < np; ++j) mx = fmaxf(mx, P.row_max[at + (size_t)j * P.rows]);
    if (mx == -INFINITY) mx = 0.f;
    for (int j = 0; j < np; ++j)
      z = fmaf(P.row_sum[at + (size_t)j * P.rows], ex2_approx(P.row_max[at + (size_t)j * P.rows] - mx), z);
    mx_out[i] = mx;
    inv_out[i] = z > 0.f ? 1.f / z : 0.f;
  }
}

// Second grid, few rows: CTA (1024 tokens, b, g); a thread takes four neighbouring tokens.
constexpr int kFinishMaxRows = 64;
__global__ void __launch_bounds__(kWeightsFinishThreads) paged_weights_scores_kernel(const WeightsParams P, int chunks);

// Second grid, many rows: CTA (partition, b, g) multiplies again.
template <int KV, int D>
__global__ void __launch_bounds__(32 * kWeightsWarps) paged_weights_keys_kernel(const WeightsParams P) {
  constexpr int NW = kWeightsWarps;
  extern __shared__ __align__(16) unsigned char weights_smem[];
  uint4* qs = reinterpret_cast<uint4*>(weights_smem);
  float* row_mx = reinterpret_cast<float*>(qs + P.q_tiles * (D / 16) * 32);
  float* row_inv = row_mx + 16 * P.q_tiles;
  const int j = blockIdx.x % P.np, bg = blockIdx.x / P.np;
  const int g = bg % P.num_kv_heads, b = bg / P.num_kv_heads;
  const int L = clamped_len(P.context_lens, b, P.block_size, P.max_blocks_per_seq, nullptr);
  const int t0 = j * P.part, t1 = min(L, t0 + P.part);
  if (t0 >= L) return;
  const int start = P.start_lens ? P.start_lens[b] : L;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
  const int G = P.rows / P.q_len;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int first = 0; first < P.rows; first += 16 * P.q_tiles) {
    const int tiles = min(P.q_tiles, (P.rows - first + 15) / 16);
    KeyStream<KV, D> keys;
    keys.request(P, b, g, t0 + 16 * warp, t1);
    __syncthreads();  // the rows before are done with
    load_query_tiles<KV, D>(P, qs, b, g, first / 16, tiles);
    merge_rows(P, bg, L, first, min(16 * tiles, P.rows - first), row_mx, row_inv);
    for (int i = P.rows - first + threadIdx.x; i < 16 * tiles; i += 32 * NW) row_mx[i] = row_inv[i] = 0.f;
    __syncthreads();
    for (int t = t0 + 16 * warp; t < t1; t += 16 * NW) {
      uint32_t b0[D / 8], b1[D / 8];
      keys.next[0].fragments(b0, P.bases);
      keys.next[1].fragments(b1, P.bases);
      const bool ok = keys.next_ok;
      keys.request(P, b, g, t + 16 * NW, t1);
      float sum[4] = {0.f, 0.f, 0.f, 0.f};  // tokens 2c, 2c + 1, 8 + 2c, 9 + 2c over the lane's rows
      for (int k = 0; k < tiles; ++k) {
        int lim[2];
        float mu[2], iz[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int i = 16 * k + r + 8 * hf;
          lim[hf] = ok && first + i < P.rows ? min(L - P.q_len + (first + i) / G + 1, t1) - t : 0;
          mu[hf] = row_mx[i];
          iz[hf] = row_inv[i];
        }
        float sc[2][4];
        tile_scores<D>(qs + k * (D / 16) * 32, b0, b1, P.scale_log2, lim, sc);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sum[2 * nt + e % 2] = fmaf(ex2_approx(sc[nt][e] - mu[e / 2]), iz[e / 2], sum[2 * nt + e % 2]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], k);
      if (r < 4 && ok) {  // row group r writes the lane's token r
        const float w = r == 0 ? sum[0] : (r == 1 ? sum[1] : (r == 2 ? sum[2] : sum[3]));
        const int tok = t + 2 * c + (r & 1) + 8 * (r >> 1);
        if (tok < t1) {
          const int pb = P.block_tables[(size_t)b * P.max_blocks_per_seq + tok / P.block_size];
          float* o = P.weights + ((size_t)pb * P.num_kv_heads + g) * P.block_size + tok % P.block_size;
          if (first > 0)
            *o += w;
          else
            *o = tok < start && P.decay != 0.f ? fmaf(P.decay, *o, w) : w;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Choice of tokens: CTA (b, g).  Weights as ordered 32-bit keys (equal values
// equal keys, larger ones larger, not a number the largest, no block the
// smallest); the need-th largest key of the candidates by four passes of 256
// bins; then every warp writes the chosen tokens of its own stretch, ascending.
struct TokenSelectParams {
  const float* weights;
  const int32_t *block_tables, *context_lens;
  int32_t *kept, *kept_lens;
  int num_seqs, num_kv_heads, block_size, num_blocks, max_blocks_per_seq, max_kept, sink, recent;
  int cached;  // keys held in shared memory
  int* error_word;
};

constexpr int kTokenSelectThreads = 512;

__device__ __forceinline__ uint32_t ordered_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// ---------------------------------------------------------------------------
// Copy of kept rows: CTA (64 new rows, b, g).  Threads look up where the rows
// come from and go to, then all copy 16-byte pieces, K's and V's, eight in flight.
struct CompactParams {
  uint8_t *k_cache, *v_cache;
  float* weights;
  const int32_t *block_tables, *context_lens, *kept, *kept_lens, *new_tables;
  int num_seqs, num_kv_heads, num_blocks, block_size, max_blocks_per_seq, max_kept, max_new_blocks, chunks;
  int* error_word;
};

constexpr int kCompactRows = 64, kCompactThreads = 256;

template <int KV, int D>
__global__ void __launch_bounds__(kCompactThreads) paged_kv_compact_kernel(const CompactParams P) {
  // pieces of a row in one cache: 16 bytes each; 4-bit rows: D / 32 of codes, and the scales
  constexpr int PIECES = KV == kKvFp16 ? D / 8 : (KV == kKvE4m3 ? D / 16 : D / 32 + 1);
  __shared__ int src_block[kCompactRows], src_row[kCompactRows], dst_block[kCompactRows];
  const int chunk = blockIdx.x % P.chunks, bg = blockIdx.x / P.chunks;
  const int g = bg % P.num_kv_heads, b = bg / P.num_kv_heads;
  const int i0 = chunk * kCompactRows;
  const int room = min(P.max_kept, (int)min((long long)P.max_new_blocks * P.block_size, 0x7fffffffLL));
  const int n = min(P.kept_lens[b], room) - i0;
  if (n <= 0) {
    if (chunk == 0 && g == 0 && threadIdx.x == 0 && P.kept_lens[b] < 0) record_error(P.error_word, kErrBadBlock);
    return;
  }
  if (chunk == 0 && g == 0 && threadIdx.x == 0 && P.kept_lens[b] > room) record_error(P.error_word, kErrBadBlock);
  const int BS = P.block_size, rows = min(n, kCompactRows);
  if (threadIdx.x < rows) {
    const int i = i0 + threadIdx.x;
    const int t = P.kept[(size_t)bg * P.max_kept + i];
    const int to = P.new_tables[(size_t)b * P.max_new_blocks + i / BS];
    int from = -1;
    if (t >= 0 && t < P.context_lens[b] && t / BS < P.max_blocks_per_seq)
      from = P.block_tables[(size_t)b * P.max_blocks_per_seq + t / BS];
    if (from < 0 || from >= P.num_blocks || to < 0 || to >= P.num_blocks) {
      record_error(P.error_word, kErrBadBlock);
      from = -1;
    }
    src_block[threadIdx.x] = from;
    src_row[threadIdx.x] = t % BS;
    dst_block[threadIdx.x] = to;
    if (from >= 0 && P.weights)
      P.weights[((size_t)to * P.num_kv_heads + g) * BS + i % BS] =
          P.weights[((size_t)from * P.num_kv_heads + g) * BS + t % BS];
  }
  __syncthreads();
  constexpr int U = 8;
  const int items = rows * 2 * PIECES;
  for (int at = threadIdx.x; at < items; at += U * kCompactThreads) {
    uint4 x[U];
    uint8_t* to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int it = at + u * kCompactThreads;
      to[u] = nullptr;
      if (it >= items) continue;
      const int piece = it % PIECES, kv = it / PIECES % 2, i = it / (2 * PIECES);
      if (src_block[i] < 0) continue;
      uint8_t* cache = kv ? P.v_cache : P.k_cache;
      const size_t from_tile = (size_t)src_block[i] * P.num_kv_heads + g;
      const size_t to_tile = (size_t)dst_block[i] * P.num_kv_heads + g;
      const int from_row = src_row[i], to_row = (i0 + i) % BS;
      if constexpr (KV == kKvInt4) {
        const size_t TILE = (size_t)BS * D * 9 / 16;
        if (piece < D / 32) {
          x[u] = *reinterpret_cast<const uint4*>(cache + from_tile * TILE + (piece * BS + from_row) * 16);
          to[u] = cache + to_tile * TILE + (piece * BS + to_row) * 16;
        } else {
          const uint8_t* s = cache + from_tile * TILE + BS * (D / 2) + from_row * (D / 16);
          uint8_t* o = cache + to_tile * TILE + BS * (D / 2) + to_row * (D / 16);
          if constexpr (D == 128)
            *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(s);
          else
            *reinterpret_cast<uint32_t*>(o) = *reinterpret_cast<const uint32_t*>(s);
        }
      } else {
        x[u] = *reinterpret_cast<const uint4*>(cache + ((from_tile * BS + from_row) * PIECES + piece) * 16);
        to[u] = cache + ((to_tile * BS + to_row) * PIECES + piece) * 16;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u]) *reinterpret_cast<uint4*>(to[u]) = x[u];
  }
}

}  // namespace pkd
