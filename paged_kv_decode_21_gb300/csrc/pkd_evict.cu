// pkd_evict.cu -- C entry points of the gathered attention weights, the choice
// of tokens and the copy of kept rows: argument checks, the split and launches.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/paged_decode.h"
#include "pkd_evict.cuh"

namespace pkd {

__global__ void __launch_bounds__(kWeightsFinishThreads) paged_weights_scores_kernel(const WeightsParams P,
                                                                                     int chunks) {
  __shared__ float row_off[kFinishMaxRows];
  const int chunk = blockIdx.x % chunks, bg = blockIdx.x / chunks;
  const int g = bg % P.num_kv_heads, b = bg / P.num_kv_heads;
  const int L = min(clamped_len(P.context_lens, b, P.block_size, P.max_blocks_per_seq, nullptr),
                    (int)min(P.score_stride, 0x7fffffffLL));
  const int t = 4 * (chunk * kWeightsFinishThreads + (int)threadIdx.x);
  if (4 * chunk * kWeightsFinishThreads >= L) return;
  const int start = P.start_lens ? P.start_lens[b] : L;
  int pb = -1;
  if (t < L) pb = P.block_tables[(size_t)b * P.max_blocks_per_seq + t / P.block_size];
  const bool mine = pb >= 0 && pb < P.num_blocks;
  float* o = P.weights + ((size_t)(mine ? pb : 0) * P.num_kv_heads + g) * P.block_size + t % P.block_size;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the old weights and the first rows' scores along with the statistics
  constexpr int U = 4;
  const float* s = P.scores + (size_t)bg * P.rows * P.score_stride + t;
  float4 old = make_float4(0.f, 0.f, 0.f, 0.f), x[U];
  if (mine && P.decay != 0.f) old = *reinterpret_cast<const float4*>(o);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (mine && u < P.rows) x[u] = *reinterpret_cast<const float4*>(s + (size_t)u * P.score_stride);
  merge_rows(P, bg, L, 0, P.rows, row_off, kWeightsFinishThreads);
  __syncthreads();
  if (!mine) return;
  const float before[4] = {old.x, old.y, old.z, old.w};
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = 0; i0 < P.rows; i0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= P.rows) break;
      if (i0 > 0) x[u] = *reinterpret_cast<const float4*>(s + (size_t)(i0 + u) * P.score_stride);
      const float off = row_off[i0 + u];
      w[0] += ex2_approx(x[u].x - off);
      w[1] += ex2_approx(x[u].y - off);
      w[2] += ex2_approx(x[u].z - off);
      w[3] += ex2_approx(x[u].w - off);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (t + k < start && P.decay != 0.f) w[k] = fmaf(P.decay, before[k], w[k]);
  if (t + 4 <= L) {
    *reinterpret_cast<float4*>(o) = make_float4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (t + k < L) o[k] = w[k];
  }
}

constexpr int kMaxTokens = 1 << 30;  // the longest context, and the most tokens kept
constexpr int kSelectBins = 2048;
template <int NT>
__global__ void __launch_bounds__(NT) paged_kv_token_select_kernel(const TokenSelectParams P) {
  constexpr int NWARP = NT / 32, PER = kSelectBins / NWARP / 32;  // bins a lane sums
  extern __shared__ __align__(16) uint32_t select_keys[];
  __shared__ uint32_t hist[2][kSelectBins];  // in turns, so that one is cleared while the other is filled
  __shared__ uint32_t warp_bins[NWARP];
  __shared__ uint32_t found[3];  // the bin, what remains to be found in it, and how many are in it
  __shared__ int above[NWARP], equal[NWARP];  // per warp's stretch
  const int g = blockIdx.x % P.num_kv_heads, b = blockIdx.x / P.num_kv_heads;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  // (counts of four tokens at a time stay in 32 bits)
  const int L = min(kMaxTokens, max(0, clamped_len(P.context_lens, b, P.block_size, P.max_blocks_per_seq,
                                                   g == 0 && tid == 0 ? P.error_word : nullptr)));
  const int K = P.max_kept;
  int32_t* out = P.kept + (size_t)blockIdx.x * K;
  if (g == 0 && tid == 0) P.kept_lens[b] = min(L, K);
  if (L <= K) {
    for (int i = tid; i < K; i += NT) out[i] = i < L ? i : -1;
    return;
  }
  for (int i = tid; i < kSelectBins; i += NT) hist[0][i] = 0;
  __syncthreads();
  const int lo = P.sink, hi = L - P.recent;  // candidates; more of them than are needed, as L > K
  const int32_t* table = P.block_tables + (size_t)b * P.max_blocks_per_seq;
  auto place = [&](int t) -> const float* {  // of token t's weight, or null
    const int pb = table[t / P.block_size];
    if (pb < 0 || pb >= P.num_blocks) {
      record_error(P.error_word, kErrBadBlock);
      return nullptr;
    }
    return P.weights + ((size_t)pb * P.num_kv_heads + g) * P.block_size + t % P.block_size;
  };
  // A token's key; 0 for the first and last ones, which are taken anyway: they
  // count in the lowest bin, where none that is looked for lies but tokens
  // without a block, and those are told apart again below.
  auto weigh = [&](int t) -> uint32_t {
    if (t < lo || t >= hi) return 0u;
    const float* p = place(t);
    return p ? ordered_key(*p) : 0u;
  };
  // Every key counts in the bins of its uppermost bits as it comes.
  auto count = [&](uint32_t key) { atomicAdd(&hist[0][key >> 21], 1u); };
  const int held = min(L, P.cached);
  if (P.block_shift >= 0) {
    constexpr int U = 8;
    const float* base = P.weights + (size_t)g * P.block_size;
    const size_t stride = (size_t)P.num_kv_heads << P.block_shift;
    for (int q0 = tid; 4 * q0 < held; q0 += U * NT) {
      int pb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = 4 * (q0 + u * NT);
        pb[u] = t < held ? table[t >> P.block_shift] : -1;
      }
      float4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = 4 * (q0 + u * NT);
        if ((uint32_t)pb[u] < (uint32_t)P.num_blocks)
          x[u] = *reinterpret_cast<const float4*>(base + (size_t)(uint32_t)pb[u] * stride +
                                                  (t & (P.block_size - 1)));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = 4 * (q0 + u * NT);
        if (t >= held) continue;
        uint4 k = make_uint4(0u, 0u, 0u, 0u);
        if ((uint32_t)pb[u] < (uint32_t)P.num_blocks)
          k = make_uint4(ordered_key(x[u].x), ordered_key(x[u].y), ordered_key(x[u].z), ordered_key(x[u].w));
        else
          record_error(P.error_word, kErrBadBlock);
        if (t < lo || t + 4 > hi) {
          if (t < lo || t >= hi) k.x = 0u;
          if (t + 1 < lo || t + 1 >= hi) k.y = 0u;
          if (t + 2 < lo || t + 2 >= hi) k.z = 0u;
          if (t + 3 < lo || t + 3 >= hi) k.w = 0u;
        }
        *reinterpret_cast<uint4*>(select_keys + t) = k;
        count(k.x);
        count(k.y);
        count(k.z);
        count(k.w);
      }
    }
  } else {
    for (int t = tid; t < (held + 3) / 4 * 4; t += NT) count(select_keys[t] = weigh(t));
  }
  auto one = [&](int t) { return t < P.cached ? select_keys[t] : weigh(t); };
  const int need = K - P.sink - P.recent;
  uint32_t T = 0xFFFFFFFFu;
  uint32_t take = 0;  // of those equal to T, the first so many
  bool ties = false;
  if (need > 0) {
    for (int t = P.cached + tid; t < hi; t += NT) count(weigh(t));
    uint32_t prefix = 0;
    take = need;
    // bits 31..21, 20..10, 9..0: the first pass tells signs, exponents and two
    // more bits apart, so that few of a warp's additions meet in one bin
    for (int pass = 0; pass < 3; ++pass) {
      uint32_t* bins = hist[pass % 2];
      const int bits = pass == 2 ? 10 : 11;
      if (pass > 0) {
        const int shift = pass == 1 ? 10 : 0;
        auto look = [&](uint32_t k) {
          if ((k >> (shift + bits)) == prefix) atomicAdd(&bins[(k >> shift) & ((1u << bits) - 1)], 1u);
        };
        const uint4* quads = reinterpret_cast<const uint4*>(select_keys);
        const int nq = (min(hi, P.cached) + 3) / 4;
        constexpr int U = 4;
        for (int q0 = tid; q0 < nq; q0 += U * NT) {
          uint4 k[U];
#pragma unroll
          for (int u = 0; u < U; ++u) k[u] = quads[min(q0 + u * NT, nq - 1)];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (q0 + u * NT >= nq) break;
            look(k[u].x);
            look(k[u].y);
            look(k[u].z);
            look(k[u].w);
          }
        }
        for (int t = P.cached + tid; t < hi; t += NT) look(weigh(t));
      }
      __syncthreads();
      // From the largest bin down: warp w has bins kSelectBins - 1 - 32 PER w
      // downwards, its lane l the PER of them from 32 PER w + PER l on.
      uint32_t n[PER], mine = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) mine += n[k] = bins[kSelectBins - 1 - (warp * 32 + lane) * PER - k];
      for (int i = tid; i < kSelectBins; i += NT) hist[(pass + 1) % 2][i] = 0;
      uint32_t upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += x;
      }
      if (lane == 31) warp_bins[warp] = upto;
      __syncthreads();
      uint32_t before = upto - mine + __reduce_add_sync(0xffffffffu, lane < warp ? warp_bins[lane] : 0u);
      if (before < take && before + mine >= take) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          if (before < take && before + n[k] >= take) {
            found[0] = kSelectBins - 1 - (warp * 32 + lane) * PER - k;
            found[1] = take - before;
            found[2] = n[k];
          }
          before += n[k];
        }
      }
      __syncthreads();
      prefix = (prefix << bits) | found[0];
      take = found[1];
      // Where the whole bin is taken, the bits below and equal keys need no telling
      // apart: as a rule after two passes or three.
      ties = found[2] != take || prefix == 0;
      if (!ties) {
        T = (prefix << (pass == 0 ? 21 : (pass == 1 ? 10 : 0))) - 1;
        take = 0;
        break;
      }
    }
    if (ties) T = prefix;
  }
  // The chosen: first and last ones, keys above T, the first `take` equal to T.
  // Every warp counts those of its stretch, then writes them behind those before
  // it.  A lane has 32 neighbouring tokens as a word of bits (votes over keys that
  // lie side by side): counting and ranking by token instead took four times as
  // long, bound by its bit counts.
  const int seg = ((L + NWARP - 1) / NWARP + 31) / 32 * 32;  // tokens a warp
  const int s0 = min(L, warp * seg), s1 = min(L, s0 + seg);
  // of tokens t0 + 32 lane ..: wa those above T, and the first and last ones, we those equal to T
  auto words = [&](int t0, uint32_t& wa, uint32_t& we) {
    wa = we = 0;
    const int groups = min(32, (s1 - t0 + 31) / 32);
    constexpr int G = 4;
    for (int i0 = 0; i0 < groups; i0 += G) {
      const int t = t0 + 32 * i0 + lane;
      uint32_t k[G];
      if (t - lane >= lo && t - lane + 32 * G <= min(hi, P.cached)) {
#pragma unroll
        for (int i = 0; i < G; ++i) k[i] = select_keys[t + 32 * i];
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const uint32_t ma = __ballot_sync(0xffffffffu, k[i] > T);
          if (lane == i0 + i) wa = ma;
        }
        if (ties) {
#pragma unroll
          for (int i = 0; i < G; ++i) {
            const uint32_t me = __ballot_sync(0xffffffffu, k[i] == T);
            if (lane == i0 + i) we = me;
          }
        }
      } else {
        for (int i = 0; i < G; ++i) {
          const int at = t + 32 * i;
          const bool inside = at >= lo && at < hi;
          const uint32_t key = inside ? one(at) : 0u;
          const uint32_t ma = __ballot_sync(0xffffffffu, inside ? key > T : at < L),
                         me = __ballot_sync(0xffffffffu, ties && inside && key == T);
          if (lane == i0 + i) {
            wa = ma;
            we = me;
          }
        }
      }
    }
    // (groups behind the stretch's last, of the last four, are the next warp's)
    if (lane >= groups) wa = we = 0;
  };
  uint32_t wa = 0, we = 0;
  int na = 0, ne = 0;
  for (int t0 = s0; t0 < s1; t0 += 1024) {
    words(t0, wa, we);
    na += __popc(wa);
    ne += __popc(we);
  }
  na = (int)__reduce_add_sync(0xffffffffu, (unsigned)na);
  ne = (int)__reduce_add_sync(0xffffffffu, (unsigned)ne);
  if (lane == 0) {
    above[warp] = na;
    equal[warp] = ne;
  }
  __syncthreads();
  // before this warp's stretch
  int a0 = (int)__reduce_add_sync(0xffffffffu, lane < warp ? (unsigned)above[lane] : 0u);
  int e0 = (int)__reduce_add_sync(0xffffffffu, lane < warp ? (unsigned)equal[lane] : 0u);
  for (int t0 = s0; t0 < s1; t0 += 1024) {
    if (seg > 1024) words(t0, wa, we);
    const uint32_t mine = (uint32_t)__popc(wa) | ((uint32_t)__popc(we) << 16);
    uint32_t upto = mine;  // both counts at once: at most 1024 each
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += y;
    }
    const int e = e0 + (int)((upto - mine) >> 16);
    const int at = a0 + (int)((upto - mine) & 0xFFFFu) + min(e, (int)take);
    uint32_t same = we;
    for (int over = e + __popc(we) - (int)take; over > 0 && same; --over) same &= ~(0x80000000u >> __clz(same));
    const uint32_t w = wa | same;
    // Few to a word: every lane its own, one after the other.  Many: the warp a word
    // at a time (1024 of 1150 tokens, 256 rows: 7.9 us instead of 9.6; but 2048 of
    // 8000-32768 47.0 instead of 44.1).
    if (K < L / 4) {
      for (uint32_t x = w, to = at; x; x &= x - 1, ++to)
        if ((int)to < K) out[to] = t0 + 32 * lane + __ffs(x) - 1;
    } else {
      const int groups = min(32, (s1 - t0 + 31) / 32);
#pragma unroll 4
      for (int i = 0; i < groups; ++i) {
        const uint32_t x = __shfl_sync(0xffffffffu, w, i);
        const int to = __shfl_sync(0xffffffffu, at, i) + __popc(x & ((1u << lane) - 1));
        if ((x >> lane & 1) && to < K) out[to] = t0 + 32 * i + lane;
      }
    }
    const uint32_t sum = __shfl_sync(0xffffffffu, upto, 31);
    a0 += (int)(sum & 0xFFFFu);
    e0 += (int)(sum >> 16);
  }
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
pkd_status launched() { return cudaGetLastError() == cudaSuccess ? PKD_OK : PKD_ERR_LAUNCH; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int sms() {
  int n = 0, dev = 0;
  if (failed(cudaGetDevice(&dev)) || failed(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) || n <= 0)
    n = 148;
  return n;
}

constexpr unsigned long long kWaitBudgetNs = 100ull * 1000ull * 1000ull;  // 100 ms per bounded wait
constexpr int kRowTiles = 8;     // row tiles of a CTA of the first grid, where there is more than one
constexpr int kQueryTiles = 16;  // and of Q in shared memory in the second

struct WeightsPlan {
  long long rows;   // per (b, g)
  int part, np, row_tiles, row_chunks;
  bool scores;
  long long score_stride;
  size_t stats, total;
};

pkd_status check_weights(int num_seqs, int q_len, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                         int max_context_len) {
  if (num_seqs < 0 || q_len < 1 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      max_context_len < 0 || max_context_len > kMaxTokens || num_q_heads % num_kv_heads != 0)
    return PKD_ERR_SHAPE;
  if (num_q_heads / num_kv_heads > 8 || (head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32))
    return PKD_ERR_UNSUPPORTED;
  if ((long long)num_seqs * q_len * num_q_heads > 0x7fffffffLL) return PKD_ERR_SHAPE;
  return PKD_OK;
}

// The split does not depend on the cache's type, so that one workspace size
// serves a shape: partitions of 128 to 4096 tokens that make four CTAs an SM of
// the second grid, whose CTAs take every row of their tokens (the first has one for
// every chunk of rows besides; counted by those, 448 rows of 32 (b, g) with 4000-16384
// tokens made one second-grid CTA for every SM: 702 us instead of 282, 65536 rows of 2
// with 8192 tokens 109 ms instead of 10).  Twice or three times as many CTAs: 112 rows
// 91 us instead of 89, 448 rows 291 instead of 282; half as many about 140 and 433.
// (128 tokens only where the first grid stays within that too: 256 rows of 8 (b, g) with
// 8192 tokens 74 us, with 256 tokens 56, as every CTA loads all the queries.)
// Sixteen CTAs an SM where rows are few, as those read and wait more.
//
// Scores are kept for up to 16 rows, whatever a key weighs: 8 bytes a row and
// token written and read against reading the keys again, 72 bytes of 128 dims in 4
// bits.  Past 9 rows the scores are the more bytes, but the second reading is bound
// by its products, not by bytes.  64 x 512-4096 tokens x 8 heads, scores against keys
// again: 4 bits, 4 rows 48 and 129 us, 16 rows 70 and 130 (64 dims 56 and 107);
// E4M3 68 and 119, fp16 87 and 160; 16 x 16K-32K tokens, 16 rows, 4 bits 161 and 259.
WeightsPlan plan_weights(int num_seqs, int q_len, int num_q_heads, int num_kv_heads, int max_context_len) {
  WeightsPlan p{};
  p.rows = (long long)q_len * (num_q_heads / num_kv_heads);
  p.row_tiles = p.rows <= 8 ? 0 : (p.rows <= 16 ? 1 : kRowTiles);
  p.row_chunks = p.row_tiles < 2 ? 1 : (int)((p.rows + 16 * p.row_tiles - 1) / (16 * p.row_tiles));
  const long long bg = (long long)num_seqs * num_kv_heads;
  long long part = 128;
  const long long want = (p.rows <= kFinishMaxRows ? 16LL : 4LL) * sms();  // CTAs
  auto ctas = [&](long long each) { return each * ((max_context_len + part - 1) / part); };
  while (part < 4096 && (ctas(bg) > want || (part < 256 && ctas(bg * p.row_chunks) > want))) part *= 2;
  p.part = (int)part;
  p.np = (int)std::max(1LL, (max_context_len + part - 1) / part);
  p.scores = p.rows <= kFinishMaxRows;
  p.score_stride = (long long)round_up((size_t)p.np * p.part, 64);
  p.stats = round_up((size_t)bg * p.np * p.rows * sizeof(float), 256);
  p.total = 2 * p.stats + (p.scores ? round_up((size_t)bg * p.rows * p.score_stride * sizeof(float), 256) : 0);
  return p;
}

template <int KV, int D>
pkd_status launch_weights(const WeightsPlan& plan, WeightsParams p, cudaStream_t stream) {
  const long long bg = (long long)p.num_seqs * p.num_kv_heads;
  const long long grid = bg * plan.np * plan.row_chunks;
  if (grid > 0x7fffffffLL) return PKD_ERR_SHAPE;
  auto smem = [](int tiles) { return tiles * ((D / 16) * 32 * 16 + 16 * 4); };
  // (the attributes belong to the kernels: what the largest call needs, the same for all)
  if (plan.row_tiles < 2) {
    auto* fn = plan.row_tiles == 0 ? paged_weights_few_kernel<KV, D, 1> : paged_weights_few_kernel<KV, D, 2>;
    constexpr int bytes = WeightsRing<KV, D>::SMEM;
    if (failed(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes))) return PKD_ERR_LAUNCH;
    fn<<<(unsigned)grid, 32 * kWeightsWarps, bytes, stream>>>(p, kWaitBudgetNs);
  } else {
    paged_weights_rows_kernel<KV, D, kRowTiles><<<(unsigned)grid, 32 * kWeightsWarps, smem(kRowTiles), stream>>>(p);
  }
  if (cudaGetLastError() != cudaSuccess) return PKD_ERR_LAUNCH;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (plan.scores) {
    const int chunks = (int)((plan.score_stride + 4 * kWeightsFinishThreads - 1) / (4 * kWeightsFinishThreads));
    if (bg * chunks > 0x7fffffffLL) return PKD_ERR_SHAPE;
    cfg.gridDim = dim3((unsigned)(bg * chunks));
    cfg.blockDim = dim3(kWeightsFinishThreads);
    return failed(cudaLaunchKernelEx(&cfg, paged_weights_scores_kernel, p, chunks)) ? PKD_ERR_LAUNCH : PKD_OK;
  }
  auto* fn = paged_weights_keys_kernel<KV, D>;
  if (failed(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem(kQueryTiles))))
    return PKD_ERR_LAUNCH;
  p.q_tiles = (int)std::min<long long>(kQueryTiles, (plan.rows + 15) / 16);
  cfg.gridDim = dim3((unsigned)(bg * plan.np));
  cfg.blockDim = dim3(32 * kWeightsWarps);
  cfg.dynamicSmemBytes = smem(p.q_tiles);
  return failed(cudaLaunchKernelEx(&cfg, fn, p)) ? PKD_ERR_LAUNCH : PKD_OK;
}

}  // namespace
}  // namespace pkd

using namespace pkd;

extern "C" {

size_t paged_kv_attention_weights_workspace_size(int num_seqs, int q_len, int num_q_heads, int num_kv_heads,
                                                 int head_dim, int block_size, int max_context_len) {
  if (check_weights(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len) != PKD_OK)
    return 0;
  if (num_seqs == 0 || max_context_len == 0) return 0;
  return plan_weights(num_seqs, q_len, num_q_heads, num_kv_heads, max_context_len).total;
}

pkd_status paged_kv_attention_weights(const void* q, const void* k_cache, const int32_t* block_tables,
                                      const int32_t* context_lens, const int32_t* start_lens, float* weights,
                                      int num_seqs, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                                      int block_size, int num_blocks, int max_blocks_per_seq, int max_context_len,
                                      float scale, float k_scale, float decay, int kv_type, void* workspace,
                                      size_t workspace_bytes, int* error_word, cudaStream_t stream) {
  const pkd_status st =
      check_weights(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len);
  if (st != PKD_OK) return st;
  if (num_blocks <= 0 || max_blocks_per_seq <= 0 ||
      (long long)max_context_len > (long long)max_blocks_per_seq * block_size)
    return PKD_ERR_SHAPE;
  if (!std::isfinite(scale) || !std::isfinite(k_scale) || k_scale <= 0.f || !(decay >= 0.f && decay <= 1.f))
    return PKD_ERR_SHAPE;
  if (kv_type < PKD_KV_FP16 || kv_type > PKD_KV_INT4) return PKD_ERR_SHAPE;
  const float s = scale * k_scale * 1.4426950408889634f * (kv_type == PKD_KV_INT4 ? kInt4Unscale : 1.f);
  if (!std::isfinite(s)) return PKD_ERR_SHAPE;
  if (num_seqs == 0 || max_context_len == 0) return PKD_OK;
  if (!q || !k_cache || !block_tables || !context_lens || !weights) return PKD_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(weights, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(start_lens, 4) || !aligned(error_word, 4))
    return PKD_ERR_ALIGN;
  const WeightsPlan plan = plan_weights(num_seqs, q_len, num_q_heads, num_kv_heads, max_context_len);
  if (!workspace) return PKD_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return PKD_ERR_ALIGN;
  if (workspace_bytes < plan.total) return PKD_ERR_WORKSPACE;
  WeightsParams p{};
  p.q = static_cast<const __half*>(q);
  p.k_cache = k_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.start_lens = start_lens;
  p.weights = weights;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.row_max = reinterpret_cast<float*>(ws);
  p.row_sum = reinterpret_cast<float*>(ws + plan.stats);
  p.scores = plan.scores ? reinterpret_cast<float*>(ws + 2 * plan.stats) : nullptr;
  p.score_stride = plan.score_stride;
  p.num_seqs = num_seqs;
  p.q_len = q_len;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.rows = (int)plan.rows;
  p.part = plan.part;
  p.np = plan.np;
  p.row_chunks = plan.row_chunks;
  p.q_sign = s < 0.f ? 0x80008000u : 0u;
  // (a scale of 0, equal weights: one too small to tell, so that -inf times it stays -inf)
  p.scale_log2 = std::max(std::fabs(s), 1e-30f);
  p.decay = decay;
  p.error_word = error_word;
  p.bases = kInt4Bases;
  switch (kv_type) {
    case PKD_KV_FP16:
      return head_dim == 128 ? launch_weights<kKvFp16, 128>(plan, p, stream)
                             : launch_weights<kKvFp16, 64>(plan, p, stream);
    case PKD_KV_E4M3:
      return head_dim == 128 ? launch_weights<kKvE4m3, 128>(plan, p, stream)
                             : launch_weights<kKvE4m3, 64>(plan, p, stream);
    default:
      return head_dim == 128 ? launch_weights<kKvInt4, 128>(plan, p, stream)
                             : launch_weights<kKvInt4, 64>(plan, p, stream);
  }
}

pkd_status paged_kv_token_select(const float* weights, const int32_t* block_tables, const int32_t* context_lens,
                                 int32_t* kept, int32_t* kept_lens, int num_seqs, int num_kv_heads, int block_size,
                                 int num_blocks, int max_blocks_per_seq, int max_context_len, int max_kept,
                                 int sink_tokens, int recent_tokens, int* error_word, cudaStream_t stream) {
  if (num_seqs < 0 || num_kv_heads <= 0 || block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 ||
      max_context_len < 0 || max_context_len > kMaxTokens || max_kept < 1 || max_kept > kMaxTokens ||
      sink_tokens < 0 || recent_tokens < 0 ||
      (long long)sink_tokens + recent_tokens > max_kept ||
      (long long)max_context_len > (long long)max_blocks_per_seq * block_size)
    return PKD_ERR_SHAPE;
  const long long grid = (long long)num_seqs * num_kv_heads;
  if (grid > 0x7fffffffLL) return PKD_ERR_SHAPE;
  if (num_seqs == 0) return PKD_OK;
  if (!weights || !block_tables || !context_lens || !kept || !kept_lens) return PKD_ERR_NULL;
  if (!aligned(weights, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(kept, 4) ||
      !aligned(kept_lens, 4) || !aligned(error_word, 4))
    return PKD_ERR_ALIGN;
  TokenSelectParams p{};
  p.weights = weights;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.kept = kept;
  p.kept_lens = kept_lens;
  p.num_seqs = num_seqs;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_kept = max_kept;
  p.sink = sink_tokens;
  p.recent = recent_tokens;
  p.error_word = error_word;
  // keys of longer contexts are read again in every pass
  constexpr int kMostCached = 48 * 1024;
  p.cached = max_context_len <= max_kept ? 0 : (int)round_up((size_t)std::min(max_context_len, kMostCached), 4);
  p.block_shift = -1;
  if (block_size % 4 == 0 && (block_size & (block_size - 1)) == 0 && aligned(weights, 16))
    for (p.block_shift = 2; 1 << p.block_shift < block_size;) ++p.block_shift;
  // a thread has one round of eight loads of four keys, up to 1024 of them
  const bool wide = p.cached > 8192;
  auto* fn = wide ? paged_kv_token_select_kernel<1024> : paged_kv_token_select_kernel<256>;
  if (failed(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kMostCached)))
    return PKD_ERR_LAUNCH;
  fn<<<(unsigned)grid, wide ? 1024 : 256, 4 * p.cached, stream>>>(p);
  return launched();
}

pkd_status paged_kv_compact(void* k_cache, void* v_cache, float* weights, const int32_t* block_tables,
                            const int32_t* context_lens, const int32_t* kept, const int32_t* kept_lens,
                            const int32_t* new_tables, int num_seqs, int num_kv_heads, int head_dim, int block_size,
                            int num_blocks, int max_blocks_per_seq, int max_kept, int max_new_blocks, int kv_type,
                            int* error_word, cudaStream_t stream) {
  if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0 || max_kept < 1 || max_kept > kMaxTokens || max_new_blocks < 1)
    return PKD_ERR_SHAPE;
  if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32)) return PKD_ERR_UNSUPPORTED;
  if (kv_type < PKD_KV_FP16 || kv_type > PKD_KV_INT4) return PKD_ERR_SHAPE;
  if (num_seqs == 0) return PKD_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !kept || !kept_lens || !new_tables)
    return PKD_ERR_NULL;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(weights, 4) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(kept, 4) || !aligned(kept_lens, 4) || !aligned(new_tables, 4) ||
      !aligned(error_word, 4))
    return PKD_ERR_ALIGN;
  CompactParams p{};
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.weights = weights;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.kept = kept;
  p.kept_lens = kept_lens;
  p.new_tables = new_tables;
  p.num_seqs = num_seqs;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_kept = max_kept;
  p.max_new_blocks = max_new_blocks;
  p.error_word = error_word;
  const long long most = std::min<long long>(max_kept, (long long)max_new_blocks * block_size);
  const KvType kv = kv_type == PKD_KV_FP16 ? kKvFp16 : (kv_type == PKD_KV_E4M3 ? kKvE4m3 : kKvInt4);
  const int rows = compact_rows(kv, head_dim) * (kCompactThreads / 32);
  p.chunks = (int)((most + rows - 1) / rows);
  const long long grid = (long long)num_seqs * num_kv_heads * p.chunks;
  if (grid > 0x7fffffffLL) return PKD_ERR_SHAPE;
#define PKD_COMPACT(KV_) (head_dim == 128 ? paged_kv_compact_kernel<KV_, 128> : paged_kv_compact_kernel<KV_, 64>)
  auto* fn = kv_type == PKD_KV_FP16   ? PKD_COMPACT(kKvFp16)
             : kv_type == PKD_KV_E4M3 ? PKD_COMPACT(kKvE4m3)
                                      : PKD_COMPACT(kKvInt4);
#undef PKD_COMPACT
  fn<<<(unsigned)grid, kCompactThreads, 0, stream>>>(p);
  return launched();
}

}  // extern "C"
