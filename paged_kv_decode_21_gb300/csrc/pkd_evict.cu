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
  __shared__ uint32_t hist[kSelectBins];
  __shared__ uint32_t warp_bins[NWARP];
  __shared__ uint32_t found[2];  // the bin, and what remains to be found in it
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
      }
    }
  } else {
    for (int t = tid; t < (held + 3) / 4 * 4; t += NT) select_keys[t] = weigh(t);
  }
  // keys of tokens 4 q .. 4 q + 3
  auto quad = [&](int q, uint32_t (&k)[4]) {
    if (4 * q + 4 <= P.cached) {
      const uint4 x = *reinterpret_cast<const uint4*>(select_keys + 4 * q);
      k[0] = x.x; k[1] = x.y; k[2] = x.z; k[3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i] = weigh(4 * q + i);
    }
  };
  const int need = K - P.sink - P.recent;
  uint32_t T = 0xFFFFFFFFu;
  uint32_t take = 0;  // of those equal to T, the first so many
  if (need > 0) {
    uint32_t prefix = 0;
    take = need;
    // bits 31..21, 20..10, 9..0: the first pass tells signs, exponents and two
    // more bits apart, so that few of a warp's additions meet in one bin
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kSelectBins; i += NT) hist[i] = 0;
      __syncthreads();
      for (int q = tid; 4 * q < hi; q += NT) {
        uint32_t k[4];
        quad(q, k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (pass == 0 || (k[i] >> (shift + bits)) == prefix)
            atomicAdd(&hist[(k[i] >> shift) & ((1u << bits) - 1)], 1u);
      }
      __syncthreads();
      // From the largest bin down: warp w has bins kSelectBins - 1 - 32 PER w
      // downwards, its lane l the PER of them from 32 PER w + PER l on.
      uint32_t n[PER], mine = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) mine += n[k] = hist[kSelectBins - 1 - (warp * 32 + lane) * PER - k];
      uint32_t upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += x;
      }
      if (lane == 31) warp_bins[warp] = upto;
      __syncthreads();
      uint32_t before = upto - mine;
      for (int w = 0; w < warp; ++w) before += warp_bins[w];
      if (before < take && before + mine >= take) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          if (before < take && before + n[k] >= take) {
            found[0] = kSelectBins - 1 - (warp * 32 + lane) * PER - k;
            found[1] = take - before;
          }
          before += n[k];
        }
      }
      __syncthreads();
      prefix = (prefix << bits) | found[0];
      take = found[1];
    }
    T = prefix;
  }
  // The chosen: first and last ones, keys above T, the first `take` equal to T.
  // Per quad: 2 bits a token, 2: chosen, 1: equal to T
  const int seg = ((L + NWARP - 1) / NWARP + 127) / 128 * 32;  // quads a warp
  const int s0 = min((L + 3) / 4, warp * seg), s1 = min((L + 3) / 4, s0 + seg);
  auto kinds = [&](int q) {
    uint32_t k[4], x = 0;
    const int t = 4 * q;
    if (need > 0 && t < hi && t + 4 > lo) {
      quad(q, k);
#pragma unroll
      for (int i = 0; i < 4; ++i) x |= (k[i] > T ? 2u << (2 * i) : 0u) | (k[i] == T ? 1u << (2 * i) : 0u);
    }
    if (t < lo || t + 4 > hi) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t + i < lo || t + i >= hi) x = (x & ~(3u << (2 * i))) | (t + i < L ? 2u << (2 * i) : 0u);
      }
    }
    return x;
  };
  auto counts = [](uint32_t x) { return (uint32_t)__popc(x & 0xAAu) | ((uint32_t)__popc(x & 0x55u) << 16); };
  __syncthreads();
  int na = 0, ne = 0;
  for (int q = s0 + lane; q < s1; q += 32) {
    const uint32_t x = kinds(q);
    na += __popc(x & 0xAAu);
    ne += __popc(x & 0x55u);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    na += __shfl_xor_sync(0xffffffffu, na, d);
    ne += __shfl_xor_sync(0xffffffffu, ne, d);
  }
  if (lane == 0) {
    above[warp] = na;
    equal[warp] = ne;
  }
  __syncthreads();
  int a0 = 0, e0 = 0;  // before this warp's stretch
  for (int w = 0; w < warp; ++w) {
    a0 += above[w];
    e0 += equal[w];
  }
  for (int q0 = s0; q0 < s1; q0 += 32) {
    const uint32_t x = q0 + lane < s1 ? kinds(q0 + lane) : 0u;
    const uint32_t mine = counts(x);
    uint32_t upto = mine;  // both counts at once: at most 128 each
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += y;
    }
    int a = a0 + (int)((upto - mine) & 0xFFFFu), e = e0 + (int)((upto - mine) >> 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t kind = (x >> (2 * i)) & 3u;
      if (kind == 2u || (kind == 1u && e < (int)take)) {
        const int at = a + min(e, (int)take);
        if (at < K) out[at] = 4 * (q0 + lane) + i;
      }
      a += kind == 2u;
      e += kind == 1u;
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
// serves a shape.
WeightsPlan plan_weights(int num_seqs, int q_len, int num_q_heads, int num_kv_heads, int max_context_len) {
  WeightsPlan p{};
  p.rows = (long long)q_len * (num_q_heads / num_kv_heads);
  p.row_tiles = p.rows <= 8 ? 0 : (p.rows <= 16 ? 1 : kRowTiles);
  p.row_chunks = p.row_tiles < 2 ? 1 : (int)((p.rows + 16 * p.row_tiles - 1) / (16 * p.row_tiles));
  const long long bg = (long long)num_seqs * num_kv_heads;
  long long part = 128;
  const long long want = (p.rows <= kFinishMaxRows ? 16LL : 4LL) * sms();  // CTAs
  while (part < 4096 && bg * p.row_chunks * ((max_context_len + part - 1) / part) > want) part *= 2;
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
  const float s = scale * k_scale * 1.4426950408889634f * (kv_type == PKD_KV_INT4 ? kInt4Unscale : 1.f);
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
      max_context_len < 0 || max_context_len > kMaxTokens || max_kept < 1 || max_kept > kMaxTokens || sink_tokens < 0 || recent_tokens < 0 ||
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
  const int rows = compact_rows(kv, head_dim);
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
