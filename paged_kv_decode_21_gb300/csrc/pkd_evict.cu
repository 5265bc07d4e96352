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
  __shared__ float row_mx[kFinishMaxRows], row_inv[kFinishMaxRows];
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
  merge_rows(P, bg, L, 0, P.rows, row_mx, row_inv);
  __syncthreads();
  if (!mine) return;
  float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
  if (P.decay != 0.f) old = *reinterpret_cast<const float4*>(o);
  const float before[4] = {old.x, old.y, old.z, old.w};
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  const float* s = P.scores + (size_t)bg * P.rows * P.score_stride + t;
  for (int i = 0; i < P.rows; ++i) {
    const float4 x = *reinterpret_cast<const float4*>(s + (size_t)i * P.score_stride);
    w[0] = fmaf(ex2_approx(x.x - row_mx[i]), row_inv[i], w[0]);
    w[1] = fmaf(ex2_approx(x.y - row_mx[i]), row_inv[i], w[1]);
    w[2] = fmaf(ex2_approx(x.z - row_mx[i]), row_inv[i], w[2]);
    w[3] = fmaf(ex2_approx(x.w - row_mx[i]), row_inv[i], w[3]);
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

__global__ void __launch_bounds__(kTokenSelectThreads) paged_kv_token_select_kernel(const TokenSelectParams P) {
  constexpr int NT = kTokenSelectThreads, NWARP = NT / 32;
  extern __shared__ uint32_t select_keys[];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];               // the bin, and what remains to be found in it
  __shared__ int above[NWARP], equal[NWARP];  // per warp's stretch
  const int g = blockIdx.x % P.num_kv_heads, b = blockIdx.x / P.num_kv_heads;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int L = max(0, clamped_len(P.context_lens, b, P.block_size, P.max_blocks_per_seq,
                                   g == 0 && tid == 0 ? P.error_word : nullptr));
  const int K = P.max_kept;
  int32_t* out = P.kept + (size_t)blockIdx.x * K;
  if (g == 0 && tid == 0) P.kept_lens[b] = min(L, K);
  if (L <= K) {
    for (int i = tid; i < K; i += NT) out[i] = i < L ? i : -1;
    return;
  }
  const int lo = P.sink, hi = L - P.recent;  // candidates; more of them than are needed, as L > K
  auto weigh = [&](int t) -> uint32_t {
    const int pb = P.block_tables[(size_t)b * P.max_blocks_per_seq + t / P.block_size];
    if (pb < 0 || pb >= P.num_blocks) {
      record_error(P.error_word, kErrBadBlock);
      return 0u;
    }
    return ordered_key(P.weights[((size_t)pb * P.num_kv_heads + g) * P.block_size + t % P.block_size]);
  };
  for (int t = lo + tid; t < hi && t < P.cached; t += NT) select_keys[t] = weigh(t);
  auto key = [&](int t) { return t < P.cached ? select_keys[t] : weigh(t); };
  const int need = K - P.sink - P.recent;
  uint32_t T = 0xFFFFFFFFu;
  uint32_t take = 0;  // of those equal to T, the first so many
  if (need > 0) {
    uint32_t prefix = 0;
    take = need;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += NT) hist[i] = 0;
      __syncthreads();
      for (int t = lo + tid; t < hi; t += NT) {
        const uint32_t k = key(t);
        if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp == 0) {
        // lane l has bins 255 - 8l .. 248 - 8l: from the largest down
        uint32_t n[8], mine = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) mine += n[k] = hist[255 - 8 * lane - k];
        uint32_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += x;
        }
        uint32_t before = upto - mine;
        if (before < take && upto >= take) {
          for (int k = 0; k < 8; ++k) {
            if (before + n[k] >= take) {
              found[0] = 255 - 8 * lane - k;
              found[1] = take - before;
              break;
            }
            before += n[k];
          }
        }
      }
      __syncthreads();
      prefix = (prefix << 8) | found[0];
      take = found[1];
    }
    T = prefix;
  }
  // The chosen: first and last ones, keys above T, the first `take` equal to T
  const int seg = ((L + NWARP - 1) / NWARP + 31) / 32 * 32;
  const int s0 = min(L, warp * seg), s1 = min(L, s0 + seg);
  auto kind = [&](int t) {  // 2: chosen, 1: equal to T, 0: neither
    if (t < lo || t >= hi) return 2;
    if (need == 0) return 0;
    const uint32_t k = key(t);
    return k > T ? 2 : (k == T ? 1 : 0);
  };
  __syncthreads();
  int na = 0, ne = 0;
  for (int t = s0 + lane; t < s1; t += 32) {
    const int k = kind(t);
    na += k == 2;
    ne += k == 1;
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
  const unsigned below = (1u << lane) - 1u;
  for (int t0 = s0; t0 < s1; t0 += 32) {
    const int t = t0 + lane;
    const int k = t < s1 ? kind(t) : 0;
    const unsigned ma = __ballot_sync(0xffffffffu, k == 2), me = __ballot_sync(0xffffffffu, k == 1);
    const int a = a0 + __popc(ma & below), e = e0 + __popc(me & below);
    if (k == 2 || (k == 1 && e < (int)take)) {
      const int at = a + min(e, (int)take);
      if (at < K) out[at] = t;
    }
    a0 += __popc(ma);
    e0 += __popc(me);
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

constexpr int kMaxTokens = 1 << 30;
constexpr int kRowTiles = 4;    // row tiles of a CTA of the first grid, where there is more than one
constexpr int kQueryTiles = 16; // and of Q in shared memory in the second

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
  p.row_tiles = p.rows <= 16 ? 1 : kRowTiles;
  p.row_chunks = (int)((p.rows + 16 * p.row_tiles - 1) / (16 * p.row_tiles));
  const long long bg = (long long)num_seqs * num_kv_heads;
  const long long want = 8LL * sms();  // CTAs
  long long part = 128;
  while (part < 4096 && bg * p.row_chunks * ((max_context_len + part - 1) / part) > want) part *= 2;
  p.part = (int)part;
  p.np = (int)std::max(1LL, (max_context_len + part - 1) / part);
  p.scores = p.rows <= 16;
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
  if (plan.row_tiles == 1)
    paged_weights_rows_kernel<KV, D, 1><<<(unsigned)grid, 32 * kWeightsWarps, 0, stream>>>(p);
  else
    paged_weights_rows_kernel<KV, D, kRowTiles><<<(unsigned)grid, 32 * kWeightsWarps, 0, stream>>>(p);
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
  auto smem = [](int tiles) { return tiles * ((D / 16) * 32 * 16 + 2 * 16 * 4); };
  // (the attribute belongs to the kernel: what the largest call needs, the same for all)
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
  p.scale_log2 = scale * k_scale * 1.4426950408889634f * (kv_type == PKD_KV_INT4 ? kInt4Unscale : 1.f);
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
      max_context_len < 0 || max_kept < 1 || sink_tokens < 0 || recent_tokens < 0 ||
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
  p.cached = max_context_len <= max_kept ? 0 : std::min(max_context_len, kMostCached);
  if (failed(cudaFuncSetAttribute(paged_kv_token_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  4 * kMostCached)))
    return PKD_ERR_LAUNCH;
  paged_kv_token_select_kernel<<<(unsigned)grid, kTokenSelectThreads, 4 * p.cached, stream>>>(p);
  return launched();
}

pkd_status paged_kv_compact(void* k_cache, void* v_cache, float* weights, const int32_t* block_tables,
                            const int32_t* context_lens, const int32_t* kept, const int32_t* kept_lens,
                            const int32_t* new_tables, int num_seqs, int num_kv_heads, int head_dim, int block_size,
                            int num_blocks, int max_blocks_per_seq, int max_kept, int max_new_blocks, int kv_type,
                            int* error_word, cudaStream_t stream) {
  if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0 || max_kept < 1 || max_new_blocks < 1)
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
  p.chunks = (int)((most + kCompactRows - 1) / kCompactRows);
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
