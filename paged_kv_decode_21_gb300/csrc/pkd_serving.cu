// pkd_serving.cu -- C entry points of the rotated append, the block bounds and
// the block choice: argument checks and launches.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/paged_decode.h"
#include "pkd_serving.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

pkd_status launched() { return cudaGetLastError() == cudaSuccess ? PKD_OK : PKD_ERR_LAUNCH; }

constexpr int kMaxRopeHeadDim = 512;  // 16 dims a thread, at least four heads in flight

pkd_status append_rope(const void* q, const void* k_new, const void* v_new, long long q_stride, long long k_stride,
                       long long v_stride, const float* rope_table, const int32_t* token_starts,
                       const int32_t* positions, const int32_t* block_tables, const int32_t* context_lens, void* q_out,
                       long long q_out_stride, void* k_cache, void* v_cache, int num_tokens, int num_seqs,
                       int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim, int interleaved,
                       int max_positions, int block_size, int num_blocks, int max_blocks_per_seq, bool fp8,
                       float k_scale, float v_scale, int* error_word, cudaStream_t stream) {
  if (num_tokens < 0 || num_seqs < 0 || num_q_heads < 0 || num_kv_heads <= 0 || head_dim <= 0 || rotary_dim < 0 ||
      block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0)
    return PKD_ERR_SHAPE;
  if (head_dim % 16 != 0 || head_dim > kMaxRopeHeadDim || rotary_dim % 16 != 0 || rotary_dim > head_dim)
    return PKD_ERR_SHAPE;
  if (rotary_dim > 0 && max_positions <= 0) return PKD_ERR_SHAPE;
  if (fp8 && !(std::isfinite(k_scale) && std::isfinite(v_scale) && k_scale > 0.f && v_scale > 0.f))
    return PKD_ERR_SHAPE;
  if (num_tokens == 0 || num_seqs == 0) return PKD_OK;
  if (!token_starts && num_tokens % num_seqs != 0) return PKD_ERR_SHAPE;
  const long long q_row = (long long)num_q_heads * head_dim, kv_row = (long long)num_kv_heads * head_dim;
  if (num_q_heads > 0 && (q_stride < q_row || q_out_stride < q_row)) return PKD_ERR_SHAPE;
  if (k_stride < kv_row || v_stride < kv_row) return PKD_ERR_SHAPE;
  if (!k_new || !v_new || !block_tables || !context_lens || !k_cache || !v_cache) return PKD_ERR_NULL;
  if (num_q_heads > 0 && (!q || !q_out)) return PKD_ERR_NULL;
  if (rotary_dim > 0 && !rope_table) return PKD_ERR_NULL;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(rope_table, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
      !aligned(token_starts, 4) || !aligned(positions, 4) || !aligned(error_word, 4) || k_stride % 8 != 0 ||
      v_stride % 8 != 0)
    return PKD_ERR_ALIGN;
  if (num_q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16) || q_stride % 8 != 0 || q_out_stride % 8 != 0))
    return PKD_ERR_ALIGN;
  // rotated in place, every token's row is its own
  if (num_q_heads > 0 && num_tokens > 1 && q == q_out && q_stride != q_out_stride) return PKD_ERR_SHAPE;
  pkd::RopeAppendParams p{};
  p.q = static_cast<const __half*>(q);
  p.k = static_cast<const __half*>(k_new);
  p.v = static_cast<const __half*>(v_new);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.table = rope_table;
  p.token_starts = token_starts;
  p.positions = positions;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.q_out = static_cast<__half*>(q_out);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.num_tokens = num_tokens;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.rotary_dim = rotary_dim;
  p.max_positions = max_positions;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.error_word = error_word;
  auto* fn = fp8 ? (interleaved ? pkd::paged_kv_append_rope_kernel<true, true>
                                : pkd::paged_kv_append_rope_kernel<true, false>)
                 : (interleaved ? pkd::paged_kv_append_rope_kernel<false, true>
                                : pkd::paged_kv_append_rope_kernel<false, false>);
  fn<<<(unsigned)num_tokens, pkd::kRopeThreads, 0, stream>>>(p);
  return launched();
}

// Dynamic shared memory of the choice among `blocks` blocks: scores, a bit per block.
constexpr int select_smem(int blocks) { return 4 * (blocks + (blocks + 31) / 32) + 16; }

pkd_status check_blocks(int num_seqs, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                        int max_blocks_per_seq) {
  if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0)
    return PKD_ERR_SHAPE;
  if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32)) return PKD_ERR_UNSUPPORTED;
  return PKD_OK;
}

}  // namespace

extern "C" {

pkd_status paged_kv_append_rope(const void* q, const void* k_new, const void* v_new, long long q_stride,
                                long long k_stride, long long v_stride, const float* rope_table,
                                const int32_t* token_starts, const int32_t* positions, const int32_t* block_tables,
                                const int32_t* context_lens, void* q_out, long long q_out_stride, void* k_cache,
                                void* v_cache, int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads,
                                int head_dim, int rotary_dim, int interleaved, int max_positions, int block_size,
                                int num_blocks, int max_blocks_per_seq, int* error_word, cudaStream_t stream) {
  return append_rope(q, k_new, v_new, q_stride, k_stride, v_stride, rope_table, token_starts, positions, block_tables,
                     context_lens, q_out, q_out_stride, k_cache, v_cache, num_tokens, num_seqs, num_q_heads,
                     num_kv_heads, head_dim, rotary_dim, interleaved, max_positions, block_size, num_blocks,
                     max_blocks_per_seq, false, 1.f, 1.f, error_word, stream);
}

pkd_status paged_kv_append_rope_fp8(const void* q, const void* k_new, const void* v_new, long long q_stride,
                                    long long k_stride, long long v_stride, const float* rope_table,
                                    const int32_t* token_starts, const int32_t* positions,
                                    const int32_t* block_tables, const int32_t* context_lens, void* q_out,
                                    long long q_out_stride, void* k_cache, void* v_cache, int num_tokens, int num_seqs,
                                    int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim, int interleaved,
                                    int max_positions, int block_size, int num_blocks, int max_blocks_per_seq,
                                    float k_scale, float v_scale, int* error_word, cudaStream_t stream) {
  return append_rope(q, k_new, v_new, q_stride, k_stride, v_stride, rope_table, token_starts, positions, block_tables,
                     context_lens, q_out, q_out_stride, k_cache, v_cache, num_tokens, num_seqs, num_q_heads,
                     num_kv_heads, head_dim, rotary_dim, interleaved, max_positions, block_size, num_blocks,
                     max_blocks_per_seq, true, k_scale, v_scale, error_word, stream);
}

pkd_status paged_kv_block_bounds(const void* k_cache, const int32_t* block_tables, const int32_t* context_lens,
                                 const int32_t* start_lens, void* bounds, int num_seqs, int num_kv_heads, int head_dim,
                                 int block_size, int num_blocks, int max_blocks_per_seq, int max_new_tokens,
                                 int kv_fp8, int* error_word, cudaStream_t stream) {
  const pkd_status st = check_blocks(num_seqs, num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq);
  if (st != PKD_OK) return st;
  if (max_new_tokens < 0) return PKD_ERR_SHAPE;
  if (num_seqs == 0 || max_new_tokens == 0) return PKD_OK;
  if (!k_cache || !block_tables || !context_lens || !bounds) return PKD_ERR_NULL;
  if (!aligned(k_cache, 16) || !aligned(bounds, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
      !aligned(start_lens, 4) || !aligned(error_word, 4))
    return PKD_ERR_ALIGN;
  pkd::BlockBoundsParams p{};
  p.k_cache = k_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.start_lens = start_lens;
  p.bounds = bounds;
  p.num_seqs = num_seqs;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.error_word = error_word;
  // blocks that max_new_tokens tokens can touch, from anywhere inside a block
  // on; from token 0 when no starts are given
  p.grid_blocks = start_lens ? (int)(((long long)max_new_tokens + block_size - 2) / block_size + 1)
                             : (int)(((long long)max_new_tokens + block_size - 1) / block_size);
  p.grid_blocks = std::min(p.grid_blocks, max_blocks_per_seq);
  // A warp's kv heads: up to eight, whose tiles stream one behind the other,
  // while 32 warps an SM remain (32 prompts of up to 8192 tokens, 8 heads: 78
  // us, against 128 with one head a warp); one where the call is small.
  int sms = 0, dev = 0;
  if (pkd::failed(cudaGetDevice(&dev)) ||
      pkd::failed(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) || sms <= 0)
    sms = 148;
  const long long blocks = (long long)num_seqs * p.grid_blocks;
  p.heads_per_warp = 1;
  while (p.heads_per_warp < 8 && p.heads_per_warp < num_kv_heads &&
         blocks * num_kv_heads >= 2LL * p.heads_per_warp * 32 * sms)
    p.heads_per_warp *= 2;
  const long long units = blocks * ((num_kv_heads + p.heads_per_warp - 1) / p.heads_per_warp);
  const long long grid = (units + pkd::kBoundsWarps - 1) / pkd::kBoundsWarps;
  if (grid > 0x7fffffffLL) return PKD_ERR_SHAPE;
  auto* fn = kv_fp8 ? (head_dim == 128 ? pkd::paged_kv_block_bounds_kernel<128, 1>
                                       : pkd::paged_kv_block_bounds_kernel<64, 1>)
                    : (head_dim == 128 ? pkd::paged_kv_block_bounds_kernel<128, 2>
                                       : pkd::paged_kv_block_bounds_kernel<64, 2>);
  fn<<<(unsigned)grid, 32 * pkd::kBoundsWarps, 0, stream>>>(p);
  return launched();
}

pkd_status paged_kv_block_select(const void* q, const void* bounds, const int32_t* block_tables,
                                 const int32_t* context_lens, int32_t* block_lists, int32_t* list_lens, int num_seqs,
                                 int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                 int max_blocks_per_seq, int max_context_len, int max_selected, int sink_blocks,
                                 int recent_blocks, int kv_fp8, int* error_word, cudaStream_t stream) {
  if (num_q_heads <= 0 || max_context_len < 0 || max_selected <= 0 || sink_blocks < 0 || recent_blocks < 0 ||
      num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
      (long long)sink_blocks + recent_blocks > max_selected)
    return PKD_ERR_SHAPE;
  const pkd_status st = check_blocks(num_seqs, num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq);
  if (st != PKD_OK) return st;
  if (num_q_heads / num_kv_heads > 8) return PKD_ERR_UNSUPPORTED;
  if ((long long)max_context_len > (long long)max_blocks_per_seq * block_size) return PKD_ERR_SHAPE;
  const int max_blocks = (int)(((long long)max_context_len + block_size - 1) / block_size);
  if (max_blocks > PKD_MAX_SELECT_BLOCKS) return PKD_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKD_OK;
  if (!q || !bounds || !block_tables || !context_lens || !block_lists || !list_lens) return PKD_ERR_NULL;
  if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
      !aligned(block_lists, 4) || !aligned(list_lens, 4) || !aligned(error_word, 4))
    return PKD_ERR_ALIGN;
  pkd::BlockSelectParams p{};
  p.q = static_cast<const __half*>(q);
  p.bounds = bounds;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.lists = block_lists;
  p.list_lens = list_lens;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_blocks = max_blocks;
  p.max_selected = max_selected;
  p.sink = sink_blocks;
  p.recent = recent_blocks;
  p.error_word = error_word;
  // Rows (sequence, kv head) are what runs side by side.  Many rows: one CTA
  // each, of 128 threads, so that four rows share an SM and one's selection
  // runs beside another's pass (1024 rows of 256 blocks: 33 us, against 43 with
  // 256 threads).  Few: clusters, until they would fill the GPU twice over or a
  // warp would be without a tile of 16 blocks (8 rows of 2048 blocks: 11 us
  // with 16 CTAs a row, 23 with one; 256 rows: 46 with one, 50 with two, 68
  // with eight).  Sixteen need a GPC that holds them all at once, so they are
  // left to score arrays of which an SM holds two.
  int sms = 0, dev = 0;
  if (pkd::failed(cudaGetDevice(&dev)) ||
      pkd::failed(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) || sms <= 0)
    sms = 148;
  const long long rows = (long long)num_seqs * num_kv_heads;
  const int tiles = (max_blocks + 15) / 16;
  const int smem = select_smem(max_blocks);
  const bool narrow = rows > 2LL * sms;
  const int most = smem <= 64 * 1024 ? pkd::kSelMaxCluster : 8;
  p.cluster = 1;
  while (!narrow && p.cluster < most && rows * 2 * p.cluster <= 2LL * sms &&
         2 * p.cluster * pkd::kSelMaxWarps <= tiles)
    p.cluster *= 2;
  const long long grid = rows * p.cluster;
  if (grid > 0x7fffffffLL) return PKD_ERR_SHAPE;
  const int nt = narrow ? 128 : 256;
#define PKD_SELECT(D_, KVB_) \
  (narrow ? pkd::paged_kv_block_select_kernel<D_, KVB_, 128> : pkd::paged_kv_block_select_kernel<D_, KVB_, 256>)
  auto* fn = kv_fp8 ? (head_dim == 128 ? PKD_SELECT(128, 1) : PKD_SELECT(64, 1))
                    : (head_dim == 128 ? PKD_SELECT(128, 2) : PKD_SELECT(64, 2));
#undef PKD_SELECT
  // (The attribute belongs to the kernel, not to the call: what the largest call
  // needs, the same for all, so that a call of another host thread in between
  // changes nothing.)
  if (pkd::failed(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       select_smem(PKD_MAX_SELECT_BLOCKS))))
    return PKD_ERR_LAUNCH;
  if (p.cluster > 8 && pkd::failed(cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)))
    return PKD_ERR_LAUNCH;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)nt);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (pkd::failed(cudaLaunchKernelEx(&cfg, fn, p))) return PKD_ERR_LAUNCH;
  return launched();
}

}  // extern "C"
