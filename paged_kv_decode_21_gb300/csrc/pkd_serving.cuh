// pkd_serving.cuh -- kernels of the steps around a decode call: the rotated
// append of new tokens, the key bounds of cache blocks, and the choice of
// blocks by those bounds.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>
#include "pkd_decode_mma.cuh"
#include "pkd_int4.cuh"

namespace pkd {

constexpr uint32_t kErrBadPosition = 8u;  // a rotation position outside the table

// A cache's scale, and its reciprocal less and more 2^-21 of it, made on the host
// once a call: the IEEE quotient x / scale lies between x times the two (each off by
// 2^-24 at most), and the conversion to E4M3 is monotone, so where both products give
// the same codes, the quotient does too.  (under = 0: a scale whose reciprocal is not
// far inside fp32's range.)
struct E4m3Scale {
  float scale, under, over;
};
inline E4m3Scale e4m3_scale(float scale) {
  const float inv = scale > 1e-30f && scale < 1e30f ? 1.f / scale : 0.f;
  return {scale, inv * (1.f - 0x1p-21f), inv * (1.f + 0x1p-21f)};
}

// ---------------------------------------------------------------------------
// Rotated append.  With c_i = cos(p theta_i), s_i = sin(p theta_i) from row p
// of the table, pair i of a head turns as
//   y_a = x_a c_i - x_b s_i,   y_b = x_b c_i + x_a s_i
// (a, b) = (i, i + R/2), or (2i, 2i + 1) when the pairs are interleaved; dims
// from R on pass through.  Products and sums in fp32, rounded once to fp16 (or
// divided by the cache's scale and rounded once to E4M3).
//
// One CTA per token: thread (head slot, c) owns the 16 dims of two 16-byte
// chunks that rotate together, loads its 8 cosines and sines once, and walks
// the token's q, k and v heads with them.  The first head's data is requested
// before the token's sequence, position and block are looked up, so that chain
// of dependent loads hides behind it.
//
// Bound by HBM: every byte is moved once.  CTAs of 128 threads, sixteen heads
// at D = 128, keep more tokens in different phases on an SM than 256: prompts
// of 28842 tokens, 40 q and 8 kv heads, 133 against 155 us, 6.2 TB/s.
//
// AXES: pair i goes by the position on axis pair_axes[i], so the token's cosines
// come from several rows of the table: looked up once a token, a thread a pair,
// and shared.
//
// KVB 0 (4-bit caches): a group of 16 dims is a thread's two chunks, or, where
// they are R/2 apart, one chunk of each of two neighbouring lanes, which
// exchange their maxima.  Every operation is rounded by itself, so that the
// codes do not depend on which products a compiler fuses.
struct RopeAppendParams {
  const __half *q, *k, *v;         // token t's heads at q + t * q_stride (elements), head_dim apart
  long long q_stride, k_stride, v_stride, q_out_stride;
  const float* table;              // [max_positions][R]: R/2 cosines, then R/2 sines
  const int32_t* token_starts;     // [num_seqs + 1], or null: num_tokens / num_seqs tokens each
  const int32_t* positions;        // [num_tokens], or null: the logical position; AXES: [num_axes][num_tokens]
  const int32_t* pair_axes;        // AXES: [R / 2]
  const int32_t *block_tables, *context_lens;
  __half* q_out;
  void *k_cache, *v_cache;
  int num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, rotary_dim, max_positions, block_size, num_blocks,
      max_blocks_per_seq, num_axes;
  float k_scale, v_scale;
  E4m3Scale k8, v8;
  int* error_word;
};

// Eight fp32 values as codes 8 + clamp(rint(x / step), -7, 7), value k in bits 4k
// ..  Adding 1.5 2^23 + 8 in one fused multiply-add rounds x / step to an integer
// and leaves the code in the low bits.  The quotient by a reciprocal is within
// 2^-20 of the exact one where it is below 8 and the IEEE quotient within 2^-21,
// so they round alike unless the first is nearer than 2e-5 to halfway: then IEEE
// division decides (one value in 25000), as it does where `edge` says so: for scales
// that are subnormal or saturated, which alone let quotients pass 7.5, and for cache
// scales at the ends of fp32's range, where a step's reciprocal is infinite or
// subnormal.
__device__ __forceinline__ uint32_t pack8_int4(const float (&x)[8], float step, bool edge) {
  if (!(step > 0.f)) return 0x88888888u;
  constexpr float kMagic = 12582912.f + 8.f;
  const float inv = __frcp_rn(step);
  uint32_t w = 0;
  float off = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float r = fmaf(x[k], inv, kMagic);
    off = fmaxf(off, fabsf(fmaf(x[k], inv, kMagic - r)));
    w |= (__float_as_uint(r) & 15u) << (4 * k);
  }
  if (edge || !(off <= 0.49998f)) {
    w = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      w |= (uint32_t)((int)fminf(fmaxf(rintf(__fdiv_rn(x[k], step)), -7.f), 7.f) + 8) << (4 * k);
  }
  return w;
}
__device__ __forceinline__ float absmax8(const float (&x)[8]) {
  float a = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) a = fmaxf(a, fabsf(x[k]));
  return a;
}
// The scale byte of a group whose largest magnitude is a, and its step.
__device__ __forceinline__ uint32_t int4_scale_byte(float a, float scale, float& step) {
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(__fdiv_rn(a, __fmul_rn(7.f, scale))));
  const uint32_t byte = two & 0xFFu;
  step = __fmul_rn(__half2float(__ushort_as_half((unsigned short)(byte << 7))) * kInt4Unscale, scale);
  return byte;
}

// Four fp32 values over `scale` as E4M3 codes.
__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d, float scale) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(__fdiv_rn(b, scale)), "f"(__fdiv_rn(a, scale)));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(__fdiv_rn(d, scale)), "f"(__fdiv_rn(c, scale)));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ uint32_t cvt4_e4m3(float a, float b, float c, float d, float by) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * by), "f"(a * by));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * by), "f"(c * by));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// The same for eight of them (E4m3Scale).
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], const E4m3Scale& s) {
  if (s.under > 0.f) {
    const uint2 a = make_uint2(cvt4_e4m3(x[0], x[1], x[2], x[3], s.under), cvt4_e4m3(x[4], x[5], x[6], x[7], s.under));
    const uint2 b = make_uint2(cvt4_e4m3(x[0], x[1], x[2], x[3], s.over), cvt4_e4m3(x[4], x[5], x[6], x[7], s.over));
    if (a.x == b.x && a.y == b.y) return a;
  }
  return make_uint2(pack4_e4m3(x[0], x[1], x[2], x[3], s.scale), pack4_e4m3(x[4], x[5], x[6], x[7], s.scale));
}

__device__ __forceinline__ void unpack8(const uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
}

constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 8;  // an SM
constexpr int kMaxRopePairs = 256;  // of the largest head_dim
// A thread's place: which 16 dims (two chunks that rotate together, from e0 and e1 on) of which head slot.
struct RopeLane {
  int c, slot, slots, e0, e1;
  bool rot;
};
template <bool PAIRS>
__device__ __forceinline__ RopeLane rope_lane(const RopeAppendParams& P) {
  const int units = P.head_dim / 16;
  RopeLane l;
  l.slots = kRopeThreads / units;  // heads in flight
  l.c = threadIdx.x % units;
  l.slot = threadIdx.x / units;
  l.rot = l.c < P.rotary_dim / 16;
  l.e0 = l.rot && !PAIRS ? 8 * l.c : 16 * l.c;
  l.e1 = l.rot && !PAIRS ? P.rotary_dim / 2 + 8 * l.c : 16 * l.c + 8;
  return l;
}
// Head h of token t: q heads, then k heads, then v heads.
__device__ __forceinline__ const __half* rope_source(const RopeAppendParams& P, int t, int h) {
  if (h < P.num_q_heads) return P.q + t * P.q_stride + (long long)h * P.head_dim;
  h -= P.num_q_heads;
  if (h < P.num_kv_heads) return P.k + t * P.k_stride + (long long)h * P.head_dim;
  return P.v + t * P.v_stride + (long long)(h - P.num_kv_heads) * P.head_dim;
}
// The thread's 16 dims (u0, u1) of head h: turned, and stored into q_out or into row `in` of the block's tiles.
template <int KVB, bool PAIRS>
__device__ __forceinline__ void rope_head(const RopeAppendParams& P, const RopeLane& lane, const float (&cs)[8],
                                          const float (&sn)[8], const uint4 u0, const uint4 u1, int h, int t,
                                          size_t tile0, int in) {
  constexpr bool F8 = KVB == 1, I4 = KVB == 0;
  const int D = P.head_dim, units = D / 16, c = lane.c, e0 = lane.e0, e1 = lane.e1;
  const bool rot = lane.rot;
  const bool is_q = h < P.num_q_heads, is_v = h >= P.num_q_heads + P.num_kv_heads;
  const bool turn = rot && !is_v;
  float x[8], y[8];
  if (turn || (KVB != 2 && !is_q)) {
    unpack8(u0, x);
    unpack8(u1, y);
  }
  if (turn) {
    // y_a = a cos - d sin, y_b = d cos + a sin
    auto turned = [](float& a, float& d, float co, float si) {
      const float a0 = a, d0 = d;
      if constexpr (I4) {
        a = __fsub_rn(__fmul_rn(a0, co), __fmul_rn(d0, si));
        d = __fadd_rn(__fmul_rn(d0, co), __fmul_rn(a0, si));
      } else {
        a = fmaf(a0, co, -d0 * si);
        d = fmaf(d0, co, a0 * si);
      }
    };
    if constexpr (PAIRS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        turned(x[2 * i], x[2 * i + 1], cs[i], sn[i]);
        turned(y[2 * i], y[2 * i + 1], cs[4 + i], sn[4 + i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) turned(x[i], y[i], cs[i], sn[i]);
    }
  }
  if (is_q) {
    __half* o = P.q_out + t * P.q_out_stride + (long long)h * D;
    *reinterpret_cast<uint4*>(o + e0) = turn ? pack8(x) : u0;
    *reinterpret_cast<uint4*>(o + e1) = turn ? pack8(y) : u1;
  } else {
    const int g = h - P.num_q_heads - (is_v ? P.num_kv_heads : 0);
    const size_t row = ((tile0 + g) * P.block_size + in) * D;
    if constexpr (I4) {
      const float sc = is_v ? P.v_scale : P.k_scale;
      const int BS = P.block_size;
      uint8_t* tile = static_cast<uint8_t*>(is_v ? P.v_cache : P.k_cache) +
                      (tile0 + g) * ((size_t)BS * D * 9 / 16);
      uint8_t* scales = tile + (size_t)BS * D / 2 + in * units;
      // (a scale byte's value lies in 2^-9 .. 448, so steps and reciprocals of the others are normal)
      const bool far = !(sc > 0x1p-110f && sc < 0x1p110f);
      auto codes = [&](int e) { return reinterpret_cast<uint32_t*>(tile + ((e / 32) * BS + in) * 16 + e % 32 / 2); };
      float ax = absmax8(x), ay = absmax8(y), sx, sy;
      uint32_t bx, by;
      if (rot && !PAIRS) {
        // the other halves of both groups are the neighbouring lane's
        const unsigned both = 3u << (threadIdx.x & 30);
        ax = fmaxf(ax, __shfl_xor_sync(both, ax, 1));
        ay = fmaxf(ay, __shfl_xor_sync(both, ay, 1));
        bx = int4_scale_byte(ax, sc, sx);
        by = int4_scale_byte(ay, sc, sy);
        if (c % 2 == 0) {
          scales[e0 / 16] = (uint8_t)bx;
          scales[e1 / 16] = (uint8_t)by;
        }
      } else {
        bx = by = int4_scale_byte(fmaxf(ax, ay), sc, sx);
        sy = sx;
        scales[e0 / 16] = (uint8_t)bx;
      }
      *codes(e0) = pack8_int4(x, sx, far || bx < 8 || bx == 0x7E);
      *codes(e1) = pack8_int4(y, sy, far || by < 8 || by == 0x7E);
    } else if constexpr (F8) {
      uint8_t* o = static_cast<uint8_t*>(is_v ? P.v_cache : P.k_cache) + row;
      *reinterpret_cast<uint2*>(o + e0) = pack8_e4m3(x, is_v ? P.v8 : P.k8);
      *reinterpret_cast<uint2*>(o + e1) = pack8_e4m3(y, is_v ? P.v8 : P.k8);
    } else {
      __half* o = static_cast<__half*>(is_v ? P.v_cache : P.k_cache) + row;
      *reinterpret_cast<uint4*>(o + e0) = turn ? pack8(x) : u0;
      *reinterpret_cast<uint4*>(o + e1) = turn ? pack8(y) : u1;
    }
  }
}

// (One axis into E4M3 caches: seven CTAs an SM, as 64 registers spill.  1, 256, 1024 and 8192 tokens of 32/8 heads 3.0,
// 3.7, 5.3 and 36 us; eight 3.1, 3.8, 5.45 and 34.5.)
template <int KVB, bool PAIRS, bool AXES>
__global__ void __launch_bounds__(kRopeThreads, KVB == 1 && !AXES ? 7 : kRopeCtas)
    paged_kv_append_rope_kernel(const RopeAppendParams P) {
  const RopeLane lane = rope_lane<PAIRS>(P);
  const int R = P.rotary_dim, c = lane.c, slots = lane.slots, e0 = lane.e0, e1 = lane.e1;
  const bool rot = lane.rot;
  const int heads = P.num_q_heads + 2 * P.num_kv_heads;
  const int t = blockIdx.x;
  auto source = [&](int h) { return rope_source(P, t, h); };
  int h = lane.slot;
  const bool mine = lane.slot < slots;
  uint4 u0 = make_uint4(0u, 0u, 0u, 0u), u1 = u0;
  if (mine && h < heads) {
    const __half* s = source(h);
    u0 = *reinterpret_cast<const uint4*>(s + e0);
    u1 = *reinterpret_cast<const uint4*>(s + e1);
  }
  // AXES: a thread a pair looks up the pair's axis, the position there and the
  // table's entries, once for all heads
  __shared__ __align__(16) float turn_cos[AXES ? kMaxRopePairs : 4], turn_sin[AXES ? kMaxRopePairs : 4];
  bool off = false;
  if constexpr (AXES) {
    for (int i = threadIdx.x; i < R / 2; i += kRopeThreads) {
      const int axis = P.pair_axes[i];
      const int p = axis >= 0 && axis < P.num_axes ? P.positions[(size_t)axis * P.num_tokens + t] : -1;
      if (p >= 0 && p < P.max_positions) {
        turn_cos[i] = P.table[(long long)p * R + i];
        turn_sin[i] = P.table[(long long)p * R + R / 2 + i];
      } else {
        off = true;
      }
    }
  }
  // the token's sequence b and its place j in it
  int b, j;
  if (P.token_starts) {
    b = find_segment(P.token_starts, P.num_seqs, t);
    if (b >= P.num_seqs) return;  // past the last sequence: left as it is
    j = t - P.token_starts[b];
    if (j < 0) return;
  } else {
    const int per = P.num_tokens / P.num_seqs;
    b = t / per;
    j = t - b * per;
  }
  const int L = P.context_lens[b];
  // logical position and its block (of a length that is not negative: below 2^32)
  const long long at = (long long)L + j;
  const long long lb = (uint32_t)at / (uint32_t)P.block_size;
  const long long pos = P.positions && !AXES ? P.positions[t] : at;
  int block = -1;
  if (L >= 0 && lb < P.max_blocks_per_seq) block = P.block_tables[(size_t)b * P.max_blocks_per_seq + lb];
  uint32_t err = 0;
  if (block < 0 || block >= P.num_blocks) err |= kErrBadBlock;
  float cs[8], sn[8];
  if constexpr (AXES) {
    if (__syncthreads_or(off)) err |= kErrBadPosition;
  } else {
    if (R > 0 && (pos < 0 || pos >= P.max_positions)) err |= kErrBadPosition;
  }
  if (err) {
    if (threadIdx.x == 0) record_error(P.error_word, err);
    return;
  }
  if (AXES && rot) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 a = reinterpret_cast<const float4*>(turn_cos)[2 * c + i];
      const float4 d = reinterpret_cast<const float4*>(turn_sin)[2 * c + i];
      cs[4 * i] = a.x; cs[4 * i + 1] = a.y; cs[4 * i + 2] = a.z; cs[4 * i + 3] = a.w;
      sn[4 * i] = d.x; sn[4 * i + 1] = d.y; sn[4 * i + 2] = d.z; sn[4 * i + 3] = d.w;
    }
  }
  if (!AXES && rot) {
    const float4* row = reinterpret_cast<const float4*>(P.table + pos * R + 8 * c);
    const float4* row2 = reinterpret_cast<const float4*>(P.table + pos * R + R / 2 + 8 * c);
    const float4 a = row[0], a2 = row[1], s = row2[0], s2 = row2[1];
    cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w; cs[4] = a2.x; cs[5] = a2.y; cs[6] = a2.z; cs[7] = a2.w;
    sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w; sn[4] = s2.x; sn[5] = s2.y; sn[6] = s2.z; sn[7] = s2.w;
  }
  const size_t tile0 = (size_t)block * P.num_kv_heads;
  const int in = (int)(at - lb * P.block_size);
  if (!mine) return;
  for (; h < heads;) {
    const int hn = h + slots;
    uint4 n0 = u0, n1 = u1;
    if (hn < heads) {
      const __half* s = source(hn);
      n0 = *reinterpret_cast<const uint4*>(s + e0);
      n1 = *reinterpret_cast<const uint4*>(s + e1);
    }
    rope_head<KVB, PAIRS>(P, lane, cs, sn, u0, u1, h, t, tile0, in);
    h = hn;
    u0 = n0;
    u1 = n1;
  }
}

// Whether a position that token t's pairs first, first + step .. go by lies outside the table.
__device__ __forceinline__ bool off_table(const RopeAppendParams& P, int t, int first, int step) {
  bool off = false;
  for (int i = first; i < P.rotary_dim / 2; i += step) {
    const int axis = P.pair_axes[i];
    const int p = axis >= 0 && axis < P.num_axes ? P.positions[(size_t)axis * P.num_tokens + t] : -1;
    off |= p < 0 || p >= P.max_positions;
  }
  return off;
}

// The same for many tokens, kRopeRun of them a CTA: their sequences, positions,
// blocks and cosines are looked up side by side first and kept in shared memory,
// so that those chains of dependent loads are paid once a run, not once a token;
// then the CTA walks the heads of all of them.  Where codes are written, a thread's
// heads come by asynchronous copies into places of its own, three ahead of the
// one it turns; fp16 rows, which need no more instructions than the copies leave
// room for, come one ahead in registers.
//
// Prompts of 28842 tokens, 40 q and 8 kv heads, three axes: 4-bit caches 137 us, 5.4
// TB/s (one ahead in registers 156); 20082 tokens, 32 and 8, E4M3, three axes: 82
// us, 5.5 TB/s (97).  fp16, 28842 tokens, three axes: 139 us; one axis 134, as with a
// token a CTA (with the copies 172).  Which calls come here: takes_runs.  Two ahead
// 83 and 138, five 91 and 153; runs of eight tokens 91 and 153, seven CTAs an SM 84
// and 135, ten 142 and 287.  The quotients that codes are rounded from go by
// reciprocals where both neighbours of the reciprocal give the same codes, else by
// IEEE divisions (all by divisions, a token a CTA: 125 for E4M3).
constexpr int kRopeRun = 4;
constexpr int kRopeAhead = 4;  // places a thread has for heads on their way
__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int KVB, bool PAIRS, bool AXES>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) paged_kv_append_rope_run_kernel(const RopeAppendParams P) {
  static_assert(kRopeRun <= kRopeThreads / 32, "a warp looks up a token");
  constexpr bool RING = KVB != 2;
  __shared__ __align__(16) float turn[kRopeRun][2 * kMaxRopePairs];  // cosines, then sines
  __shared__ int block_of[kRopeRun], row_of[kRopeRun], pos_of[kRopeRun];
  const RopeLane lane = rope_lane<PAIRS>(P);
  const int R = P.rotary_dim, heads = P.num_q_heads + 2 * P.num_kv_heads;
  const int first = blockIdx.x * kRopeRun, n = min(kRopeRun, P.num_tokens - first);
  int k = 0, h = lane.slot;    // token of the run, head
  int ka = 0, ha = lane.slot;  // and those to request next
  const bool mine = lane.slot < lane.slots;
  auto settle = [&](int& k, int& h) {
    while (h >= heads && k < n) {
      h -= heads;
      ++k;
    }
  };
  settle(k, h);
  settle(ka, ha);
  __shared__ uint4 ring[RING ? kRopeAhead : 1][2][kRopeThreads];  // a thread's own places
  uint4 n0 = make_uint4(0u, 0u, 0u, 0u), n1 = n0;                  // without a ring: the next head
  uint32_t slot = 0;  // the next request's
  auto request = [&]() {
    if (mine && ka < n) {
      const __half* s = rope_source(P, first + ka, ha);
      if constexpr (RING) {
        cp_async_16(&ring[slot][0][threadIdx.x], s + lane.e0);
        cp_async_16(&ring[slot][1][threadIdx.x], s + lane.e1);
      } else {
        n0 = *reinterpret_cast<const uint4*>(s + lane.e0);
        n1 = *reinterpret_cast<const uint4*>(s + lane.e1);
      }
      ha += lane.slots;
      settle(ka, ha);
    }
    if constexpr (RING) {
      cp_async_commit();
      slot = slot + 1 == kRopeAhead ? 0 : slot + 1;
    }
  };
#pragma unroll
  for (int i = 0; i + 1 < (RING ? kRopeAhead : 2); ++i) request();
  const int w = threadIdx.x / 32;
  if (w < n) {
    const int t = first + w;
    int b, j = -1, block = -1, row = 0, pos = -1;
    if (P.token_starts) {
      b = find_segment(P.token_starts, P.num_seqs, t);
      if (b < P.num_seqs) j = t - P.token_starts[b];
    } else {
      const int per = P.num_tokens / P.num_seqs;
      b = t / per;
      j = t - b * per;
    }
    uint32_t err = 0;
    if (j >= 0) {  // (past the last sequence: left as it is)
      const int L = P.context_lens[b];
      const long long at = (long long)L + j;  // of a length that is not negative: below 2^32
      const long long lb = (uint32_t)at / (uint32_t)P.block_size;
      if (L >= 0 && lb < P.max_blocks_per_seq) block = P.block_tables[(size_t)b * P.max_blocks_per_seq + lb];
      row = (int)(at - lb * P.block_size);
      if (block < 0 || block >= P.num_blocks) err |= kErrBadBlock;
      if constexpr (!AXES) {
        const long long p = P.positions ? P.positions[t] : at;
        if (R > 0 && (p < 0 || p >= P.max_positions))
          err |= kErrBadPosition;
        else
          pos = (int)p;
      }
      if (err) block = -1;
      if constexpr (AXES) {
        // a token without a block is looked at here, as it is skipped below
        if (err && __any_sync(0xffffffffu, off_table(P, t, threadIdx.x % 32, 32))) err |= kErrBadPosition;
      }
    }
    if (threadIdx.x % 32 == 0) {
      if (err) record_error(P.error_word, err);
      block_of[w] = block;
      row_of[w] = row;
      pos_of[w] = pos;
    }
  }
  __syncthreads();
  bool off = false;
  for (int i = threadIdx.x; i < n * (R / 2); i += kRopeThreads) {
    const int x = i / (R / 2), pair = i % (R / 2);
    if (block_of[x] < 0) continue;
    int p = pos_of[x];
    if constexpr (AXES) {
      const int axis = P.pair_axes[pair];
      p = axis >= 0 && axis < P.num_axes ? P.positions[(size_t)axis * P.num_tokens + first + x] : -1;
      if (p < 0 || p >= P.max_positions) {
        row_of[x] = -1;  // (block_of may still be read by others)
        off = true;
        continue;
      }
    }
    turn[x][pair] = P.table[(long long)p * R + pair];
    turn[x][kMaxRopePairs + pair] = P.table[(long long)p * R + R / 2 + pair];
  }
  if (AXES && __syncthreads_or(off)) {
    if (threadIdx.x == 0) record_error(P.error_word, kErrBadPosition);
  }
  if (!AXES) __syncthreads();
  if (!mine) return;  // (nothing of its own in flight)
  float cs[8], sn[8];
  int turned_for = -1;
  uint32_t at = 0;
  while (k < n) {
    uint4 u0 = n0, u1 = n1;
    if constexpr (RING) {
      cp_async_wait<kRopeAhead - 2>();
      u0 = ring[at][0][threadIdx.x];
      u1 = ring[at][1][threadIdx.x];
      at = at + 1 == kRopeAhead ? 0 : at + 1;
    }
    request();
    if (lane.rot && k != turned_for) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 a = reinterpret_cast<const float4*>(turn[k])[2 * lane.c + i];
        const float4 d = reinterpret_cast<const float4*>(turn[k] + kMaxRopePairs)[2 * lane.c + i];
        cs[4 * i] = a.x; cs[4 * i + 1] = a.y; cs[4 * i + 2] = a.z; cs[4 * i + 3] = a.w;
        sn[4 * i] = d.x; sn[4 * i + 1] = d.y; sn[4 * i + 2] = d.z; sn[4 * i + 3] = d.w;
      }
      turned_for = k;
    }
    if (block_of[k] >= 0 && row_of[k] >= 0)
      rope_head<KVB, PAIRS>(P, lane, cs, sn, u0, u1, h, first + k, (size_t)block_of[k] * P.num_kv_heads, row_of[k]);
    h += lane.slots;
    settle(k, h);
  }
}

// ---------------------------------------------------------------------------
// Key bounds: for a cache block's tokens t (those before the sequence's
// length) and every dim d, lo_d = min_t k[t][d] and hi_d = max_t k[t][d], in
// the cache's own type: both are cache values, so nothing is rounded.  A key that
// is not a number makes both so.
//
// A warp takes up to eight kv heads of one (sequence, block): their tiles lie
// behind one another, a warp-wide load of 16 bytes a lane covers several whole
// rows, all of a step's loads are independent and the next step's are
// requested first, and the row groups meet in a butterfly.  Bound by HBM: 32
// prompts of 4000-8192 tokens, 8 heads, 78 us, 5.8 TB/s (one head a warp: 128,
// and 90 without the next step's loads).
struct BlockBoundsParams {
  const void* k_cache;
  const int32_t *block_tables, *context_lens;
  const int32_t* start_lens;  // nullable: blocks before start_lens[b] / block_size are left as they are
  void* bounds;               // [num_blocks][num_kv_heads][2][D]: lo, then hi
  int num_seqs, num_kv_heads, block_size, num_blocks, max_blocks_per_seq, grid_blocks;
  int heads_per_warp;
  int* error_word;
};

__device__ __forceinline__ uint32_t hmin2_u(uint32_t a, uint32_t b) {
  const __half2 r = __hmin2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmax2_u(uint32_t a, uint32_t b) {
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmin2_nan_u(uint32_t a, uint32_t b) {
  const __half2 r = __hmin2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmax2_nan_u(uint32_t a, uint32_t b) {
  const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmax2_abs(uint32_t a, uint32_t b) {  // max(a, |b|)
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), __habs2(*reinterpret_cast<const __half2*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// d = A . B for one m16n8k16 tile, from zero.
__device__ __forceinline__ void mma_16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Two fp16 pairs that hold E4M3 values -> the four codes (exact).
__device__ __forceinline__ uint32_t f16x2x2_to_e4m3x4(uint32_t lo, uint32_t hi) {
  uint16_t a, b;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(lo));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(hi));
  return (uint32_t)a | ((uint32_t)b << 16);
}

// The 16 bytes of a cache row as fp16 pairs: WORDS = 4 (fp16) or 8 (E4M3).
template <int KVB>
__device__ __forceinline__ void cache_words(const uint4 u, uint32_t (&w)[KVB == 2 ? 4 : 8]) {
  if constexpr (KVB == 2) {
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else {
    e4m3x4_to_f16x2x2(u.x, w[0], w[1]);
    e4m3x4_to_f16x2x2(u.y, w[2], w[3]);
    e4m3x4_to_f16x2x2(u.z, w[4], w[5]);
    e4m3x4_to_f16x2x2(u.w, w[6], w[7]);
  }
}
template <int KVB>
__device__ __forceinline__ uint4 words_to_cache(const uint32_t (&w)[KVB == 2 ? 4 : 8]) {
  if constexpr (KVB == 2) {
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    return make_uint4(f16x2x2_to_e4m3x4(w[0], w[1]), f16x2x2_to_e4m3x4(w[2], w[3]), f16x2x2_to_e4m3x4(w[4], w[5]),
                      f16x2x2_to_e4m3x4(w[6], w[7]));
  }
}

constexpr int kBoundsWarps = 8;
constexpr int kBoundsLoads = 8;  // loads in flight a lane
template <int D, int KVB>
__global__ void __launch_bounds__(32 * kBoundsWarps) paged_kv_block_bounds_kernel(const BlockBoundsParams P) {
  constexpr int CPR = D * KVB / 16;  // 16-byte chunks per row
  constexpr int RP = 32 / CPR;       // rows per warp-wide load
  constexpr int W = KVB == 2 ? 4 : 8;
  constexpr int U = kBoundsLoads;
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
  const int runs = (P.num_kv_heads + P.heads_per_warp - 1) / P.heads_per_warp;
  const int g0 = (int)(unit % runs) * P.heads_per_warp;
  const long long bi = unit / runs;
  const int b = (int)(bi / P.grid_blocks);
  if (b >= P.num_seqs) return;
  const int L = P.context_lens[b];
  const int start = P.start_lens ? max(P.start_lens[b], 0) : 0;
  const long long i = start / P.block_size + bi % P.grid_blocks;
  if (i * P.block_size >= L) return;
  int p = -1;
  if (i < P.max_blocks_per_seq) p = P.block_tables[(size_t)b * P.max_blocks_per_seq + i];
  if (p < 0 || p >= P.num_blocks) {
    if (lane == 0) record_error(P.error_word, kErrBadBlock);
    return;
  }
  const int valid = min(P.block_size, (int)(L - i * P.block_size));
  const int c = lane % CPR, r0 = lane / CPR;
  const size_t tile0 = (size_t)p * P.num_kv_heads + g0;
  const uint4* src = static_cast<const uint4*>(P.k_cache) + tile0 * P.block_size * CPR + c;
  uint4* dst = static_cast<uint4*>(P.bounds) + tile0 * 2 * CPR;
  // The warp's tiles (kv heads of one block) lie behind one another; steps of
  // U loads a lane run over them, the next step's loads requested before this
  // step's values are used.
  const int steps = (P.block_size + U * RP - 1) / (U * RP);  // per tile
  const int heads = min(P.heads_per_warp, P.num_kv_heads - g0);
  uint4 next[U];
  auto request = [&](int s) {  // step s: rows (s % steps) * U * RP + k * RP + r0 of tile s / steps
    const uint4* t = src + (size_t)(s / steps) * P.block_size * CPR;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int r = (s % steps) * U * RP + k * RP + r0;
      if (r < valid) next[k] = t[(size_t)r * CPR];
    }
  };
  request(0);
  uint32_t lo[W], hi[W];
  for (int s = 0; s < heads * steps; ++s) {
    uint4 u[U];
#pragma unroll
    for (int k = 0; k < U; ++k) u[k] = next[k];
    if (s + 1 < heads * steps) request(s + 1);
    if (s % steps == 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        lo[w] = 0x7C007C00u;  // +inf
        hi[w] = 0xFC00FC00u;  // -inf
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int r = (s % steps) * U * RP + k * RP + r0;
      if (r < valid) {
        uint32_t x[W];
        cache_words<KVB>(u[k], x);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          lo[w] = hmin2_nan_u(lo[w], x[w]);
          hi[w] = hmax2_nan_u(hi[w], x[w]);
        }
      }
    }
    if (s % steps == steps - 1) {
#pragma unroll
      for (int m = CPR; m < 32; m <<= 1)
#pragma unroll
        for (int w = 0; w < W; ++w) {
          lo[w] = hmin2_nan_u(lo[w], __shfl_xor_sync(0xffffffffu, lo[w], m));
          hi[w] = hmax2_nan_u(hi[w], __shfl_xor_sync(0xffffffffu, hi[w], m));
        }
      if (r0 == 0) dst[(size_t)(s / steps) * 2 * CPR + c] = words_to_cache<KVB>(lo);
      if (r0 == 1) dst[(size_t)(s / steps) * 2 * CPR + CPR + c] = words_to_cache<KVB>(hi);
    }
  }
}

// ---------------------------------------------------------------------------
// Choice of blocks.  The score of block i for kv head g is the largest score
// that any key inside the block's bounds could have with any of the group's
// queries,
//   S_i = max_h sum_d max(q_hd lo_id, q_hd hi_id)
//       = max_h (sum_d min(q_hd, 0) lo_id + sum_d max(q_hd, 0) hi_id),
// a product of [blocks x 2D] bounds with [2D x heads] queries: mma.m16n8k16
// with 16 blocks as rows and the group's heads as columns, bounds going from
// global memory straight into A fragments (a lane's 16 bytes of a row are its
// k slots of two steps; the query fragments follow the same order of dims).
// The first `sink` and the last `recent` blocks are always taken, and of the
// others the best, ties to the lowest index, as if scores were exact.  A bound
// that is not finite makes one of its two products +inf or not a number whatever
// the query's sign (0 * inf is not a number): its block counts as the best.
//
// The scores are sums of 2D exact products in fp32, off by at most E.  If tau
// is the k-th largest of them, blocks above tau + 2E are chosen and those below
// tau - 2E are not, whatever the rounding did; those between are scored again
// in fp64.  One pass of 2048 bins over the scores' range finds the bin of tau;
// the blocks of that bin and of those within 2E of it, a handful, are ranked
// directly.  Where they are many (equal blocks, a wide E) the general way
// takes over: radix selection finds tau, the blocks between are scored in
// fp64, and the same step runs again on their distances from tau, kept as fp32
// in the places of their scores, until the distances are exact in fp64's last
// bit.
//
// One cluster per (sequence, kv head): its CTAs share the pass over the
// bounds, which is bandwidth, and write scores into the shared memory of CTA
// 0, which selects.  The others leave, so one row's selection runs beside
// other rows' passes.
//
// What bounds it: the bounds are read once (32 sequences of 16K-32K tokens, 8
// heads, fp16: 203 MB in 44.5 us, 4.6 TB/s), at 16 warps an SM with 8 KiB each
// in flight; the selection itself takes 4-5 us after a row's last score, a
// chain of a few shared-memory passes, and the longest row ends the grid.
// (Requesting lo and hi rows alternately, a tile ahead: 48.7 us; 24 warps with
// 4 KiB each: 55.)
struct BlockSelectParams {
  const __half* q;      // [B][Hq][D]
  const void* bounds;   // [num_blocks][Hkv][2][D]
  const int32_t *block_tables, *context_lens;
  int32_t* lists;       // [B][Hkv][max_selected]
  int32_t* list_lens;   // [B][Hkv]
  int num_seqs, num_q_heads, num_kv_heads, block_size, num_blocks, max_blocks_per_seq, max_blocks, max_selected, sink,
      recent, cluster;
  int* error_word;
};

constexpr int kSelBinBits = 11, kSelBins = 1 << kSelBinBits;
constexpr int kSelMaxCluster = 16;
constexpr int kSelMaxWarps = 8;  // CTAs of 128 or 256 threads
// The bound of a score's error, relative to sum_d |q_d| max |bound|: one step
// adds 16 exact products, each cut at worst at 2^-23 of the largest, so 2^-19
// of its terms' magnitudes; every step starts from zero, and the up to 16
// results are summed in fp32 (2^-20 of all): 1.5 x 2^-19.
constexpr float kSelErr = 1.5f / 524288.f;

// The largest score, which also stands for +inf and for one that is not a
// number: finite, so that such blocks are ranked, counted and tied as any other.
// Its negative is the lowest: a head of -inf, a block outside the pool.  Finite
// fp16 scores end at 2^9 * 2^32.
constexpr float kSelTop = 3.0e38f;
constexpr uint32_t kHalfMax2 = 0x7BFF7BFFu;  // 65504, twice

__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// The block's score in fp64 (one below kSelTop: a block that reached it is not
// scored again), from its bounds at `lo` (then hi) and the group's
// queries; whole warp, the same value in every lane.
template <int D, int KVB>
__device__ __forceinline__ double exact_score(const char* lo, const __half* q, int G) {
  constexpr int DPC = 16 / KVB;
  const int lane = threadIdx.x & 31, h = lane / 4, c = lane % 4;  // four lanes a head, D / 4 dims each
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  if (h < G) {
#pragma unroll
    for (int jj = 0; jj < D / (4 * DPC); ++jj) {
      const int d0 = DPC * (4 * jj + c);
      uint32_t wl[DPC / 2], wh[DPC / 2];
      cache_words<KVB>(*reinterpret_cast<const uint4*>(lo + d0 * KVB), wl);
      cache_words<KVB>(*reinterpret_cast<const uint4*>(lo + (size_t)(D + d0) * KVB), wh);
#pragma unroll
      for (int w = 0; w < DPC / 2; ++w) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(q + (size_t)h * D + d0 + 2 * w));
        const float2 l = __half22float2(*reinterpret_cast<const __half2*>(&wl[w]));
        const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&wh[w]));
        // the larger of the two products of each dim, exact in fp32
        s[(2 * w) % 4] += (double)(x.x * (x.x < 0.f ? l.x : u.x));
        s[(2 * w + 1) % 4] += (double)(x.y * (x.y < 0.f ? l.y : u.y));
      }
    }
  }
  double t = (s[0] + s[1]) + (s[2] + s[3]);
  t += __shfl_xor_sync(0xffffffffu, t, 1);
  t += __shfl_xor_sync(0xffffffffu, t, 2);
  t = h < G ? fmax(t, -(double)kSelTop) : -(double)kSelTop;
#pragma unroll
  for (int m = 4; m < 32; m <<= 1) t = fmax(t, __shfl_xor_sync(0xffffffffu, t, m));
  return t;
}

// Exclusive sum over the CTA's WARPS warps of one count per thread; *tot is the total.
template <int WARPS>
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, s, k);
    if (lane >= k) s += x;
  }
  __syncthreads();  // the previous use of warp_sums is over
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const int x = warp_sums[w];
    base += w < warp ? x : 0;
    all += x;
  }
  *tot = all;
  return base + s - v;
}

// What a warp of the cluster hands to CTA 0 with its scores.
struct SelWarpStats {
  float kmax;        // largest |bound| it read
  float smin, smax;  // range of its scores that are to choose from
};

template <int D, int KVB, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) paged_kv_block_select_kernel(const BlockSelectParams P) {
  constexpr int NW = NT / 32;
  constexpr int DPC = 16 / KVB;      // dims per 16-byte chunk
  constexpr int JJ = D / (4 * DPC);  // chunks per lane and row
  constexpr int W = DPC / 2;         // fp16 pairs per chunk
  constexpr int ROWB = D * KVB;      // bytes of lo (and of hi)
  constexpr int PER = kSelBins / NT;
  // blocks around the border are ranked directly where they are NT or fewer, one a thread
  extern __shared__ __align__(16) float s_score[];  // CTA 0: [max_blocks], then a bit per block
  __shared__ __align__(16) int s_hist[kSelBins];
  __shared__ SelWarpStats s_stats[kSelMaxCluster * NW];
  __shared__ int s_sums[NW];
  __shared__ uint32_t s_red[2 * NW];
  __shared__ int s_found[2], s_n;
  __shared__ float s_tau;
  __shared__ float s_ws[NT];   // blocks around the border: score,
  __shared__ int s_wi[NT];     // index,
  __shared__ double s_wd[NT];  // exact score where it counts

  const int row = blockIdx.x / P.cluster, rank = blockIdx.x % P.cluster;
  const int b = row / P.num_kv_heads, g = row % P.num_kv_heads;
  const int G = P.num_q_heads / P.num_kv_heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane / 4, c = lane % 4;
  const int K = P.max_selected;
  const int32_t* bt = P.block_tables + (size_t)b * P.max_blocks_per_seq;
  int32_t* list = P.lists + (size_t)row * K;

  const int L = P.context_lens[b];
  int nblk = L > 0 ? (int)(((long long)L + P.block_size - 1) / P.block_size) : 0;
  if (nblk > P.max_blocks) {  // past the host's bound or the table row
    if (threadIdx.x == 0 && rank == 0) record_error(P.error_word, kErrBadBlock);
    nblk = P.max_blocks;
  }
  if (nblk <= K) {  // every block is taken
    if (rank == 0) {
      for (int i = threadIdx.x; i < K; i += NT) list[i] = i < nblk ? i : -1;
      if (threadIdx.x == 0) P.list_lens[row] = nblk;
    }
    return;
  }
  if (P.cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int i0 = P.sink, i1 = nblk - P.recent;  // the blocks to choose from
  int need = K - P.sink - P.recent;             // of which so many are taken: < i1 - i0

  // ---- scores
  uint32_t qlo[JJ * W], qhi[JJ * W];  // min(q, 0), max(q, 0) of head r (zero past the group)
  const __half* qrow = P.q + ((size_t)b * P.num_q_heads + g * G) * D;
  float qsum = 0.f;
#pragma unroll
  for (int jj = 0; jj < JJ; ++jj)
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint32_t x =
          r < G ? *reinterpret_cast<const uint32_t*>(qrow + (size_t)r * D + DPC * (4 * jj + c) + 2 * w) : 0u;
      qlo[jj * W + w] = hmin2_nan_u(x, 0u);
      qhi[jj * W + w] = hmax2_nan_u(x, 0u);
      const uint32_t a = hmin2_u(x & 0x7FFF7FFFu, kHalfMax2);  // what is not finite does not widen the error bound
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a));
      qsum += f.x + f.y;
    }
  const char* base = static_cast<const char*>(P.bounds) + (size_t)g * 2 * ROWB + 16 * c;
  const size_t block_stride = (size_t)P.num_kv_heads * 2 * ROWB;
  // a warp takes TT tiles of 16 blocks at a time: 8 KiB of bounds in flight (D = 128)
  constexpr int TT = KVB == 2 ? 1 : 2;
  const int tiles = (nblk + 15) / 16;
  const int step = P.cluster * NW;
  uint32_t kabs = 0;  // running maximum of |bound|, fp16 pair
  float smin = INFINITY, smax = -INFINITY;
  uint32_t score0, stats0;  // CTA 0's arrays in the cluster's shared window
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(score0) : "r"(smem_u32(s_score)));
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(stats0) : "r"(smem_u32(s_stats)));
  bool joined = P.cluster == 1;
  int id[TT][2];
  auto load_ids = [&](int tile) {
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int i = (tile + t * step) * 16 + 8 * f + r;
        id[t][f] = i < nblk ? bt[i] : -1;
      }
  };
  int tile = rank * NW + warp;
  load_ids(tile);
  if (rank == 0) {  // the bins start empty
#pragma unroll
    for (int k = 0; k < PER / 4; ++k) reinterpret_cast<int4*>(s_hist)[threadIdx.x + NT * k] = make_int4(0, 0, 0, 0);
    if (threadIdx.x == 0) s_found[0] = s_found[1] = s_n = 0;
  }
  for (; tile < tiles; tile += TT * step) {
    uint4 a[TT][2][2][JJ];  // [tile][row half][lo, hi][chunk]
    bool ok[TT][2];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        ok[t][f] = id[t][f] >= 0 && id[t][f] < P.num_blocks;
        const char* src = base + (size_t)(ok[t][f] ? id[t][f] : 0) * block_stride;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int jj = 0; jj < JJ; ++jj)
            a[t][f][e][jj] =
                ok[t][f] ? *reinterpret_cast<const uint4*>(src + e * ROWB + 64 * jj) : make_uint4(0u, 0u, 0u, 0u);
      }
    load_ids(tile + TT * step);
    float2 sum[TT][2];  // [row half]: heads 2c, 2c + 1
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      sum[t][0] = sum[t][1] = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int jj = 0; jj < JJ; ++jj) {
          uint32_t w0[W], w1[W];
          cache_words<KVB>(a[t][0][e][jj], w0);
          cache_words<KVB>(a[t][1][e][jj], w1);
#pragma unroll
          for (int w = 0; w < W; ++w) kabs = hmax2_abs(hmax2_abs(kabs, w0[w]), w1[w]);
#pragma unroll
          for (int s = 0; s < W / 2; ++s) {
            const uint32_t* qv = (e == 0 ? qlo : qhi) + jj * W + 2 * s;
            float acc[4];
            mma_16816_zero(acc, w0[2 * s], w1[2 * s], w0[2 * s + 1], w1[2 * s + 1], qv[0], qv[1]);
            sum[t][0] = __fadd2_rn(sum[t][0], make_float2(acc[0], acc[1]));
            sum[t][1] = __fadd2_rn(sum[t][1], make_float2(acc[2], acc[3]));
          }
        }
    }
    if (!joined) {  // CTA 0 has started: its shared memory may be written
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      joined = true;
    }
#pragma unroll
    for (int u = 0; u < 2 * TT; ++u) {
      const int t = u / 2, f = u % 2;
      // heads 2c and 2c + 1 of block row r + 8f; heads past the group do not count
      const float s0 = 2 * c < G ? sum[t][f].x : -INFINITY;
      const float s1 = 2 * c + 1 < G ? sum[t][f].y : -INFINITY;
      float s = fmax_nan(s0, s1);
      s = fmax_nan(s, __shfl_xor_sync(0xffffffffu, s, 1));
      s = fmax_nan(s, __shfl_xor_sync(0xffffffffu, s, 2));
      s = fmaxf(fminf(s, kSelTop), -kSelTop);  // not a number: kSelTop
      const int i = (tile + t * step) * 16 + 8 * f + r;
      if (c == 0 && i < nblk) {
        if (!ok[t][f]) {
          record_error(P.error_word, kErrBadBlock);
          s = -kSelTop;  // a block outside the pool comes last
        }
        if (i >= i0 && i < i1) {
          smin = fminf(smin, s);
          smax = fmaxf(smax, s);
        }
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(score0 + 4 * i), "f"(s) : "memory");
      }
    }
  }
  if (!joined) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) {
    kabs = hmax2_u(kabs, __shfl_xor_sync(0xffffffffu, kabs, k));
    smin = fminf(smin, __shfl_xor_sync(0xffffffffu, smin, k));
    smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, k));
  }
  if (lane == 0) {
    kabs = hmin2_u(kabs, kHalfMax2);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&kabs));
    const uint32_t at = stats0 + (uint32_t)(rank * NW + warp) * (uint32_t)sizeof(SelWarpStats);
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(fmaxf(f.x, f.y)) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4), "f"(smin) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 8), "f"(smax) : "memory");
  }
  if (P.cluster > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank != 0) return;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }

  // ---- selection, CTA 0
  // every warp has sum_d |q_hd| of head r in its lanes of that row
  qsum += __shfl_xor_sync(0xffffffffu, qsum, 1);
  qsum += __shfl_xor_sync(0xffffffffu, qsum, 2);
  SelWarpStats st = {0.f, INFINITY, -INFINITY};
  for (int i = lane; i < step; i += 32) {
    st.kmax = fmaxf(st.kmax, s_stats[i].kmax);
    st.smin = fminf(st.smin, s_stats[i].smin);
    st.smax = fmaxf(st.smax, s_stats[i].smax);
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) {
    qsum = fmaxf(qsum, __shfl_xor_sync(0xffffffffu, qsum, k));
    st.kmax = fmaxf(st.kmax, __shfl_xor_sync(0xffffffffu, st.kmax, k));
    st.smin = fminf(st.smin, __shfl_xor_sync(0xffffffffu, st.smin, k));
    st.smax = fmaxf(st.smax, __shfl_xor_sync(0xffffffffu, st.smax, k));
  }
  float E = st.kmax * qsum * kSelErr;
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(s_score + P.max_blocks);  // a bit per chosen block
  const int words = (nblk + 31) / 32;
  auto bounds_of = [&](int pb) { return static_cast<const char*>(P.bounds) + (size_t)pb * block_stride + (size_t)g * 2 * ROWB; };
  auto exact = [&](int i) {
    const int pb = bt[i];
    return pb >= 0 && pb < P.num_blocks ? exact_score<D, KVB>(bounds_of(pb), qrow, G) : -(double)kSelTop;
  };
  bool settled = false;
  int ties = 0;  // of the blocks in the second mask (s_hist), the first `ties` are chosen too

  // bin of a score: non-decreasing in it, 0 .. kSelBins - 1
  const float bin_scale = (float)kSelBins / (st.smax - st.smin);
  auto bin_of = [&](float s) { return min(kSelBins - 1, (int)((s - st.smin) * bin_scale)); };
  const float reach = 2.f * E * bin_scale + 2.f;  // bins that 2E reaches, one more for the rounding of a place
  if (need > 0 && st.smax > st.smin && bin_scale < INFINITY && reach < 64.f) {
    const int delta = (int)reach;
    for (int i = i0 + threadIdx.x; i < i1; i += NT) atomicAdd(&s_hist[bin_of(s_score[i])], 1);
    __syncthreads();
    // this thread's bins, from the highest down
    int bins[PER];
#pragma unroll
    for (int k = 0; k < PER / 4; ++k) {
      const int4 x = reinterpret_cast<const int4*>(s_hist)[kSelBins / 4 - 1 - (int)threadIdx.x * (PER / 4) - k];
      bins[4 * k] = x.w;
      bins[4 * k + 1] = x.z;
      bins[4 * k + 2] = x.y;
      bins[4 * k + 3] = x.x;
    }
    int mine = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) mine += bins[k];
    int tot;
    int above = block_scan<NW>(mine, s_sums, &tot);
    if (above < need && need <= above + mine) {  // the need-th largest is in one of this thread's bins
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        if (above < need && need <= above + bins[k]) {
          const int bin = kSelBins - 1 - (threadIdx.x * PER + k);
          const int top = min(kSelBins - 1, bin + delta);
          int higher = above;  // blocks in bins past top
          for (int t = bin + 1; t <= top; ++t) higher -= s_hist[t];
          s_found[0] = bin;
          s_found[1] = higher;
        }
        above += bins[k];
      }
    }
    __syncthreads();
    const int top = s_found[0] + delta, bottom = s_found[0] - delta;
    // mark the blocks that are in whatever the border's order; gather those around it
    for (int w = warp; w < words; w += NW) {
      const int i = 32 * w + lane;
      bool in = i < nblk && (i < i0 || i >= i1);
      if (i >= i0 && i < i1) {
        const float s = s_score[i];
        const int bin = bin_of(s);
        in = bin > top;
        if (!in && bin >= bottom) {
          const int at = atomicAdd(&s_n, 1);
          if (at < NT) {
            s_ws[at] = s;
            s_wi[at] = i;
          }
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (lane == 0) s_mask[w] = m;
    }
    __syncthreads();
    const int n = s_n, left = need - s_found[1];  // 0 < left <= n
    if (n <= NT) {
      settled = true;
      // one block a thread: its rank by (score, then index), which fixes tau
      const bool in = (int)threadIdx.x < n;
      const float s = in ? s_ws[threadIdx.x] : 0.f;
      const int idx = in ? s_wi[threadIdx.x] : 0;
      int rank_s = 0;
      if (32 * warp < n)
        for (int k = 0; k < n; ++k) rank_s += s_ws[k] > s || (s_ws[k] == s && s_wi[k] < idx);
      if (in && rank_s == left - 1) s_tau = s;
      __syncthreads();
      const float wlo = __fsub_rd(s_tau, 2.f * E), whi = __fadd_ru(s_tau, 2.f * E);
      const bool sure = in && s > whi;
      const bool open = in && s <= whi && s >= wlo;
      const int n_sure = __syncthreads_count(sure), n_open = __syncthreads_count(open);
      bool take = sure;
      if (n_sure + n_open == left) {
        take = sure || open;
      } else if (E == 0.f) {
        take = in && rank_s < left;
      } else {
        // the open ones, a warp each in turn
        int at = 0;
        for (int k0 = 0; k0 < n; k0 += 32) {
          const float sk = k0 + lane < n ? s_ws[k0 + lane] : -INFINITY;
          for (unsigned todo = __ballot_sync(0xffffffffu, sk <= whi && sk >= wlo); todo; todo &= todo - 1, ++at) {
            if (at % NW != warp) continue;
            const int k = k0 + __ffs(todo) - 1;
            const double x = s_ws[k] < kSelTop ? exact(s_wi[k]) : (double)kSelTop;
            if (lane == 0) s_wd[k] = x;
          }
        }
        __syncthreads();
        if (open) {
          const double x = s_wd[threadIdx.x];
          int ahead = 0;
          for (int k = 0; k < n; ++k)
            if (s_ws[k] <= whi && s_ws[k] >= wlo) ahead += s_wd[k] > x || (s_wd[k] == x && s_wi[k] < idx);
          take = ahead < left - n_sure;
        }
      }
      if (take) atomicOr(&s_mask[idx >> 5], 1u << (idx & 31));
    }
  }

  if (!settled) {
    // the general way: chosen are scores >= thr and the first `ties` of those equal to tie
    float thr = INFINITY, tie = INFINITY;
    double center = 0.0;
    for (int round = 0; need > 0; ++round) {
      // tau: the need-th largest of the finite scores, by radix selection on their order
      uint32_t kmin = 0xffffffffu, kmx = 0u;
      for (int i = i0 + threadIdx.x; i < i1; i += NT) {
        const float s = s_score[i];
        if (fabsf(s) < INFINITY) {
          kmin = min(kmin, order_key(s));
          kmx = max(kmx, order_key(s));
        }
      }
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) {
        kmin = min(kmin, __shfl_xor_sync(0xffffffffu, kmin, k));
        kmx = max(kmx, __shfl_xor_sync(0xffffffffu, kmx, k));
      }
      __syncthreads();
      if (lane == 0) {
        s_red[warp] = kmin;
        s_red[NW + warp] = kmx;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        kmin = min(kmin, s_red[w]);
        kmx = max(kmx, s_red[NW + w]);
      }
      uint32_t lo = kmin, span = kmx >= kmin ? kmx - kmin : 0u;  // tau's key lies in [lo, lo + span]
      int left = need;
      while (span > 0) {
        const int bits = 32 - __clz(span);
        const int shift = bits > kSelBinBits ? bits - kSelBinBits : 0;
        __syncthreads();
        for (int i = threadIdx.x; i < kSelBins; i += NT) s_hist[i] = 0;
        __syncthreads();
        for (int i = i0 + threadIdx.x; i < i1; i += NT) {
          const float s = s_score[i];
          const uint32_t k = order_key(s) - lo;
          if (fabsf(s) < INFINITY && k <= span) atomicAdd(&s_hist[k >> shift], 1);
        }
        __syncthreads();
        int mine = 0, tot;
#pragma unroll
        for (int k = 0; k < PER; ++k) mine += s_hist[kSelBins - 1 - (threadIdx.x * PER + k)];
        int above = block_scan<NW>(mine, s_sums, &tot);
        if (above < left && left <= above + mine) {
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            const int bin = kSelBins - 1 - (threadIdx.x * PER + k);
            const int x = s_hist[bin];
            if (above < left && left <= above + x) {
              s_found[0] = bin;
              s_found[1] = above;
            }
            above += x;
          }
        }
        __syncthreads();
        lo += (uint32_t)s_found[0] << shift;
        left -= s_found[1];
        span = (1u << shift) - 1u;
      }
      const float tau = key_value(lo);
      const float wlo = __fsub_rd(tau, 2.f * E), whi = __fadd_ru(tau, 2.f * E);
      int n_above = 0, n_in = 0, above, inside;  // the window's, of this thread and of all
      for (int i = i0 + threadIdx.x; i < i1; i += NT) {
        const float s = s_score[i];
        if (fabsf(s) < INFINITY) {
          n_above += s > whi;
          n_in += s >= wlo && s <= whi;
        }
      }
      block_scan<NW>(n_above, s_sums, &above);
      block_scan<NW>(n_in, s_sums, &inside);
      if (above + inside == need) {  // the whole window is in
        thr = wlo;
        break;
      }
      if (E == 0.f) {  // equal scores: the lowest indices
        tie = tau;
        ties = need - above;
        // those above are chosen: mark them
        for (int i = i0 + threadIdx.x; i < i1; i += NT)
          if (s_score[i] > tau) s_score[i] = INFINITY;
        break;
      }
      // score the window again, exactly, as distances from tau
      const double next = center + (double)tau;
      for (int ib = i0 + 32 * warp; ib < i1; ib += NT) {
        const int i = ib + lane;
        const float s = i < i1 ? s_score[i] : -INFINITY;
        const bool in = s >= wlo && s <= whi;
        if (i < i1 && !in) s_score[i] = s > whi ? INFINITY : -INFINITY;
        for (unsigned todo = __ballot_sync(0xffffffffu, in); todo; todo &= todo - 1) {
          const int k = ib + __ffs(todo) - 1;
          const float sk = __shfl_sync(0xffffffffu, s, k - ib);
          const double x = center + (double)sk < (double)kSelTop ? exact(k) : (double)kSelTop;
          if (lane == 0) s_score[k] = (float)(x - next);
        }
      }
      __syncthreads();
      center = next;
      need -= above;
      // a distance is at most a few E; its rounding to fp32 is off by 2^-24 of it.  The
      // next round's distances from a point this near are exact.
      E = round == 0 ? E * (1.f / (1 << 21)) : 0.f;
    }
    __syncthreads();
    for (int w = warp; w < words; w += NW) {
      const int i = 32 * w + lane;
      const float s = i < nblk ? s_score[i] : -INFINITY;
      const bool in = i < nblk && (i < i0 || i >= i1 || s >= thr || s == INFINITY);
      const unsigned m = __ballot_sync(0xffffffffu, in);
      const unsigned e = __ballot_sync(0xffffffffu, i < nblk && !in && ties > 0 && s == tie);
      if (lane == 0) {
        s_mask[w] = m;
        s_hist[w] = (int)e;
      }
    }
  }
  __syncthreads();

  // ---- the chosen blocks in ascending order: a run of mask words a thread
  const int per = (words + NT - 1) / NT;
  const int from = min(words, (int)threadIdx.x * per), to = min(words, from + per);
  int all_eq;
  if (ties > 0) {  // the first `ties` of the equal ones join
    int n_eq = 0;
    for (int w = from; w < to; ++w) n_eq += __popc((uint32_t)s_hist[w]);
    int before = block_scan<NW>(n_eq, s_sums, &all_eq);
    for (int w = from; w < to; ++w)
      for (uint32_t e = (uint32_t)s_hist[w]; e && before < ties; e &= e - 1, ++before) s_mask[w] |= e & (0u - e);
  }
  int n_in = 0, count;
  for (int w = from; w < to; ++w) n_in += __popc(s_mask[w]);
  int place = block_scan<NW>(n_in, s_sums, &count);
  for (int w = from; w < to; ++w)
    for (uint32_t m = s_mask[w]; m; m &= m - 1, ++place)
      if (place < K) list[place] = 32 * w + __ffs(m) - 1;
  if (threadIdx.x == 0) P.list_lens[row] = K;  // count, always: more than K blocks, all scores finite
}

}  // namespace pkd
