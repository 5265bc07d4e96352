// pkd_shared_tc.cuh -- attention of many query rows over one shared context,
// both products on the fifth-generation tensor cores (tcgen05).
//
// A group of sequences that share a prefix asks, for every kv head, for
//   S = Q K^T,  P = softmax(scale S),  O = P V
// over one [tokens x D] K and V and all the group's query rows (sequences x
// new tokens x heads of the kv head's group): a dense product whose
// arithmetic intensity grows with the rows, so past about 300 rows it is the
// tensor cores that bound it and not the cache read.  Results leave as fp32
// partials (unnormalised O, maximum, sum) for the merge with each sequence's
// own context.
//
// Work split: one CTA per (chunk of up to 256 query rows, partition of the
// shared context, kv head), one CTA per SM.  The rows are two tiles of 128
// (tensor-memory lanes), A and B, that share every K and V tile of 64 tokens;
// while the softmax of one runs, the tensor cores work for the other.
//   tensor memory   O of A and B (128 columns each); two S buffers of 64
//                   columns each for A and for B, P as fp16 pairs over S
//   shared memory   Q of both tiles; rings of K and V tiles
// Two S buffers per row tile let Q K^T of the tile after next run behind the
// softmax of the next.
//
// What bounds it.  Per 64 tokens both row tiles together need 512 cycles of
// tensor math for Q K^T and 512 for P V.  Q K^T with both operands in shared
// memory reads 6 KiB per 32-cycle step at N = 64, so it takes 48; with that,
// 1280 cycles; measured 0.74 us in a long prefix (E4M3 0.93), 1.45-1.5 thousand
// cycles: 256 x 7 rows over 32768 tokens, 4 kv heads, 112 CTAs of 128 tiles: 106
// us, the tensor pipe busy 67% of their cycles.  The rest is the chain
// P -> P V -> free S buffer -> Q K^T of one issuing warp, in which every test
// of a barrier takes over a hundred cycles while the MMAs stream operands from
// shared memory.  (One 128-token S buffer per row tile, a third less shared-
// memory traffic but S, softmax and P V in one chain, was slower: 179 us for that
// call where two of 64 first took 151.)
//
// Rounding.  P is rounded to fp16, once, for P V: kind::f16 takes fp16 operands,
// and V is fp16 (or widened to it).  That is 2^-11 of each weight, as in the other
// tensor-core decode kernels; the sums of the weights, O, the statistics and the
// partials are fp32, the sums of P before its rounding.
// A CTA's start and end take 8 us: the group's lengths 1.1, the first tiles and
// Q 4, the last 64 tokens' chain and the outputs 3.
//
// Roles:
//   warps 0-3, 4-7  softmax of tile A, B: one thread per row, as in
//                   pkd_decode_tc.cuh
//   warps 8, 9      MMA issuers of A and B: the whole warp waits on the next
//                   barriers of its chain, one elected lane issues.  (One warp
//                   polling the conditions of both chains: 2450 cycles; one for
//                   S and one for P V of both, which keeps both softmaxes in
//                   step: 2150; four warps, at 128 registers a thread: as two.)
//   warps 10, 11    K and V tiles: copies, one lane per box
//   warps 12-15     E4M3: widen the landed bytes to fp16 in place, two warps per
//                   ring (a warp that also copied took 2560 cycles a tile)
// Every wait is bounded; a role that gives up raises the abort flag.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>
#include "pkd_decode_tc.cuh"

namespace pkd {

constexpr int kSharedRows = 256;  // query rows per CTA

template <int BS, int KVB, int HD>
struct SharedTcTraits {
  static_assert(BS == 16 || BS == 32, "block_size");
  static_assert(KVB == 2 || (KVB == 1 && HD == 128), "E4M3 rows are widened at head_dim 128 only");
  static constexpr bool F8 = KVB == 1;
  static constexpr int D = HD;
  static constexpr int NH = D / 64;      // 64-dim halves of a row
  static constexpr int TN = 64;          // tokens per tile
  static constexpr int NBT = TN / BS;    // cache blocks per tile
  static constexpr int NBOX = TN / 16;   // 16-row boxes per tile and half
  // stages of the K and of the V ring.  (fp16 at D = 128: a fifth costs 4%, in
  // the issuer's chain; E4M3: the widened tiles want it, 6%)
  static constexpr int NS = HD == 64 ? 8 : KVB == 1 ? 5 : 4;
  static constexpr int ROWB = 128;       // bytes per swizzled row: 64 fp16
  static constexpr int QH = 128 * ROWB;  // one 64-dim half of a row tile's Q
  static constexpr int KVH = TN * ROWB;  // one 64-dim half of a K or V tile
  static constexpr int TILE = NH * KVH;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + 2 * NH * QH;
  static constexpr int V_OFF = K_OFF + NS * TILE;
  static constexpr int MAIN = V_OFF + NS * TILE;
  // full, kempty, vempty [NS]; sfull, pfull, pfree [2][2]; drain [2]; E4M3: kland, vland [NS]
  static constexpr int NBAR = 3 * NS + 12 + 2 + (F8 ? 2 * NS : 0);
  static constexpr int W_MMA = 8, W_K = 10, W_V = 11, W_WIDE = 12;
  // fp16: three warps per scheduler, 168 registers a thread.  E4M3: four more
  // that widen, at 128 registers and a few spilled bytes
  static constexpr int WIDENERS = F8 ? 2 : 0;  // per ring
  static constexpr int THREADS = F8 ? 512 : 384;
  static constexpr int TAIL = NBAR * 8 + 8 + NS * 4 + 4;
  static constexpr int SMEM_BYTES = MAIN + ((TAIL + 15) / 16) * 16;
  static_assert(SMEM_BYTES <= 227 * 1024, "one CTA per SM");
  static_assert(2 * SMEM_BYTES > 227 * 1024, "never two: a second one's tensor-memory allocation would wait");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t O_COL = 0, S_COL = 256;  // tile x: + 128 x; S buffer h: + 64 h
  static constexpr uint32_t IDESC_S = tc_idesc_f16(128, TN, false);
  static constexpr uint32_t IDESC_O = tc_idesc_f16(128, D, true);
};

template <int BS, int KVB, int HD>
__global__ void __launch_bounds__(SharedTcTraits<BS, KVB, HD>::THREADS, 1)
    paged_shared_tc_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                           const DecodeParams P) {
  using T = SharedTcTraits<BS, KVB, HD>;
  constexpr bool F8 = T::F8;
  constexpr int NS = T::NS, TN = T::TN, D = T::D;
  extern __shared__ __align__(1024) unsigned char smem_sh[];
  unsigned char* smem = smem_sh;
  const uint32_t sbase = smem_u32(smem);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (sbase & 1023u) {  // the swizzled operands need 1024-byte aligned groups
    if (threadIdx.x == 0) record_error(P.error_word, kErrLayout);
    return;
  }
  // full: K tile n and V tile n - 2 (with its bad-block mask) are in shared
  // memory: what an issuer needs next, when it has P of tile n - 2.  One test a
  // tile instead of two; n runs to ntiles + 1, with no V for n < 2 and no K for
  // the last two.
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + T::MAIN);  // [NS]
  uint64_t* kempty = full + NS;    // [NS] S of the tile computed, for every row tile
  uint64_t* vempty = kempty + NS;  // [NS] P V of the tile completed, for every row tile
  uint64_t* sfull = vempty + NS;   // [2][2] S of a tile is in buffer h of row tile x
  uint64_t* pfull = sfull + 4;     // [2][2] P of a tile is over its S columns
  uint64_t* pfree = pfull + 4;     // [2][2] P V of a tile completed (the buffer free, O stable)
  uint64_t* drain = pfree + 4;     // [2] every MMA of an issuer completed
  uint64_t* kland = drain + 2;     // E4M3: [NS] a tile's bytes landed
  uint64_t* vland = kland + NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2 + (F8 ? 2 * NS : 0));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* vbad = reinterpret_cast<volatile uint32_t*>(tmem_slot + 2);  // [NS]
  volatile int* bad_flag = reinterpret_cast<volatile int*>(tmem_slot + 2 + NS);

  // Work item: row chunk fastest (its CTAs read the same K and V), then
  // partition, then kv head.  Where all CTAs run at once the chunks go slowest:
  // those past the last row, whose CTAs leave at once, are then the last CTAs
  // and leave pairs of SMs (TPCs) free, not one SM here and there, because own
  // contexts beside a CTA in its TPC slow it down by a third (48 x 4 x 28/4
  // rows in two groups over 8192 E4M3 tokens: CTAs of 28 us, 37 so).
  const int G = P.num_q_heads / P.num_kv_heads;
  const int others = P.max_partitions * P.num_kv_heads;
  const int rest = P.chunks_outer ? blockIdx.x % others : blockIdx.x / P.q_chunks;
  const int j = rest % P.max_partitions, g = rest / P.max_partitions;
  GroupChunk ch;
  if (!find_group_chunk(P.group_starts, P.context_lens, P.num_groups, P.num_seqs, P.q_len * G, P.rows_per_chunk,
                        P.chunks_outer ? blockIdx.x / others : blockIdx.x % P.q_chunks, &ch))
    return;
  const int rows = min(P.rows_per_chunk, ch.tokens - ch.first);
  const size_t tok0 = (size_t)(ch.base / G);  // the group's first query token over the batch
  const int Hq = P.num_q_heads;
  auto out_row = [&](int rr) {
    const int r = ch.first + rr;
    return (tok0 + r / G) * Hq + g * G + r % G;
  };
  int L = ch.len;
  if (past_row<BS>(P, L)) {
    if (threadIdx.x == 0) record_error(P.error_word, kErrBadBlock);
    L = P.max_blocks_per_seq * BS;
  }
  const int PS = P.partition_size;
  const int t0 = j * PS;
  if (t0 >= L) return;  // the merge reads no partial past the context
  const int t1 = min(t0 + PS, L);
  const int ntiles = (t1 - t0 + TN - 1) / TN;
  const int nblk = (t1 - t0 + BS - 1) / BS;
  const int32_t* bt = P.block_tables + (size_t)ch.group * P.max_blocks_per_seq + t0 / BS;
  const int nx = rows > 128 ? 2 : 1;  // row tiles in use
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], F8 ? 2 * 32 * T::WIDENERS : 2);  // the K warps and the V warps
      mbar_init(&kempty[s], nx);
      mbar_init(&vempty[s], nx);
      if (F8) {
        mbar_init(&kland[s], 1);
        mbar_init(&vland[s], 1);
      }
    }
    for (int x = 0; x < 2; ++x) {
      const int live_warps = min(4, max(1, (rows - 128 * x + 31) / 32));
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sfull[2 * x + h], 1);
        mbar_init(&pfull[2 * x + h], 32 * live_warps);
        mbar_init(&pfree[2 * x + h], 1);
      }
      mbar_init(&drain[x], 1);
    }
    *abort_flag = 0;
    *bad_flag = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  // From here the copies run, beside the loading of Q by the softmax warps.
  uint32_t tmem = 0;
  bool any_bad = false;
  if (warp < T::W_K) {
    if (warp == T::W_MMA) {
      tmem_alloc(tmem_slot, T::TMEM_COLS);
      tmem_relinquish();
    }
    if (warp < 8) {
      // Q rows into the 64-dim halves of their tile, 128-byte swizzled; unused rows
      // zero.  Asynchronous copies of the warp's 32 rows, one or two whole rows
      // each, from a short loop: the code of a call is cold after the caches took
      // its data, and unrolled loads took 3 us here.
      constexpr int CPR = D / 8, RP = 32 / CPR;  // 16-byte chunks per row, rows per copy
      const int c = lane % CPR;
      const uint32_t qrow = (uint32_t)out_row(min((int)threadIdx.x, rows - 1));
      const __half* src = P.q + 8 * c;
      const uint32_t dst = sbase + T::Q_OFF + ((warp / 4) * T::NH + c / 8) * T::QH + (warp % 4) * 32 * T::ROWB;
#pragma unroll 1
      for (int i = lane / CPR; i < 32; i += RP) {
        const uint32_t at = __shfl_sync(0xffffffffu, qrow, i);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * T::ROWB + (((c % 8) ^ (i % 8)) << 4)),
                     "l"(src + (size_t)at * D), "r"(32 * warp + i < rows ? 16 : 0)
                     : "memory");
      }
      // Whether any block id of the partition is bad: where none is, as always but
      // for a caller's mistake, the softmax need not read the tiles' masks (a
      // shared-memory read costs it over a hundred cycles a tile).
      int wrong_id = 0;
      for (int k = threadIdx.x; k < nblk; k += 256) wrong_id |= bt[k] < 0 || bt[k] >= P.num_blocks;
      if (wrong_id) *bad_flag = 1;
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
    }
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(32 * T::W_K) : "memory");  // the softmax and issuing warps
    tc_fence_after();
    tmem = *tmem_slot;
    any_bad = *bad_flag != 0;
  }

  if (warp >= T::W_K) {
    // ------------------------------------------------------------ K, V tiles
    const bool is_k = warp % 2 == T::W_K % 2;
    uint64_t* empty = is_k ? kempty : vempty;
    const int lead = is_k ? 0 : 2;  // tile t's full barrier is number t + lead
    const uint32_t ring = is_k ? T::K_OFF : T::V_OFF;
    // fp16: the copies complete on the full barrier; E4M3: on a landing barrier
    auto land_bar = [&](int t) -> uint64_t* {
      if constexpr (F8) return is_k ? &kland[t % NS] : &vland[t % NS];
      return &full[(t + lead) % NS];
    };
    auto land_parity = [&](int t) -> uint32_t { return F8 ? (t / NS) & 1 : ((t + lead) / NS) & 1; };
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, mbar_wait_or_abort(bar, parity, P.timeout_ns, abort_flag));
    };
    // A stage is free for tile t once the tile NS before it was used; and an
    // arrival for full barrier n may only follow the completion of its number
    // n - NS, which that implies but for the first V tiles.
    auto wait_free = [&](int t) {
      if (t >= NS)
        wait(&empty[t % NS], ((t / NS) - 1) & 1);
      else if (t + lead >= NS)
        wait(&full[(t + lead) % NS], 0);
    };
    // The arrivals for full barriers without a tile of this ring: the first
    // two (V), the last two (K).
    auto idle_arrivals = [&](int from) {
      for (int n = from; n < from + 2 && ok; ++n) {
        wait_free(n - lead);
        if (ok && (F8 || lane == 0)) mbar_arrive(&full[n % NS]);
      }
    };
    int issued = 0;
    if (!F8 || warp < T::W_WIDE) {
      // Copies: lane l copies box l % NBOX of 64-dim half l / NBOX (E4M3: one
      // box holds whole rows); its block id is read one tile ahead.
      const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
      const L2Hints l2h = make_l2_hints(false);
      const int box = lane % T::NBOX, h = lane / T::NBOX;
      const bool mine = lane < (F8 ? 1 : T::NH) * T::NBOX;
      auto block_of = [&](int i) {
        const int k = i * T::NBT + box * 16 / BS;
        return mine && i < ntiles && k < nblk ? bt[k] : -1;
      };
      int id = block_of(0);
      if (!F8 && !is_k) idle_arrivals(0);
      for (; issued < ntiles; ++issued) {
        wait_free(issued);
        if (!ok) break;
        const int st = issued % NS;
        const bool in = mine && issued * T::NBT + box * 16 / BS < nblk;
        const bool good = in && id >= 0 && id < P.num_blocks;
        const unsigned wrong = __ballot_sync(0xffffffffu, in && !good && h == 0);
        const int boxes = __popc(__ballot_sync(0xffffffffu, good));
        if (lane == 0) {
          uint32_t bad = 0;
#pragma unroll
          for (int kk = 0; kk < T::NBT; ++kk) bad |= ((wrong >> (kk * BS / 16)) & 1u) << kk;
          // the mask is read by threads that waited for the tile's full barrier
          if (!is_k) vbad[st] = bad;
          if (is_k && bad) record_error(P.error_word, kErrBadBlock);
          mbar_arrive_expect_tx(land_bar(issued), (uint32_t)boxes * 16 * 128);
        }
        __syncwarp();
        if (good)
          tma_load_3d(sbase + ring + st * T::TILE + (F8 ? 0 : h * T::KVH) + box * 16 * T::ROWB, map,
                      land_bar(issued), F8 ? 0 : 64 * h, g * BS + (box * 16) % BS, id, l2h);
        id = block_of(issued + 1);
      }
      if (!F8 && is_k) idle_arrivals(ntiles);
    } else {
      // E4M3: widen this warp's rows of every tile.  Row r's 128 bytes landed
      // at its place in the first 64-dim half; every lane reads its chunks
      // before any writes both halves.
      const int part = (warp - T::W_WIDE) / 2;
      if (!is_k) idle_arrivals(0);
      for (int t = 0; t < ntiles; ++t) {
        wait(land_bar(t), land_parity(t));
        if (!ok) break;
        unsigned char* stg = smem + ring + (t % NS) * T::TILE;
        constexpr int CH = TN * 8 / 32 / (F8 ? T::WIDENERS : 1);  // 16-byte chunks a lane
        uint4 in[CH];
#pragma unroll
        for (int k = 0; k < CH; ++k)
          in[k] = *reinterpret_cast<const uint4*>(stg + 16 * (32 * CH * part + lane + 32 * k));
        __syncwarp();
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int q = 32 * CH * part + lane + 32 * k, r = q >> 3;
          const int c = (q & 7) ^ (r & 7);  // dims 16 c .. 16 c + 15 of row r
          uint4 lo, hi;
          e4m3x4_to_f16x2x2(in[k].x, lo.x, lo.y);
          e4m3x4_to_f16x2x2(in[k].y, lo.z, lo.w);
          e4m3x4_to_f16x2x2(in[k].z, hi.x, hi.y);
          e4m3x4_to_f16x2x2(in[k].w, hi.z, hi.w);
          unsigned char* row = stg + (c >> 2) * T::KVH + r * T::ROWB;
          *reinterpret_cast<uint4*>(row + ((((2 * c) & 7) ^ (r & 7)) << 4)) = lo;
          *reinterpret_cast<uint4*>(row + ((((2 * c + 1) & 7) ^ (r & 7)) << 4)) = hi;
        }
        fence_proxy_async_smem();  // visible to the tensor cores
        mbar_arrive(&full[(t + lead) % NS]);
      }
      if (is_k && ok) idle_arrivals(ntiles);
    }
    if (!ok) {
      if (lane == 0 && !*abort_flag) record_error(P.error_word, kErrTimeout);
      *abort_flag = 1;
    }
    __syncwarp();
    if (*abort_flag && lane == 0)  // let the copies in flight land before the CTA exits
      for (int t = max(0, issued - NS); t < issued; ++t)
        mbar_wait_bounded(land_bar(t), land_parity(t), P.timeout_ns);
  } else if (warp >= T::W_MMA && warp - T::W_MMA < nx) {
    // ------------------------------------------------------------ MMA issuer of row tile x
    const int x = warp - T::W_MMA;
    const uint32_t qs = sbase + T::Q_OFF + x * T::NH * T::QH;
    const uint32_t scol = tmem + T::S_COL + 128 * x, ocol = tmem + T::O_COL + 128 * x;
    bool ok = true;
    // (A test of a barrier costs over a hundred cycles while the MMAs stream
    // their operands from shared memory: three a tile is what is needed.)
    auto await = [&](uint64_t* bar, uint32_t parity, uint64_t* bar2, uint32_t parity2) {
      const bool second = lane & 1;
      ok = __all_sync(0xffffffffu, ok && mbar_wait_or_abort(second ? bar2 : bar, second ? parity2 : parity,
                                                            P.timeout_ns, abort_flag));
      tc_fence_after();
    };
    auto issue_qk = [&](int s) {
      if (ok && elect_one()) {
        const uint32_t ks = sbase + T::K_OFF + (s % NS) * T::TILE;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma_f16(scol + 64 * (s & 1), sw128_desc(qs + (k / 4) * T::QH + (k % 4) * 32, 16, 1024),
                     sw128_desc(ks + (k / 4) * T::KVH + (k % 4) * 32, 16, 1024), T::IDESC_S, k > 0 ? 1u : 0u);
        tc_commit(&sfull[2 * x + (s & 1)]);
        tc_commit(&kempty[s % NS]);
      }
      __syncwarp();
    };
    await(&full[0], 0, &full[0], 0);
    issue_qk(0);
    if (ntiles > 1) {
      await(&full[1], 0, &full[1], 0);
      issue_qk(1);
    }
    for (int s = 0; s < ntiles && ok; ++s) {
      // P and V of this tile, and K of the tile after next
      await(&pfull[2 * x + (s & 1)], (s >> 1) & 1, &full[(s + 2) % NS], ((s + 2) / NS) & 1);
      if (ok && elect_one()) {
        const uint32_t vs = sbase + T::V_OFF + (s % NS) * T::TILE;
        const uint32_t pa = scol + 64 * (s & 1);  // P: 8 columns per 16 tokens
#pragma unroll
        for (int k = 0; k < TN / 16; ++k)
          tc_mma_f16_ts(ocol, pa + 8 * k, sw128_desc(vs + k * 16 * T::ROWB, T::KVH, 1024), T::IDESC_O,
                        (s > 0 || k > 0) ? 1u : 0u);
        tc_commit(&pfree[2 * x + (s & 1)]);
        tc_commit(&vempty[s % NS]);
      }
      __syncwarp();
      if (s + 2 < ntiles && ok) {
        // the S buffer is free once P V, which reads P from it, completed
        await(&pfree[2 * x + (s & 1)], (s >> 1) & 1, &pfree[2 * x + (s & 1)], (s >> 1) & 1);
        issue_qk(s + 2);
      }
    }
    if (!ok) {
      if (lane == 0 && !*abort_flag) record_error(P.error_word, kErrTimeout);
      *abort_flag = 1;
    }
    // every MMA completes before tensor memory is freed
    if (elect_one()) tc_commit(&drain[x]);
    __syncwarp();
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&drain[x], 0, P.timeout_ns))) {
      if (lane == 0) record_error(P.error_word, kErrTimeout);
      *abort_flag = 1;
    }
  } else if (warp < 8 && warp * 32 < rows) {
    // ------------------------------------------------------------ softmax
    const int rr = threadIdx.x, x = warp / 4;
    const bool live = rr < rows;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = tl + T::O_COL + 128 * x, tsx = tl + T::S_COL + 128 * x;
    const int xthreads = 32 * min(4, (rows - 128 * x + 31) / 32);  // live threads of this row tile
    float m = -INFINITY, mt = -INFINITY, l = 0.f;                  // running shift, exact maximum, sum of p
    bool ok = true;
    for (int s = 0; s < ntiles; ++s) {
      const int h = s & 1, sv = s % NS;
      ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&sfull[2 * x + h], (s >> 1) & 1, P.timeout_ns, abort_flag));
      if (!ok) break;
      tc_fence_after();
      float sc[2][32];
      tmem_ld32(tsx + 64 * h, sc[0]);
      tmem_ld32(tsx + 64 * h + 32, sc[1]);
      const int nv = t1 - (t0 + s * TN);  // tokens of the tile inside the partition
      uint32_t bad = 0;
      if (any_bad || nv < TN) {  // the tile's V and its bad-block mask are needed below
        ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&full[(s + 2) % NS], ((s + 2) / NS) & 1, P.timeout_ns, abort_flag));
        bad = vbad[sv];
      }
      tmem_ld_wait();
      if (!ok) break;
      const bool raw = nv >= TN && bad == 0 && P.scale_log2 >= 0.f;
      if (!raw) {
#pragma unroll
        for (int e = 0; e < TN; ++e)
          sc[e / 32][e % 32] =
              (e < nv && !((bad >> (e / BS)) & 1u)) ? sc[e / 32][e % 32] * P.scale_log2 : -INFINITY;
      }
      float mx[8];
#pragma unroll
      for (int a = 0; a < 8; ++a) {
        const float* v = &sc[a / 4][(a % 4) * 8];
        mx[a] = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
      }
      float tmax = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                         fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
      const float f = raw ? P.scale_log2 : 1.f;  // the scale still to apply
      if (raw) tmax *= f;
      mt = fmaxf(mt, tmax);
      const bool rescale = __any_sync(0xffffffffu, tmax > m + kLazyTau);
      float alpha = 1.f;
      if (rescale) {
        const float mn = fmaxf(m, tmax);
        alpha = (mn == -INFINITY) ? 1.f : ex2_approx(m - mn);
        l *= alpha;
        m = mn;
      }
      const float mu = m == -INFINITY ? 0.f : m;  // nothing seen yet: masked scores give p = 0
      const float2 f2 = make_float2(f, f), nmu2 = make_float2(-mu, -mu);
      float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t pk[TN / 2];
#pragma unroll
      for (int e = 0; e < TN / 2; ++e) {
        const float2 y = ffma2(make_float2(sc[e / 16][(2 * e) % 32], sc[e / 16][(2 * e + 1) % 32]), f2, nmu2);
        const float2 pp = make_float2(ex2_approx(y.x), ex2_approx(y.y));
        acc[e % 4] = __fadd2_rn(acc[e % 4], pp);
        pk[e] = pack_half2(pp.x, pp.y);
      }
      const float2 at = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
      l += at.x + at.y;
      // O holds the tiles before once P V of the last of them completed: rescale it in place
      if (s > 0 && rescale) {
        ok = __all_sync(0xffffffffu,
                        mbar_wait_bounded(&pfree[2 * x + ((s - 1) & 1)], ((s - 1) >> 1) & 1, P.timeout_ns));
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(to + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= alpha;
          tmem_st32(to + 32 * c, o);
        }
      }
      tmem_st32u(tsx + 64 * h, pk);
      tmem_st_wait();
      if (nv < TN || bad) {
        // V rows that hold no token of the partition, or a bad block's: p = 0
        // there, and 0 * NaN would not be 0.  (The other row tile writes the
        // same zeros for itself.)
        unsigned char* vt = smem + T::V_OFF + sv * T::TILE;
        for (int y = rr - 128 * x; y < T::NH * TN * 8; y += xthreads) {
          const int hh = y / (TN * 8), r = (y / 8) % TN, c = y % 8;
          if (r >= nv || ((bad >> (r / BS)) & 1u))
            *reinterpret_cast<uint4*>(vt + hh * T::KVH + r * T::ROWB + c * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      mbar_arrive(&pfull[2 * x + h]);
    }
    if (ok)
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&pfree[2 * x + ((ntiles - 1) & 1)], ((ntiles - 1) >> 1) & 1,
                                                     P.timeout_ns));
    if (!ok) {
      if (lane == 0) record_error(P.error_word, kErrTimeout);
      *abort_flag = 1;
    } else {
      tc_fence_after();
      // partials relative to the exact maximum mt; O and l to the shift m
      const uint32_t orow = live ? (uint32_t)out_row(rr) : 0u;
      const size_t pidx = (size_t)orow * P.max_partitions + j;
      const float f = m == -INFINITY ? 0.f : ex2_approx(m - mt);
      const float fo = f * P.v_scale;
      // O leaves through the row tile's part of Q's place (its last product is
      // complete), 32 rows x CC columns a warp and pass, so that a store covers
      // whole 128-byte lines of a row or two: a store of 16 bytes from each of
      // 32 rows took 6 us for 256 rows in 140 CTAs at once.
      constexpr int CC = 32 * T::NH, CPR = CC / 4;
      unsigned char* stage = smem + T::Q_OFF + x * T::NH * T::QH + (warp & 3) * (T::NH * T::QH / 4);
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += CC) {
#pragma unroll
        for (int cc = 0; cc < CC; cc += 32) {
          float o[32];
          tmem_ld32(to + c0 + cc, o);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(stage + lane * 16 * CPR + (((cc / 4 + q) ^ (lane & 7)) << 4)) =
                make_float4(o[4 * q] * fo, o[4 * q + 1] * fo, o[4 * q + 2] * fo, o[4 * q + 3] * fo);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
          const int r = (32 * i + lane) / CPR, q = lane % CPR;
          const uint32_t at = __shfl_sync(0xffffffffu, orow, r);
          const float4 v = *reinterpret_cast<const float4*>(stage + r * 16 * CPR + ((q ^ (r & 7)) << 4));
          if (32 * warp + r < rows)
            *reinterpret_cast<float4*>(P.tmp_out + ((size_t)at * P.max_partitions + j) * D + c0 + 4 * q) = v;
        }
        __syncwarp();
      }
      if (live) {
        P.max_logits[pidx] = mt * 0.69314718055994530942f;
        P.exp_sums[pidx] = l * f;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == T::W_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, T::TMEM_COLS);
  }
}

}  // namespace pkd
