// pkd_append_rule.h -- which of its two kernels a rotated append takes (host code alone).
#pragma once

namespace pkd {

constexpr int kRopeRunTokens = 16;      // tokens an SM from which the append takes runs of them where tokens are
constexpr long long kRopeFewDims = 1536;  // of few dims,
constexpr int kRopeRunTokensWide = 24;  // and where they are of more

// Whether tokens are taken in runs of four instead of one a CTA: `per_sm` tokens
// an SM, of `dims` elements (all heads; a CTA's threads hold 2048 at once),
// `kv_dims` of them written into caches of `kv` (a pkd_kv_type).  A run pays the
// chain of look-ups once for four tokens, so it gains where a token is little
// work behind that chain or the chain is long (several axes); but it hands its
// heads out one behind the other, and its copies of codes' heads take twice the
// requests where a thread's two 16-byte chunks lie side by side (`pairs`, and
// heads that mostly do not turn).  Time of runs over that of a token a CTA, at
// 4096, 8192 and 28842 tokens:
//   fp16, one axis    1280 dims .82 .84 .79, 2304 .85 .92 .86, 2816 .91 .98 .91,
//                     3584 1.03 1.03 .97, 4096 1.08 1.09 1.01, 6144 1.09 1.09 1.01
//   fp16, axes        2304 .84 .82 .75, 3584 .92 .94 .89, 4096 .98 1.02 .95, 6144 1.02 1.05 .98
//   E4M3, one axis    2304 .87 .91 .79, 3584 .95 .96 .89, 4096 1.09 1.03 .96, 6144 1.11 1.06 .97
//   E4M3, axes        2304 .77 .75 .67, 4096 .91 .88 .79, 6144 .90 .92 .82, 8192 .98 .96 .86
//   4 bits, one axis  2304 .92 .97 .85, 4096 1.10 1.09 .97, 6144 1.06 1.05 .98
//   4 bits, axes      2304 .82 .84 .73, 4096 1.00 .93 .84, 6144 .96 .94 .86; with as many kv
//                     heads as q heads 6144 1.04 1.03 .94, 12288 1.15 1.12 1.04
//   E4M3, pairs       one axis 1280 .92 .89 .92, 1536 1.00 .98 .99, 2304 1.02 1.06 .92, 6144
//                     1.30 1.30 1.23; axes 2304 1.00 .94 .85, 4096 1.21 1.19 1.09
//   E4M3, half turns  one axis 2304 1.00 1.02 .89, 6144 1.14 1.09 1.03; axes 3584 .91 .93 .83,
//                     6144 1.05 1.01 .91
// At 2500 tokens 1280 dims .93 (fp16) to .79, 2304 1.00, 4096 dims and more 1.09 to 1.19.
inline bool takes_runs(int per_sm, long long dims, long long kv_dims, int kv, bool pairs, bool mostly_turned,
                       bool axes) {
  if (per_sm < (dims <= kRopeFewDims ? kRopeRunTokens : kRopeRunTokensWide)) return false;
  const bool many = per_sm >= 128, much_kv = 2 * kv_dims > dims;
  if (kv == 0) return dims <= (axes ? 3584 : 2816) || (axes && many);
  if (pairs) return dims <= (axes || many ? 2560 : kRopeFewDims);
  if (!mostly_turned) return dims <= (axes ? 3584 : (many ? 2560 : kRopeFewDims)) || (axes && many && !much_kv);
  if (kv == 2 && much_kv) return dims <= (axes && many ? 6144 : 2560);
  return dims <= 3584 || axes || many;
}

}  // namespace pkd
