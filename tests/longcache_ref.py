"""References of the operators around long caches (4-bit caches, positions of several axes, gathered
weights, eviction), written from their definitions: the quantiser in IEEE fp32 with every operation
rounded by itself, everything else in torch double."""
import math

import torch

from serving_ref import E4M3, gathered

LOG2E = 1.4426950408889634


def tile_parts(cache, D):
    """(codes [NB][H][D/32][BS][16], scales [NB][H][BS][D/16]) views of a 4-bit cache."""
    BS = cache.shape[2]
    flat = cache.reshape(cache.shape[0], cache.shape[1], -1)
    return (flat[:, :, :BS * D // 2].unflatten(2, (D // 32, BS, 16)),
            flat[:, :, BS * D // 2:].unflatten(2, (BS, D // 16)))


def int4_values(cache, D, scale):
    """double [NB][H][BS][D] of a 4-bit cache, dim by dim."""
    codes, scales = tile_parts(cache, D)
    out = torch.empty((*cache.shape[:3], D), dtype=torch.float64, device=cache.device)
    s = (scales & 0x7F).contiguous().view(E4M3).double()
    for d in range(D):
        byte = codes[:, :, d // 32, :, d % 32 // 2].to(torch.int64)
        u = byte % 16 if d % 2 == 0 else byte // 16
        out[..., d] = (u - 8).double() * s[..., d // 16] * scale
    return out


def int4_rows(x, scale):
    """(codes uint8 [.., D] one a dim, scale bytes [.., D/16]) of fp32 CPU rows."""
    assert x.dtype == torch.float32 and not x.is_cuda
    k = torch.tensor(scale, dtype=torch.float32)
    g = x.reshape(*x.shape[:-1], -1, 16)
    top = g.abs().amax(-1) / (torch.tensor(7.0) * k)
    byte = top.clamp(max=448.0).to(E4M3)
    step = byte.float() * k
    q = torch.where(step[..., None] > 0, torch.round(g / step[..., None].clamp(min=1e-45)).clamp(-7, 7),
                    torch.zeros(()))
    return (q + 8).to(torch.uint8).reshape(x.shape), byte.view(torch.uint8)


def rotate32(x, cos, sin, R, pairs):
    """fp32 CPU rotation, each product and sum rounded by itself; x [T][H][D], cos and sin [T][R/2]."""
    x = x.float()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., :R // 2], x[..., R // 2:R])
    c, s = cos[:, None], sin[:, None]
    ya, yb = a * c - b * s, b * c + a * s
    y = x.clone()
    if pairs:
        y[..., 0:R:2], y[..., 1:R:2] = ya, yb
    else:
        y[..., :R // 2], y[..., R // 2:R] = ya, yb
    return y


def rows_of(table, positions, axes, R):
    """cos, sin [T][R/2] by a position per axis ([A][T]) and an axis per pair."""
    half = R // 2
    if not half:
        return table.new_zeros(positions.shape[1], 0), table.new_zeros(positions.shape[1], 0)
    at = torch.stack([positions[int(a)] for a in axes.tolist()], 1).long()
    i = torch.arange(half)
    return table[at, i], table[at, half + i]


def write_int4(cache, D, block, row, codes, scales):
    """Codes [H][D] and scale bytes [H][D/16] of one token into a CPU cache."""
    c, s = tile_parts(cache, D)
    two = codes.reshape(codes.shape[0], D // 32, 16, 2)
    c[block, :, :, row] = two[..., 0] | (two[..., 1] << 4)
    s[block, :, row] = scales


def random_int4(shape, D, seed, lo=0x20, hi=0x48, device="cuda"):
    """A cache of random codes (every one of the 16) and random scale bytes in [lo, hi]."""
    NB, H, BS = shape
    g = torch.Generator(device=device).manual_seed(seed)
    cache = torch.randint(0, 256, (NB, H, BS, 9 * D // 16), generator=g, device=device, dtype=torch.int32).to(torch.uint8)
    _, s = tile_parts(cache, D)
    s.copy_(torch.randint(lo, hi + 1, s.shape, generator=g, device=device, dtype=torch.int32).to(torch.uint8))
    return cache


def weights_after(q, k, bt, lens, weights, scale, start, decay, block):
    """weights after the call, double, and the largest sum |q k| scale log2(e) of any score; k double
    [NB][H][BS][D] values; q [B][ql][Hq][D]."""
    B, ql, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    out, most = weights.double().clone(), 0.0
    for b in range(B):
        for g in range(H):
            kk = gathered(k, bt[b], lens[b], g, block)
            if not lens[b]:
                continue
            x = q[b, :, g * G:(g + 1) * G].double()
            s = (x @ kk.t()) * scale
            most = max(most, float(((x.abs() @ kk.abs().t()) * abs(scale) * LOG2E).max()))
            t = torch.arange(lens[b], device=q.device)
            seen = t <= (lens[b] - ql + torch.arange(ql, device=q.device))[:, None]
            s = s.masked_fill(~seen[:, None], -math.inf)
            p = torch.softmax(s, -1)
            p = torch.where(seen.any(1)[:, None, None], p, 0.0).sum((0, 1))
            at, row = bt[b, t // block].long(), t % block
            first = lens[b] if start is None else start[b]
            old = torch.where((t < first) & (torch.tensor(decay, device=q.device) != 0),
                              weights[at, g, row].double() * decay, 0.0)
            out[at, g, row] = old + p
    return out, most


def weights_bound(D, rows, tokens, most):
    """Relative error of a gathered weight.  A score is a sum of D exact products in fp32 and two roundings
    of its scaling, off by at most (D + 2) 2^-24 of sum |q k| in log2 units, so a p by ln 2 times that; a
    row's sum by as much; sums over `tokens` terms and over `rows` by 2^-24 a term; each ex2 (four of them:
    p, a shift of the running sum, two merges) by 2^-22; the reciprocal and products by 2^-22 together."""
    return 2 * math.log(2) * (D + 2) * 2.0 ** -24 * most + (tokens + rows + 16) * 2.0 ** -24 + 5 * 2.0 ** -22


def token_select(weights, bt, lens, K, sink, recent, block):
    """kept, kept_lens by sorting in Python: descending weight, then position; NaN first."""
    w = weights.cpu()
    B, H = bt.shape[0], w.shape[1]
    kept = torch.full((B, H, K), -1, dtype=torch.int32)
    for b in range(B):
        n = lens[b]
        for g in range(H):
            if n <= K:
                pick = list(range(n))
            else:
                t = torch.arange(n)
                x = w[bt[b].cpu()[t // block].long(), g, t % block].tolist()
                always = list(range(sink)) + list(range(n - recent, n))
                rest = sorted(range(sink, n - recent),
                              key=lambda i: (-math.inf if math.isnan(x[i]) else -x[i], not math.isnan(x[i]), i))
                pick = sorted(always + rest[:K - sink - recent])
            kept[b, g, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return kept, torch.tensor([min(n, K) for n in lens], dtype=torch.int32)
