"""64-bit references of the serving-step operators (rotated append, shared-prefix attention, block
bounds, block choice, attention over listed blocks), written from their definitions in torch
double, and the element bounds of their tests."""
import torch

from paged_kv_decode_21_gb300 import workloads

E4M3 = torch.float8_e4m3fn


def values(x):
    """Cache elements as double (bytes: the E4M3 code's value)."""
    return (x.view(E4M3).float() if x.dtype == torch.uint8 else x).double()


def make_cache(shape, seed, fp8, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return workloads.rand_e4m3(shape, g, device) if fp8 else workloads.randn_f16(shape, g, device)


def deal_tables(lens, block, width, pool, seed, device="cuda", skip=0):
    """Block tables of a seeded permutation of the pool (its first `skip` entries left out), -1 past each length."""
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(pool, generator=g)[skip:].to(torch.int32)
    bt = torch.full((len(lens), max(1, width)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // block)
        bt[b, :m] = perm[at:at + m]
        at += m
    assert at <= perm.numel()
    return bt.to(device), perm[at:]


def gathered(cache, row, n, g, block):
    """The first n tokens of a table row for kv head g, as double [n][D]."""
    m = -(-n // block)
    return values(cache[row[:m].long(), g]).reshape(-1, cache.shape[-1])[:n]


def attend(q, k, v, scale):
    """(softmax(scale q k^T) v, softmax(..) |v|) for q [r][D]; zeros where there is no key."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], v.shape[-1], dtype=torch.float64, device=q.device)
        return z, z.clone()
    p = torch.softmax(q.double() @ k.t() * scale, -1)
    return p @ v, p @ v.abs()


def attention_bound(ref, absref, tokens, vmax):
    """Largest error of the tensor-core paths: every weight is rounded to fp16 once (2^-11 of it, or
    2^-25 where it is subnormal, the largest weight being at least 1 before normalisation), the result
    once (2^-11 of it, or 2^-25), and fp32 arithmetic elsewhere stays below an eighth of the first term
    (scores of a few units, each a sum of 128 products: 2^-24 * 128 * 8 = 2^-14)."""
    return 1.25 * 2.0 ** -11 * absref + 2.0 ** -11 * ref.abs() + 2.0 ** -25 * (1 + tokens * vmax)


def check(out, ref, absref, tokens, vmax, what=""):
    got = out.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = ((got - ref).abs() / attention_bound(ref, absref, tokens, vmax)).max().item() if ref.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"
    return worst


def prefix_attention(q, kc, vc, ptab, plens, gstarts, bt, lens, scale, ks, vs, block):
    """q [B][ql][Hq][D] -> (out, weights over |V|)."""
    B, ql, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    plens, gstarts, lens = plens.tolist(), gstarts.tolist(), lens.tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    for b in range(B):
        y = [i for i in range(len(plens)) if gstarts[i] <= b < gstarts[i + 1]]
        for g in range(Hkv):
            k, v = gathered(kc, bt[b], lens[b], g, block), gathered(vc, bt[b], lens[b], g, block)
            n0 = 0
            if y:
                n0 = plens[y[0]]
                k = torch.cat((gathered(kc, ptab[y[0]], n0, g, block), k))
                v = torch.cat((gathered(vc, ptab[y[0]], n0, g, block), v))
            for j in range(ql):
                seen = n0 + max(0, lens[b] - ql + 1 + j)
                o, a = attend(q[b, j, g * G:(g + 1) * G], k[:seen], v[:seen], scale * ks)
                out[b, j, g * G:(g + 1) * G], mag[b, j, g * G:(g + 1) * G] = o * vs, a * vs
    return out, mag


def block_bounds(kc, bt, lens, start, bounds, block):
    """bounds after the call, as double."""
    out = values(bounds)
    for b, n in enumerate(lens):
        for i in range(start[b] // block, -(-n // block)):
            p = int(bt[b, i])
            x = values(kc[p, :, :min(block, n - i * block)])
            out[p, :, 0], out[p, :, 1] = x.amin(1), x.amax(1)
    return out


def block_select(q, bounds, bt, lens, K, sink, recent, block):
    """The lists by the exact scores, ties to the lowest index (Python integers and fp64)."""
    B, Hq, D = q.shape
    Hkv = bounds.shape[1]
    G = Hq // Hkv
    lists = torch.full((B, Hkv, K), -1, dtype=torch.int32)
    counts = torch.zeros((B, Hkv), dtype=torch.int32)
    for b in range(B):
        m = -(-lens[b] // block)
        for g in range(Hkv):
            if m <= K:
                pick = list(range(m))
            else:
                e = values(bounds[bt[b, :m].long(), g])
                x = q[b, g * G:(g + 1) * G].double()[:, None]
                s = torch.maximum(x * e[:, 0], x * e[:, 1]).sum(-1).amax(0).tolist()
                always = list(range(sink)) + list(range(m - recent, m))
                rest = sorted((i for i in range(sink, m - recent)), key=lambda i: (-s[i], i))
                pick = sorted(always + rest[:K - sink - recent])
            lists[b, g, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
            counts[b, g] = len(pick)
    return lists, counts


def listed_attention(q, kc, vc, bt, lens, lists, counts, scale, ks, vs, block):
    B, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    lists, counts = lists.cpu(), counts.cpu()
    for b in range(B):
        for g in range(Hkv):
            pick = lists[b, g, :int(counts[b, g])].tolist()
            k = [values(kc[int(bt[b, i]), g, :min(block, lens[b] - i * block)]) for i in pick]
            v = [values(vc[int(bt[b, i]), g, :min(block, lens[b] - i * block)]) for i in pick]
            if pick:
                o, a = attend(q[b, g * G:(g + 1) * G], torch.cat(k), torch.cat(v), scale * ks)
                out[b, g * G:(g + 1) * G], mag[b, g * G:(g + 1) * G] = o * vs, a * vs
    return out, mag
