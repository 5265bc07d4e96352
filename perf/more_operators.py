"""Cases of the operators around caches that are too long for 16 bits a value, or for all their tokens: their inputs,
their plain forms in elementary torch operations, and the library's calls.

Kinds of case:
  axes     rotation of q and k by positions of several axes (time, height, width), and the write of k and v into the cache
  append4  the rotated append into a cache of 4-bit codes, and the new rows read back as the cache holds them
  attn4    decode attention over a cache of 4-bit codes
  weights  every cached token's softmax weight, summed over the queries, added to what it has gathered so far
  evict    the choice of the tokens with the largest gathered weights, and their rows copied into blocks of their own
"""
import math

import torch

own = False  # set from outside: the library's kernels instead of the plain forms

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
F16, F8, I4 = "fp16", "e4m3", "int4"  # what a cache holds
BYTES = {F16: 2.0, F8: 1.0, I4: 9 / 16}  # a value: 4 bits and a sixteenth of a scale byte


# ------------------------------------------------------------------ cases
def _axes(name, seqs, lo, hi, past, q_heads, kv_heads, head_dim=128, rotary=128, block=16, kind=F16, pairs=False,
          turns=False):
    return {"name": name, "kind": "axes", "seqs": seqs, "new_lo": lo, "new_hi": hi, "past": past, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "rotary": rotary, "block": block, "cache": kind,
            "pairs": pairs, "turns": turns}


def _append4(name, seqs, lo, hi, past, q_heads, kv_heads, head_dim=128, rotary=128, block=16, pairs=False,
             several=False):
    return {"name": name, "kind": "append4", "seqs": seqs, "new_lo": lo, "new_hi": hi, "past": past,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "rotary": rotary, "block": block,
            "cache": I4, "pairs": pairs, "several": several}


def _attn4(name, seqs, q_len, lo, hi, q_heads, kv_heads, head_dim=128, block=16):
    return {"name": name, "kind": "attn4", "seqs": seqs, "q_len": q_len, "len_lo": lo, "len_hi": hi,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "block": block, "cache": I4}


def _weights(name, seqs, q_len, lo, hi, q_heads, kv_heads, head_dim=128, block=16, kind=F16, decay=1.0):
    return {"name": name, "kind": "weights", "seqs": seqs, "q_len": q_len, "len_lo": lo, "len_hi": hi,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "block": block, "cache": kind,
            "decay": decay}


def _evict(name, seqs, lo, hi, keep, sink, recent, kv_heads, head_dim=128, block=16, kind=F16):
    return {"name": name, "kind": "evict", "seqs": seqs, "len_lo": lo, "len_hi": hi, "keep": keep, "sink": sink,
            "recent": recent, "kv_heads": kv_heads, "head_dim": head_dim, "block": block, "cache": kind}


def listed():
    return [
        # one token for each sequence of a batch that began with images
        _axes("axes_token", 64, 1, 1, 2000, 28, 4),
        # ragged prompts of text and images over E4M3 caches, the axes in turns over the frequencies
        _axes("axes_prompts_e4m3", 9, 300, 4096, 0, 32, 8, kind=F8, turns=True),
        # one token for each sequence of a full decode batch
        _append4("append4_token", 128, 1, 1, 1023, 32, 8),
        # ragged prompts written in one go and read back for their own dense attention, images among the text
        _append4("append4_prompts", 13, 17, 4096, 0, 40, 8, several=True),
        # a few requests: latency
        _attn4("attn4_few", 4, 1, 500, 2000, 32, 8),
        # a ragged chat batch
        _attn4("attn4_batch", 128, 1, 512, 4096, 32, 8),
        # draft tokens verified
        _attn4("attn4_verify", 48, 4, 2000, 8192, 28, 4),
        # the long contexts that 4 bits make room for
        _attn4("attn4_long", 32, 1, 16384, 32768, 40, 8),
        # the weights of one decode step
        _weights("weights_step", 64, 1, 512, 4096, 32, 8),
        # the weights that the last 16 tokens of fresh prompts give to the prompts, over E4M3 caches
        _weights("weights_window_e4m3", 8, 16, 4000, 16384, 28, 4, kind=F8),
        # a batch that has outgrown its budget by a few blocks
        _evict("evict_step", 32, 1100, 1152, 1024, 4, 256, 8),
        # long prompts cut to a budget, over E4M3 caches
        _evict("evict_prompts_e4m3", 48, 8000, 32768, 2048, 16, 128, 8, kind=F8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((32, 32), (32, 8), (28, 4), (40, 8), (4, 4), (8, 1), (18, 3))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        what = rng.choice(("axes", "append4", "attn4", "attn4", "attn4", "weights", "weights", "evict", "evict"))
        hq, hkv = rng.choice(HEADS)
        d, block = rng.choice((64, 128, 128)), rng.choice((16, 16, 32))
        kind = rng.choice((F16, F8, I4))
        seqs = _log(rng, 1, 256)
        if what in ("axes", "append4"):
            hi = _log(rng, 1, 4096) if rng.random() < 0.6 else 1
            lo, past, r = max(1, hi // rng.randint(1, 9)), _log(rng, 1, 8000), rng.choice((d, d, 32))
            if seqs * hi > 60000:
                continue
            if what == "axes":
                c = _axes("", seqs, lo, hi, past, hq, hkv, d, r, block, rng.choice((F16, F8)), rng.random() < 0.4,
                          rng.random() < 0.5)
            else:
                c = _append4("", seqs, lo, hi, past, hq, hkv, d, r, block, rng.random() < 0.4, rng.random() < 0.5)
        elif what == "attn4":
            hi = _log(rng, 1, 32768)
            ql = rng.choice((1, 1, 1, 2, 5))
            c = _attn4("", seqs, ql, max(ql, hi // rng.randint(1, 9)), max(ql, hi), hq, hkv, d, block)
        elif what == "weights":
            hi = _log(rng, 1, 32768)
            ql = rng.choice((1, 1, 3, 16, 32))
            c = _weights("", seqs, ql, max(ql, hi // rng.randint(1, 9)), max(ql, hi), hq, hkv, d, block, kind,
                         rng.choice((1.0, 1.0, 0.75, 0.0)))
            if seqs * ql * hq * c["len_hi"] > 4e8:
                continue
        else:
            hi, keep = _log(rng, 1, 32768), _log(rng, 1, 4096)
            c = _evict("", seqs, max(1, hi // rng.randint(1, 9)), hi, keep, rng.randint(0, min(16, keep // 2)),
                       rng.randint(0, keep // 2), hkv, d, block, rng.choice((F16, F8)))
        held = seqs * max(c.get("len_hi", 0) + c.get("keep", 0), c.get("past", 0) + c.get("new_hi", 0))
        if held * hkv * d <= 8e8 and _cost(c) <= most:
            del c["name"]
            return c


# ------------------------------------------------------------------ sizes
def _spread(lo, hi, n):
    """n lengths from lo to hi in a fixed mixed order (the golden-ratio sequence)."""
    return [lo + int((hi - lo + 1) * ((k * 0.6180339887498949 + 0.37) % 1.0)) if hi > lo else lo for k in range(n)]


def work(c):
    e, d, hkv, n = BYTES[c["cache"]], c["head_dim"], c["kv_heads"], c["seqs"]
    if c["kind"] in ("axes", "append4"):
        t, hq = sum(_spread(c["new_lo"], c["new_hi"], n)), c["q_heads"]
        positions = min(t, c["past"] + c["new_hi"])
        byt = t * d * (hq * 4 + hkv * 2 * (2 + e)) + positions * c["rotary"] * 4 + t * 4
        if c["kind"] == "axes" or c["several"]:
            byt += t * 12
        if c["kind"] == "append4":  # the rows once more, and their values
            byt += t * d * hkv * 2 * (e + 2)
        return {"bytes": byt, "flops": 3 * t * (hq + hkv) * c["rotary"]}
    lens = _spread(c["len_lo"], c["len_hi"], n)
    if c["kind"] == "evict":
        kept = sum(min(x, c["keep"]) for x in lens)
        cut = sum(x for x in lens if x > c["keep"])  # where no more tokens are there than are kept, no weight is needed
        return {"bytes": hkv * (4 * cut + kept * (4 * d * e + 8 + 4)), "flops": hkv * cut}
    rows, hq = c["q_len"] * c["q_heads"], c["q_heads"]
    if c["kind"] == "weights":
        byt = sum(lens) * hkv * (d * e + (8 if c["decay"] else 4)) + n * rows * d * 2
        return {"bytes": byt, "flops": 2 * d * sum(lens) * rows}
    return {"bytes": sum(lens) * hkv * d * 2 * e + 2 * n * rows * d * 2, "flops": 4 * d * sum(lens) * rows}


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


# ------------------------------------------------------------------ caches
def _normal(shape, g):
    out = torch.empty(shape, dtype=torch.float16, device=DEV)
    flat = out.view(-1)
    for s in range(0, flat.numel(), 1 << 26):
        e = min(flat.numel(), s + (1 << 26))
        flat[s:e] = torch.randn(e - s, generator=g, device=DEV)
    return out


def _parts(cache, d):
    """Views of a 4-bit cache [blocks][kv heads][block][9 d / 16]: codes [..][d / 32][block][16 bytes], two dims a
    byte, the lower nibble first, and E4M3 scales [..][block][d / 16]."""
    block = cache.shape[2]
    flat = cache.flatten(2)
    return flat[:, :, :block * d // 2].unflatten(2, (d // 32, block, 16)), flat[:, :, block * d // 2:].unflatten(
        2, (block, d // 16))


def _quantized(x, scale):
    """(codes [.., d / 32, 16], scale bytes [.., d / 16]) of fp32 rows x [.., d]."""
    x = x.unflatten(-1, (-1, 16))
    top = torch.full((), 7.0, device=DEV) * scale
    s = (x.abs().amax(-1) / top).clamp(max=448).to(E4M3)
    step = (s.float() * scale)[..., None]
    q = torch.where(step > 0, (x / step).round().clamp(-7, 7), 0.0)
    u = (q + 8).to(torch.uint8).flatten(-2)
    return (u[..., 0::2] | (u[..., 1::2] << 4)).unflatten(-1, (-1, 16)), s.view(torch.uint8)


def _cache(pool, hkv, block, d, kind, g, scale):
    """Caches of ~N(0,1) values; bytes: the codes of N(0,1) / scale."""
    if kind == F16:
        return _normal((pool, hkv, block, d), g)
    out = torch.empty((pool, hkv, block, d if kind == F8 else 9 * d // 16), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (hkv * block * d))
    for a in range(0, pool, step):
        e = min(pool, a + step)
        x = torch.randn((e - a, hkv, block, d), generator=g, device=DEV)
        if kind == F8:
            out[a:e] = (x / scale).clamp_(-448, 448).to(E4M3).view(torch.uint8)
        else:
            codes, scales = _parts(out[a:e], d)
            u, s = _quantized(x, scale)
            codes.copy_(u.transpose(2, 3))
            scales.copy_(s)
    return out


def _tables(lens, block, extra, g):
    """Block tables of a seeded permutation of a pool a tenth larger than needed, `extra` blocks of it left over."""
    per = [-(-x // block) for x in lens]
    pool = max(1, -(-(sum(per) + extra) * 11 // 10))
    perm = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int32)
    return _dealt(per, perm), pool, perm[sum(per):]


def _dealt(per, blocks):
    need = torch.tensor(per, device=DEV)
    i = torch.arange(max(1, max(per)), device=DEV)
    start = (need.cumsum(0) - need)[:, None] + i
    return torch.where(i < need[:, None], blocks[start.clamp(max=blocks.numel() - 1)], -1).to(torch.int32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ inputs
def _grid_positions(past, new):
    """[3][tokens] positions of the new tokens: text, whose axes go together, an image of rows and columns in its
    middle third (where there is room for one), and text after it, from the image's largest position on."""
    out = []
    for p, n in zip(past, new):
        a, m = n // 3, n // 3
        if m < 16:
            out.append(torch.arange(p, p + n).expand(3, n))
            continue
        wide = max(2, int(math.sqrt(m)))
        i = torch.arange(m)
        image = torch.stack((torch.full((m,), p + a), p + a + i // wide, p + a + i % wide))
        after = int(image.max()) + 1
        out.append(torch.cat((torch.arange(p, p + a).expand(3, a), image,
                              torch.arange(after, after + n - a - m).expand(3, n - a - m)), 1))
    return torch.cat(out, 1).to(torch.int32).to(DEV)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    d, hkv, n, block, kind = c["head_dim"], c["kv_heads"], c["seqs"], c["block"], c["cache"]
    one = {F16: 1.0, F8: 1 / 64.0, I4: 1 / 16.0}[kind]
    s = dict(c=c, ks=one, vs=one, scale=1.0 / math.sqrt(d), err=torch.zeros(1, dtype=torch.int32, device=DEV), ws=None)
    if c["kind"] in ("axes", "append4"):
        new, hq, r = _spread(c["new_lo"], c["new_hi"], n), c["q_heads"], c["rotary"]
        past = _spread(c["past"] // 2, c["past"], n)
        t = sum(new)
        s["bt"], pool, _ = _tables([a + b for a, b in zip(past, new)], block, 0, g)
        qkv = _normal((t, (hq + 2 * hkv) * d), g)  # the fused projection's rows
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        pos = torch.arange(max(a + b for a, b in zip(past, new)), device=DEV, dtype=torch.float64)
        ang = pos[:, None] * 10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
        s["rope"] = torch.cat((ang.cos(), ang.sin()), 1).float()
        s["starts"] = _ints([0] + torch.tensor(new).cumsum(0).tolist())
        s["lens"] = _ints(past)
        s["positions"] = s["axes"] = None
        if c["kind"] == "axes" or c["several"]:
            i = torch.arange(r // 2, device=DEV)
            edge = (r // 8, r // 8 + 3 * r // 16)  # a quarter of the frequencies for time, three eighths a side
            s["axes"] = (i % 3 if c.get("turns") else (i >= edge[0]).int() + (i >= edge[1]).int()).to(torch.int32)
            s["positions"] = _grid_positions(past, new)
        row = 9 * d // 16 if kind == I4 else d
        dtype = torch.float16 if kind == F16 else torch.uint8
        s["kc"] = torch.zeros((pool, hkv, block, row), dtype=dtype, device=DEV)
        s["vc"] = torch.zeros((pool, hkv, block, row), dtype=dtype, device=DEV)
        s["q_out"] = torch.zeros((t, hq, d), dtype=torch.float16, device=DEV)
        if c["kind"] == "append4":
            s["k_out"] = torch.zeros((t, hkv, d), dtype=torch.float16, device=DEV)
            s["v_out"] = torch.zeros((t, hkv, d), dtype=torch.float16, device=DEV)
        return s
    lens = _spread(c["len_lo"], c["len_hi"], n)
    s["lens"], s["max_len"] = _ints(lens), max(lens)
    kept = [-(-min(x, c["keep"]) // block) for x in lens] if c["kind"] == "evict" else [0]
    s["bt"], pool, rest = _tables(lens, block, sum(kept), g)
    s["kc"] = _cache(pool, hkv, block, d, kind, g, s["ks"])
    if c["kind"] in ("weights", "evict"):
        # a few tokens gather most of the weight, many next to none
        s["weights"] = torch.rand((pool, hkv, block), generator=g, device=DEV) ** 8
    if c["kind"] == "evict":
        s["vc"] = _cache(pool, hkv, block, d, kind, g, s["vs"])
        s["new_bt"] = _dealt(kept, rest)
        s["kept"] = torch.empty((n, hkv, c["keep"]), dtype=torch.int32, device=DEV)
        s["kept_lens"] = torch.empty((n,), dtype=torch.int32, device=DEV)
        return s
    s["q"] = _normal((n, c["q_len"], c["q_heads"], d), g)
    if c["kind"] == "weights":
        s["first"] = _ints([x - c["q_len"] for x in lens])
    else:
        s["vc"] = _cache(pool, hkv, block, d, kind, g, s["vs"])
        s["out"] = torch.empty_like(s["q"])
    return s


def _shown(x):
    """A cache as its values: byte caches as E4M3 numbers."""
    return x.view(E4M3) if x.dtype == torch.uint8 else x


# ------------------------------------------------------------------ one pass
def run(s):
    return (_RUN_OWN if own else _RUN_PLAIN)[s["c"]["kind"]](s)


def _own_axes(s):
    from paged_kv_decode_21_gb300 import ops
    kw = dict(token_starts=s["starts"], interleaved=s["c"]["pairs"], q_out=s["q_out"], error_word=s["err"])
    if s["c"]["cache"] == F8:
        ops.paged_kv_append_rope_axes_fp8(s["q"], s["k"], s["v"], s["rope"], s["axes"], s["positions"], s["bt"],
                                          s["lens"], s["kc"], s["vc"], s["ks"], s["vs"], **kw)
    else:
        ops.paged_kv_append_rope_axes(s["q"], s["k"], s["v"], s["rope"], s["axes"], s["positions"], s["bt"],
                                      s["lens"], s["kc"], s["vc"], **kw)
    return {"q": s["q_out"], "k": _shown(s["kc"]), "v": _shown(s["vc"])}


def _places(s):
    """(sequence, logical position) of every new token."""
    t = torch.arange(s["q"].shape[0], device=DEV, dtype=torch.int32)
    b = torch.searchsorted(s["starts"][1:], t, right=True)
    return b, (s["lens"][b] + t - s["starts"][b]).long()


def _rotated(x, cos, sin, r, pairs):
    x = x.to(cos.dtype)
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., :r // 2], x[..., r // 2:r])
    y, z = a * cos - b * sin, b * cos + a * sin
    rot = torch.stack((y, z), -1).flatten(-2) if pairs else torch.cat((y, z), -1)
    return torch.cat((rot, x[..., r:]), -1)


def _turned(s, logical):
    """fp32 q and k, rotated: pair i by the token's position on the pair's axis."""
    c, half = s["c"], s["c"]["rotary"] // 2
    if s["axes"] is None:
        cos, sin = s["rope"][logical, :half], s["rope"][logical, half:]
    else:
        at = s["positions"].long()[s["axes"].long()].t()  # tokens, pairs
        i = torch.arange(half, device=DEV)
        cos, sin = s["rope"][at, i], s["rope"][at, half + i]
    return tuple(_rotated(x, cos[:, None], sin[:, None], c["rotary"], c["pairs"]) for x in (s["q"], s["k"]))


def _plain_axes(s):
    block, fp8 = s["c"]["block"], s["c"]["cache"] == F8
    b, pos = _places(s)
    q, k = _turned(s, pos)
    v = s["v"].float()
    s["q_out"].copy_(q)
    if fp8:
        k = (k / s["ks"]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        v = (v / s["vs"]).clamp(-448, 448).to(E4M3).view(torch.uint8)
    at = s["bt"][b, pos // block].long()
    s["kc"][at, :, pos % block] = k if fp8 else k.half()
    s["vc"][at, :, pos % block] = v if fp8 else v.half()
    return {"q": s["q_out"], "k": _shown(s["kc"]), "v": _shown(s["vc"])}


def _own_append4(s):
    from paged_kv_decode_21_gb300 import ops
    ops.paged_kv_append_rope_int4(s["q"], s["k"], s["v"], s["rope"], s["bt"], s["lens"], s["kc"], s["vc"], s["ks"],
                                  s["vs"], token_starts=s["starts"], positions=s["positions"], pair_axes=s["axes"],
                                  interleaved=s["c"]["pairs"], q_out=s["q_out"], error_word=s["err"])
    ops.paged_kv_read_int4(s["kc"], s["vc"], s["bt"], s["lens"], s["ks"], s["vs"], s["k_out"], s["v_out"],
                           token_starts=s["starts"], error_word=s["err"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _opened(codes, scales, scale):
    """fp32 values [.., d] of codes [.., d / 32, 16] and scale bytes [.., d / 16]."""
    u = torch.stack((codes & 15, codes >> 4), -1).flatten(-3).float() - 8
    step = scales.view(E4M3).float() * scale
    return (u.unflatten(-1, (-1, 16)) * step[..., None]).flatten(-2)


def _plain_append4(s):
    d, block = s["c"]["head_dim"], s["c"]["block"]
    b, pos = _places(s)
    q, k = _turned(s, pos)
    s["q_out"].copy_(q)
    at = s["bt"][b, pos // block].long()
    for x, cache, scale, out in ((k, s["kc"], s["ks"], s["k_out"]), (s["v"].float(), s["vc"], s["vs"], s["v_out"])):
        codes, scales = _parts(cache, d)
        codes[at, :, :, pos % block], scales[at, :, pos % block] = _quantized(x, scale)
        out.copy_(_opened(codes[at, :, :, pos % block], scales[at, :, pos % block], scale))
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_attn4(s):
    from paged_kv_decode_21_gb300 import ops
    c = s["c"]
    if s["ws"] is None:  # a program keeps its workspace from call to call
        s["ws"] = ops.alloc_workspace(ops.paged_decode_int4_workspace_size(
            c["seqs"], c["q_len"], c["q_heads"], c["kv_heads"], c["head_dim"], c["block"], s["max_len"]), DEV)
    return ops.paged_decode_attention_int4(s["q"], s["kc"], s["vc"], s["bt"], s["lens"], s["scale"], s["ks"], s["vs"],
                                           out=s["out"], max_context_len=s["max_len"], workspace=s["ws"],
                                           error_word=s["err"])


def _rows(s, cache, scale):
    """[sequences][kv heads][tokens][d] fp32 values of whole contexts (whole blocks)."""
    c, at = s["c"], s["bt"].long().clamp(min=0)
    if c["cache"] == I4:
        codes, scales = _parts(cache, c["head_dim"])
        x = _opened(codes[at].transpose(3, 4), scales[at], scale)  # n, m, kv, block, d
    else:
        x = _shown(cache[at]).float() * scale
    return x.transpose(1, 2).flatten(2, 3)


def _scores(s):
    """Masked scores [sequences][kv heads][q_len][group][tokens]."""
    c = s["c"]
    ql, hkv = c["q_len"], c["kv_heads"]
    k = _rows(s, s["kc"], s["ks"])
    q = s["q"].float().view(c["seqs"], ql, hkv, -1, c["head_dim"]).permute(0, 2, 1, 3, 4) * s["scale"]
    sc = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).unflatten(2, (ql, -1))
    t = torch.arange(k.shape[2], device=DEV)
    seen = s["lens"].long()[:, None] - ql + 1 + torch.arange(ql, device=DEV)  # tokens that query j sees
    return sc.masked_fill_((t >= seen[:, :, None])[:, None, :, None, :], float("-inf"))


def _plain_attn4(s):
    sc = _scores(s)
    p = (sc - sc.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p.flatten(2, 3), _rows(s, s["vc"], s["vs"])).unflatten(2, p.shape[2:4]) / p.sum(-1, keepdim=True)
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(s["out"].shape))
    return s["out"]


def _own_weights(s):
    from paged_kv_decode_21_gb300 import ops
    c = s["c"]
    if s["ws"] is None:
        s["ws"] = ops.alloc_workspace(ops.paged_kv_attention_weights_workspace_size(
            c["seqs"], c["q_len"], c["q_heads"], c["kv_heads"], c["head_dim"], c["block"], s["max_len"]), DEV)
    return ops.paged_kv_attention_weights(s["q"], s["kc"], s["bt"], s["lens"], s["weights"], s["scale"],
                                          k_scale=s["ks"], start_lens=s["first"], decay=c["decay"],
                                          max_context_len=s["max_len"], workspace=s["ws"], error_word=s["err"])


def _plain_weights(s):
    c = s["c"]
    sc = _scores(s)
    p = (sc - sc.amax(-1, keepdim=True)).exp_()
    p = (p / p.sum(-1, keepdim=True)).sum((2, 3))  # n, kv, tokens
    t = torch.arange(p.shape[2], device=DEV)
    b, i = (t < s["lens"].long()[:, None]).nonzero(as_tuple=True)
    at, row = s["bt"][b, i // c["block"]].long(), i % c["block"]
    old = torch.where((i < s["first"].long()[b])[:, None], s["weights"][at, :, row] * c["decay"], 0.0)
    s["weights"][at, :, row] = old + p[b, :, i]
    return s["weights"]


def _own_evict(s):
    from paged_kv_decode_21_gb300 import ops
    c = s["c"]
    ops.paged_kv_token_select(s["weights"], s["bt"], s["lens"], c["keep"], sink_tokens=c["sink"],
                              recent_tokens=c["recent"], max_context_len=s["max_len"], kept=s["kept"],
                              kept_lens=s["kept_lens"], error_word=s["err"])
    ops.paged_kv_compact(s["kc"], s["vc"], s["bt"], s["lens"], s["kept"], s["kept_lens"], s["new_bt"],
                         weights=s["weights"], error_word=s["err"])
    return {"kept": s["kept"], "kept_lens": s["kept_lens"], "k": _shown(s["kc"]), "v": _shown(s["vc"]),
            "weights": s["weights"]}


def _plain_evict(s):
    c = s["c"]
    n, hkv, block, keep = c["seqs"], c["kv_heads"], c["block"], c["keep"]
    w = s["weights"][s["bt"].long().clamp(min=0)].transpose(1, 2).flatten(2)  # n, kv, tokens
    t, lens = torch.arange(w.shape[2], device=DEV), s["lens"].long()[:, None, None]
    w = w.masked_fill((t < c["sink"]) | (t >= lens - c["recent"]), float("inf")).masked_fill(t >= lens, float("-inf"))
    if w.shape[2] < keep:
        w = torch.nn.functional.pad(w, (0, keep - w.shape[2]), value=float("-inf"))
    chosen = w.sort(dim=2, descending=True, stable=True).indices[:, :, :keep]  # ties: the lowest index
    count, rank = s["lens"].clamp(max=keep), torch.arange(keep, device=DEV)
    valid = rank < count.long()[:, None, None]
    chosen = torch.where(valid, chosen, 1 << 30).sort(dim=2).values
    s["kept"].copy_(torch.where(valid, chosen, -1))
    s["kept_lens"].copy_(count)
    b, h, i = valid.expand(n, hkv, keep).nonzero(as_tuple=True)
    t = chosen[b, h, i]
    src, dst = s["bt"][b, t // block].long(), s["new_bt"][b, i // block].long()
    for x in (s["kc"], s["vc"], s["weights"]):
        x[dst, h, i % block] = x[src, h, t % block]
    return {"kept": s["kept"], "kept_lens": s["kept_lens"], "k": _shown(s["kc"]), "v": _shown(s["vc"]),
            "weights": s["weights"]}


_RUN_OWN = {"axes": _own_axes, "append4": _own_append4, "attn4": _own_attn4, "weights": _own_weights,
            "evict": _own_evict}
_RUN_PLAIN = {"axes": _plain_axes, "append4": _plain_append4, "attn4": _plain_attn4, "weights": _plain_weights,
              "evict": _plain_evict}


# ------------------------------------------------------------------ from the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    d, hkv, n, block, kind = c["head_dim"], c["kv_heads"], c["seqs"], c["block"], c["cache"]
    f = lambda x: (x.view(E4M3).float() if x.dtype == torch.uint8 else x).double()  # noqa: E731
    lens = s["lens"].tolist()

    def four(x, scale):
        """The values that 64-bit rows [.., d] have in 4 bits."""
        parts = []
        for x in x.split(16, -1):
            e = (x.abs().max(-1, keepdim=True).values / (7 * scale)).clamp(max=448).float().to(E4M3).double() * scale
            parts.append(torch.where(e > 0, torch.round(x / e.clamp(min=1e-300)).clamp(-7, 7) * e, 0.0))
        return torch.cat(parts, -1)

    if c["kind"] in ("axes", "append4"):
        r, half, starts = c["rotary"], c["rotary"] // 2, s["starts"].tolist()
        kind_k = [torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV) for _ in range(2)] if kind == I4 else [
            f(s["kc"]), f(s["vc"])]
        qs = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        col = torch.arange(half, device=DEV)
        for b in range(n):
            a, e = starts[b], starts[b + 1]
            pos = torch.arange(lens[b], lens[b] + e - a, device=DEV)
            rows = pos[:, None].expand(-1, half)
            if s["axes"] is not None:
                rows = torch.stack([s["positions"][int(x), a:e] for x in s["axes"].tolist()], 1).long()
            w = torch.complex(s["rope"][rows, col].double(), s["rope"][rows, half + col].double())[:, None]
            at = s["bt"][b].long()[pos // block]
            for x, cache, scale in ((s["q"], None, 1), (s["k"], kind_k[0], s["ks"]), (s["v"], kind_k[1], s["vs"])):
                y = x[a:e].double()
                if x is not s["v"]:
                    if c["pairs"]:
                        z = torch.complex(y[..., 0:r:2], y[..., 1:r:2]) * w
                        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
                    else:
                        z = torch.complex(y[..., :half], y[..., half:r]) * w
                        y[..., :half], y[..., half:r] = z.real, z.imag
                if cache is None:
                    qs[a:e] = y
                elif kind == I4:
                    cache[a:e] = four(y, scale)
                else:
                    cache[at, :, pos % block] = y / scale
        return {"q": qs, "k": kind_k[0], "v": kind_k[1]}

    def tokens(cache, b, g, length, scale):
        at = s["bt"][b, :-(-length // block)].long()
        if kind != I4:
            return f(cache[at, g]).reshape(-1, d)[:length] * scale
        raw = cache[at, g].reshape(len(at), -1).long()
        r, i = torch.arange(block, device=DEV)[:, None], torch.arange(d, device=DEV)
        u = (raw[:, (i // 32 * block + r) * 16 + i % 32 // 2] >> (i % 2 * 4)) & 15
        e = raw[:, block * d // 2 + r * (d // 16) + i // 16].to(torch.uint8).view(E4M3).double()
        return ((u - 8) * e).reshape(-1, d)[:length] * scale

    if c["kind"] == "evict":
        k, v, w = f(s["kc"]), f(s["vc"]), s["weights"].double()
        if n * hkv > 1500:
            return None
        for b in range(n):
            m = min(lens[b], c["keep"])
            t = torch.arange(lens[b], device=DEV)
            src, dst = s["bt"][b].long()[t // block], s["new_bt"][b].long()
            i = torch.arange(m, device=DEV)
            for g in range(hkv):
                x = w[src, g, t % block]
                always = (t < c["sink"]) | (t >= lens[b] - c["recent"])
                first = torch.cat((t[always], t[~always][(-x[~always]).sort(stable=True).indices]))[:m].sort().values
                pick = first if lens[b] > c["keep"] else t
                for cache in (k, v, w):
                    cache[dst[i // block], g, i % block] = cache[src[pick], g, pick % block]
        return {"kept": None, "kept_lens": None, "k": k, "v": v, "weights": w}
    ql, grp = c["q_len"], c["q_heads"] // hkv
    if n * hkv > 2500:
        return None
    q = s["q"].double().view(n, ql, hkv, grp, d)
    out = torch.zeros(n, ql, hkv, grp, d, dtype=torch.float64, device=DEV)
    w = s["weights"].double() if c["kind"] == "weights" else None
    for b in range(n):
        t = torch.arange(lens[b], device=DEV)
        hidden = (t > lens[b] - ql + torch.arange(ql, device=DEV)[:, None])[:, None]
        for g in range(hkv):
            x = (q[b, :, g] @ tokens(s["kc"], b, g, lens[b], s["ks"]).t() * s["scale"]).masked_fill(hidden, -math.inf)
            p = torch.softmax(x, -1)
            if w is None:
                out[b, :, g] = p @ tokens(s["vc"], b, g, lens[b], s["vs"])
            else:
                at = s["bt"][b].long()[t // block]
                old = w[at, g, t % block] * c["decay"]
                old[lens[b] - ql:] = 0
                w[at, g, t % block] = old + p.sum((0, 1))
    return w if w is not None else out.view(s["q"].shape)
