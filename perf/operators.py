"""Cases of the serving-step operators around paged decode attention: their inputs, their plain forms in
elementary torch operations, and the library's calls.

Kinds of case:
  append  rotation of q and k by position, and the write of k and v into the paged cache (prompts, single tokens)
  prefix  decode attention of a batch whose groups of sequences share a long prefix in the cache
  bounds  the elementwise minimum and maximum of every cache block's keys
  sparse  the choice of each sequence's most promising blocks by those bounds, and attention over them alone
"""
import math

import torch

own = False  # set from outside: the library's kernels instead of the plain forms

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def _append(name, seqs, lo, hi, past, q_heads, kv_heads, head_dim=128, rotary=128, block=16, fp8=False, pairs=False):
    return {"name": name, "kind": "append", "seqs": seqs, "new_lo": lo, "new_hi": hi, "past": past,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "rotary": rotary, "block": block,
            "fp8": fp8, "pairs": pairs}


def _prefix(name, seqs, q_len, groups, prefix, lo, hi, q_heads, kv_heads, head_dim=128, block=16, fp8=False):
    return {"name": name, "kind": "prefix", "seqs": seqs, "q_len": q_len, "groups": groups, "prefix": prefix,
            "own_lo": lo, "own_hi": hi, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "block": block, "fp8": fp8}


def _bounds(name, seqs, lo, hi, new, kv_heads, head_dim=128, block=16, fp8=False):
    return {"name": name, "kind": "bounds", "seqs": seqs, "len_lo": lo, "len_hi": hi, "new": new,
            "kv_heads": kv_heads, "head_dim": head_dim, "block": block, "fp8": fp8}


def _sparse(name, seqs, lo, hi, keep, sink, recent, q_heads, kv_heads, head_dim=128, block=16, fp8=False):
    return {"name": name, "kind": "sparse", "seqs": seqs, "len_lo": lo, "len_hi": hi, "keep": keep, "sink": sink,
            "recent": recent, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "block": block,
            "fp8": fp8}


def listed():
    return [
        # one token for each of a few sequences: the latency of a single decode step
        _append("append_token_few", 4, 1, 1, 2000, 32, 8),
        # a full decode batch over E4M3 caches
        _append("append_token_batch_e4m3", 256, 1, 1, 1023, 28, 4, fp8=True),
        # ragged prompts written in one go, half of every head rotated in adjacent pairs
        _append("append_prompts", 13, 17, 4096, 0, 40, 8, rotary=64, pairs=True),
        # a few requests over one short system prompt: latency
        _prefix("prefix_few", 4, 1, 1, 1000, 1, 128, 32, 8),
        # a chat batch over one system prompt
        _prefix("prefix_chat", 64, 1, 1, 4096, 64, 1024, 32, 8),
        # draft tokens verified over E4M3 caches, two prompts in one batch
        _prefix("prefix_verify_e4m3", 48, 4, 2, 8192, 100, 512, 28, 4, fp8=True),
        # many continuations of one long document
        _prefix("prefix_document", 256, 1, 1, 32768, 64, 512, 28, 4),
        # the blocks that one new token of each sequence touched
        _bounds("bounds_token", 128, 512, 4096, 1, 8),
        # every block of freshly written prompts
        _bounds("bounds_prompts", 32, 4000, 8192, 8192, 8),
        # one long conversation: latency
        _sparse("sparse_one", 1, 32768, 32768, 64, 1, 2, 32, 8),
        # long contexts of a batch
        _sparse("sparse_batch", 32, 16384, 32768, 128, 1, 4, 40, 8),
        # longer ones over E4M3 caches
        _sparse("sparse_long_e4m3", 64, 30000, 65536, 256, 4, 8, 28, 4, fp8=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((32, 32), (32, 8), (28, 4), (40, 8), (4, 4), (8, 1), (18, 3))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        kind = rng.choice(("append", "append", "prefix", "prefix", "prefix", "bounds", "sparse", "sparse"))
        hq, hkv = rng.choice(HEADS)
        d, block, fp8 = rng.choice((64, 128, 128)), rng.choice((16, 16, 32)), rng.random() < 0.4
        seqs = _log(rng, 1, 256)
        if kind == "append":
            hi = _log(rng, 1, 4096) if rng.random() < 0.6 else 1
            c = _append("", seqs, max(1, hi // rng.randint(1, 9)), hi, _log(rng, 1, 8000), hq, hkv, d,
                        rng.choice((d, d, 32)), block, fp8, rng.random() < 0.4)
            if seqs * hi > 60000:
                continue
        elif kind == "prefix":
            hi = _log(rng, 1, 2000)
            c = _prefix("", seqs, rng.choice((1, 1, 1, 2, 5)), min(seqs, rng.choice((1, 1, 2, 3))),
                        _log(rng, 40, 32768), max(1, hi // rng.randint(1, 9)), hi, hq, hkv, d, block, fp8)
            c["own_lo"], c["own_hi"] = max(c["own_lo"], c["q_len"]), max(c["own_hi"], c["q_len"])
            if seqs * c["q_len"] > 512:
                continue
        elif kind == "bounds":
            hi = _log(rng, 1, 8192)
            c = _bounds("", seqs, max(1, hi // rng.randint(1, 9)), hi, rng.choice((1, 5, hi)), hkv, d, block, fp8)
        else:
            hi = _log(rng, 200, 65536)
            keep = _log(rng, 8, 300)
            c = _sparse("", seqs, max(1, hi // rng.randint(1, 9)), hi, keep, rng.randint(0, 2), rng.randint(1, 4),
                        hq, hkv, d, block, fp8)
        size = seqs * max(c.get("own_hi", 0), c.get("len_hi", 0), c.get("past", 0)) * hkv * d * 4
        if size <= 6e9 and _cost(c) <= most:
            del c["name"]
            return c


# ------------------------------------------------------------------ sizes
def _spread(lo, hi, n):
    """n lengths from lo to hi in a fixed mixed order (the golden-ratio sequence)."""
    return [lo + int((hi - lo + 1) * ((k * 0.6180339887498949 + 0.37) % 1.0)) if hi > lo else lo for k in range(n)]


def _group_sizes(c):
    n, k = c["seqs"], c["groups"]
    return [n // k + (1 if i < n % k else 0) for i in range(k)]


def _prefix_lens(c):
    return [max(1, c["prefix"] - 37 * i) for i in range(c["groups"])]


def work(c):
    e = 1 if c["fp8"] else 2
    d, hkv, n = c["head_dim"], c["kv_heads"], c["seqs"]
    if c["kind"] == "append":
        t = sum(_spread(c["new_lo"], c["new_hi"], n))
        positions = min(t, c["past"] + c["new_hi"])
        byt = t * d * (c["q_heads"] * 4 + hkv * 2 * (2 + e)) + positions * c["rotary"] * 4 + t * 4
        return {"bytes": byt, "flops": 3 * t * (c["q_heads"] + hkv) * c["rotary"]}
    if c["kind"] == "bounds":
        first = [max(0, x - c["new"]) // c["block"] * c["block"] for x in _spread(c["len_lo"], c["len_hi"], n)]
        toks = sum(x - f for x, f in zip(_spread(c["len_lo"], c["len_hi"], n), first))
        blocks = sum(-(-(x - f) // c["block"]) for x, f in zip(_spread(c["len_lo"], c["len_hi"], n), first))
        return {"bytes": (toks + 2 * blocks) * hkv * d * e + 4 * blocks, "flops": 2 * toks * hkv * d}
    hq = c["q_heads"]
    if c["kind"] == "prefix":
        rows = [s * c["q_len"] * hq for s in _group_sizes(c)]
        pre, own_t = _prefix_lens(c), sum(_spread(c["own_lo"], c["own_hi"], n))
        byt = (sum(pre) + own_t) * hkv * d * 2 * e + 2 * n * c["q_len"] * hq * d * 2
        return {"bytes": byt, "flops": 4 * d * (sum(r * p for r, p in zip(rows, pre)) + own_t * c["q_len"] * hq)}
    lens = _spread(c["len_lo"], c["len_hi"], n)
    blocks = [-(-x // c["block"]) for x in lens]
    kept = sum(min(b, c["keep"]) for b in blocks)
    # where a sequence has no more blocks than are kept, nothing has to be scored
    scored = sum(b for b in blocks if b > c["keep"])
    byt = (scored * 2 * d * e + kept * c["block"] * d * 2 * e) * hkv + 2 * n * hq * d * 2 + 4 * kept * hkv
    return {"bytes": byt, "flops": (4 * d * scored + 4 * d * kept * c["block"]) * hq}


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


# ------------------------------------------------------------------ inputs
def _normal(shape, g, scale=1.0):
    out = torch.empty(shape, dtype=torch.float16, device=DEV)
    flat = out.view(-1)
    for s in range(0, flat.numel(), 1 << 26):
        e = min(flat.numel(), s + (1 << 26))
        flat[s:e] = torch.randn(e - s, generator=g, device=DEV) * scale
    return out


def _cache(shape, g, fp8):
    """~N(0,1) values; E4M3: codes of N(0,1) / scale at a per-cache scale of 1/64."""
    if not fp8:
        return _normal(shape, g)
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = out.view(-1)
    for s in range(0, flat.numel(), 1 << 26):
        e = min(flat.numel(), s + (1 << 26))
        x = torch.randn(e - s, generator=g, device=DEV) * 64.0
        flat[s:e] = x.clamp_(-448, 448).to(E4M3).view(torch.uint8)
    return out


def _tables(lens, block, extra, g):
    """Block tables of a seeded permutation of a pool a tenth larger than needed, `extra` blocks of it left over."""
    per = [-(-x // block) for x in lens]
    pool = max(1, -(-(sum(per) + extra) * 11 // 10))
    perm = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int32)
    need = torch.tensor(per, device=DEV)
    width = max(1, max(per))
    i = torch.arange(width, device=DEV)
    start = (need.cumsum(0) - need)[:, None] + i
    bt = torch.where(i < need[:, None], perm[start.clamp(max=pool - 1)], -1).to(torch.int32)
    return bt, pool, perm[sum(per):]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    d, hkv, n, block = c["head_dim"], c["kv_heads"], c["seqs"], c["block"]
    s = dict(c=c, ks=1 / 64.0, vs=1 / 64.0, scale=1.0 / math.sqrt(d), err=torch.zeros(1, dtype=torch.int32, device=DEV))
    if c["kind"] == "append":
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
        shape = (pool, hkv, block, d)
        kind = torch.uint8 if c["fp8"] else torch.float16
        s["kc"], s["vc"] = torch.zeros(shape, dtype=kind, device=DEV), torch.zeros(shape, dtype=kind, device=DEV)
        s["q_out"] = torch.zeros((t, hq, d), dtype=torch.float16, device=DEV)
        return s
    if c["kind"] == "prefix":
        own_l, pre = _spread(c["own_lo"], c["own_hi"], n), _prefix_lens(c)
        need = sum(-(-x // block) for x in pre)
        s["bt"], pool, rest = _tables(own_l, block, need, g)
        ptab = torch.full((c["groups"], -(-max(pre) // block)), -1, dtype=torch.int32, device=DEV)
        at = 0
        for i, x in enumerate(pre):
            m = -(-x // block)
            ptab[i, :m] = rest[at:at + m]
            at += m
        sizes = _group_sizes(c)
        s.update(ptab=ptab, plens=_ints(pre), gstarts=_ints([0] + torch.tensor(sizes).cumsum(0).tolist()),
                 lens=_ints(own_l), max_own=max(own_l), max_prefix=max(pre), sizes=sizes, pre=pre)
        shape = (pool, hkv, block, d)
        s["kc"], s["vc"] = _cache(shape, g, c["fp8"]), _cache(shape, g, c["fp8"])
        q = (n, c["q_len"], c["q_heads"], d) if c["q_len"] > 1 else (n, c["q_heads"], d)
        s["q"] = _normal(q, g)
        s["out"] = torch.empty_like(s["q"])
        s["ws"] = None
        return s
    lens = _spread(c["len_lo"], c["len_hi"], n)
    s["bt"], pool, _ = _tables(lens, block, 0, g)
    s["lens"], s["max_len"] = _ints(lens), max(lens)
    s["kc"] = _cache((pool, hkv, block, d), g, c["fp8"])
    kind = torch.uint8 if c["fp8"] else torch.float16
    if c["kind"] == "bounds":
        s["first"] = _ints([max(0, x - c["new"]) for x in lens])
        s["most_new"] = max(min(x, c["new"]) for x in lens)
        s["bounds"] = torch.zeros((pool, hkv, 2, d), dtype=kind, device=DEV)
        return s
    s["vc"] = _cache((pool, hkv, block, d), g, c["fp8"])
    s["bounds"] = torch.empty((pool, hkv, 2, d), dtype=kind, device=DEV)
    for a in range(0, pool, 1 << 13):  # every block, its last tokens included
        x = _values(s["kc"][a:a + (1 << 13)])
        s["bounds"][a:a + (1 << 13)] = _codes(torch.stack((x.amin(2), x.amax(2)), 2), c["fp8"])
    s["q"] = _normal((n, c["q_heads"], d), g)
    s["out"] = torch.empty_like(s["q"])
    s["lists"] = torch.empty((n, hkv, c["keep"]), dtype=torch.int32, device=DEV)
    s["counts"] = torch.empty((n, hkv), dtype=torch.int32, device=DEV)
    s["ws"] = None
    return s


def _values(x):
    """The fp32 values of cache elements (E4M3: the code's value, without the per-cache scale)."""
    return x.view(E4M3).float() if x.dtype == torch.uint8 else x.float()


def _codes(x, fp8):
    return x.to(E4M3).view(torch.uint8) if fp8 else x.half()


def _shown(x):
    """A cache as its values: byte caches as E4M3 numbers."""
    return x.view(E4M3) if x.dtype == torch.uint8 else x


# ------------------------------------------------------------------ one pass
def run(s):
    return (_RUN_OWN if own else _RUN_PLAIN)[s["c"]["kind"]](s)


def _workspace(s, nbytes, ops):
    """A program keeps its workspace from call to call."""
    if s["ws"] is None and nbytes:
        s["ws"] = ops.alloc_workspace(nbytes, DEV)
    return s["ws"]


def _own_append(s):
    from paged_kv_decode_21_gb300 import ops
    if s["c"]["fp8"]:
        ops.paged_kv_append_rope_fp8(s["q"], s["k"], s["v"], s["rope"], s["bt"], s["lens"], s["kc"], s["vc"],
                                     s["ks"], s["vs"], token_starts=s["starts"], interleaved=s["c"]["pairs"],
                                     q_out=s["q_out"], error_word=s["err"])
    else:
        ops.paged_kv_append_rope(s["q"], s["k"], s["v"], s["rope"], s["bt"], s["lens"], s["kc"], s["vc"],
                                 token_starts=s["starts"], interleaved=s["c"]["pairs"], q_out=s["q_out"],
                                 error_word=s["err"])
    return {"q": s["q_out"], "k": _shown(s["kc"]), "v": _shown(s["vc"])}


def _rotated(x, cos, sin, r, pairs):
    x = x.to(cos.dtype)
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., :r // 2], x[..., r // 2:r])
    y, z = a * cos - b * sin, b * cos + a * sin
    rot = torch.stack((y, z), -1).flatten(-2) if pairs else torch.cat((y, z), -1)
    return torch.cat((rot, x[..., r:]), -1)


def _plain_append(s):
    c, r, block = s["c"], s["c"]["rotary"], s["c"]["block"]
    t = torch.arange(s["q"].shape[0], device=DEV, dtype=torch.int32)
    b = torch.searchsorted(s["starts"][1:], t, right=True)
    pos = (s["lens"][b] + t - s["starts"][b]).long()
    cs = s["rope"][pos]
    cos, sin = cs[:, None, :r // 2], cs[:, None, r // 2:]
    s["q_out"].copy_(_rotated(s["q"], cos, sin, r, c["pairs"]))
    k, v = _rotated(s["k"], cos, sin, r, c["pairs"]), s["v"].float()
    if c["fp8"]:
        k = _codes((k / s["ks"]).clamp(-448, 448), True)
        v = _codes((v / s["vs"]).clamp(-448, 448), True)
    else:
        k, v = k.half(), v.half()
    at = s["bt"][b, pos // block].long()
    s["kc"][at, :, pos % block] = k
    s["vc"][at, :, pos % block] = v
    return {"q": s["q_out"], "k": _shown(s["kc"]), "v": _shown(s["vc"])}


def _own_prefix(s):
    from paged_kv_decode_21_gb300 import ops
    c = s["c"]
    if s["ws"] is None:
        _workspace(s, ops.paged_decode_prefix_workspace_size(
            c["seqs"], c["q_len"], c["q_heads"], c["kv_heads"], c["head_dim"], c["block"], c["groups"],
            s["max_prefix"], s["max_own"]), ops)
    kw = dict(out=s["out"], max_prefix_len=s["max_prefix"], max_context_len=s["max_own"], workspace=s["ws"],
              error_word=s["err"])
    if c["fp8"]:
        return ops.paged_decode_attention_prefix_fp8(s["q"], s["kc"], s["vc"], s["ptab"], s["plens"], s["gstarts"],
                                                     s["bt"], s["lens"], s["scale"], s["ks"], s["vs"], **kw)
    return ops.paged_decode_attention_prefix(s["q"], s["kc"], s["vc"], s["ptab"], s["plens"], s["gstarts"], s["bt"],
                                             s["lens"], s["scale"], **kw)


def _rows(cache, table, block):
    """[sequences][kv heads][tokens][head_dim] values of the blocks in `table` (whole blocks)."""
    x = _values(cache[table.long().clamp(min=0)])  # n, m, kv, block, d
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_prefix(s):
    c = s["c"]
    d, hkv, ql, block = c["head_dim"], c["kv_heads"], c["q_len"], c["block"]
    grp = c["q_heads"] // hkv
    ks, vs = (s["ks"], s["vs"]) if c["fp8"] else (1.0, 1.0)
    q = s["q"].float().view(c["seqs"], ql, hkv, grp, d).permute(0, 2, 1, 3, 4) * (s["scale"] * ks)  # n, kv, ql, grp, d
    ko, vo = _rows(s["kc"], s["bt"], block), _rows(s["vc"], s["bt"], block)
    so = torch.einsum("nkqgd,nktd->nkqgt", q, ko)
    t = torch.arange(ko.shape[2], device=DEV)
    seen = s["lens"].long()[:, None] - ql + 1 + torch.arange(ql, device=DEV)  # tokens that draft token j sees
    so = so.masked_fill((t >= seen[:, :, None])[:, None, :, None, :], float("-inf"))
    out = torch.empty(c["seqs"], ql, hkv, grp, d, device=DEV)
    at = 0
    for i, size in enumerate(s["sizes"]):  # the few groups, each with its own prefix
        e = at + size
        m = -(-s["pre"][i] // block)
        kp = _rows(s["kc"], s["ptab"][i:i + 1, :m], block)[0, :, :s["pre"][i]]
        vp = _rows(s["vc"], s["ptab"][i:i + 1, :m], block)[0, :, :s["pre"][i]]
        for g in range(hkv):  # a head at a time: the scores of all would not fit
            sp = q[at:e, g].reshape(-1, d) @ kp[g].t()
            sg = so[at:e, g].reshape(size * ql * grp, -1)
            top = torch.maximum(sp.amax(1, keepdim=True), sg.amax(1, keepdim=True))
            pp, po = (sp - top).exp_(), (sg - top).exp_()
            o = pp @ vp[g] + torch.einsum("nrt,ntd->nrd", po.view(size, ql * grp, -1), vo[at:e, g]).reshape(-1, d)
            o = o / (pp.sum(1, keepdim=True) + po.sum(1, keepdim=True))
            out[at:e, :, g] = o.view(size, ql, grp, d)
        at = e
    s["out"].copy_((out * vs).view(s["out"].shape))
    return s["out"]


def _own_bounds(s):
    from paged_kv_decode_21_gb300 import ops
    ops.paged_kv_block_bounds(s["kc"], s["bt"], s["lens"], s["bounds"], start_lens=s["first"],
                              max_new_tokens=s["most_new"], error_word=s["err"])
    return _shown(s["bounds"])


def _plain_bounds(s):
    block = s["c"]["block"]
    first, last = s["first"].long() // block, (s["lens"].long() - 1) // block
    i = first[:, None] + torch.arange((s["most_new"] + block - 2) // block + 1, device=DEV)
    i = torch.minimum(i, last[:, None])  # past the last block: the last one again
    at = s["bt"].gather(1, i).long()
    x = _values(s["kc"][at])  # n, m, kv, block, d
    tok = i[:, :, None] * block + torch.arange(block, device=DEV)
    off = (tok >= s["lens"].long()[:, None, None])[:, :, None, :, None]
    lo, hi = x.masked_fill(off, float("inf")).amin(3), x.masked_fill(off, float("-inf")).amax(3)
    s["bounds"][at] = _codes(torch.stack((lo, hi), 3), s["c"]["fp8"])
    return _shown(s["bounds"])


def _own_sparse(s):
    from paged_kv_decode_21_gb300 import ops
    c = s["c"]
    if s["ws"] is None:
        _workspace(s, ops.paged_decode_blocks_workspace_size(c["seqs"], c["q_heads"], c["kv_heads"], c["head_dim"],
                                                             c["block"], c["keep"]), ops)
    ops.paged_kv_block_select(s["q"], s["bounds"], s["bt"], s["lens"], c["keep"], block_size=c["block"],
                              sink_blocks=c["sink"], recent_blocks=c["recent"], max_context_len=s["max_len"],
                              block_lists=s["lists"], list_lens=s["counts"], error_word=s["err"])
    kw = dict(out=s["out"], workspace=s["ws"], error_word=s["err"])
    if c["fp8"]:
        ops.paged_decode_attention_blocks_fp8(s["q"], s["kc"], s["vc"], s["bt"], s["lens"], s["lists"], s["counts"],
                                              s["scale"], s["ks"], s["vs"], **kw)
    else:
        ops.paged_decode_attention_blocks(s["q"], s["kc"], s["vc"], s["bt"], s["lens"], s["lists"], s["counts"],
                                          s["scale"], **kw)
    return {"lists": s["lists"], "counts": s["counts"], "out": s["out"]}


def _plain_sparse(s):
    c = s["c"]
    n, d, hkv, block, keep = c["seqs"], c["head_dim"], c["kv_heads"], c["block"], c["keep"]
    grp = c["q_heads"] // hkv
    q = s["q"].double().view(n, hkv, grp, d)
    blocks = ((s["lens"].long() + block - 1) // block)[:, None, None]
    i = torch.arange(s["bt"].shape[1], device=DEV)
    # the largest product that any key inside the bounds can have: in 64 bits, for blocks next to the border
    e = s["bounds"][s["bt"].long().clamp(min=0)]  # n, m, kv, 2, d
    e = (e.view(E4M3).half() if c["fp8"] else e).permute(0, 2, 3, 1, 4)
    score = torch.matmul(q.clamp(max=0), e[:, :, 0].double().transpose(2, 3))
    score += torch.matmul(q.clamp(min=0), e[:, :, 1].double().transpose(2, 3))
    score = score.amax(2)
    score = score.masked_fill((i < c["sink"]) | (i >= blocks - c["recent"]), float("inf"))
    score = score.masked_fill(i >= blocks, float("-inf"))
    if score.shape[2] < keep:
        score = torch.nn.functional.pad(score, (0, keep - score.shape[2]), value=float("-inf"))
    chosen = score.sort(dim=2, descending=True, stable=True).indices[:, :, :keep]  # ties: the lowest index
    count = blocks.clamp(max=keep)
    rank = torch.arange(keep, device=DEV)
    chosen = torch.where(rank < count, chosen, 1 << 30).sort(dim=2).values
    lists = torch.where(rank < count, chosen, -1).expand(n, hkv, keep)
    at = s["bt"].long()[:, None, :].expand(n, hkv, -1).gather(2, lists.clamp(min=0)).clamp(min=0)
    h = torch.arange(hkv, device=DEV)[None, :, None]
    ks, vs = (s["ks"], s["vs"]) if c["fp8"] else (1.0, 1.0)
    k, v = _values(s["kc"][at, h]).flatten(2, 3), _values(s["vc"][at, h]).flatten(2, 3)  # n, kv, keep * block, d
    tok = (lists[..., None] * block + torch.arange(block, device=DEV)).flatten(2)
    off = (tok < 0) | (tok >= s["lens"].long()[:, None, None])
    sc = torch.matmul(q.float() * (s["scale"] * ks), k.transpose(2, 3)).masked_fill(off[:, :, None], float("-inf"))
    p = (sc - sc.amax(3, keepdim=True)).exp_()
    o = torch.matmul(p, v) * vs / p.sum(3, keepdim=True)
    s["out"].copy_(o.view(n, c["q_heads"], d))
    s["lists"].copy_(lists)
    s["counts"].copy_(count[:, :, 0].expand(n, hkv))
    return {"lists": s["lists"], "counts": s["counts"], "out": s["out"]}


_RUN_OWN = {"append": _own_append, "prefix": _own_prefix, "bounds": _own_bounds, "sparse": _own_sparse}
_RUN_PLAIN = {"append": _plain_append, "prefix": _plain_prefix, "bounds": _plain_bounds, "sparse": _plain_sparse}


# ------------------------------------------------------------------ from the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    d, hkv, n, block = c["head_dim"], c["kv_heads"], c["seqs"], c["block"]
    f = lambda x: (x.view(E4M3).float() if x.dtype == torch.uint8 else x).double()  # noqa: E731
    lens = s["lens"].tolist()
    if c["kind"] == "append":
        r, half, starts = c["rotary"], c["rotary"] // 2, s["starts"].tolist()
        caches = [f(s["kc"]), f(s["vc"])]
        qs = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        for b in range(n):
            a, e = starts[b], starts[b + 1]
            pos = torch.arange(lens[b], lens[b] + e - a, device=DEV)
            w = torch.complex(s["rope"][pos, :half].double(), s["rope"][pos, half:].double())[:, None]
            at = s["bt"][b].long()[pos // block]
            for x, cache in ((s["q"], None), (s["k"], caches[0]), (s["v"], caches[1])):
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
                else:
                    cache[at, :, pos % block] = y / (s["ks"] if cache is caches[0] else s["vs"]) if c["fp8"] else y
        return {"q": qs, "k": caches[0], "v": caches[1]}
    if c["kind"] == "bounds":
        out = f(s["bounds"])
        first = s["first"].tolist()
        for b in range(n):
            for i in range(first[b] // block, -(-lens[b] // block)) if c["new"] <= 64 else ():
                p = int(s["bt"][b, i])
                x = f(s["kc"][p, :, :min(block, lens[b] - i * block)])
                out[p, :, 0], out[p, :, 1] = x.min(1).values, x.max(1).values
            if c["new"] > 64:  # many blocks: the whole ones at once, the last alone
                lo, hi = first[b] // block, lens[b] // block
                p = s["bt"][b, lo:hi].long()
                x = f(s["kc"][p])
                out[p, :, 0], out[p, :, 1] = x.min(2).values, x.max(2).values
                if lens[b] % block:
                    p = int(s["bt"][b, hi])
                    x = f(s["kc"][p, :, :lens[b] % block])
                    out[p, :, 0], out[p, :, 1] = x.min(1).values, x.max(1).values
        return out
    ks, vs = (s["ks"], s["vs"]) if c["fp8"] else (1.0, 1.0)
    grp = c["q_heads"] // hkv

    def tokens(cache, table, length, g):
        m = -(-length // block)
        return f(cache[table[:m].long(), g]).reshape(-1, d)[:length]

    if c["kind"] == "prefix":
        ql = c["q_len"]
        if n * hkv * ql > 6000:
            return None
        out = torch.zeros(n, ql, hkv, grp, d, dtype=torch.float64, device=DEV)
        q = s["q"].double().view(n, ql, hkv, grp, d)
        of = [i for i, size in enumerate(s["sizes"]) for _ in range(size)]
        for g in range(hkv):
            shared = [(tokens(s["kc"], s["ptab"][i], x, g), tokens(s["vc"], s["ptab"][i], x, g))
                      for i, x in enumerate(s["pre"])]
            for b in range(n):
                k0, v0 = shared[of[b]]
                k = torch.cat((k0, tokens(s["kc"], s["bt"][b], lens[b], g)))
                v = torch.cat((v0, tokens(s["vc"], s["bt"][b], lens[b], g)))
                for j in range(ql):
                    seen = len(k0) + lens[b] - ql + 1 + j
                    p = torch.softmax(q[b, j, g] @ k[:seen].t() * (s["scale"] * ks), -1)
                    out[b, j, g] = p @ v[:seen] * vs
        return out.view(s["q"].shape)
    if n * hkv > 2500:
        return None
    out = torch.zeros(n, hkv, grp, d, dtype=torch.float64, device=DEV)
    q = s["q"].double().view(n, hkv, grp, d)
    for b in range(n):
        m = -(-lens[b] // block)
        p = s["bt"][b, :m].long()
        e = f(s["bounds"][p])  # m, kv, 2, d
        tail = lens[b] - (m - 1) * block
        for g in range(hkv):
            x = q[b, g][:, None]
            best = torch.maximum(x * e[:, g, 0], x * e[:, g, 1]).sum(2).amax(0)
            always = set(range(min(c["sink"], m))) | set(range(max(0, m - c["recent"]), m))
            rest = [i for i in (-best).sort(stable=True).indices.tolist() if i not in always]
            pick = sorted(list(always) + rest[:max(0, min(c["keep"], m) - len(always))]) if m > c["keep"] else list(range(m))
            at = p[torch.tensor(pick, device=DEV)]
            length = len(pick) * block - (block - tail if pick[-1] == m - 1 else 0)
            k, v = f(s["kc"][at, g]).reshape(-1, d)[:length], f(s["vc"][at, g]).reshape(-1, d)[:length]
            out[b, g] = torch.softmax(q[b, g] @ k.t() * (s["scale"] * ks), -1) @ v * vs
    return {"lists": None, "counts": None, "out": out.view(s["q"].shape)}
