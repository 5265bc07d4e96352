"""Gathered attention weights where a partition has more than a slot of every warp's ring (1024 tokens and more, as
large batches plan them), with blocks missing late in it; and softmax scales of any sign."""
import math

import pytest
import torch

import longcache_ref as ref
from serving_ref import deal_tables
from test_gpu_evict import SCALE, cache_of, doubles, i32
from test_gpu_int4_paths import ragged
from paged_kv_decode_21_gb300 import ops, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"


def up(x, a):
    return -(-x // a) * a


def planned_partition(B, ql, Hq, H, D, BS, most):
    """The partition that a call plans, from the size of its workspace (statistics of every row and partition, and
    the scores of up to 16 rows)."""
    rows = ql * Hq // H
    size = ops.paged_kv_attention_weights_workspace_size(B, ql, Hq, H, D, BS, most)
    found = []
    for part in (128, 256, 512, 1024, 2048, 4096):
        np = -(-most // part)
        total = 2 * up(4 * B * H * np * rows, 256)
        if rows <= 16:
            total += up(4 * B * H * rows * up(np * part, 64), 256)
        if total == size:
            found.append(part)
    assert len(found) == 1, found
    return found[0]


def weights_after(q, k, bt, lens, weights, scale, start, decay, BS):
    """weights after the call in double, over the tokens whose block is in the pool; k double [NB][H][BS][D]."""
    B, ql, Hq, D = q.shape
    NB, H = k.shape[:2]
    G = Hq // H
    out, most = weights.double().clone(), 0.0
    for b in range(B):
        t = torch.arange(lens[b], device=DEV)
        at = bt[b, t // BS].long()
        t, at = t[(at >= 0) & (at < NB)], at[(at >= 0) & (at < NB)]
        if not t.numel():
            continue
        seen = t <= (lens[b] - ql + torch.arange(ql, device=DEV))[:, None]
        for g in range(H):
            kk = k[at, g, t % BS]
            x = q[b, :, g * G:(g + 1) * G].double()
            s = x @ kk.t() * scale
            most = max(most, float((x.abs() @ kk.abs().t()).max()) * abs(scale) * ref.LOG2E)
            p = torch.softmax(s.masked_fill(~seen[:, None], -math.inf), -1)
            p = torch.where(seen.any(1)[:, None, None], p, 0.0).sum((0, 1))
            first = lens[b] if start is None else start[b]
            old = torch.where(t < first, weights[at, g, t % BS].double() * decay, 0.0) if decay else 0.0
            out[at, g, t % BS] = old + p
    return out, most


def run(kind, D, BS, Hq, H, ql, lens, most, seed, scale=None, start=None, decay=1.0, bad=()):
    scale = D ** -0.5 if scale is None else scale
    need = sum(-(-n // BS) for n in lens)
    bt, _ = deal_tables(lens, BS, -(-most // BS), need + 3, seed)
    NB = need + 3
    for i, (b, n) in enumerate(bad):
        bt[b, n] = (-1, NB, 2 ** 31 - 1)[i % 3]
    kc = cache_of(kind, NB, H, BS, D, seed + 1)
    g = torch.Generator(device=DEV).manual_seed(seed + 2)
    q = workloads.randn_f16((len(lens), ql, Hq, D), g, DEV)
    w = torch.rand((NB, H, BS), generator=g, device=DEV)
    before = w.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    want, size = weights_after(q, doubles(kind, kc, D), bt, lens, before, scale * SCALE[kind], start, decay, BS)
    ops.paged_kv_attention_weights(q if ql > 1 else q[:, 0].contiguous(), kc, bt, i32(*lens), w, scale,
                                   k_scale=SCALE[kind], start_lens=None if start is None else i32(*start), decay=decay,
                                   max_context_len=most, error_word=err)
    assert ops.pkd_read_device_error(err) == (ops.DEVERR_BAD_BLOCK if bad else 0)
    used = torch.zeros((NB, BS), dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        t = torch.arange(n, device=DEV)
        at = bt[b, t // BS].long()
        ok = (at >= 0) & (at < NB)
        used[at[ok], t[ok] % BS] = True
    assert (w == before).permute(0, 2, 1)[~used].all()              # nothing else was touched
    a, e = w.permute(0, 2, 1)[used].double(), want.permute(0, 2, 1)[used]
    bound = ref.weights_bound(D, ql * Hq // H, most, size)
    worst = ((a - e).abs() / (bound * e + 2.0 ** -23 * e + 1e-30)).max().item()
    assert worst <= 1.0, worst


# sequences, heads, query tokens, longest: rows 1, 4, 9-16, 40 and 320 (more than one load of queries)
LARGE = [(320, 1, 1, 1, 8192), (80, 16, 4, 1, 8192), (80, 16, 4, 4, 8192), (80, 12, 4, 3, 6000), (40, 32, 4, 5, 8192),
         (10, 32, 4, 40, 8192)]


@pytest.mark.parametrize("kind", ["fp16", "e4m3", "int4"])
@pytest.mark.parametrize("D,BS", [(128, 16), (128, 32), (64, 16), (64, 32)])
@pytest.mark.parametrize("B,Hq,H,ql,most", LARGE)
def test_long_partitions(kind, D, BS, B, Hq, H, ql, most):
    lens = ragged(B, most, B + ql)
    part = planned_partition(B, ql, Hq, H, D, BS, most)
    assert part >= 1024
    longest = sorted(range(B), key=lambda b: -lens[b])[:3]
    bad = [(longest[0], lens[longest[0]] // BS - 1), (longest[0], 900 // BS), (longest[1], 2000 // BS),
           (longest[2], 1030 // BS), (longest[2], 1030 // BS + 1), (longest[2], 500 // BS)]
    run(kind, D, BS, Hq, H, ql, lens, most, 3, start=[n - n // 3 for n in lens], decay=0.5, bad=bad)
    run(kind, D, BS, Hq, H, ql, lens, most, 4)


@pytest.mark.parametrize("kind", ["fp16", "e4m3", "int4"])
@pytest.mark.parametrize("BS", [16, 32])
@pytest.mark.parametrize("Hq,H,ql", [(8, 2, 1), (8, 2, 3), (16, 2, 2), (8, 1, 9)])
def test_the_rest_is_right_beside_missing_blocks(kind, BS, Hq, H, ql):
    lens = [130, 1, 0, 64, 300, 17]
    bad = [(0, 0), (0, 130 // BS), (1, 0), (3, 1), (4, 3), (4, 4)]    # the first, the last, the only one, two in a row
    run(kind, 128, BS, Hq, H, ql, lens, 320, 5, bad=bad, start=[50, 0, 0, 64, 0, 3], decay=0.75)


@pytest.mark.parametrize("kind", ["fp16", "e4m3", "int4"])
@pytest.mark.parametrize("scale", [-0.09, 0.0, -0.0, 1e-38, -1.0])
@pytest.mark.parametrize("Hq,H,ql", [(4, 4, 1), (8, 1, 2), (8, 1, 5)])
def test_softmax_scales(kind, scale, Hq, H, ql):
    run(kind, 128, 16, Hq, H, ql, [0, 1, 40, 700], 700, 6, scale=scale)
