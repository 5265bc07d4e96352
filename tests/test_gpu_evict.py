"""Gathered attention weights, the choice of tokens by them, the copy of the kept rows, and the three together
with the append and the decode around them."""
import math

import pytest
import torch

import longcache_ref as ref
from serving_ref import attend, attention_bound, deal_tables, make_cache, values
from paged_kv_decode_21_gb300 import ops, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = {"fp16": 1.0, "e4m3": 1 / 64, "int4": 0.125}


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def cache_of(kind, NB, H, BS, D, seed):
    if kind == "int4":
        return ref.random_int4((NB, H, BS), D, seed)
    return make_cache((NB, H, BS, D), seed, kind == "e4m3")


def doubles(kind, cache, D):
    return ref.int4_values(cache, D, 1.0) if kind == "int4" else values(cache)


LENS = [0, 1, 2, 15, 16, 17, 33, 130, 300, 1030]


def run_weights(kind, D, BS, Hq, H, ql, decay, with_start, lens=LENS, **kw):
    need = sum(-(-n // BS) for n in lens)
    NB = need + 3
    bt, _ = deal_tables(lens, BS, max(-(-n // BS) for n in lens) + 1, NB, 3)
    kc = cache_of(kind, NB, H, BS, D, 5)
    g = torch.Generator(device=DEV).manual_seed(ql)
    q = workloads.randn_f16((len(lens), ql, Hq, D), g, DEV)
    w = torch.rand((NB, H, BS), generator=g, device=DEV)
    start = [max(0, n - 1 - n // 3) for n in lens] if with_start else None
    if decay == 0.0:
        w.fill_(math.nan)
        w[:, 0] = 1.0
    elif with_start:
        for b, n in enumerate(lens):      # what was where a new token now is does not count
            for t in range(start[b], n):
                w[bt[b, t // BS].long(), :, t % BS] = math.nan
    before = w.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    k = doubles(kind, kc, D)
    want, most = ref.weights_after(q, k, bt, lens, before, D ** -0.5 * SCALE[kind], start, decay, BS)
    got = ops.paged_kv_attention_weights(q if ql > 1 else q[:, 0].contiguous(), kc, bt, i32(*lens), w, D ** -0.5,
                                         k_scale=SCALE[kind], start_lens=None if start is None else i32(*start),
                                         decay=decay, error_word=err, **kw)
    assert got is w and ops.pkd_read_device_error(err) == 0
    used = torch.zeros((NB, BS), dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        t = torch.arange(n, device=DEV)
        used[bt[b, t // BS].long(), t % BS] = True
    same = (w == before) | (w.isnan() & before.isnan())
    assert same.permute(0, 2, 1)[~used].all()                       # nothing else was touched
    a, e = w.permute(0, 2, 1)[used].double(), want.permute(0, 2, 1)[used]
    assert torch.isfinite(a).all()
    bound = ref.weights_bound(D, ql * Hq // H, max(lens), most)
    worst = ((a - e).abs() / (bound * e + 2.0 ** -23 * e + 1e-30)).max().item() if a.numel() else 0.0
    assert worst <= 1.0, worst
    return w


@pytest.mark.parametrize("kind", ["fp16", "e4m3", "int4"])
@pytest.mark.parametrize("D,BS", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("Hq,H,ql", [(4, 4, 1), (8, 2, 1), (7, 1, 3), (16, 2, 2), (5, 1, 4), (8, 1, 40), (3, 3, 17)])
def test_weights(kind, D, BS, Hq, H, ql):
    run_weights(kind, D, BS, Hq, H, ql, 1.0, True)


@pytest.mark.parametrize("kind", ["fp16", "int4"])
@pytest.mark.parametrize("ql", [1, 40])
@pytest.mark.parametrize("decay,with_start", [(1.0, False), (0.5, True), (0.5, False), (0.0, True), (0.0, False)])
def test_weights_decay_and_new_tokens(kind, ql, decay, with_start):
    run_weights(kind, 128, 16, 8, 2, ql, decay, with_start)


def test_weights_many_rows_and_long_contexts():
    """Rows past one load of queries (256), partitions past 128 tokens, one row over 70000 tokens."""
    run_weights("e4m3", 128, 16, 8, 1, 70, 1.0, True, lens=[500, 3, 900])
    run_weights("fp16", 64, 16, 2, 2, 1, 1.0, True, lens=[70001])
    run_weights("int4", 128, 32, 8, 1, 5, 1.0, True, lens=[20000, 64])


def test_weights_sum_to_the_rows():
    """Every row that sees a token gives a weight of 1 in all; the same call twice gives the same bits."""
    lens, BS, D = [5, 0, 400], 16, 128
    bt, _ = deal_tables(lens, BS, 25, 30, 3)
    kc = cache_of("fp16", 30, 2, BS, D, 1)
    q = workloads.randn_f16((3, 9, 8, D), torch.Generator(device=DEV).manual_seed(1), DEV)
    w = torch.zeros((30, 2, BS), device=DEV)
    ops.paged_kv_attention_weights(q, kc, bt, i32(*lens), w, 0.09)
    sums = w.sum((0, 2)).double()
    assert (sums - 4 * (5 + 9)).abs().max() < 1e-3
    again = torch.zeros_like(w)
    ops.paged_kv_attention_weights(q, kc, bt, i32(*lens), again, 0.09)
    assert torch.equal(w, again)


@pytest.mark.parametrize("ql", [1, 20])
def test_weights_bad_blocks(ql):
    BS, D = 16, 64
    kc = cache_of("fp16", 6, 1, BS, D, 1)
    bt = i32(0, 6, 1, 2, -1, 3, 4, 5).view(2, 4)
    q = workloads.randn_f16((2, ql, 4, D), torch.Generator(device=DEV).manual_seed(1), DEV)
    w = torch.zeros((6, 1, BS), device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.paged_kv_attention_weights(q, kc, bt, i32(64, 60), w, 0.1, error_word=err)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK and torch.isfinite(w).all()
    ops.paged_kv_attention_weights(q, kc, bt[:, :1].contiguous(), i32(16, 1 << 30), w, 0.1, max_context_len=16,
                                   error_word=err)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK


@pytest.mark.parametrize("K,sink,recent", [(1, 0, 0), (1, 1, 0), (8, 2, 3), (8, 4, 4), (40, 0, 0), (40, 1, 30),
                                           (129, 16, 16), (2000, 3, 5)])
@pytest.mark.parametrize("BS", [16, 32, 5])
def test_select(K, sink, recent, BS):
    lens = [0, 1, 7, 8, 9, 40, 41, 130, 700, 1500]
    NB, H = sum(-(-n // BS) for n in lens) + 4, 3
    bt, _ = deal_tables(lens, BS, -(-1500 // BS), NB, 8)
    g = torch.Generator(device=DEV).manual_seed(K)
    w = torch.rand((NB, H, BS), generator=g, device=DEV) ** 8
    w[:, 1] = (torch.rand((NB, BS), generator=g, device=DEV) * 6).floor() / 4 - 0.5     # many equal ones, some negative
    w[:, 2] = 0.0
    w[::3, 2] = -0.0
    w[1::5, 1, :2] = math.nan
    w[2::5, 1, :2] = math.inf
    w[3::5, 1, :2] = -math.inf
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kept, n = ops.paged_kv_token_select(w, bt, i32(*lens), K, sink, recent, error_word=err)
    want, m = ref.token_select(w, bt, lens, K, sink, recent, BS)
    assert ops.pkd_read_device_error(err) == 0
    assert torch.equal(n.cpu(), m) and torch.equal(kept.cpu(), want)


@pytest.mark.parametrize("bound", [None, 60000])
def test_select_past_the_cached_keys(bound):
    BS, n, K = 16, 60000, 5000
    NB = n // BS + 1
    bt = torch.randperm(NB, generator=torch.Generator().manual_seed(1)).to(torch.int32)[None].to(DEV)
    w = torch.rand((NB, 2, BS), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    w[:, 1] = (w[:, 1] * 100).floor()
    kept, _ = ops.paged_kv_token_select(w, bt, i32(n), K, 4, 100, max_context_len=bound)
    want, _ = ref.token_select(w, bt, [n], K, 4, 100, BS)
    assert torch.equal(kept.cpu(), want)


def test_select_bad_blocks_come_last():
    w = torch.rand((4, 1, 16), device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kept, n = ops.paged_kv_token_select(w, i32(0, 9, 2)[None].contiguous(), i32(48), 20, 0, 0, error_word=err)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK and n.tolist() == [20]
    assert not any(16 <= t < 32 for t in kept[0, 0].tolist())
    kept, n = ops.paged_kv_token_select(w, i32(0, 9, 2)[None].contiguous(), i32(1 << 30), 40, 0, 0, max_context_len=48,
                                        error_word=err)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK and n.tolist() == [40]
    assert kept[0, 0].tolist()[-1] == 47


def compacted(cache, bt, new, kept, lens, BS, D, kind):
    """The cache after the copy, row by row on the CPU."""
    out = cache.cpu().clone()
    src = cache.cpu()
    for b in range(bt.shape[0]):
        for g in range(kept.shape[1]):
            for i in range(int(lens[b])):
                t = int(kept[b, g, i])
                f, to = int(bt[b, t // BS]), int(new[b, i // BS])
                if kind == "int4":
                    for x, y in zip(ref.tile_parts(out, D), ref.tile_parts(src, D)):
                        x_, y_ = (x[to, g], y[f, g])
                        if x.dim() == 5:
                            x_[:, i % BS] = y_[:, t % BS]
                        else:
                            x_[i % BS] = y_[t % BS]
                else:
                    out[to, g, i % BS] = src[f, g, t % BS]
    return out


@pytest.mark.parametrize("kind", ["fp16", "e4m3", "int4"])
@pytest.mark.parametrize("D,BS", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("with_weights", [True, False])
def test_compact(kind, D, BS, with_weights):
    lens, K, H = [0, 1, 20, 90, 300], 70, 2
    most = -(-K // BS)
    need = sum(-(-n // BS) for n in lens)
    bt, rest = deal_tables(lens, BS, 20, need + 5 * most + 2, 3)
    new = rest[:5 * most].view(5, most).to(DEV).contiguous()
    NB = need + 5 * most + 2
    kc, vc = (cache_of(kind, NB, H, BS, D, s) for s in (1, 2))
    w = torch.rand((NB, H, BS), device=DEV)
    kept, n = ops.paged_kv_token_select(w, bt, i32(*lens), K, 2, 9)
    want_k, want_v = (compacted(x, bt, new, kept, n, BS, D, kind) for x in (kc, vc))
    want_w = compacted(w[..., None], bt, new, kept, n, BS, D, "fp16")[..., 0] if with_weights else w.cpu()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.paged_kv_compact(kc, vc, bt, i32(*lens), kept, n, new, weights=w if with_weights else None, error_word=err)
    assert ops.pkd_read_device_error(err) == 0
    assert torch.equal(kc.cpu(), want_k) and torch.equal(vc.cpu(), want_v) and torch.equal(w.cpu(), want_w)


def test_compact_skips_what_it_cannot_copy():
    BS, D = 16, 128
    kc, vc = (cache_of("fp16", 8, 1, BS, D, s) for s in (1, 2))
    before = kc.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kept = i32(0, -1, 20, 5, 17, 3).view(1, 1, 6)
    ops.paged_kv_compact(kc, vc, i32(0, 9)[None].contiguous(), i32(20), kept, i32(6), i32(4)[None].contiguous(), error_word=err)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK
    want = before.clone()
    for i, t in ((0, 0), (3, 5), (5, 3)):
        want[4, :, i] = before[0, :, t]
    assert torch.equal(kc, want)
    for new, n in ((8, 6), (-1, 6), (4, -3)):
        ops.paged_kv_compact(kc, vc, i32(0, 1)[None].contiguous(), i32(32), kept, i32(n), i32(new)[None].contiguous(),
                             error_word=err)
        assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK and torch.equal(kc, want)
    # more kept than the new row holds: the row is filled
    many = torch.arange(32, dtype=torch.int32, device=DEV).view(1, 1, 32)
    ops.paged_kv_compact(kc, vc, i32(0, 1)[None].contiguous(), i32(32), many, i32(32), i32(4)[None].contiguous(),
                         error_word=err)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK and torch.equal(kc[4], kc[0])
    assert torch.equal(kc[5:], before[5:])


@pytest.mark.parametrize("kind", ["fp16", "e4m3", "int4"])
def test_a_run_of_steps(kind):
    """Prompts with images written, decode steps that gather weights, a cut to a budget, and further steps over
    what was kept: against attention over the kept tokens in fp64."""
    D, BS, Hq, H, K = 128, 16, 8, 2, 48
    lens = [100, 30, 77]
    B, per = len(lens), 10
    NB = 2 * B * per
    bt = torch.randperm(B * per, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, per).to(DEV)
    new = (bt + B * per).contiguous()
    row = 72 if kind == "int4" else D
    kc = torch.zeros((NB, H, BS, row), dtype=torch.float16 if kind == "fp16" else torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    w = torch.full((NB, H, BS), math.nan, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    ang = torch.arange(200, dtype=torch.float64)[:, None] * 0.7 ** torch.arange(64)
    table = torch.cat((ang.cos(), ang.sin()), 1).float().to(DEV)
    axes = (torch.arange(64) % 3).to(torch.int32).to(DEV)
    one = SCALE[kind]

    def append(tables, past, runs):
        T = sum(runs)
        qkv = workloads.randn_f16((T, Hq + 2 * H, D), g, DEV)
        pos = torch.randint(0, 200, (3, T), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
        starts = i32(0, *torch.tensor(runs).cumsum(0).tolist())
        args = (qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:], table)
        kw = dict(token_starts=starts, error_word=err)
        if kind == "int4":
            return ops.paged_kv_append_rope_int4(*args, tables, past, kc, vc, one, one, positions=pos, pair_axes=axes, **kw)
        if kind == "e4m3":
            return ops.paged_kv_append_rope_axes_fp8(*args, axes, pos, tables, past, kc, vc, one, one, **kw)
        return ops.paged_kv_append_rope_axes(*args, axes, pos, tables, past, kc, vc, **kw)

    def decode(q, tables, cl):
        args = (q, kc, vc, tables, cl, D ** -0.5)
        if kind == "int4":
            return ops.paged_decode_attention_int4(*args, one, one, error_word=err)
        if kind == "e4m3":
            return ops.paged_decode_attention_fp8(*args, one, one, error_word=err)
        return ops.paged_decode_attention_ex(*args, error_word=err)

    cl = i32(*lens)
    q = append(bt, torch.zeros_like(cl), lens)
    ends = (cl.cumsum(0) - 1).long()
    ops.paged_kv_attention_weights(q[ends].contiguous(), kc, bt, cl, w, D ** -0.5, k_scale=one,
                                   start_lens=torch.zeros_like(cl), error_word=err)
    q = append(bt, cl, [1] * B)
    cl = cl + 1
    ops.paged_kv_attention_weights(q, kc, bt, cl, w, D ** -0.5, k_scale=one, start_lens=cl - 1, error_word=err)
    kept, n = ops.paged_kv_token_select(w, bt, cl, K, 2, 8, error_word=err)
    want, _ = ref.token_select(w, bt, cl.tolist(), K, 2, 8, BS)
    assert torch.equal(kept.cpu(), want)
    ops.paged_kv_compact(kc, vc, bt, cl, kept, n, new, weights=w, error_word=err)
    # the step after: one more token in the new blocks, attention over the kept tokens and it
    q = append(new, n, [1] * B)
    out = decode(q, new, n + 1).double()
    k, v = doubles(kind, kc, D) * one, doubles(kind, vc, D) * one
    for b in range(B):
        for h in range(H):
            m = int(n[b])
            t = kept[b, h, :m].long()
            at = bt[b, t // BS].long()
            tail = new[b, m // BS].long()
            kk = torch.cat((k[at, h, t % BS], k[tail, h, m % BS][None]))
            vv = torch.cat((v[at, h, t % BS], v[tail, h, m % BS][None]))
            o, a = attend(q[b, 4 * h:4 * h + 4], kk, vv, D ** -0.5)
            bound = attention_bound(o, a, m + 1, float(vv.abs().max()))
            assert ((out[b, 4 * h:4 * h + 4] - o).abs() <= bound).all()
    ops.paged_kv_attention_weights(q, kc, new, n + 1, w, D ** -0.5, k_scale=one, start_lens=n, error_word=err)
    assert ops.pkd_read_device_error(err) == 0
    for b in range(B):
        t = torch.arange(int(n[b]) + 1, device=DEV)
        assert torch.isfinite(w[new[b, t // BS].long(), :, t % BS]).all()


def test_captured_steps_and_another_stream():
    BS, D, lens, K = 16, 128, [200, 90], 64
    bt, rest = deal_tables(lens, BS, 13, 40, 4)
    new = rest[:8].view(2, 4).to(DEV).contiguous()
    kc, vc = (cache_of("fp16", 40, 2, BS, D, s) for s in (1, 2))
    q = workloads.randn_f16((2, 8, D), torch.Generator(device=DEV).manual_seed(1), DEV)
    cl = i32(*lens)
    w0 = torch.rand((40, 2, BS), device=DEV)

    def steps(kc, vc, w, ws=None, stream=None, kept=None, n=None):
        ops.paged_kv_attention_weights(q, kc, bt, cl, w, 0.1, max_context_len=200, workspace=ws, stream=stream)
        kept, n = ops.paged_kv_token_select(w, bt, cl, K, 1, 5, max_context_len=200, kept=kept, kept_lens=n, stream=stream)
        ops.paged_kv_compact(kc, vc, bt, cl, kept, n, new, weights=w, stream=stream)
        return kept, n

    want = [kc.clone(), vc.clone(), w0.clone()]
    want_kept, _ = steps(*want)
    side = torch.cuda.Stream()
    other = [kc.clone(), vc.clone(), w0.clone()]
    side.wait_stream(torch.cuda.current_stream())
    got, _ = steps(*other, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want_kept) and all(torch.equal(a, b) for a, b in zip(other, want))
    ws = ops.alloc_workspace(ops.paged_kv_attention_weights_workspace_size(2, 1, 8, 2, D, BS, 200), DEV)
    state = [kc.clone(), vc.clone(), w0.clone()]
    kept, n = torch.zeros_like(want_kept), torch.zeros_like(cl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps(*state, ws=ws, kept=kept, n=n)
    for _ in range(2):
        for x, y in zip(state, (kc, vc, w0)):
            x.copy_(y)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want_kept) and all(torch.equal(a, b) for a, b in zip(state, want))


def test_refusals():
    kc = torch.zeros((4, 2, 16, 128), dtype=torch.float16, device=DEV)
    q = torch.zeros((1, 4, 128), dtype=torch.float16, device=DEV)
    bt, cl, w = i32(0, 1).view(1, 2), i32(20), torch.zeros((4, 2, 16), device=DEV)
    ok = (q, kc, bt, cl, w, 0.1)
    ops.paged_kv_attention_weights(*ok)
    for i, bad in ((0, q.float()), (0, q[0]), (1, kc.float()), (1, kc[:, :, :, :64].contiguous()), (2, bt.long()),
                   (3, cl.long()), (4, w.half()), (4, w[:3]), (4, w.cpu())):
        with pytest.raises((ValueError, ops.PagedDecodeError)):
            ops.paged_kv_attention_weights(*ok[:i], bad, *ok[i + 1:])
    for kw in (dict(decay=1.5), dict(decay=-0.1), dict(decay=math.nan), dict(k_scale=0.0), dict(max_context_len=33)):
        with pytest.raises(ops.PagedDecodeError):
            ops.paged_kv_attention_weights(*ok, **kw)
    with pytest.raises(ops.PagedDecodeError):
        ops.paged_kv_attention_weights(*ok, workspace=torch.zeros(256, dtype=torch.uint8, device=DEV)[:16])
    for K, s, r in ((0, 0, 0), (4, 3, 2), (4, -1, 0), (4, 0, -1)):
        with pytest.raises(ops.PagedDecodeError):
            ops.paged_kv_token_select(w, bt, cl, K, s, r)
    kept, n = ops.paged_kv_token_select(w, bt, cl, 8)
    new = i32(2).view(1, 1)
    for args in ((kc, kc[:3], bt, cl, kept, n, new), (kc, kc, bt, cl, kept[:, :1].contiguous(), n, new),
                 (kc, kc.view(torch.uint8), bt, cl, kept, n, new), (kc, kc, bt, cl, kept, n.long(), new),
                 (kc, kc, bt, cl, kept, n, new[:0])):
        with pytest.raises(ValueError):
            ops.paged_kv_compact(*args)



def test_select_with_thousands_of_equal_keys_at_the_border():
    """Thousands of weights that agree in their leading bits, and thousands that are equal, at the border."""
    BS, n = 16, 30000
    NB = n // BS
    bt = torch.randperm(NB, generator=torch.Generator().manual_seed(2)).to(torch.int32)[None].to(DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    w = torch.empty((NB, 3, BS), device=DEV)
    w[:, 0] = 1.0 + torch.rand((NB, BS), generator=g, device=DEV) * 2.0 ** -4
    w[:, 1] = 0.5
    w[:, 2] = torch.where(torch.rand((NB, BS), generator=g, device=DEV) < 0.5, 0.25, 0.75)
    for K, sink, recent in ((7000, 0, 0), (20000, 5, 11), (100, 50, 50)):
        kept, _ = ops.paged_kv_token_select(w, bt, i32(n), K, sink, recent)
        want, _ = ref.token_select(w, bt, [n], K, sink, recent, BS)
        assert torch.equal(kept.cpu(), want), K


@pytest.mark.parametrize("K", [14999, 15000, 30000])
def test_select_of_long_contexts_few_and_many_kept(K):
    BS, n = 16, 60000
    NB = n // BS + 1
    bt = torch.randperm(NB, generator=torch.Generator().manual_seed(4)).to(torch.int32)[None].to(DEV)
    w = torch.rand((NB, 2, BS), generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
    w[:, 1] = (w[:, 1] * 5).floor()
    kept, _ = ops.paged_kv_token_select(w, bt, i32(n), K, 33, 70)
    want, _ = ref.token_select(w, bt, [n], K, 33, 70, BS)
    assert torch.equal(kept.cpu(), want)
