"""Rotated append with positions of several axes, into fp16 and E4M3 caches."""
import pytest
import torch

import longcache_ref as ref
from serving_ref import E4M3, deal_tables
from paged_kv_decode_21_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def setup(D, BS, R, A, seed, runs=(3, 0, 1, 21), past=(0, 5, 15, 30), Hq=5, H=2):
    g = torch.Generator().manual_seed(seed)
    T = sum(runs)
    x = torch.randn((T + 1, Hq + 2 * H, D), generator=g).half()
    p = x.to(DEV).view(T + 1, -1)
    q, k, v = p[:, :Hq * D].view(T + 1, Hq, D), p[:, Hq * D:(Hq + H) * D].view(T + 1, H, D), p[:, (Hq + H) * D:].view(
        T + 1, H, D)
    ang = torch.rand((60, max(R // 2, 1)), generator=g, dtype=torch.float64) * 6.28
    table = torch.cat((ang.cos(), ang.sin()), 1).float()[:, :R].contiguous()
    pos = torch.randint(0, 60, (A, T + 1), generator=g)
    axes = torch.randint(0, A, (R // 2,), generator=g)
    starts = [0]
    for n in runs:
        starts.append(starts[-1] + n)
    bt, _ = deal_tables([a + b for a, b in zip(past, runs)], BS, 8, 16, seed)
    return x, q, k, v, table, pos, axes, starts, bt, i32(*past)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,BS,R,pairs,A", [(128, 16, 128, False, 3), (128, 16, 128, True, 3), (64, 32, 32, False, 2),
                                            (80, 8, 48, False, 3), (80, 16, 16, True, 8), (16, 16, 16, False, 1),
                                            (512, 16, 512, False, 4), (128, 16, 0, False, 3)])
def test_against_the_formula(fp8, D, BS, R, pairs, A):
    Hq, H = 5, 2
    x, q, k, v, table, pos, axes, starts, bt, past = setup(D, BS, R, A, D + R + A)
    shape = (16, H, BS, D)
    kc = torch.full(shape, 9, dtype=torch.uint8 if fp8 else torch.float16, device=DEV)
    vc = kc.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.full(q.shape, 7.0, dtype=torch.float16, device=DEV)
    args = (q, k, v, table.to(DEV), axes.to(torch.int32).to(DEV), pos.to(torch.int32).to(DEV), bt, past, kc, vc)
    kw = dict(token_starts=i32(*starts), interleaved=pairs, q_out=q_out, error_word=err)
    if fp8:
        ops.paged_kv_append_rope_axes_fp8(*args, 0.25, 0.5, **kw)
    else:
        ops.paged_kv_append_rope_axes(*args, **kw)
    assert ops.pkd_read_device_error(err) == 0
    cos, sin = (t.double() for t in ref.rows_of(table, pos, axes, R))
    y = x.double()
    for t in range(y.shape[0] - 1):
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if pairs else (i, i + R // 2)
            xa, xb = x[t, :Hq + H, a].double(), x[t, :Hq + H, b].double()
            y[t, :Hq + H, a], y[t, :Hq + H, b] = xa * cos[t, i] - xb * sin[t, i], xb * cos[t, i] + xa * sin[t, i]
    assert (q_out[-1] == 7).all()
    got = q_out[:-1].double().cpu()
    # one rounding to fp16 (2^-11), and fp32 products and a sum before it, 2^-22 of |x|
    size = x[:-1, :Hq].double().abs().amax(-1, keepdim=True)
    assert ((got - y[:-1, :Hq]).abs() <= 2.0 ** -11 * y[:-1, :Hq].abs() + 2.0 ** -21 * size + 2.0 ** -25).all()
    seen = torch.zeros(16, BS, dtype=torch.bool)
    for b in range(4):
        for j in range(starts[b + 1] - starts[b]):
            t, p = starts[b] + j, int(past[b]) + j
            at = int(bt[b, p // BS])
            seen[at, p % BS] = True
            for cache, row, s in ((kc, y[t, Hq:Hq + H], 0.25), (vc, x[t, Hq + H:].double(), 0.5)):
                if fp8:
                    z = cache[at, :, p % BS].view(E4M3).double().cpu()
                    w = row / s
                    # half a step of E4M3 (2^-4, subnormals 2^-10), and the fp32 rotation before it
                    assert ((z - w).abs() <= 2.0 ** -4 * w.abs() * (1 + 2.0 ** -16) + 2.0 ** -10 + 2.0 ** -18).all()
                else:
                    z = cache[at, :, p % BS].double().cpu()
                    assert ((z - row).abs() <= 2.0 ** -11 * row.abs() + 2.0 ** -20 * 5 + 2.0 ** -25).all()
    for cache in (kc, vc):
        assert (cache.cpu().permute(0, 2, 1, 3)[~seen] == 9).all()


def test_one_axis_for_all_is_the_plain_append():
    x, q, k, v, table, pos, axes, starts, bt, past = setup(128, 16, 128, 3, 77)
    caches = [torch.zeros((16, 2, 16, 128), dtype=torch.float16, device=DEV) for _ in range(4)]
    tab, p, st = table.to(DEV), pos.to(torch.int32).to(DEV), i32(*starts)
    a = ops.paged_kv_append_rope_axes(q, k, v, tab, i32(*[1] * 64), p, bt, past, *caches[:2], token_starts=st)
    b = ops.paged_kv_append_rope(q, k, v, tab, bt, past, *caches[2:], token_starts=st, positions=p[1].contiguous())
    n = starts[-1]
    assert torch.equal(a[:n], b[:n]) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_bad_positions_and_refusals():
    x, q, k, v, table, pos, axes, starts, bt, past = setup(128, 16, 128, 3, 5)
    kc = torch.zeros((16, 2, 16, 128), dtype=torch.float16, device=DEV)
    vc = torch.zeros_like(kc)
    tab, st = table.to(DEV), i32(*starts)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ax = axes.to(torch.int32).to(DEV)
    bad = pos.clone()
    bad[1, 0], bad[2, 4] = 60, -1
    q_out = torch.full(q.shape, 7.0, dtype=torch.float16, device=DEV)
    ops.paged_kv_append_rope_axes(q, k, v, tab, ax, bad.to(torch.int32).to(DEV), bt, past, kc, vc, token_starts=st,
                                  q_out=q_out, error_word=err)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_POSITION
    skipped = [t for t in range(starts[-1]) if (q_out[t] == 7).all()]
    assert skipped == [0, 4] and (kc[bt[0, 0].long(), :, 0] == 0).all()
    p = pos.to(torch.int32).to(DEV)
    call = lambda ax=ax, p=p: ops.paged_kv_append_rope_axes(q, k, v, tab, ax, p, bt, past, kc, vc, token_starts=st)  # noqa: E731
    for wrong in (dict(ax=None), dict(ax=ax.long()), dict(ax=ax[:32].contiguous()), dict(p=None), dict(p=p[0]),
                  dict(p=p[:, :-1].contiguous())):
        with pytest.raises(ValueError):
            call(**wrong)
    with pytest.raises(ops.PagedDecodeError):
        call(p=p.repeat(3, 1).contiguous())                       # nine axes
    with pytest.raises(ops.PagedDecodeError):
        call(ax=torch.cat((i32(0), ax))[1:])                      # not on a 16-byte boundary


@pytest.mark.parametrize("kind", ["fp16", "e4m3", "int4"])
@pytest.mark.parametrize("axes,pairs,Hq,H,D", [(0, False, 5, 2, 128), (3, True, 0, 3, 64), (3, False, 9, 1, 128)])
def test_many_tokens_are_few_tokens_many_times(kind, axes, pairs, Hq, H, D):
    """The kernel for many tokens (thousands) against the one for few, bit for bit: odd runs, bad blocks and
    positions, rows behind the last run, in place."""
    BS, T, behind = 16, 5003, 7
    runs = [0, 1, 2000, 3, 2990, 9]
    past = [5, 30, 0, 17, 1, 100]
    assert sum(runs) == T
    g = torch.Generator().manual_seed(axes + D)
    x = torch.randn((T + behind, Hq + 2 * H, D), generator=g).half().to(DEV)
    q = x[:, :Hq] if Hq else None
    k, v = x[:, Hq:Hq + H], x[:, Hq + H:]
    ang = torch.rand((60, D // 2), generator=g, dtype=torch.float64) * 6.28
    table = torch.cat((ang.cos(), ang.sin()), 1).float().to(DEV)
    pos = torch.randint(0, 60, (max(axes, 1), T + behind), generator=g, dtype=torch.int64).to(torch.int32)
    pos[0, 17], pos[-1, 2500] = 60, -1
    which = (torch.arange(D // 2) % max(axes, 1)).to(torch.int32).to(DEV)
    bt, _ = deal_tables([a + b for a, b in zip(past, runs)], BS, 190, 400, 3)
    bt[2, 7], bt[4, 11] = -1, 400
    row = 9 * D // 16 if kind == "int4" else D
    dtype = torch.float16 if kind == "fp16" else torch.uint8
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(k, v, q, pos, starts, past, bt, kc, vc):
        kw = dict(token_starts=i32(*starts), interleaved=pairs, q_out=q, error_word=err)
        p = pos.contiguous().to(DEV)
        scales = () if kind == "fp16" else (0.25, 0.3)
        if kind == "int4":
            ops.paged_kv_append_rope_int4(q, k, v, table, bt, past, kc, vc, *scales,
                                          positions=p if axes else p[0], pair_axes=which if axes else None, **kw)
        elif axes:
            fn = ops.paged_kv_append_rope_axes if kind == "fp16" else ops.paged_kv_append_rope_axes_fp8
            fn(q, k, v, table, which, p, bt, past, kc, vc, *scales, **kw)
        else:
            fn = ops.paged_kv_append_rope if kind == "fp16" else ops.paged_kv_append_rope_fp8
            fn(q, k, v, table, bt, past, kc, vc, *scales, positions=p[0], **kw)
        return ops.pkd_read_device_error(err)

    a = [torch.full((400, H, BS, row), 3, dtype=dtype, device=DEV) for _ in range(2)]
    b = [t.clone() for t in a]
    starts = [0]
    for n in runs:
        starts.append(starts[-1] + n)
    qa = x[:, :Hq].clone() if Hq else None
    bits = call(k, v, qa, pos, starts, i32(*past), bt, *a)
    assert bits == ops.DEVERR_BAD_BLOCK | ops.DEVERR_BAD_POSITION
    qb = x[:, :Hq].clone() if Hq else None
    seen = 0
    for i, n in enumerate(runs):                   # the same, at most 1000 tokens a call
        for j in range(0, n, 1000):
            m = min(1000, n - j)
            s = slice(starts[i] + j, starts[i] + j + m)
            seen |= call(k[s], v[s], qb[s] if Hq else None, pos[:, s], [0, m], i32(past[i] + j), bt[i:i + 1], *b)
    assert seen == bits
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert Hq == 0 or torch.equal(qa, qb)
