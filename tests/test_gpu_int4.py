"""4-bit caches on the GPU: the rotated append against the quantiser's definition, bit for bit; the read-back
of rows; decode attention against fp64."""
import math

import pytest
import torch

import longcache_ref as ref
from serving_ref import attend, attention_bound, deal_tables, gathered
from paged_kv_decode_21_gb300 import ops, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def rope(n, R):
    g = torch.Generator().manual_seed(n + R)
    ang = torch.rand((n, R // 2), generator=g, dtype=torch.float64) * 6.28
    return torch.cat((ang.cos(), ang.sin()), 1).float()


def new_rows(T, Hq, H, D, seed):
    """q, k, v as slices of one projection, with rows that meet the quantiser's edges."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, Hq + 2 * H, D), generator=g)
    if T > 2:
        x[0] = 0                                  # no scale
        x[1] *= 2.0 ** -10                        # subnormal scales, and scales that round to 0
        x[2, :, ::16] *= 1000                     # a value that takes the whole range
        x[T - 1] *= 900                           # scales past 448
    x = x.half()
    p = x.to(DEV).view(T, -1)
    return x, p[:, :Hq * D].view(T, Hq, D), p[:, Hq * D:(Hq + H) * D].view(T, H, D), p[:, (Hq + H) * D:].view(T, H, D)


@pytest.mark.parametrize("D,BS,R,pairs,axes", [
    (128, 16, 128, False, 0), (128, 32, 128, True, 3), (128, 16, 64, False, 3), (64, 16, 64, False, 2),
    (64, 32, 32, True, 0), (128, 16, 0, False, 0), (64, 16, 32, False, 8)])
def test_append_is_the_quantiser_bit_for_bit(D, BS, R, pairs, axes):
    Hq, H, runs, past = 6, 3, [5, 0, 1, 40], [0, 7, 31, 14]
    T, behind = sum(runs), 2
    scale = (1 / 16, 0.3)
    x, q, k, v = new_rows(T + behind, Hq, H, D, D + R)
    table = rope(97, max(R, 2))[:, :R].contiguous()
    starts = [0, 5, 5, 6, 46]
    bt, _ = deal_tables([a + b for a, b in zip(past, runs)], BS, 8, 24, 3)
    kc = torch.full((24, H, BS, 9 * D // 16), 0xA5, dtype=torch.uint8, device=DEV)
    vc = kc.clone()
    g = torch.Generator().manual_seed(9)
    logical = torch.zeros(T + behind, dtype=torch.int64)
    for b, n in enumerate(runs):
        logical[starts[b]:starts[b] + n] = past[b] + torch.arange(n)
    pos = torch.randint(0, 97, (max(axes, 1), T + behind), generator=g) if axes else logical[None]
    which = torch.randint(0, max(axes, 1), (R // 2,), generator=g)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.full((T + behind, Hq, D), 7.0, dtype=torch.float16, device=DEV)
    kw = dict(pair_axes=which.to(torch.int32).to(DEV), positions=pos.to(torch.int32).to(DEV)) if axes else {}
    out = ops.paged_kv_append_rope_int4(q, k, v, table.to(DEV), bt, i32(*past), kc, vc, *scale,
                                        token_starts=i32(*starts), interleaved=pairs, q_out=q_out, error_word=err, **kw)
    assert out is q_out and ops.pkd_read_device_error(err) == 0
    cos, sin = ref.rows_of(table, pos, which, R)
    y = ref.rotate32(x[:, :Hq + H], cos, sin, R, pairs) if R else x[:, :Hq + H].float()
    want_k = torch.full(kc.shape, 0xA5, dtype=torch.uint8)
    want_v = want_k.clone()
    for b, n in enumerate(runs):
        for j in range(n):
            t, p = starts[b] + j, past[b] + j
            at = int(bt[b, p // BS])
            ref.write_int4(want_k, D, at, p % BS, *ref.int4_rows(y[t, Hq:], scale[0]))
            ref.write_int4(want_v, D, at, p % BS, *ref.int4_rows(x[t, Hq + H:].float(), scale[1]))
    assert torch.equal(kc.cpu(), want_k) and torch.equal(vc.cpu(), want_v)
    assert torch.equal(q_out[T:].cpu(), torch.full((behind, Hq, D), 7.0).half())   # rows behind the last run
    assert torch.equal(q_out[:T].cpu(), y[:T, :Hq].half())
    # in place, and one run of one length a sequence
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(kc)
    one = [1] * 4
    ops.paged_kv_append_rope_int4(None, k[:4], v[:4], table.to(DEV), bt, i32(*past), kc2, vc2, *scale,
                                  positions=i32(3, 5, 7, 9))
    for b, n in enumerate(one):
        at, p = int(bt[b, past[b] // BS]) if past[b] // BS < bt.shape[1] else -1, past[b]
        if at < 0:
            continue
        got = ref.tile_parts(vc2.cpu(), D)
        c, s = ref.int4_rows(x[b, Hq + H:].float(), scale[1])
        assert torch.equal(got[1][at, :, p % BS], s)


def test_append_skips_bad_tokens():
    D, BS, H = 128, 16, 2
    x, q, k, v = new_rows(4, 2, H, D, 1)
    table = rope(50, D).to(DEV)
    bt = i32(0, 1, 99, 2, -1, 3).view(3, 2)
    kc = torch.full((4, H, BS, 72), 1, dtype=torch.uint8, device=DEV)
    vc = kc.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = lambda **kw: ops.paged_kv_append_rope_int4(q[:3], k[:3], v[:3], table, bt, i32(0, 3, 2), kc, vc, 1.0, 1.0,  # noqa: E731
                                                      error_word=err, **kw)
    call()
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK
    assert (kc[1:] == 1).all() and (vc[1:] == 1).all() and not (kc[0] == 1).all()
    kc.fill_(1)
    axes = torch.zeros(64, dtype=torch.int32, device=DEV)
    axes[5] = 1
    for pos, ax in (([[0, 0, 0], [50, 0, 0]], axes), ([[0, 0, 0], [-1, 0, 0]], axes), ([[0, 0, 0]] * 2, axes * 2),
                    ([[0, 0, 0]] * 2, axes - 1)):
        call(positions=i32(*sum(pos, [])).view(2, 3), pair_axes=ax.contiguous())
        assert ops.pkd_read_device_error(err) & ops.DEVERR_BAD_POSITION
        assert (kc == 1).all()
    # a position outside the table on an axis that no pair goes by does not matter
    call(positions=i32(0, 0, 0, 50, 0, 0).view(2, 3), pair_axes=torch.zeros(64, dtype=torch.int32, device=DEV))
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK and not (kc[0] == 1).all()


@pytest.mark.parametrize("D,BS", [(64, 16), (64, 32), (128, 16), (128, 32)])
def test_read_back(D, BS):
    H, NB, runs, past = 3, 30, [0, 1, 33, 9], [4, 0, 20, 15]
    kc, vc = (ref.random_int4((NB, H, BS), D, s, 0, 0x7E) for s in (1, 2))
    bt, _ = deal_tables([a + b for a, b in zip(past, runs)], BS, 6, NB, 5)
    T, starts = sum(runs), [0, 0, 1, 34, 43]
    big = torch.full((T + 2, 2 * H + 1, D), 3.0, dtype=torch.float16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ko, vo = big[:, :H], big[:, H:2 * H]
    ops.paged_kv_read_int4(kc, vc, bt, i32(*past), 1 / 64, 1 / 128, ko, vo, token_starts=i32(*starts), error_word=err)
    assert ops.pkd_read_device_error(err) == 0
    kv, vv = ref.int4_values(kc, D, 1 / 64), ref.int4_values(vc, D, 1 / 128)
    for b, n in enumerate(runs):
        p = past[b] + torch.arange(n, device=DEV)
        at = bt[b, p // BS].long()
        s = slice(starts[b], starts[b] + n)
        assert torch.equal(ko[s].double(), kv[at, :, p % BS]) and torch.equal(vo[s].double(), vv[at, :, p % BS])
    assert (big[T:] == 3).all() and (big[:, 2 * H:] == 3).all()
    out = torch.zeros((4, H, D), dtype=torch.float16, device=DEV)
    ops.paged_kv_read_int4(kc, vc, i32(0, 1, -1, NB).view(4, 1), i32(0, BS - 1, 0, 0), 1.0, 1.0, out, out.clone(),
                           error_word=err)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK
    assert torch.equal(out[1].double(), ref.int4_values(kc, D, 1.0)[1, :, BS - 1]) and (out[2:] == 0).all()


def attention(q, kv, vv, bt, lens, scale, BS):
    B, ql, Hq, D = q.shape
    H = kv.shape[1]
    G = Hq // H
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(out)
    for b in range(B):
        for g in range(H):
            k, v = gathered(kv, bt[b], lens[b], g, BS), gathered(vv, bt[b], lens[b], g, BS)
            for j in range(ql):
                n = max(0, lens[b] - ql + 1 + j)
                out[b, j, g * G:(g + 1) * G], mag[b, j, g * G:(g + 1) * G] = attend(q[b, j, g * G:(g + 1) * G], k[:n],
                                                                                    v[:n], scale)
    return out, mag


def check(q, kc, vc, bt, lens, ks, vs, BS, part=0, **kw):
    D = q.shape[-1]
    qm = q if q.dim() == 4 else q[:, None]
    kv, vv = ref.int4_values(kc, D, ks), ref.int4_values(vc, D, vs)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = ops.paged_decode_attention_int4(q, kc, vc, bt, i32(*lens), D ** -0.5, ks, vs, partition_size=part,
                                          error_word=err, **kw)
    assert ops.pkd_read_device_error(err) == 0
    want, mag = attention(qm, kv, vv, bt, lens, D ** -0.5, BS)
    got = out.view(qm.shape).double()
    assert torch.isfinite(got).all()
    bound = attention_bound(want, mag, max(lens + [1]), float(vv.abs().max()))
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())
    return out


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 64, 130, 515, 1100]


@pytest.mark.parametrize("D,BS", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("Hq,H", [(4, 4), (8, 2), (7, 1), (16, 2), (15, 3)])
@pytest.mark.parametrize("ql,part", [(1, 0), (1, -1), (1, 32), (2, 64), (5, 0), (5, -1), (17, 96)])
def test_decode(D, BS, Hq, H, ql, part):
    lens = LENS if ql < 17 else LENS[::3]
    bt, _ = deal_tables(lens, BS, -(-1100 // BS) + 1, sum(-(-n // BS) for n in lens) + 5, D + ql)
    NB = sum(-(-n // BS) for n in lens) + 5
    kc, vc = (ref.random_int4((NB, H, BS), D, s) for s in (11, 12))
    g = torch.Generator(device=DEV).manual_seed(ql)
    q = workloads.randn_f16((len(lens), ql, Hq, D), g, DEV)
    check(q[:, 0].contiguous() if ql == 1 else q, kc, vc, bt, lens, 0.125, 0.25, BS, part)


@pytest.mark.parametrize("lo,hi,ks,vs", [(0x7E, 0x7E, 2.0 ** -9, 2.0 ** -12), (0x00, 0x07, 8.0, 32.0), (0, 0, 1.0, 1.0)])
def test_decode_at_the_scales_ends(lo, hi, ks, vs):
    """Largest scales, subnormal ones, none at all."""
    BS, D, lens = 16, 128, [40, 300]
    bt, _ = deal_tables(lens, BS, 20, 24, 2)
    kc, vc = (ref.random_int4((24, 2, BS), D, s, lo, hi) for s in (21, 22))
    q = workloads.randn_f16((2, 8, D), torch.Generator(device=DEV).manual_seed(1), DEV)
    check(q, kc, vc, bt, lens, ks, vs, BS)


def test_rows_that_were_never_written_do_not_count():
    """Bytes 0xff behind the length, in the last block and in blocks of no sequence."""
    BS, D, lens = 32, 128, [33, 5, 70]
    bt, _ = deal_tables(lens, BS, 3, 7, 4)
    kc, vc = (ref.random_int4((7, 2, BS), D, s) for s in (31, 32))
    clean = [kc.clone(), vc.clone()]
    for x in (kc, vc):
        c, s = ref.tile_parts(x, D)
        used = torch.zeros(7, BS, dtype=torch.bool, device=DEV)
        for b, n in enumerate(lens):
            for t in range(n):
                used[bt[b, t // BS].long(), t % BS] = True
        c.permute(0, 3, 1, 2, 4)[~used] = 255
        s.permute(0, 2, 1, 3)[~used] = 255
    q = workloads.randn_f16((3, 3, 16, D), torch.Generator(device=DEV).manual_seed(1), DEV)
    kw = dict(max_context_len=70)
    a = ops.paged_decode_attention_int4(q, kc, vc, bt, i32(*lens), 0.1, 0.1, 0.1, **kw)
    b = ops.paged_decode_attention_int4(q, *clean, bt, i32(*lens), 0.1, 0.1, 0.1, **kw)
    assert torch.isfinite(a).all() and torch.equal(a, b)


def test_bad_blocks_and_lengths_past_the_row():
    BS, D = 16, 128
    kc, vc = (ref.random_int4((8, 2, BS), D, s) for s in (1, 2))
    q = workloads.randn_f16((3, 8, D), torch.Generator(device=DEV).manual_seed(1), DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    bt = i32(0, 1, 2, 8, 4, -5).view(3, 2)
    out = ops.paged_decode_attention_int4(q, kc, vc, bt, i32(32, 32, 32), 0.1, 0.1, 0.1, error_word=err)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK
    want, _ = attention(q[:1, None], ref.int4_values(kc, D, 0.1), ref.int4_values(vc, D, 0.1), bt[:1], [32], 0.1, BS)
    assert (out[0].double() - want[0, 0]).abs().max() < 4e-3
    ops.paged_decode_attention_int4(q, kc, vc, bt[:, :1].contiguous(), i32(3, 1 << 30, 16), 0.1, 0.1, 0.1,
                                    max_context_len=16, error_word=err)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK


def test_pool_past_32_bits():
    """Tiles whose byte offsets pass 2^32."""
    BS, D, H = 32, 128, 8
    NB = (1 << 32) // (H * BS * 72) + 300
    kc = torch.zeros((NB, H, BS, 72), dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    last = torch.arange(NB - 9, NB, device=DEV, dtype=torch.int32)
    for x, s in ((kc, 1), (vc, 2)):
        x[NB - 9:] = ref.random_int4((9, H, BS), D, s)
    q = workloads.randn_f16((1, 32, D), torch.Generator(device=DEV).manual_seed(1), DEV)
    lens = i32(280)
    got = ops.paged_decode_attention_int4(q, kc, vc, last[None], lens, 0.1, 0.1, 0.1)
    near = ops.paged_decode_attention_int4(q, kc[NB - 9:].clone(), vc[NB - 9:].clone(),
                                           torch.arange(9, device=DEV, dtype=torch.int32)[None], lens, 0.1, 0.1, 0.1)
    assert torch.equal(got, near)
    k_new = workloads.randn_f16((2, H, D), torch.Generator(device=DEV).manual_seed(3), DEV)
    ops.paged_kv_append_rope_int4(None, k_new[:1], k_new[:1], rope(300, D).to(DEV), last[None], i32(281), kc, vc, 1.0,
                                  1.0)
    out = torch.zeros((2, H, D), dtype=torch.float16, device=DEV)
    ops.paged_kv_read_int4(kc, vc, last[None], i32(280), 1.0, 1.0, torch.zeros_like(out), out)
    c, s = ref.int4_rows(k_new[0].float().cpu(), 1.0)
    assert torch.equal(out[1].double().cpu(), (c.double() - 8) * s.view(ref.E4M3).double().repeat_interleave(16, -1))


def test_captured_and_on_another_stream():
    BS, D, lens = 16, 128, [700, 90]
    bt, _ = deal_tables(lens, BS, 44, 60, 4)
    kc, vc = (ref.random_int4((60, 2, BS), D, s) for s in (41, 42))
    q = workloads.randn_f16((2, 2, 8, D), torch.Generator(device=DEV).manual_seed(1), DEV)
    cl = i32(*lens)
    want = ops.paged_decode_attention_int4(q, kc, vc, bt, cl, 0.1, 0.1, 0.1)
    ws = ops.alloc_workspace(ops.paged_decode_int4_workspace_size(2, 2, 8, 2, D, BS, 700), DEV)
    assert ws is not None
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.paged_decode_attention_int4(q, kc, vc, bt, cl, 0.1, 0.1, 0.1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.paged_decode_attention_int4(q, kc, vc, bt, cl, 0.1, 0.1, 0.1, out=out, max_context_len=700, workspace=ws)
    for _ in range(2):
        out.zero_()
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    kc = torch.zeros((4, 2, 16, 72), dtype=torch.uint8, device=DEV)
    q = torch.zeros((1, 4, 128), dtype=torch.float16, device=DEV)
    bt, cl = i32(0, 1).view(1, 2), i32(20)
    ok = (q, kc, kc, bt, cl, 0.1, 1.0, 1.0)
    ops.paged_decode_attention_int4(*ok)
    for i, bad in ((0, q.float()), (0, q.cpu()), (0, q[0]), (0, torch.zeros((1, 4, 64), dtype=torch.float16, device=DEV)),
                   (1, kc.view(torch.int8)), (1, kc[:, :, :, :64].contiguous()), (2, kc[:2]), (3, bt.long()),
                   (3, bt.expand(2, 2)), (4, cl.float())):
        with pytest.raises((ValueError, ops.PagedDecodeError, AttributeError)):
            ops.paged_decode_attention_int4(*ok[:i], bad, *ok[i + 1:])
    for i, bad in ((6, 0.0), (6, math.inf), (7, -1.0), (5, math.nan)):
        with pytest.raises(ops.PagedDecodeError):
            ops.paged_decode_attention_int4(*ok[:i], bad, *ok[i + 1:])
    for kw in (dict(partition_size=48), dict(partition_size=-2), dict(max_context_len=33)):
        with pytest.raises(ops.PagedDecodeError):
            ops.paged_decode_attention_int4(*ok, **kw)
    k = torch.zeros((1, 2, 128), dtype=torch.float16, device=DEV)
    table = rope(8, 128).to(DEV)
    for R in (48, 16):     # half a group of 16 dims rotates with another
        with pytest.raises(ops.PagedDecodeError):
            ops.paged_kv_append_rope_int4(None, k, k, table[:, :R].contiguous(), bt, cl, kc, kc, 1.0, 1.0)
    with pytest.raises(ValueError):
        ops.paged_kv_append_rope_int4(None, k, k, table, bt, cl, kc, kc, 1.0, 1.0,
                                      pair_axes=torch.zeros(64, dtype=torch.int32, device=DEV), positions=i32(0))
