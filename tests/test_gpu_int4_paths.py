"""Decode over 4-bit caches where contexts are long or grids large: pieces walked longest first, the automatic plan
past one wave of CTAs, block ids of more than one run a warp, and softmax scales of any sign."""
import pytest
import torch

import longcache_ref as ref
from serving_ref import deal_tables
from test_gpu_corrupt_lengths import int4_plan
from test_gpu_int4 import attention, check
from serving_ref import attention_bound
from paged_kv_decode_21_gb300 import ops, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def problem(lens, ql, Hq, H, D, BS, seed, most):
    """A table of `most` tokens a row whose blocks may be shared by sequences (a pool of 400)."""
    NB = 400
    g = torch.Generator(device=DEV).manual_seed(seed)
    bt = torch.randint(0, NB, (len(lens), -(-most // BS)), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    kc, vc = (ref.random_int4((NB, H, BS), D, seed + i) for i in (1, 2))
    q = workloads.randn_f16((len(lens), ql, Hq, D), g, DEV)
    return q if ql > 1 else q[:, 0].contiguous(), kc, vc, bt


def ragged(B, most, seed, few=6):
    """Lengths of which a few are long, some zero, ties among them."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, 130, (B,), generator=g)
    lens[torch.randperm(B, generator=g)[:few]] = torch.randint(most // 2, most + 1, (few,), generator=g)
    lens[1], lens[B // 2], lens[B - 1], lens[2] = most, 0, 0, 1
    lens[B // 3] = lens[B // 4] = most - 17
    return lens.tolist()


# (sequences, query tokens, heads, longest) and the automatic plan: partitions, pieces of that many tokens
ORDERED = [(160, 1, 32, 8, 1536, -1), (32, 1, 32, 8, 8192, 2048), (20, 1, 32, 8, 32768, 4096), (70, 4, 28, 4, 8192, 4096),
           (200, 4, 28, 4, 1500, -1), (130, 2, 32, 4, 2048, -1)]


@pytest.mark.parametrize("D,BS", [(128, 16), (128, 32), (64, 16)])
@pytest.mark.parametrize("B,ql,Hq,H,most,part", ORDERED)
def test_longest_first_is_the_plain_order(D, BS, B, ql, Hq, H, most, part):
    """The same pieces in another order: the same bits, with the order, with a workspace that has no room for it, and
    again and again; and right by the definition."""
    lens = ragged(B, most, B + ql)
    q, kc, vc, bt = problem(lens, ql, Hq, H, D, BS, 7, most)
    np, ordered = int4_plan(B, ql, Hq, H, D, BS, most)
    assert ordered and np == (1 if part < 0 else -(-most // part)), (np, ordered)
    kw = dict(max_context_len=most)
    cl = i32(lens)
    call = lambda **k: ops.paged_decode_attention_int4(q, kc, vc, bt, cl, 0.09, 0.125, 0.25, **kw, **k)  # noqa: E731
    plain = call(partition_size=part)
    size = ops.paged_decode_int4_workspace_size(B, ql, Hq, H, D, BS, most)
    less = ops.paged_decode_int4_workspace_size(B, ql, Hq, H, D, BS, most, part)
    assert size == less + -(-4 * B * np // 256) * 256
    space = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    assert torch.equal(call(workspace=space), plain)
    for _ in range(3):
        assert torch.equal(call(), plain)
    if less:
        assert torch.equal(call(workspace=space[:less]), plain)
    else:
        assert torch.equal(call(workspace=space[:16]), plain)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    call(error_word=err)
    assert ops.pkd_read_device_error(err) == 0
    qm = q if ql > 1 else q[:, None]
    pick = sorted(range(B), key=lambda b: -lens[b])[:4] + [0, 2, B // 2, B - 1]
    want, mag = attention(qm[pick], ref.int4_values(kc, D, 0.125), ref.int4_values(vc, D, 0.25), bt[pick],
                          [lens[b] for b in pick], 0.09, BS)
    got = plain.view(qm.shape)[pick].double()
    bound = attention_bound(want, mag, most, float(ref.int4_values(vc, D, 0.25).abs().max()))
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())


@pytest.mark.parametrize("D,BS", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("Hq,H,ql", [(4, 2, 1), (8, 1, 2), (7, 1, 4)])
@pytest.mark.parametrize("part", [-1, 4096, 8192])
def test_long_partitions(D, BS, Hq, H, ql, part):
    """More than one run of block ids a warp: past 2048 (blocks of 16) and 4096 tokens (of 32)."""
    lens = [9001, 4096, 4097, 5000, 8192, 3]
    q, kc, vc, bt = problem(lens, ql, Hq, H, D, BS, 9, 9001)
    check(q, kc, vc, bt, lens, 0.125, 0.25, BS, part, max_context_len=9001)


@pytest.mark.parametrize("part", [0, -1])
def test_bad_blocks_late_in_a_partition(part):
    """Blocks outside the pool in slots that have been used before: only their tokens are left out."""
    D, BS, Hq, H = 128, 16, 8, 2
    lens = [6000, 700]
    q, kc, vc, bt = problem(lens, 1, Hq, H, D, BS, 11, 6000)
    kv, vv = ref.int4_values(kc, D, 0.125), ref.int4_values(vc, D, 0.25)
    hit = [(0, 300), (0, 301), (0, 374), (0, 7), (1, 40)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for i, (b, n) in enumerate(hit):
        bt[b, n] = (-1, 400, 2 ** 31 - 1)[i % 3]
    out = ops.paged_decode_attention_int4(q, kc, vc, bt, i32(lens), 0.09, 0.125, 0.25, partition_size=part, error_word=err)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK
    for b, n in enumerate(lens):
        good = [i for i in range(-(-n // BS)) if (b, i) not in hit]
        left = n - sum(min(BS, n - i * BS) for x, i in hit if x == b)
        row = bt[b:b + 1, good].contiguous()
        want, mag = attention(q[b:b + 1, None], kv, vv, row, [left], 0.09, BS)
        bound = attention_bound(want, mag, n, float(vv.abs().max()))
        assert ((out[b].double() - want[0, 0]).abs() <= bound[0, 0]).all()


@pytest.mark.parametrize("scale", [-0.09, 0.0, -0.0, 1e-38, -2.0])
@pytest.mark.parametrize("Hq,H,ql", [(4, 4, 1), (8, 1, 2), (16, 2, 4), (7, 1, 5)])
@pytest.mark.parametrize("part", [0, -1])
def test_softmax_scales(scale, Hq, H, ql, part):
    D, BS, lens = 128, 16, [0, 1, 40, 700]
    bt, _ = deal_tables(lens, BS, 44, 60, 2)
    kc, vc = (ref.random_int4((60, H, BS), D, s) for s in (1, 2))
    q = workloads.randn_f16((4, ql, Hq, D), torch.Generator(device=DEV).manual_seed(1), DEV)
    kv, vv = ref.int4_values(kc, D, 0.125), ref.int4_values(vc, D, 0.25)
    want, mag = attention(q, kv, vv, bt, lens, scale, BS)
    out = ops.paged_decode_attention_int4(q if ql > 1 else q[:, 0].contiguous(), kc, vc, bt, i32(lens), scale, 0.125, 0.25,
                                          partition_size=part).view(q.shape).double()
    # a score is a sum of D exact products in fp32 and two roundings of its scaling: (D + 2) 2^-24 of the sum of
    # their sizes; a weight is off by that, relatively, and so is the sum it is divided by
    big = float((q.double().abs().amax(1).amax(1) @ kv.abs().amax(0).amax(0).amax(0)).max()) * abs(scale)
    bound = attention_bound(want, mag, 700, float(vv.abs().max())) + 2 * (D + 2) * 2.0 ** -24 * big * mag
    assert ((out - want).abs() <= bound).all(), float(((out - want).abs() / bound).max())
