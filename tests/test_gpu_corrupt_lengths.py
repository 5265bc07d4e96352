"""Lengths near INT_MAX, or negative, among good ones, on grids that walk their pieces longest first: reported, cut to
the table row, and nothing written outside the workspace that the call asked for."""
import pytest
import torch

import longcache_ref as ref
from serving_ref import make_cache
from paged_kv_decode_21_gb300 import ops, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
INT_MAX = 2 ** 31 - 1
BAD = {1: INT_MAX, 4: INT_MAX - 100, 7: INT_MAX - 8192, 9: 1 << 30, 11: -1, 12: -(1 << 31)}  # by sequence


def round_up(x, a):
    return -(-x // a) * a


def int4_plan(B, ql, Hq, H, D, BS, most):
    """(partitions, whether the order is made) of the automatic plan, from the workspace's size."""
    auto = ops.paged_decode_int4_workspace_size(B, ql, Hq, H, D, BS, most)
    for part in (-1, 128, 256, 512, 1024, 2048, 4096, 8192):
        n = 1 if part < 0 or part >= most else -(-most // part)
        plain = ops.paged_decode_int4_workspace_size(B, ql, Hq, H, D, BS, most, part)
        if auto - plain == round_up(4 * B * n, 256):
            return n, True
    return 0, False


def problem(kind, B, ql, Hq, H, most, seed):
    """Every row of the tables is full, with blocks that sequences share; lengths from 0 to most."""
    D, BS, NB = 128, 16, 300
    g = torch.Generator(device=DEV).manual_seed(seed)
    bt = torch.randint(0, NB, (B, most // BS), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    lens = torch.randint(0, most + 1, (B,), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    lens[0], lens[2], lens[3] = most, 0, 1
    if kind == "int4":
        kc, vc = (ref.random_int4((NB, H, BS), D, seed + i) for i in (1, 2))
    else:
        kc, vc = (make_cache((NB, H, BS, D), seed + i, kind == "e4m3") for i in (1, 2))
    q = workloads.randn_f16((B, ql, Hq, D), g, DEV)
    return q, kc, vc, bt, lens


@pytest.mark.parametrize("kind,B,ql,Hq,H,most,np", [
    ("int4", 160, 1, 32, 8, 1536, 1), ("int4", 32, 1, 32, 8, 8192, 4), ("int4", 70, 4, 28, 4, 8192, 2),
    ("fp16", 160, 1, 32, 8, 1536, 1), ("e4m3", 160, 1, 32, 8, 1536, 1), ("fp16", 200, 8, 28, 4, 2048, 1),
    ("e4m3", 200, 8, 28, 4, 2048, 1)])
def test_lengths_that_no_row_holds(kind, B, ql, Hq, H, most, np):
    D, BS = 128, 16
    q, kc, vc, bt, good = problem(kind, B, ql, Hq, H, most, B + ql)
    bad, cut = good.clone(), good.clone()
    for b, n in BAD.items():
        bad[b], cut[b] = n, min(max(n, 0), most)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    if kind == "int4":
        assert int4_plan(B, ql, Hq, H, D, BS, most) == (np, True)
        size = ops.paged_decode_int4_workspace_size(B, ql, Hq, H, D, BS, most)
    else:
        n, part, order, variant, *_ = ops.paged_decode_call_plan(B, ql, Hq, H, D, BS, most, kv_fp8=kind == "e4m3")
        assert order, (n, part, variant)
        size = ops.paged_decode_multi_workspace_size(B, ql, Hq, H, D, BS, most)
    assert size > 0
    space = torch.full((size + (1 << 20),), 0xA5, dtype=torch.uint8, device=DEV)

    def call(lens):
        kw = dict(max_context_len=most, workspace=space[:size], error_word=err, out=torch.full_like(q, 7.0))
        if kind == "int4":
            return ops.paged_decode_attention_int4(q, kc, vc, bt, lens, 0.09, 0.1, 0.1, **kw)
        if kind == "e4m3":
            return ops.paged_decode_attention_fp8(q, kc, vc, bt, lens, 0.09, 1 / 64, 1 / 64, **kw)
        return ops.paged_decode_attention_multi(q, kc, vc, bt, lens, 0.09, **kw)

    want = call(cut)
    assert ops.pkd_read_device_error(err) == 0
    got = call(bad)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK
    assert (space[size:] == 0xA5).all()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", ["fp16", "e4m3"])
def test_split_tails_of_such_lengths(kind):
    """The tcgen05 path's order that also splits its shortest sequences in two."""
    D, BS, ql, Hq, H, most = 128, 16, 8, 28, 4, 2048
    size = lambda B: ops.paged_decode_multi_workspace_size(B, ql, Hq, H, D, BS, most)  # noqa: E731
    B = next(B for B in range(160, 400) if size(B) > 1 << 20)    # (partials: the tail is split)
    n, part, order, variant, *_ = ops.paged_decode_call_plan(B, ql, Hq, H, D, BS, most, kv_fp8=kind == "e4m3")
    assert part == -1 and order and variant.startswith("tcgen05")
    q, kc, vc, bt, good = problem(kind, B, ql, Hq, H, most, 5)
    good[:] = torch.where(good > most // 2, good, most - good)   # all long enough to be split
    bad, cut = good.clone(), good.clone()
    for b, n in BAD.items():
        bad[b], cut[b] = n, min(max(n, 0), most)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    space = torch.full((size(B) + (1 << 20),), 0xA5, dtype=torch.uint8, device=DEV)

    def call(lens):
        kw = dict(max_context_len=most, workspace=space[:size(B)], error_word=err, out=torch.full_like(q, 7.0))
        if kind == "e4m3":
            return ops.paged_decode_attention_fp8(q, kc, vc, bt, lens, 0.09, 1 / 64, 1 / 64, **kw)
        return ops.paged_decode_attention_multi(q, kc, vc, bt, lens, 0.09, **kw)

    want = call(cut)
    assert ops.pkd_read_device_error(err) == 0
    got = call(bad)
    assert ops.pkd_read_device_error(err) == ops.DEVERR_BAD_BLOCK
    assert (space[size(B):] == 0xA5).all()
    # Which sequences are split goes by the lengths, and a split row's softmax weights are rounded to fp16 against
    # another maximum (2^-11 of each, twice), its output once more (2^-11): of values below 6.
    assert torch.isfinite(got).all() and (got.float() - want.float()).abs().max() <= 4 * 6 * 2.0 ** -11
