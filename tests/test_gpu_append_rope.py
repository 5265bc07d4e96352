"""paged_kv_append_rope(_fp8) against the definition in 64 bits: rotated queries and keys within one
rounding, values and pass-through dims bit for bit, and every other cache row untouched."""
import pytest
import torch

from paged_kv_decode_21_gb300 import ops, workloads
from serving_ref import deal_tables, make_cache, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_21_gb300 import build
    build.build()
    ops.lib()


def rope_table(n, R, base=10000.0):
    a = torch.arange(n, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    return torch.cat((a.cos(), a.sin()), 1).float().cuda()


def turned(x, table, pos, R, pairs):
    """(rotated x, sum of the terms' magnitudes) in double, from the fp32 table."""
    x = x.double().clone()
    mag = x.abs()
    if R:
        c, s = table[pos, :R // 2].double()[:, None], table[pos, R // 2:].double()[:, None]
        ia = torch.arange(0, R, 2, device=x.device) if pairs else torch.arange(R // 2, device=x.device)
        ib = ia + (1 if pairs else R // 2)
        a, b = x[..., ia].clone(), x[..., ib].clone()
        x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return x, mag


def near_f16(got, want, mag):
    # one rounding to fp16 (2^-11, or 2^-25 absolute below the normal range), three in fp32
    bound = 2.0 ** -11 * want.abs() + 2.0 ** -25 + 3 * 2.0 ** -24 * mag
    err = (got.double() - want).abs()
    assert (err <= bound).all(), (err / bound).max().item()


def near_e4m3(codes, want, mag, scale):
    """One rounding to E4M3 of want / scale: half a step (2^-4, or 2^-10 absolute), saturating."""
    x = want / scale
    got = values(codes)
    bound = 2.0 ** -4 * x.abs() + 2.0 ** -10 + 4 * 2.0 ** -24 * mag / scale
    big = x.abs() > 448
    assert torch.equal(got[big], 448.0 * torch.sign(x[big]))
    err = (got - x).abs()[~big]
    assert (err <= bound[~big]).all(), (err / bound[~big]).max().item()


def problem(news, past, Hq, Hkv, D, R, BS, seed, fp8=False, pad=0, extra_rows=3):
    T = sum(news) + extra_rows
    g = torch.Generator(device="cuda").manual_seed(seed)
    row = (Hq + 2 * Hkv) * D + pad
    qkv = workloads.randn_f16((T, row), g, "cuda")
    q = qkv[:, :Hq * D].view(T, Hq, D) if Hq else None
    k = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    v = qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(T, Hkv, D)
    ends = [a + b for a, b in zip(past, news)]
    pool = sum(-(-e // BS) for e in ends) + 3
    bt, _ = deal_tables(ends, BS, max(1, -(-max(ends) // BS)), pool, seed)
    kc, vc = make_cache((pool, Hkv, BS, D), seed + 1, fp8), make_cache((pool, Hkv, BS, D), seed + 2, fp8)
    starts = torch.tensor([0] + torch.tensor(news).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    return qkv, q, k, v, bt, kc, vc, starts, torch.tensor(past, dtype=torch.int32, device="cuda")


def run_and_check(news, past, Hq, Hkv, D, R, BS, pairs, seed, fp8=False, pad=0, positions=None, in_place=False):
    qkv, q, k, v, bt, kc, vc, starts, lens = problem(news, past, Hq, Hkv, D, R, BS, seed, fp8, pad)
    T, n = k.shape[0], sum(news)
    b = torch.repeat_interleave(torch.arange(len(news)), torch.tensor(news)).cuda()
    at = (lens[b] + torch.arange(n, device="cuda") - starts[b]).long()
    pos = at
    given = None
    if positions is not None:
        given = torch.randint(0, positions, (T,), dtype=torch.int32, device="cuda",
                              generator=torch.Generator(device="cuda").manual_seed(seed + 9))
        pos = given[:n].long()
    table = rope_table(int(pos.max()) + 1 if n else 1, R) if R else torch.zeros((1, 0), device="cuda")
    ks, vs = 0.0213, 0.0171
    k_ref, v_ref = values(kc), values(vc)
    q_ref, q_mag = turned(q[:n], table, pos, R, pairs) if Hq else (None, None)
    k_new, k_mag = turned(k[:n], table, pos, R, pairs)
    v_new = v[:n].double()
    kc0, vc0 = kc.clone(), vc.clone()
    q_out = q if in_place else (torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda") if Hq else None)
    tail = q[n:].clone() if in_place else None
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(token_starts=starts, positions=given, interleaved=pairs, q_out=q_out, error_word=ew)
    if fp8:
        got = ops.paged_kv_append_rope_fp8(q, k, v, table, bt, lens, kc, vc, ks, vs, **kw)
    else:
        got = ops.paged_kv_append_rope(q, k, v, table, bt, lens, kc, vc, **kw)
    assert ops.pkd_read_device_error(ew) == 0
    if Hq:
        near_f16(got[:n], q_ref, q_mag)
        assert torch.equal(got[:n, :, R:], q[:n, :, R:])
        # rows behind the last sequence stay as they were
        assert torch.equal(got[n:], tail) if in_place else (got[n:] == 7.0).all()
    phys, slot = bt[b, at // BS].long(), at % BS
    if fp8:
        near_e4m3(kc[phys, :, slot], k_new, k_mag, ks)
        near_e4m3(vc[phys, :, slot], v_new, v_new.abs(), vs)
    else:
        near_f16(kc[phys, :, slot], k_new, k_mag)
        assert torch.equal(kc[phys, :, slot][..., R:], k[:n, :, R:])
        assert torch.equal(vc[phys, :, slot], v[:n])
    kc[phys, :, slot] = kc0[phys, :, slot]
    vc[phys, :, slot] = vc0[phys, :, slot]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,R,BS", [(8, 2, 128, 128, 16), (4, 4, 64, 32, 32), (7, 1, 96, 96, 16),
                                           (3, 3, 16, 16, 1), (40, 8, 128, 64, 16), (2, 1, 512, 128, 5)])
def test_ragged_tokens(Hq, Hkv, D, R, BS, pairs, fp8):
    # no token, one, a block's worth, block boundaries on both sides, a long run
    run_and_check([0, 1, BS, 17, 0, 130, 3], [5, 0, BS - 1, BS, 9, 2 * BS + 1, 1000], Hq, Hkv, D, R, BS, pairs,
                  seed=D + R, fp8=fp8)


@pytest.mark.parametrize("seqs", [1, 31, 32, 33, 65, 1025])
def test_every_sequence_is_found(seqs):
    run_and_check([(i * 7) % 3 for i in range(seqs)] if seqs > 1 else [1], [i % 20 for i in range(seqs)], 4, 2, 64, 64,
                  16, False, seed=seqs)


def test_strided_rows_in_place_and_given_positions():
    run_and_check([5, 1, 40], [3, 100, 0], 8, 2, 128, 128, 16, False, 3, pad=24, positions=5000, in_place=True)
    run_and_check([5, 1, 40], [3, 100, 0], 8, 2, 128, 64, 16, True, 4, fp8=True, pad=8, positions=3)


def test_keys_and_values_alone_and_no_rotation():
    run_and_check([3, 4], [0, 31], 0, 2, 64, 64, 16, False, 5)
    run_and_check([3, 4], [0, 31], 4, 2, 64, 0, 16, False, 6)
    run_and_check([3, 4], [0, 31], 4, 2, 64, 0, 16, False, 7, fp8=True)


def test_uniform_runs_need_no_starts():
    _, q, k, v, bt, kc, vc, starts, lens = problem([2] * 6, [4, 15, 16, 0, 30, 7], 4, 2, 128, 128, 16, 8,
                                                   extra_rows=0)
    table = rope_table(64, 128)
    kc2, vc2 = kc.clone(), vc.clone()
    a = ops.paged_kv_append_rope(q, k, v, table, bt, lens, kc, vc, token_starts=starts)
    b = ops.paged_kv_append_rope(q, k, v, table, bt, lens, kc2, vc2)
    assert torch.equal(a, b) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_zero_rotation_matches_the_plain_append():
    # position 0 turns nothing: cos 1, sin 0
    _, q, k, v, bt, kc, vc, starts, lens = problem([1] * 5, [4, 15, 16, 0, 30], 4, 2, 128, 128, 16, 9, extra_rows=0)
    table = rope_table(1, 128)
    kc2, vc2 = kc.clone(), vc.clone()
    zero = torch.zeros(5, dtype=torch.int32, device="cuda")
    out = ops.paged_kv_append_rope(q, k, v, table, bt, lens, kc, vc, positions=zero)
    ops.paged_kv_append(k.contiguous(), v.contiguous(), bt, lens, kc2, vc2)
    assert torch.equal(out, q) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_far_positions_and_offsets_past_32_bits():
    # token strides whose last token starts past 2^31 elements, far rotation positions
    Hkv, D, BS, T = 1, 16, 16, 3
    stride = (1 << 30) + 8 * 5
    big = torch.zeros(2 * stride + D, dtype=torch.float16, device="cuda")
    k = torch.as_strided(big, (T, Hkv, D), (stride, D, 1))
    g = torch.Generator(device="cuda").manual_seed(1)
    k.copy_(workloads.randn_f16((T, Hkv, D), g, "cuda"))
    table = rope_table(1 << 20, D)
    bt = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((2, Hkv, BS, D), dtype=torch.float16, device="cuda") for _ in range(2))
    pos = torch.tensor([0, 524287, 1048575], dtype=torch.int32, device="cuda")
    ops.paged_kv_append_rope(None, k, k, table, bt, torch.zeros(1, dtype=torch.int32, device="cuda"), kc, vc,
                             positions=pos)
    want, mag = turned(k, table, pos.long(), D, False)
    near_f16(kc[1, :, :T].transpose(0, 1), want, mag)
    assert torch.equal(vc[1, :, :T].transpose(0, 1), k)


def test_bad_tokens_are_skipped_and_reported():
    news, past = [2, 2, 2, 2], [0, 47, 5, 3]
    _, q, k, v, bt, kc, vc, starts, lens = problem(news, past, 4, 2, 64, 64, 16, 11)
    bt = bt.clone()
    bt[2, 0] = kc.shape[0]       # outside the pool
    lens[3] = -1                 # no such length
    # sequence 1: position 47 fits its row of four blocks, 48 has no block (-1)
    bt[1, 3] = -1
    table = rope_table(47, 64)   # and position 47 no row of the table
    q_out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    kc0, vc0 = kc.clone(), vc.clone()
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.paged_kv_append_rope(q, k, v, table, bt, lens, kc, vc, token_starts=starts, q_out=q_out, error_word=ew)
    assert ops.pkd_read_device_error(ew) == ops.DEVERR_BAD_BLOCK | ops.DEVERR_BAD_POSITION
    assert (q_out[2:] == 7.0).all() and not (q_out[:2] == 7.0).all()
    p = int(bt[0, 0])
    assert torch.equal(vc[p, :, :2].transpose(0, 1), v[:2])
    kc[p, :, :2], vc[p, :, :2] = kc0[p, :, :2], vc0[p, :, :2]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)


def test_refusals_of_the_binding():
    _, q, k, v, bt, kc, vc, starts, lens = problem([1, 1], [0, 0], 4, 2, 64, 64, 16, 12, extra_rows=0)
    table = rope_table(4, 64)
    with pytest.raises(ValueError):
        ops.paged_kv_append_rope(q.float(), k, v, table, bt, lens, kc, vc)
    with pytest.raises(ValueError):
        ops.paged_kv_append_rope(q, k[:, :, ::2], v, table, bt, lens, kc, vc)
    with pytest.raises(ValueError):
        ops.paged_kv_append_rope(q, k, v, table.double(), bt, lens, kc, vc)
    with pytest.raises(ValueError):
        ops.paged_kv_append_rope(q, k, v, table, bt, lens, kc, vc, token_starts=starts[:2])
    with pytest.raises(ops.PagedDecodeError):
        ops.paged_kv_append_rope(q, k, v, table[:, :24].contiguous(), bt, lens, kc, vc)   # rotary_dim 24
    with pytest.raises(ops.PagedDecodeError):
        ops.paged_kv_append_rope_fp8(q, k, v, table, bt, lens, kc.view(torch.uint8)[..., :64].contiguous(),
                                     kc.view(torch.uint8)[..., :64].contiguous(), 0.0, 1.0)
