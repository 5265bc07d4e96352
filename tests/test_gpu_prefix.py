"""paged_decode_attention_prefix(_fp8) against 64-bit attention over prefix and own tokens together."""
import pytest
import torch

from paged_kv_decode_21_gb300 import ops, workloads
from serving_ref import check, deal_tables, make_cache, prefix_attention, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_21_gb300 import build
    build.build()
    ops.lib()


def problem(sizes, plens, lens, q_len, Hq, Hkv, D, BS, seed, fp8=False, outside=0):
    """Groups of the given sizes (and `outside` sequences behind the last group)."""
    B = sum(sizes) + outside
    assert len(lens) == B
    pool = sum(-(-n // BS) for n in list(lens) + list(plens)) + 2
    bt, rest = deal_tables(lens, BS, -(-max(list(lens) + [1]) // BS), pool, seed)
    ptab = torch.full((len(plens), max(1, -(-max(list(plens) + [1]) // BS))), -1, dtype=torch.int32)
    at = 0
    for y, n in enumerate(plens):
        m = -(-n // BS)
        ptab[y, :m] = rest[at:at + m]
        at += m
    shape = (pool, Hkv, BS, D)
    kc, vc = make_cache(shape, seed + 1, fp8), make_cache(shape, seed + 2, fp8)
    g = torch.Generator(device="cuda").manual_seed(seed + 3)
    q = workloads.randn_f16((B, q_len, Hq, D), g, "cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    starts = i32([0] + torch.tensor(sizes).cumsum(0).tolist() if sizes else [0])
    return q, kc, vc, ptab.cuda(), i32(list(plens)), starts, bt, i32(list(lens))


def run_and_check(p, BS, fp8=False, what="", **kw):
    q, kc, vc, ptab, plens, starts, bt, lens = p
    D = q.shape[-1]
    scale = D ** -0.5
    ks, vs = workloads.E4M3_SCALES["full"] if fp8 else (1.0, 1.0)
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    if fp8:
        out = ops.paged_decode_attention_prefix_fp8(q, kc, vc, ptab, plens, starts, bt, lens, scale, ks, vs,
                                                    error_word=ew, **kw)
    else:
        out = ops.paged_decode_attention_prefix(q, kc, vc, ptab, plens, starts, bt, lens, scale, error_word=ew, **kw)
    assert ops.pkd_read_device_error(ew) == 0
    ref, mag = prefix_attention(q, kc, vc, ptab, plens, starts, bt, lens, scale, ks, vs, BS)
    longest = int(plens.max() if plens.numel() else 0) + int(lens.max())
    check(out, ref, mag, longest, values(vc).abs().max().item() * vs, what)
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,BS", [(8, 2, 128, 16), (4, 4, 64, 16), (7, 1, 128, 32), (16, 2, 64, 32),
                                         (10, 2, 128, 16), (3, 3, 128, 32)])
@pytest.mark.parametrize("q_len", [1, 3])
def test_groups_of_every_size(Hq, Hkv, D, BS, q_len, fp8):
    # one sequence, several, no prefix, one token of prefix, a prefix that ends inside a block
    sizes, plens = [1, 7, 2, 3, 40], [100, 333, 0, 1, 2 * BS]
    lens = [q_len + (i * 37) % 90 for i in range(sum(sizes))]
    lens[3], lens[4] = 0, 1  # no own token, or fewer than new ones
    run_and_check(problem(sizes, plens, lens, q_len, Hq, Hkv, D, BS, seed=Hq + D, fp8=fp8), BS, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("plen", [1, 15, 64, 65, 127, 129, 1000, 4097])
@pytest.mark.parametrize("B", [1, 5, 33, 70])
def test_prefix_lengths_and_batches(B, plen, fp8):
    lens = [1 + (i * 53) % 200 for i in range(B)]
    run_and_check(problem([B], [plen], lens, 1, 8, 2, 128, 16, seed=B + plen, fp8=fp8), 16, fp8)


@pytest.mark.parametrize("G", range(1, 9))
@pytest.mark.parametrize("D", [64, 128])
def test_every_group_size_of_heads(G, D):
    run_and_check(problem([50, 3], [700, 90], [5 + i for i in range(53)], 1, 2 * G, 2, D, 16, seed=G), 16)


def test_many_groups_and_sequences_outside_them():
    sizes = [(i * 5) % 4 for i in range(70)]   # empty groups among them
    plens = [(i * 29) % 150 for i in range(70)]
    B = sum(sizes) + 3
    run_and_check(problem(sizes, plens, [1 + (i * 13) % 40 for i in range(B)], 1, 4, 2, 64, 16, seed=2, outside=3), 16)


def test_no_groups_is_plain_decode():
    p = problem([], [], [9, 100, 33], 1, 8, 2, 128, 16, seed=3, outside=3)
    out = run_and_check(p, 16)
    q, kc, vc, _, _, _, bt, lens = p
    plain = ops.paged_decode_attention(q[:, 0].contiguous(), kc, vc, bt, lens, 128 ** -0.5)
    assert (out[:, 0].double() - plain.double()).abs().max() <= 2.0 ** -9


def test_nothing_to_attend_to_gives_zeros():
    p = problem([2, 1], [0, 0], [0, 0, 0], 1, 8, 2, 128, 16, seed=4)
    assert (run_and_check(p, 16, max_prefix_len=16, max_context_len=16) == 0).all()
    assert (run_and_check(p, 16, max_prefix_len=0, max_context_len=0) == 0).all()


def test_prefix_alone_matches_decode_over_it():
    # every sequence's own context empty: each row attends to the prefix only
    p = problem([6], [300], [0] * 6, 1, 8, 2, 128, 16, seed=5)
    run_and_check(p, 16)


def test_rows_past_the_lengths_are_not_read():
    # whatever lies behind the last token of a block (prefix or own) does not count, NaN included
    p = problem([5], [1000], [7, 20, 33, 50, 1], 1, 28, 4, 128, 16, seed=6)
    q, kc, vc, ptab, plens, starts, bt, lens = p
    want = run_and_check(p, 16)
    for row, n in [(ptab[0], 1000)] + [(bt[b], int(lens[b])) for b in range(5)]:
        if n % 16:
            blk = int(row[n // 16])
            kc[blk, :, n % 16:] = float("nan")
            vc[blk, :, n % 16:] = float("inf")
    out = ops.paged_decode_attention_prefix(q, kc, vc, ptab, plens, starts, bt, lens, 128 ** -0.5)
    assert torch.equal(out, want)


def test_large_scores_stay_finite():
    p = problem([40], [500], [30] * 40, 1, 8, 2, 128, 16, seed=7)
    q = p[0]
    q.mul_(60.0)
    out = ops.paged_decode_attention_prefix(*p[:8], 1.0)
    ref, _ = prefix_attention(*p, 1.0, 1.0, 1.0, 16)
    assert torch.isfinite(out).all()
    # scores of thousands: weights are all but one-hot, and a fp32 score is off by 2^-24 * 128 terms of ~60 * 4
    assert (out.double() - ref).abs().max() <= 0.05


@pytest.mark.parametrize("B,Hq,Hkv,plen,own,fp8,q_len", [(64, 32, 8, 4096, 300, False, 1), (48, 28, 4, 3000, 90, True, 4),
                                                         (256, 28, 4, 2100, 40, False, 1)])
def test_larger_batches(B, Hq, Hkv, plen, own, fp8, q_len):
    lens = [q_len + (i * 71) % own for i in range(B)]
    run_and_check(problem([B], [plen], lens, q_len, Hq, Hkv, 128, 16, seed=8, fp8=fp8), 16, fp8)


def test_long_own_contexts_split():
    run_and_check(problem([2], [600], [5000, 3001], 1, 8, 2, 128, 16, seed=9), 16)
    run_and_check(problem([2], [600], [5000, 3001], 5, 28, 4, 128, 16, seed=10, fp8=True), 16, True)


def test_repeats_bit_for_bit_on_a_stream_and_in_a_graph():
    p = problem([20, 12], [900, 77], [4 + (i * 11) % 120 for i in range(32)], 1, 28, 4, 128, 16, seed=11)
    q, kc, vc, ptab, plens, starts, bt, lens = p
    lens -= 3  # room to grow into
    most = bt.shape[1] * 16
    kw = dict(max_prefix_len=900, max_context_len=most)
    want = run_and_check(p, 16, **kw)
    ws = ops.alloc_workspace(ops.paged_decode_prefix_workspace_size(32, 1, 28, 4, 128, 16, 2, 900, most), "cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q)
    ops.paged_decode_attention_prefix(*p, 128 ** -0.5, out=out, workspace=ws, stream=side, **kw)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.paged_decode_attention_prefix(*p, 128 ** -0.5, out=out, workspace=ws, **kw)
    # the graph follows lengths and groups that change between replays
    for shift in (0, 3):
        lens.copy_(lens + shift)
        starts.copy_(torch.tensor([0, 20 - shift, 32], dtype=torch.int32))
        out.zero_()
        graph.replay()
        ref, mag = prefix_attention(*p, 128 ** -0.5, 1.0, 1.0, 16)
        check(out, ref, mag, 1030, values(vc).abs().max().item())


@pytest.mark.parametrize("seed", range(30))
def test_random_shapes(seed):
    import random
    r = random.Random(1000 + seed)
    Hkv = r.choice((1, 2, 4, 8))
    Hq, D, BS, fp8, q_len = Hkv * r.randint(1, 8), r.choice((64, 128, 128)), r.choice((16, 32)), r.random() < 0.5, r.choice((1, 1, 2, 7))
    sizes = [r.randint(0, 40) for _ in range(r.randint(1, 4))]
    outside = r.randint(0 if sum(sizes) else 1, 3)
    plens = [r.choice((r.randint(0, 70), r.randint(0, 3000))) for _ in sizes]
    lens = [r.choice((0, r.randint(0, 20), r.randint(0, 700))) for _ in range(sum(sizes) + outside)]
    run_and_check(problem(sizes, plens, lens, q_len, Hq, Hkv, D, BS, seed, fp8, outside), BS, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_negative_and_zero_scales(fp8):
    p = problem([40], [300], [20] * 40, 1, 8, 2, 128, 16, seed=15, fp8=fp8)
    ks, vs = workloads.E4M3_SCALES["full"] if fp8 else (1.0, 1.0)
    for scale in (-0.05, 0.0):
        out = (ops.paged_decode_attention_prefix_fp8(*p, scale, ks, vs) if fp8
               else ops.paged_decode_attention_prefix(*p, scale))
        ref, mag = prefix_attention(*p, scale, ks, vs, 16)
        check(out, ref, mag, 320, values(p[2]).abs().max().item() * vs)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("before,size,after", [(0, 3, 61), (70, 40, 5), (1500, 9, 600)])
def test_more_groups_than_sequences(before, size, after, fp8):
    # a table of fixed size whose other groups are empty
    plens = [17] * before + [1500] + [300] * after
    p = problem([0] * before + [size] + [0] * after, plens, [30 + i for i in range(size)], 1, 8, 2, 128, 16,
                seed=19, fp8=fp8)
    run_and_check(p, 16, fp8)


@pytest.mark.parametrize("sizes,fp8", [([330], False), ([300], True), ([100, 0, 171, 30], False)])
def test_more_row_chunks_than_sms(sizes, fp8):
    # 8 kv heads x 20 and more chunks of rows: the shared part's grid takes more than one wave
    B = sum(sizes)
    p = problem(sizes, [1300 + 10 * y for y in range(len(sizes))], [4 + i % 30 for i in range(B)], 4, 32, 8, 128, 16,
                seed=21, fp8=fp8)
    run_and_check(p, 16, fp8)


@pytest.mark.parametrize("which", ["torch", "raw"])
def test_temporaries_of_a_call_on_another_stream_stay_its_own(which, monkeypatch):
    """The workspace allocated inside a call on a given stream is not handed out again while that
    stream has yet to run the call."""
    p = problem([40], [1000], [200] * 40, 1, 8, 2, 128, 16, seed=20)
    want = ops.paged_decode_attention_prefix(*p, 0.1, max_prefix_len=1000, max_context_len=200)
    spaces, alloc = [], ops.alloc_workspace

    def noted(n, dev):
        t = alloc(n, dev)
        spaces.append((t.data_ptr(), n))
        return t

    monkeypatch.setattr(ops, "alloc_workspace", noted)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # 0.1 s
    out = ops.paged_decode_attention_prefix(*p, 0.1, max_prefix_len=1000, max_context_len=200,
                                            stream=side if which == "torch" else side.cuda_stream)
    later = [torch.empty(spaces[0][1] + 256, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query()
    at, n = spaces[0]
    assert all(x.data_ptr() + x.numel() <= at or at + n <= x.data_ptr() for x in later)
    side.synchronize()
    assert torch.equal(out, want)


def test_groups_that_reach_past_the_batch_stay_inside_it():
    # group starts past the batch (or below zero) are cut to it
    p = list(problem([5, 3], [200, 100], [30] * 8, 1, 8, 2, 128, 16, seed=16))
    want = ops.paged_decode_attention_prefix(*p, 0.1)
    p[5] = torch.tensor([-4, 5, 1000], dtype=torch.int32, device="cuda")
    assert torch.equal(ops.paged_decode_attention_prefix(*p, 0.1), want)


@pytest.mark.parametrize("fp8,q_len", [(False, 1), (True, 1), (False, 5), (True, 5)])
def test_calls_back_to_back_on_one_workspace(fp8, q_len):
    """The two grids of a call overlap, and the merge starts early: calls in a row on one stream and one
    workspace, each on other queries, give what each gives alone."""
    p = problem([60], [3000], [q_len + (i * 37) % 300 for i in range(60)], q_len, 28, 4, 128, 16, seed=17, fp8=fp8)
    ks, vs = workloads.E4M3_SCALES["full"] if fp8 else (1.0, 1.0)
    g = torch.Generator(device="cuda").manual_seed(18)
    qs = [workloads.randn_f16(p[0].shape, g, "cuda") for _ in range(4)]
    kw = dict(max_prefix_len=3000, max_context_len=p[6].shape[1] * 16)

    def call(q, **more):
        if fp8:
            return ops.paged_decode_attention_prefix_fp8(q, *p[1:], 0.09, ks, vs, **kw, **more)
        return ops.paged_decode_attention_prefix(q, *p[1:], 0.09, **kw, **more)

    alone = []
    for q in qs:
        alone.append(call(q))
        torch.cuda.synchronize()
    ws = ops.alloc_workspace(
        ops.paged_decode_prefix_workspace_size(60, q_len, 28, 4, 128, 16, 1, 3000, kw["max_context_len"]), "cuda")
    outs = [torch.empty_like(qs[0]) for _ in range(40)]
    for i, out in enumerate(outs):
        call(qs[i % 4], out=out, workspace=ws)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, alone[i % 4]), i


def test_bad_blocks_are_reported_and_nothing_else_is_read():
    p = problem([3], [100], [40, 40, 40], 1, 8, 2, 128, 16, seed=12)
    q, kc, vc, ptab, plens, starts, bt, lens = p
    ptab[0, 2] = kc.shape[0] + 5
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.paged_decode_attention_prefix(*p, 0.1, error_word=ew)
    assert ops.pkd_read_device_error(ew) == ops.DEVERR_BAD_BLOCK and torch.isfinite(out).all()


def test_refusals_of_the_binding():
    p = list(problem([3], [100], [40, 40, 40], 1, 8, 2, 128, 16, seed=13))
    with pytest.raises(ValueError):
        ops.paged_decode_attention_prefix(*p[:5], p[5][:1], *p[6:], 0.1)      # too few group starts
    with pytest.raises(ValueError):
        ops.paged_decode_attention_prefix(p[0].float(), *p[1:], 0.1)
    with pytest.raises(ops.PagedDecodeError):
        ops.paged_decode_attention_prefix(*p, float("nan"))
    with pytest.raises(ops.PagedDecodeError):
        ops.paged_decode_attention_prefix(*p, 0.1, max_prefix_len=7 * 16 + 1)  # longer than its table row
    with pytest.raises(ops.PagedDecodeError):
        ops.paged_decode_attention_prefix(*p, 0.1, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
