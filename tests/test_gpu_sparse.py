"""Block bounds, the choice of blocks and attention over the chosen ones, against 64 bits; and the whole
serving step (rotated append, bounds, choice, attention) as a user runs it."""
import pytest
import torch

from paged_kv_decode_21_gb300 import ops, workloads
from serving_ref import (block_bounds, block_select, check, deal_tables, listed_attention, make_cache, values)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_21_gb300 import build
    build.build()
    ops.lib()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def new_bounds(pool, Hkv, D, fp8, fill=1.0):
    b = torch.full((pool, Hkv, 2, D), fill, dtype=torch.float16, device="cuda")
    return b.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else b


def problem(lens, Hq, Hkv, D, BS, seed, fp8=False):
    pool = sum(-(-n // BS) for n in lens) + 2
    bt, _ = deal_tables(lens, BS, -(-max(lens) // BS), pool, seed)
    kc, vc = make_cache((pool, Hkv, BS, D), seed + 1, fp8), make_cache((pool, Hkv, BS, D), seed + 2, fp8)
    g = torch.Generator(device="cuda").manual_seed(seed + 3)
    q = workloads.randn_f16((len(lens), Hq, D), g, "cuda")
    return q, kc, vc, bt, i32(lens)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,BS,Hkv", [(128, 16, 2), (64, 16, 3), (128, 32, 1), (64, 32, 8)])
def test_bounds_are_exact(D, BS, Hkv, fp8):
    lens = [0, 1, BS - 1, BS, BS + 1, 5 * BS + 3, 700]
    q, kc, vc, bt, cl = problem([max(n, 1) for n in lens], Hkv, Hkv, D, BS, D + BS, fp8)
    cl = i32(lens)
    # whatever lies behind a sequence's last token does not count
    for b, n in enumerate(lens):
        if n % BS and not fp8:
            kc[int(bt[b, n // BS]), :, n % BS:] = float("nan")
    bounds = new_bounds(kc.shape[0], Hkv, D, fp8)
    want = block_bounds(kc, bt, lens, [0] * len(lens), bounds, BS)
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.paged_kv_block_bounds(kc, bt, cl, bounds, error_word=ew)
    assert ops.pkd_read_device_error(ew) == 0
    assert torch.equal(values(bounds), want)
    # only the blocks from start_lens on are written again
    start = [0, 0, BS - 1, 0, BS, 3 * BS + 1, 699]
    again = new_bounds(kc.shape[0], Hkv, D, fp8, 2.0)
    want = block_bounds(kc, bt, lens, start, again, BS)
    ops.paged_kv_block_bounds(kc, bt, cl, again, start_lens=i32(start), max_new_tokens=3 * BS, error_word=ew)
    assert ops.pkd_read_device_error(ew) == 0
    assert torch.equal(values(again), want)


def test_bounds_report_bad_blocks():
    q, kc, vc, bt, cl = problem([50, 40], 2, 2, 64, 16, 1)
    bounds = new_bounds(kc.shape[0], 2, 64, False)
    bt[1, 1] = kc.shape[0]
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.paged_kv_block_bounds(kc, bt, cl, bounds, error_word=ew)
    assert ops.pkd_read_device_error(ew) == ops.DEVERR_BAD_BLOCK
    ops.paged_kv_block_bounds(kc, bt, i32([50, 16 * bt.shape[1] + 1]), bounds, max_new_tokens=80, error_word=ew)
    assert ops.pkd_read_device_error(ew) == ops.DEVERR_BAD_BLOCK


def full_bounds(kc, bt, cl, fp8):
    b = new_bounds(kc.shape[0], kc.shape[1], kc.shape[3], fp8)
    ops.paged_kv_block_bounds(kc, bt, cl, b)
    return b


def select_and_check(q, bounds, bt, lens, K, sink, recent, BS, **kw):
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    lists, counts = ops.paged_kv_block_select(q, bounds, bt, i32(lens), K, BS, sink, recent, error_word=ew, **kw)
    assert ops.pkd_read_device_error(ew) == 0
    want, wn = block_select(q, bounds, bt, lens, K, sink, recent, BS)
    assert torch.equal(counts.cpu(), wn)
    assert torch.equal(lists.cpu(), want)
    return lists, counts


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,BS", [(8, 2, 128, 16), (4, 4, 64, 16), (7, 1, 128, 32), (16, 2, 64, 32), (3, 1, 128, 16)])
@pytest.mark.parametrize("K,sink,recent", [(1, 0, 0), (4, 1, 1), (9, 4, 5), (40, 0, 3), (64, 3, 0)])
def test_choice_is_that_of_exact_scores(Hq, Hkv, D, BS, K, sink, recent, fp8):
    lens = [0, 1, K * BS, K * BS + 1, 1500, 3001, 40 * BS - 1]
    q, kc, vc, bt, cl = problem([max(n, 1) for n in lens], Hq, Hkv, D, BS, K + D, fp8)
    select_and_check(q, full_bounds(kc, bt, i32(lens), fp8), bt, lens, K, sink, recent, BS)


@pytest.mark.parametrize("blocks", [15, 255, 256, 257, 511, 513, 1024, 2047, 4099])
def test_choice_over_any_number_of_blocks(blocks):
    q, kc, vc, bt, cl = problem([16 * blocks - 3, 16 * (blocks // 2) + 1], 4, 2, 64, 16, blocks)
    select_and_check(q, full_bounds(kc, bt, cl, False), bt, cl.tolist(), 13, 1, 2, 16)


def tied(kind, blocks, Hkv, D, seed):
    """Bounds whose scores are equal, nearly so, or apart only far below fp32."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    b = workloads.randn_f16((blocks, Hkv, 2, D), g, "cuda")
    b = torch.stack((torch.minimum(b[:, :, 0], b[:, :, 1]), torch.maximum(b[:, :, 0], b[:, :, 1])), 2)
    if kind == "all":
        b[:] = b[:1].clone()
    elif kind == "few":
        b[:] = b[torch.arange(blocks, device="cuda") % 5].clone()
    elif kind == "near":  # one dim apart by a fp16 step of a small number, others equal
        b[:] = b[:1].clone()
        b[:, :, 0, 0] = -4.0
        b[:, :, 1, 0] = (1.0 + torch.randint(0, 9, (blocks,), generator=g, device="cuda") * 2.0 ** -10).half()[:, None]
        b[:, :, 1, 0] *= 2.0 ** -13
    elif kind == "zero":
        b[:] = 0
    return b.contiguous()


@pytest.mark.parametrize("kind", ["all", "few", "near", "zero"])
@pytest.mark.parametrize("blocks,K", [(40, 7), (700, 33), (3000, 500)])
def test_equal_and_nearly_equal_scores(kind, blocks, K):
    Hq, Hkv, D = 6, 2, 128
    bounds = tied(kind, blocks, Hkv, D, blocks)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = workloads.randn_f16((2, Hq, D), g, "cuda")
    q[1, :3] = 0  # a group whose queries are all zero
    bt = torch.stack([torch.randperm(blocks, generator=torch.Generator().manual_seed(i)) for i in range(2)]).int().cuda()
    select_and_check(q, bounds, bt, [16 * blocks, 16 * blocks - 5], K, 2, 1, 16)


def test_choice_with_large_outliers():
    # one dim a thousand times the others: the error bound is wide, the choice still exact
    q, kc, vc, bt, cl = problem([20000, 777], 8, 2, 128, 16, 21)
    bounds = full_bounds(kc, bt, cl, False)
    bounds[..., 7] = torch.tensor([-3000.0, 3000.0], device="cuda", dtype=torch.float16)
    select_and_check(q, bounds, bt, cl.tolist(), 50, 1, 1, 16)


def test_choice_at_the_largest_number_of_blocks():
    blocks = ops.MAX_SELECT_BLOCKS
    g = torch.Generator(device="cuda").manual_seed(3)
    pool = 4096
    b = workloads.randn_f16((pool, 1, 2, 64), g, "cuda")
    bounds = torch.stack((torch.minimum(b[:, :, 0], b[:, :, 1]), torch.maximum(b[:, :, 0], b[:, :, 1])), 2)
    q = workloads.randn_f16((1, 8, 64), g, "cuda")
    bt = (torch.arange(blocks, device="cuda") % pool)[None].int()  # blocks again and again: ties by the dozen
    lists, counts = ops.paged_kv_block_select(q, bounds, bt, i32([16 * blocks]), 100, 16, 1, 1)
    e = bounds[:, 0].double()
    s = torch.maximum(q[0].double()[:, None] * e[:, 0], q[0].double()[:, None] * e[:, 1]).sum(-1).amax(0)
    s = s[bt[0].long()]
    s[0] = s[-1] = float("inf")
    want = s.sort(descending=True, stable=True).indices[:100].sort().values
    assert int(counts) == 100 and torch.equal(lists[0, 0].long(), want)
    with pytest.raises(ops.PagedDecodeError):
        ops.paged_kv_block_select(q, bounds, torch.zeros((1, blocks + 1), dtype=torch.int32, device="cuda"),
                                  i32([5]), 100, 16, max_context_len=16 * blocks + 1)


def test_choice_avoids_and_reports_blocks_outside_the_pool():
    q, kc, vc, bt, cl = problem([900, 700], 8, 2, 128, 16, 31)
    bounds = full_bounds(kc, bt, cl, False)
    bad = bt.clone()
    bad[0, 7], bad[0, 30], bad[1, 11] = kc.shape[0], -1, 1 << 30
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    lists, counts = ops.paged_kv_block_select(q, bounds, bad, cl, 20, 16, 1, 1, error_word=ew)
    assert ops.pkd_read_device_error(ew) == ops.DEVERR_BAD_BLOCK
    # as if those blocks scored below all others (whose bounds have zero inside)
    low = torch.cat((bounds, torch.zeros_like(bounds[:1])))
    good = torch.where((bad < 0) | (bad >= kc.shape[0]), kc.shape[0], bad)
    want, _ = block_select(q, low, good, cl.tolist(), 20, 1, 1, 16)
    assert torch.equal(lists.cpu(), want) and (counts == 20).all()
    # chosen all the same where there is nothing else
    lists, counts = ops.paged_kv_block_select(q, bounds, bad, cl, 55, 16, 1, 1, error_word=ew)
    assert ops.pkd_read_device_error(ew) == ops.DEVERR_BAD_BLOCK
    assert counts.tolist() == [[55, 55], [44, 44]]
    assert not {7, 30} & set(lists[0].flatten().tolist())


def test_lengths_past_the_callers_bound_are_reported():
    q, kc, vc, bt, cl = problem([900, 700], 8, 2, 128, 16, 32)
    bounds = full_bounds(kc, bt, cl, False)
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    lists, counts = ops.paged_kv_block_select(q, bounds, bt, cl, 10, 16, 1, 1, max_context_len=800, error_word=ew)
    assert ops.pkd_read_device_error(ew) == ops.DEVERR_BAD_BLOCK
    want, _ = block_select(q, bounds, bt, [800, 700], 10, 1, 1, 16)
    assert torch.equal(lists.cpu(), want)


@pytest.mark.parametrize("fp8", [False, True])
def test_blocks_past_32_bits_of_a_large_pool(fp8):
    """A pool of more than 2^31 elements: the sequences' blocks lie at both ends of it."""
    Hq, Hkv, D, BS, lens = 32, 8, 128, 16, [600, 333]
    pool = (1 << 31) // (Hkv * BS * D) + 5000
    per = [-(-n // BS) for n in lens]
    ids = torch.cat((torch.arange(40), torch.arange(pool - sum(per) + 40, pool)))
    bt = torch.full((2, max(per)), -1, dtype=torch.int32)
    bt[0, :per[0]], bt[1, :per[1]] = ids[:per[0]].int(), ids[per[0]:].flip(0).int()
    kind = torch.uint8 if fp8 else torch.float16
    kc, vc = (torch.empty((pool, Hkv, BS, D), dtype=kind, device="cuda") for _ in range(2))
    kc[ids.cuda()], vc[ids.cuda()] = (make_cache((len(ids), Hkv, BS, D), k, fp8) for k in (1, 2))
    bt, cl = bt.cuda(), i32(lens)
    bounds = torch.empty((pool, Hkv, 2, D), dtype=kind, device="cuda")
    ops.paged_kv_block_bounds(kc, bt, cl, bounds)
    small = torch.zeros((pool,), dtype=torch.bool, device="cuda")
    small[ids.cuda()] = True
    for b, n in enumerate(lens):
        for i in (0, per[b] - 1):
            x = values(kc[int(bt[b, i]), :, :min(BS, n - i * BS)])
            got = values(bounds[int(bt[b, i])])
            assert torch.equal(got[:, 0], x.amin(1)) and torch.equal(got[:, 1], x.amax(1))
    g = torch.Generator(device="cuda").manual_seed(3)
    q = workloads.randn_f16((2, Hq, D), g, "cuda")
    lists, counts = select_and_check(q, bounds, bt, lens, 12, 1, 1, BS)
    attend_and_check(q, kc, vc, bt, lens, lists, counts, BS, fp8)
    # and a prefix at the far end
    from serving_ref import prefix_attention
    ptab = bt[1:, :per[1]].contiguous()
    ks, vs = workloads.E4M3_SCALES["full"] if fp8 else (1.0, 1.0)
    q4 = workloads.randn_f16((3, 1, Hq, D), g, "cuda")
    args = (q4, kc, vc, ptab, i32([lens[1]]), i32([0, 3]), bt[[0, 0, 0]].contiguous(), i32([600, 1, 17]))
    out = (ops.paged_decode_attention_prefix_fp8(*args, D ** -0.5, ks, vs) if fp8
           else ops.paged_decode_attention_prefix(*args, D ** -0.5))
    ref, mag = prefix_attention(*args, D ** -0.5, ks, vs, BS)
    check(out, ref, mag, 1000, 448 * vs if fp8 else 6.0)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    import random
    r = random.Random(seed)
    Hkv = r.choice((1, 2, 3, 8))
    Hq, D, BS, fp8 = Hkv * r.randint(1, 8), r.choice((64, 128)), r.choice((16, 32)), r.random() < 0.5
    lens = [r.choice((1, r.randint(1, 60), r.randint(1, 6000))) for _ in range(r.randint(1, 40))]
    K = r.choice((1, 2, 7, 31, 64, 130))
    sink = r.randint(0, min(2, K))
    recent = r.randint(0, K - sink)
    q, kc, vc, bt, cl = problem(lens, Hq, Hkv, D, BS, seed, fp8)
    lists, counts = select_and_check(q, full_bounds(kc, bt, cl, fp8), bt, lens, K, sink, recent, BS)
    attend_and_check(q, kc, vc, bt, lens, lists, counts, BS, fp8)


def test_calls_on_another_stream_repeat_bit_for_bit():
    q, kc, vc, bt, cl = problem([3000, 1501, 40], 28, 4, 128, 16, 33)
    bounds = full_bounds(kc, bt, cl, False)
    lists, counts = ops.paged_kv_block_select(q, bounds, bt, cl, 50, 16)
    out = ops.paged_decode_attention_blocks(q, kc, vc, bt, cl, lists, counts, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the current stream
        b2 = new_bounds(kc.shape[0], 4, 128, False)
        ops.paged_kv_block_bounds(kc, bt, cl, b2)
    l2, c2 = ops.paged_kv_block_select(q, b2, bt, cl, 50, 16, stream=side)  # a given one
    o2 = ops.paged_decode_attention_blocks(q, kc, vc, bt, cl, l2, c2, 0.1, stream=side)
    side.synchronize()
    used = torch.unique(bt[bt >= 0]).long()
    assert torch.equal(bounds[used], b2[used]) and torch.equal(lists, l2) and torch.equal(counts, c2)
    assert torch.equal(out, o2)


def attend_and_check(q, kc, vc, bt, lens, lists, counts, BS, fp8, **kw):
    ks, vs = workloads.E4M3_SCALES["full"] if fp8 else (1.0, 1.0)
    scale = q.shape[-1] ** -0.5
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    if fp8:
        out = ops.paged_decode_attention_blocks_fp8(q, kc, vc, bt, i32(lens), lists, counts, scale, ks, vs,
                                                    error_word=ew, **kw)
    else:
        out = ops.paged_decode_attention_blocks(q, kc, vc, bt, i32(lens), lists, counts, scale, error_word=ew, **kw)
    assert ops.pkd_read_device_error(ew) == 0
    ref, mag = listed_attention(q, kc, vc, bt, lens, lists, counts, scale, ks, vs, BS)
    check(out, ref, mag, lists.shape[-1] * BS, values(vc[torch.unique(bt[bt >= 0]).long()]).abs().max().item() * vs)
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,BS", [(8, 2, 128, 16), (4, 4, 64, 16), (7, 1, 128, 32), (16, 2, 64, 32), (10, 2, 128, 16)])
@pytest.mark.parametrize("K", [1, 5, 20, 77])
def test_attention_over_chosen_blocks(Hq, Hkv, D, BS, K, fp8):
    lens = [0, 1, BS, 300, 1501, 3000, 5 * BS - 1]
    q, kc, vc, bt, cl = problem([max(n, 1) for n in lens], Hq, Hkv, D, BS, K + D, fp8)
    for b, n in enumerate(lens):  # rows behind the last token do not count
        if n % BS and not fp8:
            kc[int(bt[b, n // BS]), :, n % BS:] = float("nan")
            vc[int(bt[b, n // BS]), :, n % BS:] = float("nan")
    lists, counts = select_and_check(q, full_bounds(kc, bt, i32(lens), fp8), bt, lens, K, 0, 1, BS)
    vc2 = torch.nan_to_num(vc) if not fp8 else vc
    kc2 = torch.nan_to_num(kc) if not fp8 else kc
    out = attend_and_check(q, kc2, vc2, bt, lens, lists, counts, BS, fp8)
    if not fp8:
        assert torch.equal(out, ops.paged_decode_attention_blocks(q, kc, vc, bt, i32(lens), lists, counts, D ** -0.5))


def test_every_block_listed_matches_dense_decode():
    lens = [700, 33, 1000]
    q, kc, vc, bt, cl = problem(lens, 28, 4, 128, 16, 3)
    K = 63
    lists = torch.arange(K, device="cuda", dtype=torch.int32).expand(3, 4, K).contiguous()
    counts = i32([[-(-n // 16)] * 4 for n in lens])
    out = attend_and_check(q, kc, vc, bt, lens, lists, counts, 16, False)
    dense = ops.paged_decode_attention(q, kc, vc, bt, cl, 128 ** -0.5)
    assert (out.double() - dense.double()).abs().max() <= 2.0 ** -9


def test_lists_in_any_order_and_of_any_length():
    lens = [700, 640, 1000]
    q, kc, vc, bt, cl = problem(lens, 8, 2, 128, 16, 4)
    g = torch.Generator().manual_seed(4)
    lists = torch.full((3, 2, 30), -7, dtype=torch.int32)
    counts = torch.zeros((3, 2), dtype=torch.int32)
    for b in range(3):
        for h in range(2):
            n = [0, 1, 30, 17, 29, 8][2 * b + h]
            pick = torch.randperm(lens[b] // 16, generator=g)[:n]
            if n and lens[b] % 16 and h:
                pick[-1] = lens[b] // 16  # the partly filled block, last
            lists[b, h, :n], counts[b, h] = pick.int(), n
    attend_and_check(q, kc, vc, bt, lens, lists.cuda(), counts.cuda(), 16, False)


def test_entries_that_break_the_list_rule_are_reported():
    lens = [100]
    q, kc, vc, bt, cl = problem(lens, 8, 2, 128, 16, 5)
    good = [0, 3, 5]
    want = None
    # none; outside the sequence; negative; the partly filled block not at the end
    for extra in ([], [7], [-1], [6]):
        row = good[:1] + extra + good[1:]
        lists = i32([[row + [-1] * (6 - len(row))] * 2])
        ew = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = ops.paged_decode_attention_blocks(q, kc, vc, bt, cl, lists, i32([[len(row)] * 2]), 0.1, error_word=ew)
        assert ops.pkd_read_device_error(ew) == (ops.DEVERR_BAD_BLOCK if extra else 0)
        want = out if want is None else want
        assert (out.double() - want.double()).abs().max() <= 2.0 ** -9


def test_serving_step_in_a_graph():
    """Rotated append, bounds of the touched blocks, choice and attention over them, captured once and
    replayed while the sequences grow across block boundaries."""
    Hq, Hkv, D, BS, K, B = 8, 2, 128, 16, 6, 3
    lens0, steps = [130, 95, 300], 20
    q, kc, vc, bt, _ = problem([n + steps for n in lens0], Hq, Hkv, D, BS, 6)
    before = i32(lens0)
    after = before + 1
    bounds = new_bounds(kc.shape[0], Hkv, D, False)
    ops.paged_kv_block_bounds(kc, bt, before, bounds)
    pos = torch.arange(512, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    table = torch.cat((pos.cos(), pos.sin()), 1).float().cuda()
    qkv = torch.zeros((B, (Hq + 2 * Hkv) * D), dtype=torch.float16, device="cuda")
    qv, kv, vv = (x.view(B, -1, D) for x in qkv.split((Hq * D, Hkv * D, Hkv * D), 1))
    q_out, out = torch.empty((B, Hq, D), dtype=torch.float16, device="cuda"), torch.empty_like(q)
    lists = torch.empty((B, Hkv, K), dtype=torch.int32, device="cuda")
    counts = torch.empty((B, Hkv), dtype=torch.int32, device="cuda")
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = ops.alloc_workspace(ops.paged_decode_blocks_workspace_size(B, Hq, Hkv, D, BS, K), "cuda")

    def step():
        ops.paged_kv_append_rope(qv, kv, vv, table, bt, before, kc, vc, q_out=q_out, error_word=ew)
        ops.paged_kv_block_bounds(kc, bt, after, bounds, start_lens=before, max_new_tokens=1, error_word=ew)
        ops.paged_kv_block_select(q_out, bounds, bt, after, K, BS, 1, 2, max_context_len=bt.shape[1] * BS,
                                  block_lists=lists, list_lens=counts, error_word=ew)
        ops.paged_decode_attention_blocks(q_out, kc, vc, bt, after, lists, counts, D ** -0.5, out=out, workspace=ws,
                                          error_word=ew)

    step()  # once eagerly, at the same lengths as the first replay
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator(device="cuda").manual_seed(7)
    for _ in range(steps):
        qkv.copy_(workloads.randn_f16(qkv.shape, g, "cuda"))
        graph.replay()
        assert ops.pkd_read_device_error(ew) == 0
        lens = after.tolist()
        want = block_bounds(kc, bt, lens, [0] * B, bounds, BS)
        used = torch.unique(torch.cat([bt[b, :-(-n // BS)] for b, n in enumerate(lens)])).long()
        assert torch.equal(values(bounds)[used], want[used])
        wl, wn = block_select(q_out, bounds, bt, lens, K, 1, 2, BS)
        assert torch.equal(lists.cpu(), wl) and torch.equal(counts.cpu(), wn)
        ref, mag = listed_attention(q_out, kc, vc, bt, lens, lists, counts, D ** -0.5, 1.0, 1.0, BS)
        check(out, ref, mag, K * BS, values(vc).abs().max().item())
        before += 1
        after += 1


def test_refusals_of_the_binding():
    q, kc, vc, bt, cl = problem([100, 50], 8, 2, 128, 16, 8)
    bounds = full_bounds(kc, bt, cl, False)
    with pytest.raises(ValueError):
        ops.paged_kv_block_bounds(kc, bt, cl, bounds[:, :, :1].contiguous())
    with pytest.raises(ValueError):
        ops.paged_kv_block_select(q, bounds.float(), bt, cl, 4, 16)
    with pytest.raises(ops.PagedDecodeError):
        ops.paged_kv_block_select(q, bounds, bt, cl, 4, 16, 3, 2)   # sink + recent above max_selected
    with pytest.raises(ops.PagedDecodeError):
        ops.paged_kv_block_select(q, bounds, bt, cl, 4, 8)
    lists, counts = ops.paged_kv_block_select(q, bounds, bt, cl, 4, 16)
    with pytest.raises(ValueError):
        ops.paged_decode_attention_blocks(q, kc, vc, bt, cl, lists.long(), counts, 0.1)
    with pytest.raises(ops.PagedDecodeError):
        ops.paged_decode_attention_blocks(q, kc, vc, bt, cl, lists, counts, float("inf"))
