"""The shared-context tcgen05 kernel at its edges: what lies behind the lengths, bad blocks, large, negative and
zero scales, empty and cut groups, against 64-bit attention; and that these calls do run that kernel."""
import pytest
import torch

from paged_kv_decode_21_gb300 import ops, workloads
from serving_ref import attend, check, gathered, prefix_attention, values
from test_gpu_prefix import problem

pytestmark = pytest.mark.gpu

# (sequences, query heads, kv heads, head_dim, block_size, E4M3).  Head and row counts whose 16-row tiles alone
# are more than the GPU's 152 SMs, so that the plan takes the shared-context kernel whatever the prefix: 8 kv
# heads x 320 / 16 and more.  CTAs of one row tile (a remainder of 64 rows) and of two are among them.
SHAPES = [(40, 64, 8, 128, 16, False), (40, 64, 8, 128, 32, True), (80, 32, 8, 128, 32, False), (80, 32, 8, 128, 16, True),
          (75, 64, 8, 64, 16, False), (75, 64, 8, 64, 32, False)]
# One kv head, 320 rows: chunks of 128 rows over prefixes of 1900 tokens and more.
NARROW = [(40, 8, 1, 128, 16, False), (40, 8, 1, 128, 32, True)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_21_gb300 import build
    build.build()
    ops.lib()


def make(shape, plens, sizes=None, q_len=1, seed=61):
    B, Hq, Hkv, D, BS, fp8 = shape
    sizes = [B] if sizes is None else sizes
    lens = [q_len + (i * 37) % 90 for i in range(B)]
    return problem(sizes, plens, lens, q_len, Hq, Hkv, D, BS, seed, fp8, outside=B - sum(sizes))


def scales(fp8):
    return workloads.E4M3_SCALES["full"] if fp8 else (1.0, 1.0)


def call(p, scale, fp8, **kw):
    if fp8:
        return ops.paged_decode_attention_prefix_fp8(*p, scale, *scales(fp8), **kw)
    return ops.paged_decode_attention_prefix(*p, scale, **kw)


def kernels_of(tmp_path, run):
    """The names of the kernels that a call launches, from a captured graph's own description."""
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        run()
    path = tmp_path / "graph.dot"
    graph.debug_dump(str(path))
    return path.read_text()


def verify(p, out, scale, BS, fp8, longest):
    ref, mag = prefix_attention(*p, scale, *scales(fp8), BS)
    check(out, ref, mag, longest, values(p[2]).abs().nan_to_num(0.0, 0.0).max().item() * scales(fp8)[1])


@pytest.mark.filterwarnings("ignore:DEBUG")  # torch's own, of the graph's description
@pytest.mark.parametrize("shape,plen", [(s, n) for s in SHAPES for n in (1, 33, 4001)]
                         + [(s, n) for s in NARROW for n in (1900, 4001)])
def test_the_calls_here_run_the_shared_context_kernel(shape, plen, tmp_path):
    p = make(shape, [plen])
    ws = ops.alloc_workspace(ops.paged_decode_prefix_workspace_size(
        shape[0], 1, shape[1], shape[2], shape[3], shape[4], 1, plen, 90), "cuda")
    out = torch.empty_like(p[0])
    names = kernels_of(tmp_path, lambda: call(p, 0.1, shape[5], out=out, workspace=ws, max_prefix_len=plen,
                                              max_context_len=90))
    assert "paged_shared_tc_kernel" in names


@pytest.mark.parametrize("shape,plen", [(s, n) for s in SHAPES for n in (1, 17, 63, 64, 65, 131, 1000, 4001)]
                         + [(s, n) for s in NARROW for n in (1900, 4001)])
def test_nothing_behind_the_last_token_counts(shape, plen):
    """NaN in the keys and infinities (E4M3: NaN, which is all it has) in the values behind the prefix's last
    token, in its block, and behind each sequence's own."""
    BS, fp8 = shape[4], shape[5]
    p = make(shape, [plen])
    q, kc, vc, ptab, plens, starts, bt, lens = p
    scale = shape[3] ** -0.5
    want = call(p, scale, fp8)
    verify(p, want, scale, BS, fp8, plen + 100)
    nan, inf = (0x7F, 0xFF) if fp8 else (float("nan"), float("inf"))
    for row, n in [(ptab[0], plen)] + [(bt[b], int(lens[b])) for b in range(shape[0])]:
        if n % BS:
            blk = int(row[n // BS])
            kc[blk, :, n % BS:] = nan
            vc[blk, :, n % BS:] = inf
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(call(p, scale, fp8, error_word=ew), want)
    assert ops.pkd_read_device_error(ew) == 0


@pytest.mark.parametrize("shape", SHAPES)
def test_unused_blocks_of_the_pool_do_not_count(shape):
    """Table entries past the lengths name blocks full of NaN."""
    BS, fp8 = shape[4], shape[5]
    p = list(make(shape, [1000 + BS // 2]))
    scale = shape[3] ** -0.5
    want = call(p, scale, fp8)
    used = torch.cat((p[3].flatten(), p[6].flatten()))
    spare = [i for i in range(p[1].shape[0]) if i not in set(used.tolist())][0]
    for c in (p[1], p[2]):
        c[spare] = 0x7F if fp8 else float("nan")
    p[3] = torch.cat((p[3], torch.full((1, 9), spare, dtype=torch.int32, device="cuda")), 1).contiguous()
    p[6] = torch.where(p[6] < 0, spare, p[6]).int()
    assert torch.equal(call(p, scale, fp8), want)


def without_blocks(p, scale, ks, vs, BS, bad_prefix, bad_own):
    """64-bit attention that passes over whole blocks of the prefix and of the sequences' own contexts."""
    q, kc, vc, ptab, plens, starts, bt, lens = p
    B, ql, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)

    def kept(row, n, bad):
        t = torch.arange(n, device="cuda")
        return torch.isin(t // BS, torch.tensor(sorted(bad), device="cuda"), invert=True) if bad else t >= 0

    def tokens(c, row, n, g):  # (a bad entry's stand-in is any block: its tokens are dropped)
        return gathered(c, row.clamp(0, c.shape[0] - 1), n, g, BS)

    n0 = int(plens[0])
    keep0 = kept(ptab[0], n0, bad_prefix)
    for g in range(Hkv):
        k0, v0 = tokens(kc, ptab[0], n0, g)[keep0], tokens(vc, ptab[0], n0, g)[keep0]
        for b in range(B):
            n = int(lens[b])
            k1, v1 = tokens(kc, bt[b], n, g), tokens(vc, bt[b], n, g)
            own = kept(bt[b], n, bad_own.get(b, ()))
            for j in range(ql):
                seen = own & (torch.arange(n, device="cuda") <= n - ql + j)
                o, a = attend(q[b, j, g * G:(g + 1) * G], torch.cat((k0, k1[seen])), torch.cat((v0, v1[seen])), scale * ks)
                out[b, j, g * G:(g + 1) * G], mag[b, j, g * G:(g + 1) * G] = o * vs, a * vs
    return out, mag


# few query rows over 16-row tiles (the mma.sync kernel) and the shapes above
@pytest.mark.parametrize("shape", [(3, 8, 2, 128, 16, False), (3, 8, 2, 128, 32, True)] + SHAPES)
@pytest.mark.parametrize("plen,bad", [(100, (0,)), (700, (2, 3, 20)), (1000, "last"), (2500, "tile"), (300, "all")])
def test_bad_blocks_are_passed_over(shape, plen, bad):
    """The error is reported and the result is attention over the blocks that are in the pool."""
    BS, fp8 = shape[4], shape[5]
    p = make(shape, [plen])
    q, kc, vc, ptab, plens, starts, bt, lens = p
    n = -(-plen // BS)
    blocks = {"last": [n - 1], "tile": list(range(256 // BS, 512 // BS)), "all": list(range(n))}.get(bad, bad)
    for i, blk in enumerate(blocks):
        ptab[0, blk] = (kc.shape[0], -1, 1 << 30, -(1 << 31))[i % 4]
    b = int((lens > BS).nonzero()[0])  # and one block of a sequence's own
    bt[b, 0] = kc.shape[0] + 7
    scale = shape[3] ** -0.5
    ks, vs = scales(fp8)
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(p, scale, fp8, error_word=ew)
    assert ops.pkd_read_device_error(ew) == ops.DEVERR_BAD_BLOCK
    ref, mag = without_blocks(p, scale, ks, vs, BS, set(blocks), {b: {0}})
    check(out, ref, mag, plen + 100, values(vc).abs().max().item() * vs)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("scale", [-0.05, 0.0])
def test_negative_and_zero_scales(shape, scale):
    p = make(shape, [777])
    verify(p, call(p, scale, shape[5]), scale, shape[4], shape[5], 900)


@pytest.mark.parametrize("shape", [s for s in SHAPES if not s[5]])
@pytest.mark.parametrize("scale", [1.0, -1.0])
def test_large_scores(shape, scale):
    """Scores of up to thousands: weights all but one-hot.  A score, a sum of D = 128 exact products in the tensor
    cores, is off by at most 1.5 * 2^-19 of sum |q k| (the bound that the choice of blocks uses), and that sum is
    128 * 60 * E|x|^2 = 4900, below 6400: 0.019; the scale and the shift add 3 * 2^-24 of 4300: 0.001.  Relative
    errors d_i of the weights move the result by sum p_i d_i (v_i - out), at most 0.02 * 2 * 6 for |v| < 6 (a
    normal value among 2^21): 0.24, and the 2^-11 roundings of weights and result add below 0.01."""
    p = make(shape, [900])
    p[0].mul_(60.0)
    out = call(p, scale, False)
    ref, _ = prefix_attention(*p, scale, 1.0, 1.0, shape[4])
    assert torch.isfinite(out).all()
    assert (out.double() - ref).abs().max() <= 0.25


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_len", [1, 3])
def test_groups_of_any_place_and_size(fp8, q_len):
    """Sequences before the first group and behind the last, groups without sequences or without a prefix, one of
    a single token, remainders of one and of two row tiles."""
    shape = (150, 32, 8, 128, 16, fp8)
    sizes, plens = [0, 41, 3, 70, 0, 20, 1], [500, 1100, 333, 0, 64, 1, 2000]
    p = list(make(shape, plens, sizes, q_len))
    p[5] = p[5] + 6  # 6 before, the rest behind
    scale = 128 ** -0.5
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(p, scale, fp8, error_word=ew)
    assert ops.pkd_read_device_error(ew) == 0
    verify(p, out, scale, 16, fp8, 2100)


@pytest.mark.parametrize("fp8", [False, True])
def test_groups_that_reach_past_the_batch(fp8):
    shape = (100, 32, 8, 128, 16, fp8)
    p = list(make(shape, [900, 2000], [60, 40]))
    want = call(p, 0.1, fp8)
    verify(p, want, 0.1, 16, fp8, 2100)
    p[5] = torch.tensor([-4, 60, 1000], dtype=torch.int32, device="cuda")
    assert torch.equal(call(p, 0.1, fp8), want)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_prefix_longer_than_its_table_row_is_cut_and_reported(fp8):
    shape = (70, 32, 8, 128, 16, fp8)
    p = list(make(shape, [640]))
    want = call(p, 0.1, fp8)
    p[4] = torch.tensor([5000], dtype=torch.int32, device="cuda")
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(p, 0.1, fp8, error_word=ew, max_prefix_len=640)
    assert ops.pkd_read_device_error(ew) == ops.DEVERR_BAD_BLOCK
    assert torch.equal(out, want)


@pytest.mark.parametrize("fp8", [False, True])
def test_repeats_bit_for_bit(fp8):
    shape = (150, 32, 8, 128, 16, fp8)
    p = make(shape, [3000])
    want = call(p, 0.1, fp8)
    for _ in range(20):
        assert torch.equal(call(p, 0.1, fp8), want)
