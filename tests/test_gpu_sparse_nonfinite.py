"""The choice of blocks where keys or queries are not finite: such blocks come first, the lists stay whole."""
import pytest
import torch

from paged_kv_decode_21_gb300 import ops, workloads
from serving_ref import values

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_21_gb300 import build
    build.build()
    ops.lib()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def ordered(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    b = workloads.randn_f16(shape, g, "cuda")
    return torch.stack((torch.minimum(b[:, :, 0], b[:, :, 1]), torch.maximum(b[:, :, 0], b[:, :, 1])), 2).contiguous()


def expected(q, bounds, bt, blocks, K, sink, recent):
    """By the definition, in 64 bits: a block with a bound that is not finite, or a score that is NaN or +inf,
    scores +inf; ties go to the lowest index."""
    B, Hq, D = q.shape
    Hkv = bounds.shape[1]
    G = Hq // Hkv
    lists = torch.full((B, Hkv, K), -1, dtype=torch.int32)
    for b in range(B):
        m = blocks[b]
        for g in range(Hkv):
            e = values(bounds[bt[b, :m].long(), g])
            x = q[b, g * G:(g + 1) * G].double()[:, None]
            s = (x.clamp(max=0) * e[:, 0] + x.clamp(min=0) * e[:, 1]).sum(-1)  # heads x blocks
            s = torch.where(torch.isnan(s), INF, s).amax(0)
            s = torch.where(torch.isfinite(e).all(-1).all(-1), s, INF).tolist()
            always = list(range(sink)) + list(range(m - recent, m))
            rest = sorted(range(sink, m - recent), key=lambda i: (-s[i], i))
            pick = sorted(always + rest[:K - sink - recent]) if m > K else list(range(m))
            lists[b, g, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return lists


def run(q, bounds, bt, blocks, K, sink, recent):
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    lists, counts = ops.paged_kv_block_select(q, bounds, bt, i32([16 * n - 3 for n in blocks]), K, 16, sink, recent,
                                              error_word=ew)
    assert ops.pkd_read_device_error(ew) == 0
    assert counts.flatten().tolist() == [min(K, n) for n in blocks for _ in range(bounds.shape[1])]
    assert torch.equal(lists.cpu(), expected(q, bounds, bt, blocks, K, sink, recent))


@pytest.mark.parametrize("how,fp8", [("hi", False), ("lo", False), ("both", False), ("nan", False), ("nan", True)])
@pytest.mark.parametrize("blocks,bad,K", [(60, 1, 9), (60, 5, 9), (60, 6, 9), (60, 30, 9), (60, 57, 9), (3000, 4, 64),
                                          (3000, 61, 64), (3000, 62, 64), (3000, 900, 64), (3000, 2997, 64)])
def test_blocks_with_bounds_that_are_not_finite_come_first(blocks, bad, K, how, fp8):
    Hq, Hkv, D, sink, recent = 8, 2, 128, 1, 2
    bounds = ordered((blocks + 3, Hkv, 2, D), blocks + bad)
    if fp8:
        bounds = bounds.to(torch.float8_e4m3fn).view(torch.uint8)
    g = torch.Generator().manual_seed(bad)
    ids = torch.randperm(blocks, generator=g)[:bad].cuda()
    dims = torch.randint(0, D, (bad,), generator=g).cuda()
    bt = torch.randperm(blocks + 3, generator=g)[None, :blocks].int().cuda().contiguous()
    at = bt[0, ids].long()
    if how in ("hi", "both"):
        bounds[at, :, 1, dims] = INF
    if how in ("lo", "both"):
        bounds[at, :, 0, dims] = -INF
    if how == "nan":
        bounds[at, :, 1, dims] = 0x7F if fp8 else NAN
    q = workloads.randn_f16((1, Hq, D), torch.Generator(device="cuda").manual_seed(7), "cuda")
    q[0, 1, ::3] = 0
    run(q, bounds, bt, [blocks], K, sink, recent)


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("heads", [[2], [0, 1, 2, 3]])
@pytest.mark.parametrize("blocks", [60, 3000])
def test_queries_that_are_not_finite(blocks, heads, value):
    """Their head scores every block +inf, NaN or -inf; the other group's choice is untouched."""
    Hq, Hkv, D = 8, 2, 128
    bounds = ordered((blocks, Hkv, 2, D), blocks)
    bt = torch.randperm(blocks, generator=torch.Generator().manual_seed(3))[None].int().cuda()
    q = workloads.randn_f16((1, Hq, D), torch.Generator(device="cuda").manual_seed(8), "cuda")
    for h in heads:
        q[0, h, 5 + h] = value
    run(q, bounds, bt, [blocks], 9, 1, 2)


def test_the_largest_finite_bounds_and_queries():
    """Scores of 128 * 65504^2 and the error bound that goes with them stay finite."""
    Hq, Hkv, D, blocks = 4, 1, 128, 400
    bounds = ordered((blocks, Hkv, 2, D), 4)
    bounds[::3, :, 1] = 65504.0
    bounds[1::3, :, 0] = -65504.0
    bt = torch.arange(blocks, device="cuda")[None].int()
    q = workloads.randn_f16((1, Hq, D), torch.Generator(device="cuda").manual_seed(9), "cuda")
    q[0, 0, ::2], q[0, 0, 1::2] = 65504.0, -65504.0
    run(q, bounds, bt, [blocks], 30, 1, 2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,BS", [(128, 16), (64, 16), (128, 32), (64, 32)])
def test_bounds_of_keys_that_are_not_finite(D, BS, fp8):
    """A NaN key makes both bounds of its dim NaN, wherever it lies among the block's tokens; infinities are
    ordinary; what lies behind the last token does not count."""
    Hkv, lens = 3, [5 * BS + 3, 1, 2 * BS]
    bt = torch.tensor([[0, 1, 2, 3, 4, 5], [6] + [-1] * 5, [7, 8] + [-1] * 4], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(D + BS)
    kc = workloads.randn_f16((9, Hkv, BS, D), g, "cuda")
    if fp8:
        kc = kc.to(torch.float8_e4m3fn).view(torch.uint8)
    nan = 0x7F if fp8 else NAN
    kc[0, 0, 0, 3], kc[1, 1, BS - 1, D - 1], kc[2, 2, 7, 40], kc[3, 0, :, 9] = nan, nan, nan, nan
    kc[5, 1, 2, 5], kc[5, 1, 3:, 6], kc[6, 0, 0, 0], kc[6, 0, 1:, 1] = nan, nan, nan, nan
    if not fp8:
        kc[7, 0, 4, 2], kc[7, 0, 5, 2], kc[8, 1, :, 8] = INF, -INF, INF
    bounds = torch.zeros((9, Hkv, 2, D), dtype=kc.dtype, device="cuda")
    ops.paged_kv_block_bounds(kc, bt, i32(lens), bounds)
    for b, n in enumerate(lens):
        for i in range(-(-n // BS)):
            p = int(bt[b, i])
            x = values(kc[p, :, :min(BS, n - i * BS)])
            got = values(bounds[p])
            for e, want in enumerate((x.amin(1), x.amax(1))):  # (amin and amax keep NaN)
                assert torch.equal(torch.isnan(got[:, e]), torch.isnan(want))
                assert torch.equal(got[:, e].nan_to_num(0.0, 1e9, -1e9), want.nan_to_num(0.0, 1e9, -1e9))
