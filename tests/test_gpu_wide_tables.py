"""Block tables whose rows hold 2^31 tokens and more."""
import pytest
import torch

from paged_kv_decode_21_gb300 import ops
from serving_ref import check, deal_tables, listed_attention, make_cache, prefix_attention, values

pytestmark = pytest.mark.gpu

WIDTH = (1 << 27) + 8  # x 16 tokens


@pytest.fixture(scope="module")
def data():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_21_gb300 import build, workloads
    build.build()
    ops.lib()
    table = torch.full((1, WIDTH), -1, dtype=torch.int32, device="cuda")
    bt, _ = deal_tables([300], 16, 19, 25, 71)
    table[:, :19] = bt
    q = workloads.randn_f16((1, 8, 128), torch.Generator(device="cuda").manual_seed(72), "cuda")
    kc, vc = make_cache((25, 2, 16, 128), 73, False), make_cache((25, 2, 16, 128), 74, False)
    return q, kc, vc, bt, table, torch.tensor([300], dtype=torch.int32, device="cuda")


def ok(ew):
    assert ops.pkd_read_device_error(ew) == 0


@pytest.mark.parametrize("variant", ["no_prefetch", "l2_prefetch", "tma_staged", "tma_mma", "tcgen05"])
def test_dense_decode(data, variant):
    q, kc, vc, bt, table, cl = data
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = ops.paged_decode_attention_ex(q, kc, vc, bt, cl, 0.09, variant=variant, error_word=ew)
    out = ops.paged_decode_attention_ex(q, kc, vc, table, cl, 0.09, variant=variant, error_word=ew)
    ok(ew)
    assert torch.equal(out, want)
    ops.paged_decode_validate_tables(table, cl, 16, kc.shape[0], ew)
    ok(ew)


@pytest.mark.parametrize("B", [1, 400])
def test_shared_prefix(data, B):
    q, kc, vc, bt, table, cl = data
    q = q.expand(B, 8, 128).contiguous()[:, None].contiguous()
    own, lens = bt[:, 17:].expand(B, -1).contiguous(), torch.full((B,), 28, dtype=torch.int32, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (kc, vc, table, i32([272]), i32([0, B]), own, lens)
    out = ops.paged_decode_attention_prefix(q, *args, 0.09, error_word=ew)
    ok(ew)
    ref, mag = prefix_attention(q[:1], kc, vc, bt, i32([272]), i32([0, 1]), own[:1], lens[:1], 0.09, 1.0, 1.0, 16)
    check(out[:1], ref, mag, 300, values(vc).abs().max().item())
    assert torch.equal(out, out[:1].expand_as(out))


def test_bounds_choice_and_listed_decode(data):
    q, kc, vc, bt, table, cl = data
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    b1, b2 = (torch.zeros((25, 2, 2, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    ops.paged_kv_block_bounds(kc, bt, cl, b1, error_word=ew)
    ops.paged_kv_block_bounds(kc, table, cl, b2, max_new_tokens=300, error_word=ew)
    assert torch.equal(b1, b2)
    ops.paged_kv_block_bounds(kc, table, cl, b2.zero_(), error_word=ew)  # the row's own length as the bound
    assert torch.equal(b1, b2)
    lists, counts = ops.paged_kv_block_select(q, b2, table, cl, 6, 16, error_word=ew)
    want = ops.paged_kv_block_select(q, b1, bt, cl, 6, 16, error_word=ew)
    assert torch.equal(lists, want[0]) and torch.equal(counts, want[1])
    out = ops.paged_decode_attention_blocks(q, kc, vc, table, cl, lists, counts, 0.09, error_word=ew)
    ok(ew)
    ref, mag = listed_attention(q, kc, vc, bt, [300], lists, counts, 0.09, 1.0, 1.0, 16)
    check(out, ref, mag, 96, values(vc).abs().max().item())
