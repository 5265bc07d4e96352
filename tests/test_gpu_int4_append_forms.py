"""The forms of the 4-bit append that take no list of starts, no positions or one position a token, and turn the
queries in place: whole caches against the quantiser's definition."""
import pytest
import torch

import longcache_ref as ref
from serving_ref import deal_tables
from test_gpu_int4 import i32, new_rows, rope
from paged_kv_decode_21_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("D,BS,R,pairs", [(128, 16, 128, False), (128, 32, 64, True), (64, 16, 64, False), (64, 32, 0, False)])
@pytest.mark.parametrize("per", [1, 3])
@pytest.mark.parametrize("given", [True, False])
def test_one_run_of_one_length_a_sequence(D, BS, R, pairs, per, given):
    Hq, H, past = 6, 3, [0, 7, 31, 14, 15]
    B, T = len(past), 5 * per
    scale = (1 / 16, 0.3)
    x, q, k, v = new_rows(T, Hq, H, D, D + per)
    table = rope(97, max(R, 2))[:, :R].contiguous()
    bt, _ = deal_tables([n + per for n in past], BS, 4, 16, 3)
    logical = torch.tensor([past[t // per] + t % per for t in range(T)])
    pos = torch.randint(0, 97, (T,), generator=torch.Generator().manual_seed(9)) if given else logical
    kc = torch.full((16, H, BS, 9 * D // 16), 0xA5, dtype=torch.uint8, device=DEV)
    vc = kc.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = ops.paged_kv_append_rope_int4(q, k, v, table.to(DEV), bt, i32(*past), kc, vc, *scale,
                                        positions=i32(*pos.tolist()) if given else None, interleaved=pairs, q_out=q,
                                        error_word=err)
    assert out is q and ops.pkd_read_device_error(err) == 0
    cos, sin = ref.rows_of(table, pos[None], torch.zeros(R // 2, dtype=torch.int64), R)
    y = ref.rotate32(x[:, :Hq + H], cos, sin, R, pairs) if R else x[:, :Hq + H].float()
    want_k = torch.full(kc.shape, 0xA5, dtype=torch.uint8)
    want_v = want_k.clone()
    for t in range(T):
        p = int(logical[t])
        at = int(bt[t // per, p // BS])
        assert at >= 0
        ref.write_int4(want_k, D, at, p % BS, *ref.int4_rows(y[t, Hq:], scale[0]))
        ref.write_int4(want_v, D, at, p % BS, *ref.int4_rows(x[t, Hq + H:].float(), scale[1]))
    assert torch.equal(kc.cpu(), want_k) and torch.equal(vc.cpu(), want_v)
    assert torch.equal(q.cpu(), y[:, :Hq].half())
