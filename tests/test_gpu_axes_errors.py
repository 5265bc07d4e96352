"""What the appends with several axes report does not depend on how many tokens a call has."""
import pytest
import torch

from paged_kv_decode_21_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("kind", ["fp16", "e4m3", "int4"])
@pytest.mark.parametrize("T", [5, 6000])
def test_a_token_with_a_bad_block_and_a_bad_position_reports_both(kind, T):
    D, BS, H = 128, 16, 1
    MB = -(-T // BS)
    k = torch.ones((T + 3, H, D), dtype=torch.float16, device=DEV)
    table = torch.ones((8, D), device=DEV)
    bt = torch.arange(MB, dtype=torch.int32, device=DEV)[None].contiguous()
    pos = torch.zeros((2, T + 3), dtype=torch.int32, device=DEV)
    axes = (torch.arange(D // 2, device=DEV) % 2).to(torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(bt, pos):
        dtype = torch.float16 if kind == "fp16" else torch.uint8
        kc, vc = (torch.full((MB, H, BS, 72 if kind == "int4" else D), 3, dtype=dtype, device=DEV) for _ in range(2))
        kw = dict(token_starts=torch.tensor([0, T], dtype=torch.int32, device=DEV), error_word=err)
        past = torch.zeros(1, dtype=torch.int32, device=DEV)
        if kind == "int4":
            ops.paged_kv_append_rope_int4(None, k, k, table, bt, past, kc, vc, 1.0, 1.0, positions=pos, pair_axes=axes, **kw)
        elif kind == "e4m3":
            ops.paged_kv_append_rope_axes_fp8(None, k, k, table, axes, pos, bt, past, kc, vc, 1.0, 1.0, **kw)
        else:
            ops.paged_kv_append_rope_axes(None, k, k, table, axes, pos, bt, past, kc, vc, **kw)
        return ops.pkd_read_device_error(err), kc, vc

    bits, kc, vc = call(bt, pos)
    assert bits == 0 and not (kc[0, 0, 0] == 3).all()
    no_block, off = bt.clone(), pos.clone()
    no_block[0, -1] = MB
    off[1, T - 1] = 8
    assert call(no_block, pos)[0] == ops.DEVERR_BAD_BLOCK
    assert call(bt, off)[0] == ops.DEVERR_BAD_POSITION
    bits, kc, vc = call(no_block, off)
    assert bits == ops.DEVERR_BAD_BLOCK | ops.DEVERR_BAD_POSITION
    assert (kc[-1] == 3).all() and (vc[-1] == 3).all()
    off[1, T - 1] = 0
    off[:, T:] = -5                                # tokens behind the last sequence are not looked at
    assert call(bt, off)[0] == 0
