"""4-bit appends whose cache scales lie at the ends of fp32's range: the quantiser's codes, bit for bit."""
import pytest
import torch

import longcache_ref as ref
from paged_kv_decode_21_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("scale,turn", [
    (1e-39, 2e-39),       # steps of about 1e-39: their reciprocals are past fp32
    (3e-41, 4e-40), (1.4e-45, 1e-43), (1e-45, 6e-45), (1e-37, 3e-37), (1e-38, 1e-38),
    (1e35, 1e36), (4e37, 1e38), (3e38, 1e38),   # 7 times the last is infinite: no scale
    (2.0 ** -110, 2.0 ** -109), (2.0 ** 110, 2.0 ** 111)])
def test_codes_of_scales_at_the_ends(scale, turn, pairs):
    """Keys of about `turn` (a table of that size turns them) over cache scales of `scale`."""
    T, H, D, BS = 64, 2, 128, 16
    g = torch.Generator().manual_seed(3)
    x = torch.randn((T, 2 * H, D), generator=g).half()
    x[0] = 0
    x[1, :, 3:] = 0
    table = (torch.rand((T, D), generator=g) - 0.5) * turn
    kc = torch.full((T // BS, H, BS, 9 * D // 16), 0xA5, dtype=torch.uint8, device=DEV)
    vc = kc.clone()
    one = float(torch.tensor(scale, dtype=torch.float32))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    bt = torch.arange(T // BS, dtype=torch.int32, device=DEV)[None]
    ops.paged_kv_append_rope_int4(None, x[:, :H].contiguous().to(DEV), x[:, H:].contiguous().to(DEV), table.to(DEV), bt,
                                  torch.zeros(1, dtype=torch.int32, device=DEV), kc, vc, one, one, interleaved=pairs,
                                  error_word=err)
    assert ops.pkd_read_device_error(err) == 0
    y = ref.rotate32(x[:, :H], table[:, :D // 2], table[:, D // 2:], D, pairs)
    want_k, want_v = torch.empty(kc.shape, dtype=torch.uint8), torch.empty(kc.shape, dtype=torch.uint8)
    for t in range(T):
        ref.write_int4(want_k, D, t // BS, t % BS, *ref.int4_rows(y[t], one))
        ref.write_int4(want_v, D, t // BS, t % BS, *ref.int4_rows(x[t, H:].float(), one))
    assert torch.equal(kc.cpu(), want_k) and torch.equal(vc.cpu(), want_v)
