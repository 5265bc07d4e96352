"""E4M3 codes of rotated appends are those of the IEEE quotient, for every fp16 value and scales of all sizes: codes go
by both neighbours of the scale's reciprocal where these agree."""
import pytest
import torch

from serving_ref import E4M3
from paged_kv_decode_21_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"

SCALES = [1.0, 1 / 64, 0.3, 1 / 3, 0.7, 1.1, 7.0, 448.0, 1e-3, 3.1e-5, 5.9e-8, 1.7e4, 1e-29, 1.1e-30, 1e-31, 9e29, 2e30,
          1e-40, 3e38, 1.0000001, 0.99999994]


@pytest.mark.parametrize("copies", [1, 40])       # 128 and 5120 tokens: a token a CTA, and runs of tokens
@pytest.mark.parametrize("shift", range(3))
def test_every_value(copies, shift):
    H, D, BS = 4, 128, 16
    bits = torch.arange(65536, dtype=torch.int32)
    x = bits.to(torch.int16).view(torch.float16)
    x = torch.where(x.isfinite(), x, torch.zeros((), dtype=torch.float16)).view(-1, H, D)
    x = x[torch.randperm(128, generator=torch.Generator().manual_seed(1))]
    k, v = x.to(DEV).repeat(copies, 1, 1), x.flip(0).to(DEV).repeat(copies, 1, 1)
    T = 128 * copies
    bt = torch.arange(T // BS, dtype=torch.int32, device=DEV)[None]
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.cat((torch.ones((T, D // 2)), torch.zeros((T, D // 2))), 1).to(DEV)     # angle 0: x cos - y sin = x
    for ks, vs in zip(SCALES[shift::3], SCALES[::-1][shift::3]):
        ks, vs = (float(torch.tensor(s, dtype=torch.float32)) for s in (ks, vs))
        kc = torch.zeros((T // BS, H, BS, D), dtype=torch.uint8, device=DEV)
        vc = torch.zeros_like(kc)
        ops.paged_kv_append_rope_fp8(None, k, v, table, bt, zero, kc, vc, ks, vs)
        for cache, rows, s in ((kc, x, ks), (vc, x.flip(0), vs)):
            quotient = rows.float() / torch.tensor(s, dtype=torch.float32)
            want = quotient.clamp(-448, 448).to(E4M3).view(torch.uint8)
            got = cache.transpose(1, 2).reshape(T, H, D).cpu().view(copies, 128, H, D)
            same = (got == want) | ((got & 0x7F == 0) & (want & 0x7F == 0) & (rows == 0))    # (0 cos - 0 sin: either zero)
            assert same.all(), (s, rows.expand(copies, -1, -1, -1)[~same][:4], got[~same][:4])
