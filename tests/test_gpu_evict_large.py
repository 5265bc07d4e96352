"""Weights, choice and compaction in pools whose byte offsets pass 2^32, and of one long sequence."""
import pytest
import torch

import longcache_ref as ref
from test_gpu_evict import SCALE, cache_of, i32
from paged_kv_decode_21_gb300 import ops, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("kind,ql", [("fp16", 1), ("fp16", 6), ("e4m3", 1), ("e4m3", 6), ("int4", 1), ("int4", 6)])
def test_pools_past_32_bits(kind, ql):
    """The pool's last blocks give what the same blocks at its beginning give."""
    D, BS, H, Hq, n, K = 128, 32, 8, 32, 600, 100
    tile = BS * D * {"fp16": 2, "e4m3": 1, "int4": 9 / 16}[kind]
    per, to = -(-n // BS), -(-K // BS)
    NB = int(2 ** 32 // (H * tile)) + 50
    row, dtype = (72 if kind == "int4" else D), (torch.float16 if kind == "fp16" else torch.uint8)
    small = [cache_of(kind, per + to, H, BS, D, s) for s in (1, 2)]
    pools = [torch.zeros((NB, H, BS, row), dtype=dtype, device=DEV) for _ in range(2)]
    for x, y in zip(pools, small):
        x[NB - per - to:] = y.view(dtype)
    g = torch.Generator(device=DEV).manual_seed(3)
    q = workloads.randn_f16((1, ql, Hq, D), g, DEV)
    w0 = torch.rand((per + to, H, BS), generator=g, device=DEV)
    big = torch.zeros((NB, H, BS), device=DEV)
    big[NB - per - to:] = w0
    near = torch.arange(per + to, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = []
    for caches, w, at in ((small, w0, near), (pools, big, near + NB - per - to)):
        bt, new = at[None, :per].contiguous(), at[None, per:].contiguous()
        ops.paged_kv_attention_weights(q, caches[0], bt, i32(n), w, 0.09, k_scale=SCALE[kind], error_word=err)
        kept, m = ops.paged_kv_token_select(w, bt, i32(n), K, 3, 20, error_word=err)
        ops.paged_kv_compact(*caches, bt, i32(n), kept, m, new, weights=w, error_word=err)
        assert ops.pkd_read_device_error(err) == 0
        got.append([kept, w[-per - to:], *(c[-per - to:].reshape(per + to, -1) for c in caches)])
    for a, b in zip(*got):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    for x in (*pools, big):
        assert not x[:NB - per - to].any()


def test_one_long_sequence():
    """One sequence of 300000 tokens: statistics of thousands of partitions, keys that do not fit, a choice among them."""
    D, BS, n, K = 64, 16, 300001, 20000
    NB = -(-n // BS)
    bt = torch.randperm(NB, generator=torch.Generator().manual_seed(1)).to(torch.int32)[None].to(DEV)
    kc = cache_of("fp16", NB, 1, BS, D, 2)
    for ql in (1, 20):
        q = workloads.randn_f16((1, ql, 2, D), torch.Generator(device=DEV).manual_seed(ql), DEV)
        w = torch.zeros((NB, 1, BS), device=DEV)
        want, most = ref.weights_after(q, kc.double(), bt, [n], w, D ** -0.5, None, 1.0, BS)
        ops.paged_kv_attention_weights(q, kc, bt, i32(n), w, D ** -0.5)
        bound = ref.weights_bound(D, 2 * ql, n, most)
        assert ((w.double() - want).abs() <= bound * want + 1e-30).all()
        kept, m = ops.paged_kv_token_select(w, bt, i32(n), K, 4, 64)
        assert torch.equal(kept.cpu(), ref.token_select(w, bt, [n], K, 4, 64, BS)[0]) and m.item() == K
