"""A query that is not a number gives a result that is not one, however the context is split, and leaves the other
rows as they are."""
import math

import pytest
import torch

import longcache_ref as ref
from serving_ref import attention_bound, deal_tables
from test_gpu_int4 import attention
from paged_kv_decode_21_gb300 import ops, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("Hq,H,ql", [(4, 4, 1), (8, 2, 1), (8, 2, 3), (16, 2, 4)])
@pytest.mark.parametrize("part", [0, -1, 64])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_queries_that_are_not_finite(Hq, H, ql, part, what):
    D, BS, lens = 128, 16, [300, 40, 0, 33]
    bt, _ = deal_tables(lens, BS, 19, 30, 2)
    kc, vc = (ref.random_int4((30, H, BS), D, s) for s in (1, 2))
    q = workloads.randn_f16((4, ql, Hq, D), torch.Generator(device=DEV).manual_seed(1), DEV)
    want, mag = attention(q, ref.int4_values(kc, D, 0.1), ref.int4_values(vc, D, 0.1), bt, lens, 0.09, BS)
    bad = [(0, 0, 1), (1, ql - 1, Hq - 1), (2, 0, 0)]
    for b, j, h in bad:
        q[b, j, h, 7] = what
    out = ops.paged_decode_attention_int4(q if ql > 1 else q[:, 0].contiguous(), kc, vc, bt,
                                          torch.tensor(lens, dtype=torch.int32, device=DEV), 0.09, 0.1, 0.1,
                                          partition_size=part).view(q.shape).double()
    for b, j, h in bad[:2]:
        assert out[b, j, h].isnan().all()
    assert (out[2] == 0).all()                      # no token: no weight, and nothing of the query
    clean = torch.ones(q.shape[:3], dtype=torch.bool, device=DEV)
    for at in bad:
        clean[at] = False
    bound = attention_bound(want, mag, 300, float(ref.int4_values(vc, D, 0.1).abs().max()))
    assert ((out - want).abs() <= bound)[clean].all()
