"""Calls around long caches from three host threads at once, each on a stream of its own, give what each gives alone."""
import pytest
import torch

from serving_ref import deal_tables
from test_gpu_evict import cache_of, i32
from test_gpu_threads import in_threads
from paged_kv_decode_21_gb300 import ops, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Work:
    """One sequence batch with caches, outputs and workspaces of its own: append, decode, weights, choice, compaction
    and read-back, over and over."""

    def __init__(self, seed, kind, lens, ql, Hq, H, K):
        self.kind, self.D, BS, self.K = kind, 128, 16, K
        g = torch.Generator(device=DEV).manual_seed(seed)
        per = -(-K // BS) + 1
        need = sum(-(-n // BS) for n in lens)
        NB, B = need + per * len(lens), len(lens)
        self.bt, rest = deal_tables(lens, BS, -(-max(lens) // BS), NB, seed)
        self.new = rest[:per * B].view(B, per).to(DEV).contiguous()
        self.caches = [cache_of(kind, NB, H, BS, self.D, seed + i) for i in (1, 2)]
        self.first = [c.clone() for c in self.caches]
        self.q = workloads.randn_f16((B, ql, Hq, self.D), g, DEV)
        self.cl, self.most = i32(*lens), max(lens)
        self.k, self.v = (workloads.randn_f16((B, H, self.D), g, DEV) for _ in range(2))
        self.table = workloads.randn_f16((self.most + 1, self.D), g, DEV).float()
        self.pos = torch.randint(0, self.most, (2, B), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
        self.axes = (torch.arange(self.D // 2, device=DEV) % 2).to(torch.int32)
        self.w0 = torch.rand((NB, H, BS), generator=g, device=DEV)
        self.w, self.ew = self.w0.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
        self.kept = torch.zeros((B, H, K), dtype=torch.int32, device=DEV)
        self.n = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.out = torch.zeros_like(self.q)
        self.rows = [torch.zeros((B, H, self.D), dtype=torch.float16, device=DEV) for _ in range(2)]
        size = ops.paged_kv_attention_weights_workspace_size(B, ql, Hq, H, self.D, BS, self.most)
        if kind == "int4":
            size = max(size, ops.paged_decode_int4_workspace_size(B, ql, Hq, H, self.D, BS, self.most))
        self.ws = ops.alloc_workspace(size, DEV)
        self.stream = torch.cuda.Stream()

    def step(self):
        for x, y in zip([*self.caches, self.w], [*self.first, self.w0]):
            x.copy_(y)
        kc, vc = self.caches
        last = self.cl - 1
        kw = dict(error_word=self.ew)
        if self.kind == "int4":
            ops.paged_kv_append_rope_int4(None, self.k, self.v, self.table, self.bt, last, kc, vc, 0.1, 0.1,
                                          positions=self.pos, pair_axes=self.axes, **kw)
            ops.paged_decode_attention_int4(self.q, kc, vc, self.bt, self.cl, 0.09, 0.1, 0.1, out=self.out,
                                            max_context_len=self.most, workspace=self.ws, **kw)
            ops.paged_kv_read_int4(kc, vc, self.bt, last, 0.1, 0.1, *self.rows, **kw)
        elif self.kind == "e4m3":
            ops.paged_kv_append_rope_axes_fp8(None, self.k, self.v, self.table, self.axes, self.pos, self.bt, last, kc, vc,
                                              0.1, 0.1, **kw)
        else:
            ops.paged_kv_append_rope_axes(None, self.k, self.v, self.table, self.axes, self.pos, self.bt, last, kc, vc, **kw)
        ops.paged_kv_attention_weights(self.q, kc, self.bt, self.cl, self.w, 0.09, k_scale=0.1, max_context_len=self.most,
                                       workspace=self.ws, **kw)
        ops.paged_kv_token_select(self.w, self.bt, self.cl, self.K, 2, 8, max_context_len=self.most, kept=self.kept,
                                  kept_lens=self.n, **kw)
        ops.paged_kv_compact(kc, vc, self.bt, self.cl, self.kept, self.n, self.new, weights=self.w, **kw)

    def state(self):
        return [x.clone() for x in [*self.caches, self.w, self.kept, self.n, self.out, *self.rows]]


def test_every_call_at_once():
    """Splits and orders of their own, choices with much and little shared memory, all three kinds of cache."""
    works = [Work(91, "int4", [40 + i * 97 % 1500 for i in range(160)], 1, 32, 8, 64),
             Work(92, "int4", [9000, 40, 3000], 3, 8, 1, 500),
             Work(93, "e4m3", [20000, 700], 1, 8, 2, 3000),
             Work(94, "fp16", [100 + 7 * i for i in range(40)], 9, 14, 2, 90)]
    want = []
    for w in works:
        w.step()
        torch.cuda.synchronize()
        assert ops.pkd_read_device_error(w.ew) == 0
        want.append(w.state())

    def body(w):
        torch.cuda.set_device(0)
        with torch.cuda.stream(w.stream):
            for _ in range(100):
                w.step()

    for _ in range(3):
        errors = in_threads([lambda w=w: body(w) for w in works])
        torch.cuda.synchronize()
        assert not errors, errors[0]
        for w, r in zip(works, want):
            assert ops.pkd_read_device_error(w.ew) == 0
            for got, x in zip(w.state(), r):
                assert torch.equal(got.view(torch.uint8), x.view(torch.uint8))
