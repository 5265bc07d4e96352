"""Calls from two host threads at once, each on a stream of its own, give what each gives alone."""
import threading

import pytest
import torch

from paged_kv_decode_21_gb300 import ops, workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_21_gb300 import build
    build.build()
    ops.lib()


def in_threads(bodies):
    """Run every body in a thread of its own, started together; the errors they raised."""
    ready, errors = threading.Barrier(len(bodies)), []

    def go(body):
        try:
            ready.wait(60)
            body()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=go, args=(b,)) for b in bodies]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


@pytest.mark.parametrize("fp8", [False, True])
def test_choices_over_long_and_short_contexts(fp8):
    """One thread chooses among 12500 blocks (their scores take 52 KB of shared memory), two others among 32, in
    the same kernel: no call may depend on what another asks for meanwhile."""
    Hq, Hkv, D, BS, K, calls = 8, 2, 128, 16, 12, 20000
    pool = 4096
    g = torch.Generator(device="cuda").manual_seed(41)
    b = workloads.randn_f16((pool, Hkv, 2, D), g, "cuda")
    bounds = torch.stack((torch.minimum(b[:, :, 0], b[:, :, 1]), torch.maximum(b[:, :, 0], b[:, :, 1])), 2).contiguous()
    if fp8:
        bounds = bounds.to(torch.float8_e4m3fn).view(torch.uint8)
    select, jobs, statuses = ops.lib().paged_kv_block_select, [], []
    for n in (200_000, 500, 500):
        q = workloads.randn_f16((1, Hq, D), g, "cuda")
        bt = (torch.arange(-(-n // BS), device="cuda") * 7 % pool)[None].int().contiguous()
        cl = torch.tensor([n], dtype=torch.int32, device="cuda")
        want = ops.paged_kv_block_select(q, bounds, bt, cl, K, BS, max_context_len=n)
        lists, lens = torch.empty_like(want[0]), torch.empty_like(want[1])
        ew, stream = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
        args = (q.data_ptr(), bounds.data_ptr(), bt.data_ptr(), cl.data_ptr(), lists.data_ptr(), lens.data_ptr(), 1, Hq,
                Hkv, D, BS, pool, bt.shape[1], n, K, 1, 1, int(fp8), ew.data_ptr(), stream.cuda_stream)
        jobs.append((args, want, lists, lens, ew, q, bt, cl, stream))
    torch.cuda.synchronize()

    def body(args):
        torch.cuda.set_device(0)
        statuses.append([select(*args) for _ in range(calls)])

    errors = in_threads([lambda a=j[0]: body(a) for j in jobs])
    torch.cuda.synchronize()
    assert not errors, errors[0]
    assert len(statuses) == 3 and not any(map(any, statuses)), [sum(map(bool, s)) for s in statuses]
    for _, want, lists, lens, ew, *_ in jobs:
        assert ops.pkd_read_device_error(ew) == 0
        assert torch.equal(lists, want[0]) and torch.equal(lens, want[1])


def test_every_call_at_once():
    """Three threads, each with streams, caches, outputs and workspaces of its own, run the whole step (append,
    bounds, choice, listed decode, shared prefix on both kernels, dense decode) over and over beside the others."""
    from test_gpu_prefix import problem

    class Work:
        def __init__(self, seed, B, Hq, q_len, plen, fp8):
            self.fp8, self.B, self.q_len = fp8, B, q_len
            lens = [q_len + (i * 37 + seed) % 300 for i in range(B)]
            self.p = problem([B], [plen], lens, q_len, Hq, 4, 128, 16, seed, fp8)
            q, kc, vc, ptab, plens, starts, bt, cl = self.p
            self.q1 = q[:, 0].contiguous()
            g = torch.Generator(device="cuda").manual_seed(seed)
            self.k, self.v = (workloads.randn_f16((B, 4, 128), g, "cuda") for _ in range(2))
            self.table = workloads.randn_f16((max(lens), 128), g, "cuda").float()
            self.before = (cl - 1).contiguous()
            self.k2, self.v2 = torch.zeros_like(kc), torch.zeros_like(vc)
            self.bounds = torch.zeros((kc.shape[0], 4, 2, 128), dtype=kc.dtype, device="cuda")
            self.most = dict(max_context_len=max(lens))
            self.plen, self.stream = plen, torch.cuda.Stream()
            self.ew = torch.zeros(1, dtype=torch.int32, device="cuda")
            nbytes = max(ops.paged_decode_prefix_workspace_size(B, q_len, Hq, 4, 128, 16, 1, plen, max(lens)),
                         ops.paged_decode_blocks_workspace_size(B, Hq, 4, 128, 16, 6),
                         ops.paged_decode_multi_workspace_size(B, 1, Hq, 4, 128, 16, max(lens)))
            self.kw = dict(workspace=ops.alloc_workspace(nbytes, "cuda"), error_word=self.ew)
            self.outs = [torch.empty_like(self.q1), torch.empty_like(self.q1), torch.empty_like(self.q1),
                         torch.empty_like(q), torch.empty((B, 4, 6), dtype=torch.int32, device="cuda"),
                         torch.empty((B, 4), dtype=torch.int32, device="cuda")]

        def step(self):
            q, kc, vc, ptab, plens, starts, bt, cl = self.p
            s = (1 / 64, 1 / 64) if self.fp8 else ()
            rot, o1, o2, o3, lists, counts = self.outs
            f = (lambda name: getattr(ops, name + "_fp8")) if self.fp8 else (lambda name: getattr(ops, name))
            f("paged_kv_append_rope")(self.q1, self.k, self.v, self.table, bt, self.before, self.k2, self.v2, *s,
                                      q_out=rot, error_word=self.ew)
            ops.paged_kv_block_bounds(kc, bt, cl, self.bounds, error_word=self.ew)
            ops.paged_kv_block_select(self.q1, self.bounds, bt, cl, 6, 16, block_lists=lists, list_lens=counts,
                                      error_word=self.ew, **self.most)
            f("paged_decode_attention_blocks")(self.q1, kc, vc, bt, cl, lists, counts, 0.09, *s, out=o1, **self.kw)
            if self.fp8:
                ops.paged_decode_attention_fp8(self.q1, kc, vc, bt, cl, 0.09, *s, out=o2, **self.most, **self.kw)
            else:
                ops.paged_decode_attention_ex(self.q1, kc, vc, bt, cl, 0.09, out=o2, **self.most, **self.kw)
            f("paged_decode_attention_prefix")(q, kc, vc, ptab, plens, starts, bt, cl, 0.09, *s, out=o3,
                                               max_prefix_len=self.plen, **self.most, **self.kw)

        def state(self):
            return [x.clone() for x in self.outs + [self.k2, self.v2, self.bounds]]

    works = [Work(81, 90, 28, 1, 3000, False), Work(82, 30, 32, 4, 2000, True), Work(83, 4, 16, 1, 500, False)]
    want = []
    for w in works:
        w.step()
        torch.cuda.synchronize()
        want.append(w.state())

    def body(w):
        torch.cuda.set_device(0)
        with torch.cuda.stream(w.stream):
            for _ in range(150):
                w.step()

    for _ in range(3):
        errors = in_threads([lambda w=w: body(w) for w in works])
        torch.cuda.synchronize()
        assert not errors, errors[0]
        for w, ref in zip(works, want):
            assert ops.pkd_read_device_error(w.ew) == 0
            for got, x in zip(w.state(), ref):
                assert torch.equal(got.view(torch.uint8), x.view(torch.uint8))
