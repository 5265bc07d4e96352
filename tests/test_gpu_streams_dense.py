"""The dense decode calls on a given stream (stream=...), as test_gpu_streams has it for the serving-step calls."""
import pytest
import torch

import test_gpu_streams as streams
from paged_kv_decode_21_gb300 import ops

pytestmark = pytest.mark.gpu


class Dense(streams.Step):
    def __init__(self):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(58)
        self.k8, self.v8 = (torch.randint(0, 127, self.kc.shape, generator=g, device="cuda", dtype=torch.uint8)
                            for _ in range(2))

    def args(self, q, lens, kc=None, vc=None):
        return (self.q if q is None else q, self.kc if kc is None else kc, self.vc if vc is None else vc, self.bt,
                self.lens if lens is None else lens, 0.1)

    def plain(self, q=None, lens=None, **kw):
        return (ops.paged_decode_attention(*self.args(q, lens), **kw),)

    def ex(self, q=None, lens=None, **kw):
        return (ops.paged_decode_attention_ex(*self.args(q, lens), partition_size=64, **kw),)

    def multi(self, q=None, lens=None, **kw):
        a = self.args(q, lens)
        return (ops.paged_decode_attention_multi(a[0].unsqueeze(1), *a[1:], partition_size=64, **kw),)

    def fp8(self, q=None, lens=None, **kw):
        return (ops.paged_decode_attention_fp8(*self.args(q, lens, self.k8, self.v8), 1 / 64, 1 / 64,
                                               partition_size=64, **kw),)

    def scratch(self, q=None, lens=None, **kw):
        return (ops.paged_decode_attention_static_scratch(*self.args(q, lens), partition_size=64, **kw),)

    def known(self, name):
        return self.most


@pytest.fixture(scope="module")
def step():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_21_gb300 import build
    build.build()
    ops.lib()
    return Dense()


CALLS = ["plain", "ex", "multi", "fp8", "scratch"]


@pytest.mark.parametrize("which", ["torch", "raw"])
@pytest.mark.parametrize("name", CALLS)
def test_buffers(step, name, which, monkeypatch):
    streams.test_buffers_of_a_call_are_not_memory_that_pending_work_uses(step, name, which, monkeypatch)


@pytest.mark.parametrize("which", ["torch", "raw"])
@pytest.mark.parametrize("name", CALLS)
def test_results(step, name, which):
    streams.test_results_freed_on_the_current_stream_are_not_reused_too_soon(step, name, which)


@pytest.mark.parametrize("which", ["torch", "raw"])
@pytest.mark.parametrize("name", CALLS)
def test_lengths(step, name, which):
    streams.test_lengths_are_read_in_the_order_of_the_given_stream(step, name, which)


@pytest.mark.parametrize("which", ["torch", "raw"])
@pytest.mark.parametrize("name", ["ex", "multi", "fp8"])
def test_workspaces_are_kept_for_the_given_stream(step, name, which, monkeypatch):
    """The workspace of a call that the given stream has yet to run is not handed out on the current one."""
    want = streams.alone(step, name)
    spaces, alloc = [], ops.alloc_workspace

    def noted(n, dev):
        t = alloc(n, dev)
        spaces.append((t.data_ptr(), n))
        return t

    monkeypatch.setattr(ops, "alloc_workspace", noted)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(streams.SLEEP)
    out = getattr(step, name)(stream=streams.given(which, side), **step.most)
    at, n = spaces[0]
    later = [torch.empty(n + 256, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(x.data_ptr() + x.numel() <= at or at + n <= x.data_ptr() for x in later)
    side.synchronize()
    for x, w in zip(out, want):
        assert torch.equal(x, w)


@pytest.mark.parametrize("which", ["torch", "raw"])
@pytest.mark.parametrize("name", CALLS)
def test_capture(step, name, which):
    streams.test_capture_of_a_call_that_makes_its_buffers(step, name, which)
