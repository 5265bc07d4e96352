"""Calls on a given stream (stream=...): the buffers that the binding makes for them, and the lengths that
it reads for them, keep to that stream's order."""
import pytest
import torch

from paged_kv_decode_21_gb300 import ops, workloads
from serving_ref import deal_tables, make_cache

pytestmark = pytest.mark.gpu

Hq, Hkv, D, BS = 28, 4, 128, 16
LENS = [200 + 3 * i for i in range(40)]
PREFIX = 1000
SLEEP = 200_000_000  # cycles: 0.1 s


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_21_gb300 import build
    build.build()
    ops.lib()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Step:
    """The inputs of every call, and the calls by name, all returning their new tensors."""

    def __init__(self):
        B = len(LENS)
        pool = sum(-(-n // BS) for n in LENS) + -(-PREFIX // BS) + 2
        self.bt, rest = deal_tables(LENS, BS, -(-max(LENS) // BS), pool, 51)
        self.ptab = rest[:-(-PREFIX // BS)][None].cuda().contiguous()
        self.kc, self.vc = make_cache((pool, Hkv, BS, D), 52, False), make_cache((pool, Hkv, BS, D), 53, False)
        g = torch.Generator(device="cuda").manual_seed(54)
        self.q = workloads.randn_f16((B, Hq, D), g, "cuda")
        self.k, self.v = (workloads.randn_f16((B, Hkv, D), g, "cuda") for _ in range(2))
        self.lens, self.plens, self.starts = i32(LENS), i32([PREFIX]), i32([0, B])
        self.table = workloads.randn_f16((max(LENS) + 1, D), g, "cuda").float()
        self.bounds = torch.zeros((pool, Hkv, 2, D), dtype=torch.float16, device="cuda")
        ops.paged_kv_block_bounds(self.kc, self.bt, self.lens, self.bounds)
        self.lists, self.counts = ops.paged_kv_block_select(self.q, self.bounds, self.bt, self.lens, 6, BS)
        self.before = self.lens - 1
        self.kc2, self.vc2 = torch.zeros_like(self.kc), torch.zeros_like(self.vc)
        self.most = dict(max_context_len=max(LENS))

    def append(self, q=None, **kw):
        return (ops.paged_kv_append_rope(self.q if q is None else q, self.k, self.v, self.table, self.bt, self.before,
                                         self.kc2, self.vc2, **kw),)

    def prefix(self, q=None, lens=None, plens=None, **kw):
        return (ops.paged_decode_attention_prefix(self.q if q is None else q, self.kc, self.vc, self.ptab,
                                                  self.plens if plens is None else plens, self.starts, self.bt,
                                                  self.lens if lens is None else lens, 0.1, **kw),)

    def select(self, q=None, lens=None, **kw):
        return ops.paged_kv_block_select(self.q if q is None else q, self.bounds, self.bt,
                                         self.lens if lens is None else lens, 6, BS, **kw)

    def blocks(self, q=None, **kw):
        return (ops.paged_decode_attention_blocks(self.q if q is None else q, self.kc, self.vc, self.bt, self.lens,
                                                  self.lists, self.counts, 0.1, **kw),)

    def known(self, name):
        """The host's bounds, so that the call reads no length itself."""
        return {"prefix": dict(max_prefix_len=PREFIX, **self.most), "select": self.most}.get(name, {})


@pytest.fixture(scope="module")
def step(_built):
    return Step()


def given(which, stream):
    return stream if which == "torch" else stream.cuda_stream


def alone(step, name, **kw):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kw.update(step.known(name))
    out = getattr(step, name)(stream=side, **kw)
    torch.cuda.synchronize()
    return [x.clone() for x in out]


CALLS = ["append", "prefix", "select", "blocks"]


@pytest.mark.parametrize("which", ["torch", "raw"])
@pytest.mark.parametrize("name", CALLS)
def test_buffers_of_a_call_are_not_memory_that_pending_work_uses(step, name, which, monkeypatch):
    """Work still pending on the current stream reads and then writes tensors that were freed behind it.  A call
    on another stream must get other memory: it would overwrite what is to be read, or be overwritten."""
    want = alone(step, name)
    sizes, alloc = [x.numel() * x.element_size() for x in want], ops.alloc_workspace

    def noted(n, dev):
        sizes.append(n + 256)
        return alloc(n, dev)

    with monkeypatch.context() as m:
        m.setattr(ops, "alloc_workspace", noted)
        alone(step, name)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes if n > 256 for _ in range(2)]
    kept = [torch.empty_like(x) for x in held]
    with torch.cuda.stream(side):  # memory of its own that a call may take without waiting for any
        spare = [torch.empty_like(x) for x in held]
    del spare
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    for x, y in zip(held, kept):
        y.copy_(x)
        x.fill_(9)
    del held, x, y
    out = getattr(step, name)(stream=given(which, side), **step.known(name))
    side.synchronize()
    busy = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert busy, "the current stream was to be still at work"
    for x, w in zip(out, want):
        assert torch.equal(x, w)
    for y in kept:
        assert (y == 7).all()


@pytest.mark.parametrize("which", ["torch", "raw"])
@pytest.mark.parametrize("name", CALLS)
def test_results_freed_on_the_current_stream_are_not_reused_too_soon(step, name, which):
    """A result is freed while work on the current stream, behind the call's, has yet to read it; the next call
    on the given stream must not write into its memory."""
    want = alone(step, name)
    q2 = step.q.flip(0).contiguous()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    out = list(getattr(step, name)(stream=given(which, side), **step.known(name)))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    kept = [x.clone() for x in out]
    del out
    later = [getattr(step, name)(q=q2, stream=given(which, side), **step.known(name)) for _ in range(3)]
    side.synchronize()
    busy = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert busy, "the current stream was to be still at work"
    assert len(later) == 3
    for x, w in zip(kept, want):
        assert torch.equal(x, w)


@pytest.mark.parametrize("which", ["torch", "raw"])
@pytest.mark.parametrize("name", ["prefix", "select"])
def test_lengths_are_read_in_the_order_of_the_given_stream(step, name, which):
    """Lengths that the given stream has yet to write: the call that reads their maximum waits for them."""
    want = alone(step, name)
    side = torch.cuda.Stream()
    late = {"lens": torch.zeros_like(step.lens)}
    if name == "prefix":
        late["plens"] = torch.zeros_like(step.plens)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
        late["lens"].copy_(step.lens)
        if name == "prefix":
            late["plens"].copy_(step.plens)
    out = getattr(step, name)(stream=given(which, side), **late)
    torch.cuda.synchronize()
    for x, w in zip(out, want):
        assert torch.equal(x, w)


@pytest.mark.parametrize("which", ["torch", "raw"])
@pytest.mark.parametrize("name", CALLS)
def test_capture_of_a_call_that_makes_its_buffers(step, name, which):
    """A call captured on the stream it is given, its results and workspace from the graph's own memory."""
    want = alone(step, name)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = getattr(step, name)(stream=given(which, side), **step.known(name))
    for _ in range(2):
        for x in out:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, w in zip(out, want):
            assert torch.equal(x, w)
