"""A launch that fails leaves nothing behind: the next call of the thread reports its own outcome."""
import ctypes

import pytest
import torch

from paged_kv_decode_21_gb300 import ops
from test_gpu_streams import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def step():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_21_gb300 import build
    build.build()
    ops.lib()
    return Step()


def calls(step):
    """Calls that launch in each of the library's ways, on the legacy default stream."""
    B = step.q.shape[0]
    out, qm = torch.empty_like(step.q), step.q.view(B, 1, *step.q.shape[1:])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    most = dict(max_context_len=max(step.lens.tolist()))
    ew = torch.zeros(1, dtype=torch.int32, device="cuda")
    lists, counts = torch.empty_like(step.lists), torch.empty_like(step.counts)
    dense = (step.q, step.kc, step.vc, step.bt, step.lens, 0.1)
    kw = dict(workspace=ws, error_word=ew, stream=0)
    return {
        "select": lambda: ops.paged_kv_block_select(step.q, step.bounds, step.bt, step.lens, 6, 16, block_lists=lists,
                                                    list_lens=counts, error_word=ew, stream=0, **most),
        "append": lambda: ops.paged_kv_append_rope(step.q, step.k, step.v, step.table, step.bt, step.before, step.kc2,
                                                   step.vc2, q_out=out, error_word=ew, stream=0),
        "bounds": lambda: ops.paged_kv_block_bounds(step.kc, step.bt, step.lens, step.bounds, error_word=ew, stream=0),
        "blocks": lambda: ops.paged_decode_attention_blocks(step.q, step.kc, step.vc, step.bt, step.lens, step.lists,
                                                            step.counts, 0.1, out=out, **kw),
        "prefix": lambda: ops.paged_decode_attention_prefix(step.q, step.kc, step.vc, step.ptab, step.plens, step.starts,
                                                            step.bt, step.lens, 0.1, out=out, max_prefix_len=1000, **most,
                                                            **kw),
        "no_prefetch": lambda: ops.paged_decode_attention_ex(*dense, out=out, variant="no_prefetch", **most, **kw),
        "tma_mma": lambda: ops.paged_decode_attention_ex(*dense, out=out, variant="tma_mma+longest_first", **most, **kw),
        "tcgen05": lambda: ops.paged_decode_attention_multi(qm, *dense[1:], out=out.view(qm.shape), variant="tcgen05",
                                                            **most, **kw),
        "validate": lambda: ops.paged_decode_validate_tables(step.bt, step.lens, 16, step.kc.shape[0], ew, stream=0),
    }


NAMES = ["select", "append", "bounds", "blocks", "prefix", "no_prefetch", "tma_mma", "tcgen05", "validate"]


@pytest.mark.parametrize("name", NAMES)
def test_a_refused_launch_is_not_reported_again(step, name):
    """While another stream is captured in global mode, the driver refuses a launch on the legacy stream (and ends
    the capture).  Every other call after it succeeds."""
    every = calls(step)
    for c in every.values():
        c()
    torch.cuda.synchronize()
    cuda = ctypes.CDLL("libcuda.so.1")
    for after in NAMES:
        stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
        assert cuda.cuStreamCreate(ctypes.byref(stream), 0) == 0
        assert cuda.cuStreamBeginCapture_v2(stream, 0) == 0
        try:
            with pytest.raises(ops.PagedDecodeError):
                every[name]()
        finally:
            assert cuda.cuStreamEndCapture(stream, ctypes.byref(graph)) != 0  # invalidated: no graph
            assert cuda.cuStreamDestroy_v2(stream) == 0
        every[after]()
    torch.cuda.synchronize()
