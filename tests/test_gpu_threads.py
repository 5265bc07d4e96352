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
