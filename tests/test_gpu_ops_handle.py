"""The operators' handle from several streams and host threads (GPU)."""
import ctypes
import threading

import pytest
import torch

import __graft_entry__

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    __graft_entry__.build()
    import mixture_experts_layer_routing_gb300 as moe
    return moe.MoeOps()


def test_no_error_is_lost_between_reading_and_clearing(ops):
    """A bad index that another stream's kernel records while the status is read comes out of that reading or the next."""
    import mixture_experts_layer_routing_gb300 as moe
    logits, bad = torch.zeros(1, 8, device="cuda"), torch.full((1, 1), 9, dtype=torch.int32, device="cuda")
    dgate, out = torch.ones(1, 1, device="cuda"), dict(dlogits=torch.empty(1, 8, device="cuda"))
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    lost = 0
    for i in range(3000):
        with torch.cuda.stream(two):
            torch.cuda._sleep(20000 + 97 * (i % 200))     # (the record meets the reading at another place each time)
            ops.gate_backward(logits, bad, dgate, out=out)
        seen = [ops.status(one) for _ in range(4)]
        two.synchronize()
        seen.append(ops.status(one))
        assert set(seen) <= {0, moe.MOE_ERR_DEVICE_INDEX}
        lost += not any(seen)
    assert lost == 0


def test_launches_of_several_host_threads_are_all_counted(ops):
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    threads, calls = 4, 20000
    y = [torch.empty_like(x) for _ in range(threads)]
    streams = [torch.cuda.Stream() for _ in range(threads)]
    torch.cuda.synchronize()
    f, before = ops._lib.moe_norm_forward, ops.launch_count()
    bad = []
    def work(i):
        arg = (ops.h, 0, x.data_ptr(), 64, None, 0, w.data_ptr(), 4, 64, 1e-6, None, y[i].data_ptr(), None, None, None,
               ctypes.c_void_p(streams[i].cuda_stream))
        bad.extend(s for s in (f(*arg) for _ in range(calls)) if s)       # (a ctypes call lets other threads run)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(threads)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    assert not bad
    assert ops.launch_count() - before == threads * calls
