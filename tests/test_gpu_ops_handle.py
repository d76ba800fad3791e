"""The operators' handle from several streams and host threads (GPU)."""

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
