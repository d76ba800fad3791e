"""The operators together (examples/fp8_expert_block.py): an expert block forward and backward against the same block
in plain fp32 torch without 8-bit operands.

Each e4m3 operand is off by up to 2^-4 of a value, uniformly over a step: 2^-4 / sqrt(3) = 3.6% at most in the root
mean square, 5.1% a product of two. Forward passes through two products (the second one's input carries the first's
error), the weights' gradients through up to four: 0.1 and 0.15 bound their relative Frobenius errors.
"""
import importlib.util
import os

import pytest
import torch

import __graft_entry__

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("fp8_expert_block", os.path.join(ROOT, "examples", "fp8_expert_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(block, x, res, idx, E):
    """The block in fp32 with autograd, on the selection idx."""
    w = {n: getattr(block, n).float().detach().requires_grad_(True) for n in ("norm_w", "Wr", "W13", "Wd")}
    xs = x.float().detach().requires_grad_(True)
    h = xs + res.float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + block.eps) * w["norm_w"]
    p = torch.sigmoid(y @ w["Wr"].t()).gather(1, idx)
    gate = block.route["route_scale"] * p / p.sum(1, keepdim=True)
    out = torch.zeros_like(h)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        g, u = (y[t] @ w["W13"][e].t()).chunk(2, 1)
        out = out.index_add(0, t, gate[t, j, None] * ((torch.nn.functional.silu(g) * u) @ w["Wd"][e].t()))
    return out, xs, w


def far(a, b):
    return ((a.float() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("T,d,f,E,k,groups,kept", [(300, 256, 128, 8, 2, 4, 2), (1, 512, 384, 16, 4, 1, 1),
                                                   (900, 384, 272, 4, 3, 1, 1)])
def test_block_forward_and_backward(example, T, d, f, E, k, groups, kept):
    block = example.Fp8ExpertBlock(d, f, E, k, groups, kept, seed=T)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res, dout = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(3))
    h, out, ctx = block.forward(x, res)
    assert torch.equal(h, (x.float() + res.float()).bfloat16())
    grads = block.backward(dout, ctx)
    assert block.ops.status() == 0
    want, xs, w = plain(block, x, res, ctx["idx"].long(), E)
    want.backward(dout.float())
    assert far(out, want.detach()) < 0.1
    for name, ref in (("dx", xs.grad), ("dnorm", w["norm_w"].grad), ("dWr", w["Wr"].grad), ("dW13", w["W13"].grad),
                      ("dWd", w["Wd"].grad)):
        assert far(grads[name], ref) < 0.15, name


def test_a_width_that_is_no_multiple_of_16_is_refused(example):
    """The down product reduces over f = 264 values, and a row of codes has to be a multiple of 16 bytes."""
    import mixture_experts_layer_routing_gb300 as moe
    block = example.Fp8ExpertBlock(384, 264, 4, 3, seed=900)
    x = torch.randn(900, 384, device="cuda").bfloat16()
    with pytest.raises(moe.MoeError) as e:
        block.forward(x, x)
    assert e.value.code == moe.MOE_ERR_UNSUPPORTED


def test_repeats_are_identical(example):
    block = example.Fp8ExpertBlock(256, 128, 8, 2, seed=5)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, res, dout = (torch.randn(500, 256, generator=g, device="cuda").bfloat16() for _ in range(3))
    a, b = block.forward(x, res), block.forward(x, res)
    assert torch.equal(a[1], b[1])
    ga, gb = block.backward(dout, a[2]), block.backward(dout, b[2])
    for n in ga:
        assert torch.equal(ga[n], gb[n]), n


def test_a_captured_backward_beside_a_live_eager_graph(example):
    """The operators in a graph while an eager autograd graph of the same inputs lives."""
    block = example.Fp8ExpertBlock(256, 128, 8, 2, seed=6)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, res, dout = (torch.randn(200, 256, generator=g, device="cuda").bfloat16() for _ in range(3))
    live = (x.float().requires_grad_(True) * 2).sum()
    eager = block.backward(dout, block.forward(x, res)[2])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block.backward(dout, block.forward(x, res)[2])
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = block.backward(dout, block.forward(x, res)[2])
    graph.replay()
    torch.cuda.synchronize()
    live.backward()
    for n in eager:
        assert torch.equal(eager[n], captured[n]), n
