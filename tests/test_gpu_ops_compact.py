"""The operators on compact storage together (examples/fp8_expert_block.py): training from 8-bit checkpoints against the
block in plain fp32 torch, decoding with 4-bit experts against the same weights in fp32.

An e4m3 operand is off by 2^-4 / sqrt(3) = 3.6% at most in the root mean square. dW13 takes in: the forward product into
g and u (two operands, 5.1%), the checkpoint of both (5.1%), the product into dact (5.1%), the codes of the gradient and
of y, and y's second quantisation (3.6% each): 10.8% as independent errors. 0.2 bounds the relative Frobenius errors of
the gradients; the forward pass is the one without checkpoints. The 4-bit layer's only rounding is bf16's, 2^-8.
"""
import importlib.util
import os

import pytest
import torch

import __graft_entry__
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("fp8_expert_block8", os.path.join(ROOT, "examples", "fp8_expert_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(block, x, res, idx, gate_of, W13, Wd):
    """The block in fp32 with autograd, on the selection idx."""
    w = {n: v.float().detach().requires_grad_(True) for n, v in (("norm_w", block.norm_w), ("Wr", block.Wr), ("W13", W13), ("Wd", Wd))}
    xs = x.float().detach().requires_grad_(True)
    h = xs + res.float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + block.eps) * w["norm_w"]
    p = torch.sigmoid(y @ w["Wr"].t()).gather(1, idx)
    gate = block.route["route_scale"] * p / p.sum(1, keepdim=True) if gate_of is None else gate_of
    out = torch.zeros_like(h)
    for e in range(W13.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        g, u = (y[t] @ w["W13"][e].t()).chunk(2, 1)
        out = out.index_add(0, t, gate[t, j, None] * ((torch.nn.functional.silu(g) * u) @ w["Wd"][e].t()))
    return out, xs, w


def far(a, b):
    return ((a.float() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("T,d,f,E,k,groups,kept", [(300, 256, 128, 8, 2, 4, 2), (1, 512, 384, 16, 4, 1, 1),
                                                   (900, 384, 256, 4, 3, 1, 1)])
def test_training_from_checkpoints(example, T, d, f, E, k, groups, kept):
    block = example.Fp8ExpertBlock(d, f, E, k, groups, kept, seed=T, save8=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res, dout = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(3))
    h, out, ctx = block.forward(x, res)
    block.save8 = False
    h2, out2, _ = block.forward(x, res)
    block.save8 = True
    assert torch.equal(h, h2) and torch.equal(out, out2)
    assert not any(n in ctx for n in ("gu", "o", "y"))
    grads = block.backward(dout, ctx)
    again = block.backward(dout, ctx)
    assert block.ops.status() == 0
    want, xs, w = plain(block, x, res, ctx["idx"].long(), None, block.W13, block.Wd)
    want.backward(dout.float())
    for name, ref in (("dx", xs.grad), ("dnorm", w["norm_w"].grad), ("dWr", w["Wr"].grad), ("dW13", w["W13"].grad),
                      ("dWd", w["Wd"].grad)):
        assert far(grads[name], ref) < 0.2, name
        assert torch.equal(grads[name], again[name]), name


def test_a_captured_backward_beside_a_live_eager_graph(example):
    block = example.Fp8ExpertBlock(256, 128, 8, 2, seed=6, save8=True)
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


@pytest.mark.parametrize("T,d,f,E,k,group,zero", [(1, 256, 128, 8, 2, 128, False), (5, 512, 384, 16, 4, 32, True),
                                                  (16, 384, 160, 4, 3, 64, False), (40, 256, 96, 8, 8, 64, True)])
def test_decoding_with_4_bit_experts(example, T, d, f, E, k, group, zero):
    block = example.Fp8ExpertBlock(d, f, E, k, seed=T)
    block.quantise4(group, zero)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, res = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    h, out = block.decode(x, res)
    n = block.ops.rms_norm(x, block.norm_w, res, block.eps, want=("y",))["y"]
    r = block.ops.gate(n.float() @ block.Wr.t(), k, bias=block.bias, dispatch=False, **block.route)

    def dense(w):
        return torch.stack([torch.from_numpy(oo.w4_values(w["codes"][e].cpu().numpy(), w["scale"][e].double().cpu().numpy(),
                                                          w["zero"][e].double().cpu().numpy() if zero else None, group))
                            for e in range(E)]).cuda()

    W13, Wd, y, want = dense(block.w13_4), dense(block.wd_4), n.double(), torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for t in range(T):
        for e, gate in zip(r["idx"][t].tolist(), r["gate"][t].double()):
            a, u = (W13[e] @ y[t]).chunk(2)
            want[t] += gate * (Wd[e] @ (torch.nn.functional.silu(a) * u))
    assert torch.equal(h, (x.float() + res.float()).bfloat16())
    assert ((out.double() - want).norm() / want.norm()).item() < 2.0 ** -8
    assert block.ops.status() == 0
    # and not far from the bf16 weights: half a step of a fifteenth of a group's range, twice, some 5-7% each
    assert far(out, plain(block, x, res, r["idx"].long(), r["gate"], block.W13, block.Wd)[0].detach()) < 0.3


def test_tensors_that_do_not_fit_are_refused():
    """By the binding, before anything is launched: nothing runs, no status is recorded."""
    import mixture_experts_layer_routing_gb300 as moe
    ops = moe.default_ops()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    w, w3, wd = ops.quant_w4(bf(64, 96), 32), ops.quant_w4(bf(3, 64, 96), 32), ops.quant_w4(bf(3, 96, 32), 32)
    x, idx, gate = bf(4, 96), i32(4, 2), f32(4, 2)
    f = ops.swiglu(bf(4, 256), want=("q", "save"))
    before = ops.launch_count()
    E = (ValueError, TypeError, RuntimeError)
    bad = [
        lambda: ops.quant_w4(bf(64, 96), 48), lambda: ops.quant_w4(bf(64, 80), 32), lambda: ops.quant_w4(bf(60, 96), 32),
        lambda: ops.quant_w4(f32(64, 96), 32), lambda: ops.quant_w4(bf(64, 192)[:, ::2], 32), lambda: ops.quant_w4(bf(96), 32),
        lambda: ops.quant_w4(bf(64, 96), 32, out=dict(codes=i32(64, 11))),
        # weights without zero points into a dict that keeps another's
        lambda: ops.quant_w4(bf(64, 96), 32, zero=False, out=dict(zero=torch.zeros(3, 64, dtype=torch.uint8, device="cuda"))),
        lambda: ops.w4_matmul(bf(4, 64), w), lambda: ops.w4_matmul(x.float(), w), lambda: ops.w4_matmul(x.cpu(), w),
        lambda: ops.w4_matmul(x, w3), lambda: ops.w4_matmul(x, w, off=i32(2)), lambda: ops.w4_matmul(x, w3, off=i32(3)),
        lambda: ops.w4_matmul(x, dict(w, group=64)), lambda: ops.w4_matmul(x, dict(codes=w["codes"], group=32)),
        lambda: ops.w4_matmul(x, dict(w, scale=w["scale"].float())), lambda: ops.w4_matmul(x, dict(w, zero=w["scale"])),
        lambda: ops.w4_matmul(x, w, out=f32(4, 63)), lambda: ops.w4_matmul(x, w, out_dtype=torch.float16),
        lambda: ops.w4_matmul(x, w, row_index=i32(4).long()), lambda: ops.w4_matmul(bf(4, 97)[:, 1:], w),
        lambda: ops.w4_matmul(x.t().contiguous().t(), w),
        lambda: ops.w4_experts(x, idx, gate, w3, w3), lambda: ops.w4_experts(x, idx.long(), gate, w3, wd),
        lambda: ops.w4_experts(x, idx, gate[:, :1], w3, wd), lambda: ops.w4_experts(x, idx, gate, w3, wd, n_shared=3),
        lambda: ops.w4_experts(x, idx, gate, w3, wd, n_shared=-1), lambda: ops.w4_experts(x, idx[0], gate, w3, wd),
        lambda: ops.w4_experts(bf(65, 96), i32(65, 2), f32(65, 2), w3, wd),
        lambda: ops.w4_experts(x, i32(4, 0), f32(4, 0), w3, wd), lambda: ops.w4_experts(x, idx, gate, w3, wd, out=bf(4, 95)),
        lambda: ops.swiglu(bf(4, 255)), lambda: ops.swiglu(bf(4, 24)), lambda: ops.swiglu(f32(4, 256)),
        lambda: ops.swiglu(bf(4, 256), out=dict(other=None)), lambda: ops.swiglu(bf(4, 256), out={}),
        lambda: ops.swiglu(bf(4, 256), out=dict(q=None)), lambda: ops.swiglu(bf(4, 256), out=dict(act=f32(4, 128))),
        lambda: ops.swiglu_backward(bf(4, 120), f["save"], f["save_scale"]),
        lambda: ops.swiglu_backward(bf(4, 128), f["save"], f["save_scale"][:, :1].contiguous()),
        lambda: ops.swiglu_backward(bf(4, 128), f["save"], f["save_scale"], gate=f32(3)),
        lambda: ops.swiglu_backward(bf(4, 128), f["save"], f["save_scale"], want=("x",)),
        lambda: ops.swiglu_backward(bf(4, 128), f["save"], f["save_scale"], out=dict(actt=None, actt_scale=None)),
        lambda: ops.swiglu_backward(bf(4, 136), torch.zeros(4, 272, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                                    f32(4, 4), want=("dq",)),
        lambda: ops.requant_cols(f["q"], f["scale"].double()), lambda: ops.requant_cols(f["q"].view(torch.uint8), f["scale"]),
        lambda: ops.requant_cols(f["q"], f["scale"], row_index=i32(4, 1)), lambda: ops.requant_cols(f["q"].t(), f["scale"]),
        lambda: ops.requant_cols(f["q"], f["scale"], out=dict(q=f["q"])),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(E):
            call()
            raise AssertionError(i)
    assert ops.launch_count() == before and ops.status() == 0


def test_backward_follows_the_forward_pass(example):
    """What a forward pass kept decides how its backward pass goes, whatever the block was switched to in between."""
    block = example.Fp8ExpertBlock(256, 128, 8, 2, seed=8, save8=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    x, res, dout = (torch.randn(70, 256, generator=g, device="cuda").bfloat16() for _ in range(3))
    ctx8 = block.forward(x, res)[2]
    want8 = block.backward(dout, ctx8)
    block.save8 = False
    ctx = block.forward(x, res)[2]
    want = block.backward(dout, ctx)
    got8 = block.backward(dout, ctx8)
    block.save8 = True
    got = block.backward(dout, ctx)
    for n in want:
        assert torch.equal(got[n], want[n]) and torch.equal(got8[n], want8[n]), n
