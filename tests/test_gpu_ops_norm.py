"""RMS norm operators against the 64-bit restatement (GPU).

Tolerances: a stored bf16 value is off by at most 2^-8 of itself, fp32 by 2^-24, e4m3 by 2^-4 (or half its smallest
step, 2^-10 scales). The fp32 sum of d <= 16384 squares goes through at most 45 additions in a row (32 in a thread,
then trees), its square root halves that error, and three products follow: under 2^-18.
"""
import numpy as np
import pytest
import torch

import __graft_entry__
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
SUMS = 2.0 ** -18


@pytest.fixture(scope="module")
def ops():
    __graft_entry__.build()
    import mixture_experts_layer_routing_gb300 as moe
    return moe.default_ops()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(T, d, dtype, seed=0, residual=True):
    g = torch.Generator().manual_seed(seed)
    chan = 1 + 20 * (torch.rand(d, generator=g) < 0.05).float()
    x = (torch.randn(T, d, generator=g) * chan).to(DT[dtype]).cuda()
    r = (3 * torch.randn(T, d, generator=g)).to(DT[dtype]).cuda() if residual else None
    w = (1 + 0.1 * torch.randn(d, generator=g)).to(DT[dtype]).cuda()
    return x, r, w


def check_forward(out, x, res, w, eps, dtype):
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    if "h" in out:
        assert torch.equal(out["h"], h)
    y, rstd = oo.rms_norm(f64(h), f64(w), eps)
    if "rstd" in out:
        assert np.all(np.abs(f64(out["rstd"]) - rstd) <= SUMS * rstd)
    if "y" in out:
        assert np.all(np.abs(f64(out["y"]) - y) <= (HALF[dtype] + 2 * SUMS) * np.abs(y))
    if "q" in out:
        s = f64(out["scale"])
        want = np.stack([np.abs(y[:, b:b + 128]).max(1) / 448 for b in range(0, y.shape[1], 128)], 1)
        assert np.all(np.abs(s - want) <= 2 * SUMS * want)
        wide = np.repeat(s, 128, 1)[:, :y.shape[1]]
        got = f64(out["q"].float()) * wide
        assert np.all(np.abs(got - y) <= (2.0 ** -4 + 4 * SUMS) * np.abs(y) + 2.0 ** -10 * wide)
        # and the codes are the nearest ones: dividing the kernel's own y would allow no other, up to its error
        assert np.mean(f64(out["q"].float()) != oo.quantise(y, 1)[0]) < 1e-3


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 64), (2, 136), (1, 7168), (5, 1408), (300, 256), (700, 2048), (2, 16384),
                                 (333, 7168), (1, 16384)])
def test_forward(ops, T, d, dtype):
    x, r, w = make(T, d, dtype, T + d)
    out = ops.rms_norm(x, w, r, want=("h", "y", "q", "rstd"))
    check_forward(out, x, r, w, 1e-6, dtype)
    assert ops.status() == 0


@pytest.mark.parametrize("want", [("h",), ("y",), ("q",), ("rstd",), ("y", "rstd")])
def test_any_output_alone_is_the_same(ops, want):
    x, r, w = make(37, 1000, "bf16", 3)
    every = ops.rms_norm(x, w, r, want=("h", "y", "q", "rstd"))
    some = ops.rms_norm(x, w, r, want=want)
    for name, t in some.items():
        assert torch.equal(t.float(), every[name].float()), name


def test_strided_rows_and_no_residual(ops):
    x, r, w = make(20, 512, "bf16", 5)
    wide = torch.full((20, 700 - 700 % 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:520] = x
    out = ops.rms_norm(wide[:, 8:520], w, want=("h", "y", "q", "rstd"), eps=1e-5)
    check_forward(out, x, None, w, 1e-5, "bf16")
    out = ops.rms_norm(x, w, wide[:, 8:520], want=("y",))
    check_forward(out, x, x, w, 1e-6, "bf16")


@pytest.mark.parametrize("which", ["x", "residual"])
def test_sum_in_place(ops, which):
    x, r, w = make(41, 768, "bf16", 6)
    want = ops.rms_norm(x, w, r, want=("h", "y"))
    h = (x if which == "x" else r)
    a, b = x.clone(), r.clone()
    h = a if which == "x" else b
    got = ops.rms_norm(a, w, b, out=dict(h=h, y=None))
    assert torch.equal(h, want["h"]) and torch.equal(got["y"], want["y"])


def test_zero_infinite_and_nan_rows(ops):
    x, _, w = make(6, 256, "bf16", 7)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 200] = float("nan")
    x[4] = 1e-30
    out = ops.rms_norm(x, w, want=("y", "q", "rstd"))
    y, q, s = out["y"].float(), out["q"].float(), out["scale"]
    assert torch.equal(y[1], torch.zeros_like(y[1])) and torch.equal(q[1], torch.zeros_like(q[1]))
    assert torch.equal(s[1], torch.zeros_like(s[1]))
    assert torch.isnan(y[2, 5]) and torch.equal(y[2, 6:], torch.zeros_like(y[2, 6:]))   # x / inf
    assert torch.isnan(y[3]).all() and torch.isnan(q[3] * s[3].repeat_interleave(128)).all()
    for t in (0, 4, 5):
        assert torch.isfinite(y[t]).all() and torch.isfinite(s[t]).all()
    check_forward({k: v[4:5] for k, v in out.items()}, x[4:5], None, w, 1e-6, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 136), (1, 7168), (64, 256), (305, 1408), (1000, 512), (33, 16384)])
@pytest.mark.parametrize("with_dh", [True, False])
def test_backward(ops, T, d, dtype, with_dh):
    h, dh, w = make(T, d, dtype, T * 3 + d)
    dy = torch.randn(T, d, generator=torch.Generator().manual_seed(9)).to(DT[dtype]).cuda()
    dh = dh if with_dh else None
    rstd = ops.rms_norm(h, w, want=("rstd",))["rstd"]
    out = ops.rms_norm_backward(dy, h, w, rstd, dh=dh)
    dx, dw, size, wsize = oo.rms_norm_backward(f64(dy), f64(h), f64(w), f64(rstd), f64(dh))
    assert np.all(np.abs(f64(out["dx"]) - dx) <= HALF[dtype] * np.abs(dx) + 2 * SUMS * size)
    # T/304 rows a CTA, then 304 parts in eight chains: under T/304 + 46 additions in a row
    assert np.all(np.abs(f64(out["dw"]) - dw) <= (T / 304 + 50) * 2.0 ** -24 * wsize)


def test_backward_in_place_and_single_outputs(ops):
    h, dh, w = make(50, 640, "bf16", 11)
    dy = torch.randn(50, 640).to(torch.bfloat16).cuda()
    rstd = ops.rms_norm(h, w, want=("rstd",))["rstd"]
    want = ops.rms_norm_backward(dy, h, w, rstd, dh=dh)
    assert torch.equal(ops.rms_norm_backward(dy, h, w, rstd, out=dict(dw=None))["dw"], want["dw"])
    got = ops.rms_norm_backward(dy, h, w, rstd, dh=dh, out=dict(dx=dh))
    assert got["dx"] is dh and torch.equal(dh, want["dx"])


def test_gradient_against_differences(ops):
    h, _, w = make(4, 64, "fp32", 12)
    dy = torch.randn(4, 64, generator=torch.Generator().manual_seed(1)).cuda()
    rstd = ops.rms_norm(h, w, want=("rstd",))["rstd"]
    got = ops.rms_norm_backward(dy, h, w, rstd)
    def loss(a, b):
        return (oo.rms_norm(f64(a), f64(b), 1e-6)[0] * f64(dy)).sum()
    for t, i in [(0, 0), (1, 17), (3, 63)]:
        step = torch.zeros_like(h)
        step[t, i] = 2.0 ** -8          # the moved values stay exact to 2^-19 of the step
        n = (loss(h.double() + step.double(), w) - loss(h.double() - step.double(), w)) / 2.0 ** -7
        assert abs(n - got["dx"][t, i].item()) <= 1e-3 * max(1.0, abs(n))     # third differences of a smooth function
    step = torch.zeros_like(w)
    step[5] = 0.125
    n = (loss(h, w.double() + step.double()) - loss(h, w.double() - step.double())) / 0.25
    assert abs(n - got["dw"][5].item()) <= 1e-4 * max(1.0, abs(n))            # linear in w


def test_no_rows(ops):
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    assert ops.rms_norm(x, w, want=("y", "q"))["q"].shape == (0, 256)
    dw = torch.full((256,), 7.0, device="cuda")
    ops.rms_norm_backward(x, x, w, torch.empty(0, device="cuda"), out=dict(dw=dw, dx=None))
    assert torch.equal(dw, torch.zeros_like(dw))


def test_offsets_past_32_bits(ops):
    T, d = 300000, 8192
    x = torch.ones(T, d, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    y = ops.rms_norm(x, w, want=("y", "rstd"))
    check_forward({k: v[-4:] for k, v in y.items()}, x[-4:], None, w, 1e-6, "bf16")
    g = ops.rms_norm_backward(y["y"], x, w, y["rstd"], out=dict(dx=None))["dx"]
    dx, _, size, _ = oo.rms_norm_backward(f64(y["y"][-4:]), f64(x[-4:]), f64(w), f64(y["rstd"][-4:]))
    assert np.all(np.abs(f64(g[-4:]) - dx) <= HALF["bf16"] * np.abs(dx) + 2 * SUMS * size)


def test_another_stream_graph_and_repeats(ops):
    x, r, w = make(200, 1024, "bf16", 13)
    want = ops.rms_norm(x, w, r, want=("h", "y", "q", "rstd"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.rms_norm(x, w, r, want=("h", "y", "q", "rstd"), stream=s)
    s.synchronize()
    for n in want:
        assert torch.equal(want[n].float(), got[n].float()), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = ops.rms_norm(x, w, r, want=("h", "y", "q", "rstd"))
        grads = ops.rms_norm_backward(x, cap["h"], w, cap["rstd"], dh=r)
    graph.replay()
    eager = ops.rms_norm_backward(x, want["h"], w, want["rstd"], dh=r)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(want[n].float(), cap[n].float()), n
    for n in eager:
        assert torch.equal(eager[n], grads[n]), n


def test_python_refusals(ops):
    x, r, w = make(4, 64, "bf16", 14)
    with pytest.raises(TypeError):
        ops.rms_norm(x.half(), w)
    with pytest.raises(ValueError):
        ops.rms_norm(x, w[:32])
    with pytest.raises(ValueError):
        ops.rms_norm(x, w, r[:2])
    with pytest.raises(ValueError):
        ops.rms_norm(x.t(), w)
    with pytest.raises(ValueError):
        ops.rms_norm(x.cpu(), w)
    with pytest.raises(ValueError):
        ops.rms_norm(x, w, want=("z",))
    with pytest.raises(RuntimeError):
        ops.rms_norm(x[:, :60], w[:60].contiguous())           # d not a multiple of 8


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_one_row_of_a_wider_array(ops, dtype):
    """A single row has no stride: the width of the array that it is a part of does not matter, nor that of its sum's."""
    x, r, w = make(3, 512, dtype, 15)
    wide = torch.zeros(3, 1021, dtype=x.dtype, device="cuda")
    wide[:1, :512], wide[2:, :] = r[:1], 1.0
    want = ops.rms_norm(x[:1], w, r[:1], want=("h", "y"))
    got = ops.rms_norm(x[:1], w, wide[:1, :512], want=("h", "y"))
    row = wide[:1, :512]
    inplace = ops.rms_norm(row, w, x[:1], out=dict(h=row, y=None))
    for n in want:
        assert torch.equal(got[n], want[n]) and torch.equal(inplace[n], want[n]), n
    if dtype == "bf16":
        q, s = ops.quant_rows(wide[:1, :512])
        wq, ws = ops.quant_rows(wide[:1, :512].clone())
        assert torch.equal(q.float(), wq.float()) and torch.equal(s, ws)
        q, s = ops.quant_cols(wide[:1, :512])
        wq, ws = ops.quant_cols(wide[:1, :512].clone())
        assert torch.equal(q.float(), wq.float()) and torch.equal(s, ws)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(1900, 512), (1501, 2048), (1217, 4096), (457, 4104), (1000, 7168), (461, 8192),
                                 (500, 16384)])
def test_backward_of_several_rows_a_cta(ops, T, d, dtype):
    """Every instance with two rows a CTA and more, the last ones uneven, dh and dw (and dx in dh's place).

    dw: a CTA adds its rows one after the other, then the parts (one a CTA) go through 32 chains and a tree of five; a
    product's own rounding is one more, rstd's and h's one. With P parts that are under T / P + 1 + P / 32 + 1 + 5 + 2
    roundings, P between 152 and 608."""
    h, dh, w = make(T, d, dtype, T + d)
    dy = torch.randn(T, d, generator=torch.Generator().manual_seed(10)).to(DT[dtype]).cuda()
    rstd = ops.rms_norm(h, w, want=("rstd",))["rstd"]
    out = ops.rms_norm_backward(dy, h, w, rstd, dh=dh)
    dx, dw, size, wsize = oo.rms_norm_backward(f64(dy), f64(h), f64(w), f64(rstd), f64(dh))
    assert np.all(np.abs(f64(out["dx"]) - dx) <= HALF[dtype] * np.abs(dx) + 2 * SUMS * size)
    chain = max(T / p + 1 + p / 32 + 1 + 5 + 2 for p in (152, 304, 456, 608))
    assert np.all(np.abs(f64(out["dw"]) - dw) <= chain * 2.0 ** -24 * wsize)
    place = dh.clone()
    got = ops.rms_norm_backward(dy, h, w, rstd, dh=place, out=dict(dx=place, dw=None))
    assert torch.equal(place, out["dx"]) and torch.equal(got["dw"], out["dw"])
    got = ops.rms_norm_backward(dy, h, w, rstd)
    dx, _, size, _ = oo.rms_norm_backward(f64(dy), f64(h), f64(w), f64(rstd))
    assert np.all(np.abs(f64(got["dx"]) - dx) <= HALF[dtype] * np.abs(dx) + 2 * SUMS * size)
    assert torch.equal(got["dw"], out["dw"]) and ops.status() == 0
