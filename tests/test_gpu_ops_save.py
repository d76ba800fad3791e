"""SwiGLU with an 8-bit checkpoint, its gradient from it and 8-bit rows quantised along the tokens, against the 64-bit
restatement (GPU).

The checkpoint's codes and scales are equal (bf16 values: every step of the definition is exact or rounded once), and so
are requantised ones (fp32 products code * scale, then the same steps). The sigmoid's fast exponential and division are
within 2^-18; oracle.ops_oracle.swiglu_backward carries that to the gradients. A code is off by half a step, 2^-4 of its
value, or half of the smallest step, 2^-10 scales.
"""
import numpy as np
import pytest
import torch

import __graft_entry__
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ops():
    __graft_entry__.build()
    import mixture_experts_layer_routing_gb300 as moe
    return moe.default_ops()


def f64(t):
    return t.float().double().cpu().numpy()


def rnd(*shape, seed=0, spread=False):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(*shape, generator=g)
    if spread:
        v = v * torch.exp2(torch.randint(-12, 3, (shape[0], 1), generator=g).float())
    return v.to(torch.bfloat16)


def make_off(cnt, first=0):
    return torch.tensor(first + np.concatenate([[0], np.cumsum(cnt)]), dtype=torch.int32).cuda()


def codes_near(q, scale, want, err, axis):
    """Codes and scales stand for `want`, known within err."""
    back = oo.values(f64(q), f64(scale), axis)
    wide = np.take(f64(scale), np.arange(back.shape[axis]) // 128, axis=axis)
    tol = 2.0 ** -4 * np.abs(want) + 1.07 * err + 2.0 ** -10 * wide
    assert np.all(np.abs(back - want) <= tol), np.max(np.abs(back - want) - tol)
    # a block's largest value sets its scale
    for b in range(f64(scale).shape[axis]):
        at = [slice(None)] * 2
        at[axis] = slice(b * 128, (b + 1) * 128)
        m, e = np.abs(want[tuple(at)]).max(axis), err[tuple(at)].max(axis)
        s = np.take(f64(scale), b, axis=axis)
        assert np.all(np.abs(s * 448 - m) <= e + 2.0 ** -22 * m)


@pytest.mark.parametrize("T,f", [(1, 8), (3, 128), (5, 136), (33, 264), (70, 200), (2, 7168), (300, 1408)])
def test_swiglu_and_checkpoint(ops, T, f):
    gu = rnd(T, 2 * f, seed=T + f, spread=True)
    gu[0, :min(f, 128)] = 0
    out = ops.swiglu(gu.cuda(), want=("act", "q", "save"))
    save, scale = oo.swiglu_save(f64(gu))
    assert np.array_equal(f64(out["save"]), save) and np.array_equal(f64(out["save_scale"]), scale)
    a = oo.swiglu(f64(gu)[:, :f], f64(gu)[:, f:])
    assert np.all(np.abs(f64(out["act"]) - a) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(a))
    q, s = ops.quant_rows(gu.cuda(), swiglu=True)
    assert torch.equal(out["q"].view(torch.uint8), q.view(torch.uint8)) and torch.equal(out["scale"], s)
    if f % 128 == 0:
        q, s = ops.quant_rows(gu.cuda())
        assert torch.equal(out["save"].view(torch.uint8), q.view(torch.uint8)) and torch.equal(out["save_scale"], s)
    for want in (("act",), ("q",), ("save_scale",)):
        one = ops.swiglu(gu.cuda(), want=want)
        assert all(torch.equal(one[n].view(torch.uint8), out[n].view(torch.uint8)) for n in one)


def test_swiglu_strided_and_not_finite(ops):
    wide = rnd(19, 1024, seed=1).cuda()
    gu = wide[:, 64:64 + 544]
    out, dense = ops.swiglu(gu, want=("act", "q", "save")), ops.swiglu(gu.contiguous(), want=("act", "q", "save"))
    assert all(torch.equal(out[n].view(torch.uint8), dense[n].view(torch.uint8)) for n in out)
    y = rnd(4, 512, seed=2)
    y[0, 3], y[1, 200], y[2, 300] = float("nan"), float("inf"), -float("inf")
    out = ops.swiglu(y.cuda(), want=("save",))
    back = f64(out["save"]) * np.repeat(f64(out["save_scale"]), 128, 1)
    bad = np.zeros((4, 4), bool)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert np.array_equal(np.isnan(back), np.repeat(bad, 128, 1))


def backward_inputs(T, f, seed, gate=True):
    gu, dact = rnd(T, 2 * f, seed=seed), rnd(T, f, seed=seed + 1, spread=True)
    gu[:, ::7] *= 4
    g = torch.rand(T, generator=torch.Generator().manual_seed(seed + 2)) - 0.1
    return gu, dact, g if gate else None


@pytest.mark.parametrize("T,f,cnt", [(1, 8, None), (5, 136, None), (128, 128, None), (129, 392, None), (300, 256, None),
                                     (300, 200, [0, 1, 127, 128, 0, 44, 0]), (257, 384, [129, 0, 128]), (77, 128, [0, 0, 77]),
                                     (140, 1024, [70, 0, 70]), (140, 1032, [70, 0, 70]), (600, 904, [1, 0, 599]), (40, 1408, None)])
@pytest.mark.parametrize("gated", [True, False])
def test_swiglu_backward(ops, T, f, cnt, gated):
    gu, dact, gate = backward_inputs(T, f, T + f, gated)
    saved = ops.swiglu(gu.cuda(), want=("save",))
    off = None if cnt is None else make_off(cnt)
    names = ("dgu", "dqt", "dgate") + (("dq",) if f % 128 == 0 else ())
    out = ops.swiglu_backward(dact.cuda(), saved["save"], saved["save_scale"], gate=None if gate is None else gate.cuda(),
                              off=off, want=names)
    g, u = oo.swiglu_saved(f64(saved["save"]), f64(saved["save_scale"]))
    dg, du, a, dgate, eg, eu, ea, size = oo.swiglu_backward(g, u, f64(dact), np.ones(T) if gate is None else f64(gate))
    dgu, err = np.concatenate([dg, du], 1), np.concatenate([eg, eu], 1)
    assert np.all(np.abs(f64(out["dgu"]) - dgu) <= err + 2.0 ** -8 * (np.abs(dgu) + err))
    # sums of up to 16 values a lane, 8 lanes, ceil(f / 128) blocks
    assert np.all(np.abs(f64(out["dgate"]) - dgate) <= (2.0 ** -17 + (24 + f / 128) * 2.0 ** -24) * size)
    if "dq" in out:
        codes_near(out["dq"], out["dq_scale"], dgu, err, 1)
    at, ends = 0, [0, T] if off is None else off.tolist()
    for lo, hi in zip(ends[:-1], ends[1:]):
        n = -(-(hi - lo) // 128) * 128
        for q, s, v, e in ((out["dqt"], out["dqt_scale"], dgu, err), (out["actt"], out["actt_scale"], a, ea)):
            pad, pe = np.zeros((n, v.shape[1])), np.zeros((n, v.shape[1]))
            pad[:hi - lo], pe[:hi - lo] = v[lo:hi], e[lo:hi]
            if n:
                codes_near(q[:, at:at + n].float().t(), s[at // 128:(at + n) // 128], pad, pe, 0)
                assert (f64(q[:, at + hi - lo:at + n]) == 0).all()
        at += n
    assert ops.status() == 0
    # any one of the outputs alone, and the same bits again
    for want in [("dgu",), ("dgate",), ("actt",)] + ([("dq",)] if f % 128 == 0 else []):
        one = ops.swiglu_backward(dact.cuda(), saved["save"], saved["save_scale"],
                                  gate=None if gate is None else gate.cuda(), off=off, want=want)
        for n in one:
            x, y = one[n].view(torch.uint8), out[n].view(torch.uint8)
            if n in ("dqt", "actt"):
                x, y = x[:, :at], y[:, :at]
            if n in ("dqt_scale", "actt_scale"):
                x, y = one[n][:at // 128], out[n][:at // 128]
            assert torch.equal(x, y), n


def test_gradient_against_differences(ops):
    """d/dgu of sum_t gate_t <act_t, dact_t>, by central differences of the function of the checkpoint's values, and
    d/dgate: within the two-sided difference's error and bf16's."""
    T, f = 4, 16
    gu, dact, gate = backward_inputs(T, f, 11)
    saved = ops.swiglu(gu.cuda(), want=("save",))
    out = ops.swiglu_backward(dact.cuda(), saved["save"], saved["save_scale"], gate=gate.cuda(), want=("dgu", "dgate"))
    g, u = oo.swiglu_saved(f64(saved["save"]), f64(saved["save_scale"]))
    x = np.concatenate([g, u], 1)
    fun = lambda z, w: (oo.swiglu(z[:, :f], z[:, f:]) * f64(dact) * w[:, None]).sum()  # noqa: E731
    for t in range(T):
        for i in range(2 * f):
            d = np.zeros_like(x)
            d[t, i] = 1e-5
            num = (fun(x + d, f64(gate)) - fun(x - d, f64(gate))) / 2e-5
            assert abs(f64(out["dgu"])[t, i] - num) <= 2.0 ** -8 * abs(num) + 1e-6 * (1 + abs(x[t, i - f] if i >= f else x[t, i + f]))
        d = np.zeros(T)
        d[t] = 1e-4
        num = (fun(x, f64(gate) + d) - fun(x, f64(gate) - d)) / 2e-4
        assert abs(f64(out["dgate"])[t] - num) <= 1e-4 * (1 + abs(num))


def test_rows_of_no_segment_stay_as_they_were(ops):
    import mixture_experts_layer_routing_gb300 as moe
    T, f = 200, 128
    gu, dact, gate = backward_inputs(T, f, 5)
    saved = ops.swiglu(gu.cuda(), want=("save",))
    off = make_off([130, 20], first=10)

    def fresh():
        new = lambda dt, *s: torch.full(s, 7.0, device="cuda").to(dt)  # noqa: E731
        Tp = (2 + 2) * 128
        return dict(dgu=new(torch.bfloat16, T, 2 * f), dq=new(F8, T, 2 * f), dq_scale=new(torch.float32, T, 2),
                    dqt=new(F8, 2 * f, Tp), dqt_scale=new(torch.float32, Tp // 128, 2 * f), actt=new(F8, f, Tp),
                    actt_scale=new(torch.float32, Tp // 128, f), dgate=new(torch.float32, T))

    out = ops.swiglu_backward(dact.cuda(), saved["save"], saved["save_scale"], gate=gate.cuda(), off=off, out=fresh())
    for n in ("dgu", "dq", "dq_scale", "dgate"):
        assert (out[n][:10].float() == 7).all() and (out[n][160:].float() == 7).all(), n
        assert not (out[n][10:160].float() == 7).all(), n
    for n in ("dqt", "actt"):
        assert (out[n][:, 384:].float() == 7).all(), n
    assert (out["dqt_scale"][3:] == 7).all() and ops.status() == 0
    for bad in ([0, 4, 2], [-1, 2, 3], [0, 2, 201]):
        out = ops.swiglu_backward(dact.cuda(), saved["save"], saved["save_scale"], gate=gate.cuda(),
                                  off=torch.tensor(bad, dtype=torch.int32).cuda(), out=fresh())
        assert all((v.float() == 7).all() for v in out.values()) and ops.status() == moe.MOE_ERR_DEVICE_INDEX


def test_backward_not_finite_and_strided(ops):
    T, f = 40, 256
    gu, dact, gate = backward_inputs(T, f, 9)
    saved = ops.swiglu(gu.cuda(), want=("save",))
    dact[3, 5], dact[7, 200] = float("nan"), float("inf")
    wide = torch.zeros(T, 640, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:64 + f] = dact.cuda()
    args = (saved["save"], saved["save_scale"])
    names = ("dgu", "dq", "dqt", "dgate")
    out = ops.swiglu_backward(wide[:, 64:64 + f], *args, gate=gate.cuda(), want=names)
    same = ops.swiglu_backward(dact.cuda(), *args, gate=gate.cuda(), want=names)
    assert all(torch.equal(out[n].view(torch.uint8), same[n].view(torch.uint8)) for n in out)
    bad = np.zeros(T, bool)
    bad[[3, 7]] = True
    assert np.array_equal(~np.isfinite(f64(out["dgate"])), bad)
    assert np.array_equal(np.isnan(f64(out["dq"]) * np.repeat(f64(out["dq_scale"]), 128, 1)).any(1), bad)
    back = f64(out["dqt"]) * np.repeat(f64(out["dqt_scale"]), 128, 0).T
    cols = np.zeros(2 * f, bool)
    cols[[5, 200, f + 5, f + 200]] = True
    assert np.array_equal(np.isnan(back).any(1), cols)


@pytest.mark.parametrize("T,C,cnt", [(1, 8, None), (128, 64, None), (129, 136, None), (300, 200, None),
                                     (300, 264, [0, 1, 127, 128, 0, 44, 0]), (257, 64, [129, 0, 128])])
@pytest.mark.parametrize("gather", [False, True])
def test_requant_cols(ops, T, C, cnt, gather):
    src = rnd(90 if gather else T, C, seed=T + C, spread=True)
    src[0, :] = 0
    index = torch.randint(0, 90, (T,), generator=torch.Generator().manual_seed(4), dtype=torch.int32)
    off = None if cnt is None else make_off(cnt)
    q8, s8 = ops.quant_rows(src.cuda())
    q, s = ops.requant_cols(q8, s8, off=off, row_index=index.cuda() if gather else None)
    v = (f64(q8).astype(np.float32) * np.repeat(f64(s8).astype(np.float32), 128, 1)[:, :C]).astype(np.float64)
    x = v[index.long().numpy()] if gather else v
    at, ends = 0, [0, T] if off is None else off.tolist()
    for lo, hi in zip(ends[:-1], ends[1:]):
        n = -(-(hi - lo) // 128) * 128
        pad = np.zeros((n, C))
        pad[:hi - lo] = x[lo:hi]
        if n:
            wq, ws = oo.quantise(pad, 0)
            assert np.array_equal(f64(q)[:, at:at + n], wq.T)
            assert np.array_equal(f64(s)[at // 128:(at + n) // 128], ws)
        at += n
    assert ops.status() == 0


def test_requant_cols_index_out_of_range(ops):
    import mixture_experts_layer_routing_gb300 as moe
    q8, s8 = ops.quant_rows(rnd(6, 64, seed=1).cuda())
    q, s = ops.requant_cols(q8, s8, row_index=torch.tensor([0, 6, 2, -1], dtype=torch.int32).cuda())
    assert (f64(q)[:, [1, 3]] == 0).all() and ops.status() == moe.MOE_ERR_DEVICE_INDEX
    # in no segment: not read
    ops.requant_cols(q8, s8, off=torch.tensor([1, 2, 3], dtype=torch.int32).cuda(),
                     row_index=torch.tensor([99, 0, 2, -1], dtype=torch.int32).cuda())
    assert ops.status() == 0


def test_streams_and_graphs_give_the_same_bits(ops):
    T, f = 260, 256
    gu, dact, gate = (t.cuda() for t in backward_inputs(T, f, 21))
    off = make_off([100, 0, 160])

    def step():
        a = ops.swiglu(gu, want=("q", "save"))
        b = ops.swiglu_backward(dact, a["save"], a["save_scale"], gate=gate, off=off, want=("dq", "dgate"))
        return [a["q"], a["scale"], b["dq"], b["dq_scale"], b["dgate"]]

    want = [t.clone() for t in step()]
    live = (gu.float().requires_grad_(True) * 2).sum()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(step())
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    live.backward()
    for o in outs:
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(o, want))
    other = ops.swiglu(gu, want=("q",), stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(other["q"].view(torch.uint8), want[0].view(torch.uint8))
