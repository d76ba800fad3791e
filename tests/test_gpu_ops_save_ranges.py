"""SwiGLU's 8-bit checkpoint, its gradient and requantised columns over the range that the calls accept (GPU): many rows,
wide ones, every cluster's size, values that are not finite, scales at both ends of fp32."""
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def f64(t):
    return t.float().double().cpu().numpy()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def inputs(T, f, seed):
    g = gen(seed)
    gu, dact = rnd(g, T, 2 * f), rnd(g, T, f)
    gu[:, ::7] *= 4
    return gu, dact, torch.rand(T, generator=g, device="cuda") - 0.1


def check_rows(out, saved, dact, gate):
    """dgu and dgate against the oracle's formulas and bounds, in 64 bits."""
    g, u = oo.swiglu_saved(f64(saved["save"]), f64(saved["save_scale"]))
    dg, du, _, dgate, eg, eu, _, size = oo.swiglu_backward(g, u, f64(dact), f64(gate))
    dgu, err = np.concatenate([dg, du], 1), np.concatenate([eg, eu], 1)
    assert np.all(np.abs(f64(out["dgu"]) - dgu) <= err + 2.0 ** -8 * (np.abs(dgu) + err))
    # sums of up to 16 values a lane, 8 lanes, ceil(f / 128) blocks
    f = dact.shape[1]
    assert np.all(np.abs(f64(out["dgate"]) - dgate) <= (2.0 ** -17 + (24 + f / 128) * 2.0 ** -24) * size)


@pytest.mark.parametrize("lo,hi", [(-1, 1), (-16, 0), (-80, -16), (0, 80)])
def test_the_gradients_sigmoid(ops, lo, hi):
    """One value a row, so that dgate is one product act * dact. In units of 2^-23: the exponential of two 2, its argument
    |g| / 2 (rounded) and |g| / 8 (log2(e) in fp32), 1 + e 0.5, its reciprocal 1, the products with g, u, dact 0.5 each."""
    T, f, g = 4096, 8, gen(hi - lo)
    gu, dact = (torch.zeros(T, n, device="cuda", dtype=torch.bfloat16) for n in (2 * f, f))
    gu[:, 0] = (torch.rand(T, generator=g, device="cuda") * (hi - lo) + lo).bfloat16()
    gu[:, f], dact[:, 0] = rnd(g, T), rnd(g, T)
    s = ops.swiglu(gu, want=("save",))
    got = ops.swiglu_backward(dact, s["save"], s["save_scale"], want=("dgate",))["dgate"].double()
    v = (s["save"].float() * s["save_scale"].repeat_interleave(f, 1)).double()
    a = v[:, 0]
    want = a * torch.special.expit(a) * v[:, f] * dact[:, 0].double()
    assert bool(((got - want).abs() <= (5 + 0.625 * a.abs()) * 2.0 ** -23 * want.abs()).all())


@pytest.mark.parametrize("T,f,cnt", [(5000, 1408, [0, 1, 1300, 128, 0, 3071, 31, 469, 0]), (5000, 1408, None),
                                     (2600, 2048, [2579, 21]), (20000, 264, [1] * 100 + [19900])])
def test_backward_of_many_tiles_without_columns(ops, T, f, cnt):
    """More tiles than run at once, so that a CTA takes a whole one; the same bits as with columns."""
    gu, dact, gate = inputs(T, f, T + f)
    saved = ops.swiglu(gu, want=("save",))
    off = None if cnt is None else torch.tensor(np.concatenate([[0], np.cumsum(cnt)]), dtype=torch.int32).cuda()
    names = ("dgu", "dgate") + (("dq",) if f % 128 == 0 else ())
    call = lambda *want: ops.swiglu_backward(dact, saved["save"], saved["save_scale"], gate=gate, off=off, want=want)  # noqa: E731
    out, cols = call(*names), call(*names, "dqt")
    assert all(same(out[n], cols[n]) for n in out)
    check_rows(out, saved, dact, gate)
    # and each alone
    for n in names:
        one = call(n)
        assert all(same(one[m], out[m]) for m in one)
    assert ops.status() == 0


@pytest.mark.parametrize("f", [8, 128, 256, 384, 512, 640, 768, 896, 1024])
@pytest.mark.parametrize("T", [1, 100, 500])
def test_gates_gradient_of_every_number_of_column_blocks(ops, T, f):
    gu, dact, gate = inputs(T, f, f)
    saved = ops.swiglu(gu, want=("save",))
    call = lambda *want: ops.swiglu_backward(dact, saved["save"], saved["save_scale"], gate=gate, want=want)  # noqa: E731
    out = call("dgu", "dgate")
    check_rows(out, saved, dact, gate)
    assert same(call("dgate", "dqt")["dgate"], out["dgate"])
    assert ops.status() == 0


@pytest.mark.parametrize("T,f", [(3, 20008), (1, 65536), (130, 8200)])
def test_wide_rows(ops, T, f):
    gu, dact, gate = inputs(T, f, f)
    out = ops.swiglu(gu, want=("act", "q", "save"))
    save, scale = oo.swiglu_save(f64(gu))
    assert np.array_equal(f64(out["save"]), save) and np.array_equal(f64(out["save_scale"]), scale)
    a = oo.swiglu(f64(gu)[:, :f], f64(gu)[:, f:])
    assert np.all(np.abs(f64(out["act"]) - a) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(a))
    back = ops.swiglu_backward(dact, out["save"], out["save_scale"], gate=gate, want=("dgu", "dgate", "dqt"))
    check_rows(back, out, dact, gate)
    # the columns' codes are those of any other width: of one block in the middle and of the last one
    for c in (4096, (f - 1) & ~127):
        n = min(128, f - c)
        part = torch.cat([gu[:, c:c + n], gu[:, f + c:f + c + n]], 1).contiguous()
        p = ops.swiglu(part, want=("save",))
        q = ops.swiglu_backward(dact[:, c:c + n].contiguous(), p["save"], p["save_scale"], gate=gate, want=("dqt",))
        for name in ("actt", "actt_scale"):
            whole = back[name][c:c + n] if name == "actt" else back[name][:, c:c + n]
            assert same(whole, q[name]), name
        assert same(torch.cat([back["dqt"][c:c + n], back["dqt"][f + c:f + c + n]]), q["dqt"])
        assert same(torch.cat([back["dqt_scale"][:, c:c + n], back["dqt_scale"][:, f + c:f + c + n]], 1), q["dqt_scale"])
    assert ops.status() == 0


def columns_of(q, s, off, index, T):
    """Codes and scales of requant_cols by the oracle, a segment at a time."""
    with np.errstate(invalid="ignore", over="ignore"):
        v = f64(q).astype(np.float32) * np.repeat(f64(s).astype(np.float32), 128, 1)[:, :q.shape[1]]
    v = v if index is None else v[index]
    parts = []
    for lo, hi in zip(off[:-1], off[1:]):
        if hi > lo:
            pad = np.zeros((-(-(hi - lo) // 128) * 128, v.shape[1]), np.float32)
            pad[:hi - lo] = v[lo:hi]
            parts.append(pad)
    return parts


@pytest.mark.parametrize("T,C,cnt", [(1100, 2056, None), (1500, 1408, [0, 700, 1, 128, 0, 671]), (3, 40008, None)])
@pytest.mark.parametrize("gather", [False, True])
def test_requant_cols_of_many_columns(ops, T, C, cnt, gather):
    g = gen(T + C)
    q, s = ops.quant_rows(rnd(g, 700 if gather else T, C) * torch.exp2(torch.randint(-20, 20, (1, C), generator=g, device="cuda").float()).bfloat16())
    index = torch.randint(0, 700, (T,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    ends = [0, T] if cnt is None else [0] + list(np.cumsum(cnt))
    off = None if cnt is None else torch.tensor(ends, dtype=torch.int32).cuda()
    qt, st = ops.requant_cols(q, s, off=off, row_index=index)
    at = 0
    for pad in columns_of(q, s, ends, None if index is None else index.cpu().numpy(), T):
        n = pad.shape[0]
        wq, ws = oo.quantise(pad, 0)
        assert np.array_equal(f64(qt)[:, at:at + n], wq.T) and np.array_equal(f64(st)[at // 128:(at + n) // 128], ws)
        at += n
    assert ops.status() == 0


@pytest.mark.parametrize("low,high", [(-149, -130), (-126, -100), (-112, -104), (100, 112), (-126, 112)])
def test_requant_cols_at_the_ends_of_the_range(ops, low, high):
    """Blocks whose maxima leave the quotients' fast path: equal codes and scales all the same."""
    T, C, g = 300, 264, gen(high - low)
    q = (torch.randn(T, C, generator=g, device="cuda") * 100).clamp(-448, 448).to(F8)
    q[:, 5] = 0
    s = torch.ldexp(torch.rand(T, 3, generator=g, device="cuda") + 1, torch.randint(low, high, (T, 3), generator=g, device="cuda"))
    qt, st = ops.requant_cols(q, s)
    (pad,) = columns_of(q, s, [0, T], None, T)
    assert np.isfinite(pad).all()
    wq, ws = oo.quantise(pad, 0)
    assert np.array_equal(f64(st), ws) and np.array_equal(f64(qt), wq.T)


def test_requant_cols_not_finite(ops):
    """A NaN or an infinity in a row's block makes NaN of the columns of that block, in its tile of tokens alone."""
    T, C = 300, 264
    src = rnd(gen(7), T, C)
    src[3, 5], src[140, 130], src[299, 263] = float("nan"), float("inf"), -float("inf")
    q, s = ops.quant_rows(src)
    qt, st = ops.requant_cols(q, s)
    back = f64(qt) * np.repeat(f64(st), 128, 0).T
    bad = np.zeros((C, 384), bool)
    bad[:128, :128] = bad[128:256, 128:256] = bad[256:, 256:] = True
    assert np.array_equal(np.isnan(back), bad)
    (pad,) = columns_of(torch.where(torch.isnan(s).repeat_interleave(128, 1)[:, :C], torch.zeros_like(q.view(torch.uint8)), q.view(torch.uint8)).view(F8),
                        torch.nan_to_num(s, nan=0.0, posinf=0.0, neginf=0.0), [0, T], None, T)
    wq, ws = oo.quantise(pad, 0)
    assert np.array_equal(f64(qt)[~bad], wq.T[~bad])
