"""CPU checks of the operators' C ABI (include/moe_ops.h): exported symbols, every refusal on the host, and the
64-bit restatements that the GPU tests compare with."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import __graft_entry__
import mixture_experts_layer_routing_gb300 as moe
from mixture_experts_layer_routing_gb300 import ops as mops
from oracle import ops_oracle as oo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ARG, UNSUP, WS = moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
P = 1 << 20          # a non-null, aligned address that no refused call looks at


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return mops._lib()


def test_every_declared_operator_is_exported_and_bound(lib):
    src = open(os.path.join(ROOT, "include", "moe_ops.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(r"^\s*moe_status\s+(moe_\w+)\s*\(", src, flags=re.M)
    assert set(names) == set(mops.OPS_EXPORTED)
    for n in names:
        assert hasattr(lib, n), n


def call(lib, name, defaults, over):
    args = dict(defaults)
    assert set(over) <= set(args), over
    args.update(over)
    return getattr(lib, name)(*args.values())


NORM = dict(ops=P, dtype=1, x=P, ld_x=256, residual=P, ld_res=256, weight=P, T=4, d=256, eps=1e-6, h=P, y=P, q=P,
            scale=P, rstd=P, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(ops=None), ARG), (dict(dtype=2), ARG), (dict(T=-1), ARG), (dict(d=0), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(x=None), ARG), (dict(weight=None), ARG),
    (dict(h=None, y=None, q=None, scale=None, rstd=None), ARG), (dict(q=None), ARG), (dict(scale=None), ARG),
    (dict(d=250), UNSUP), (dict(d=16392), UNSUP), (dict(ld_x=248), ARG), (dict(ld_res=248), ARG),
    (dict(ld_x=260), UNSUP), (dict(dtype=0, ld_x=258), UNSUP), (dict(x=P + 8), UNSUP), (dict(y=P + 2), UNSUP),
    (dict(q=P + 4), UNSUP), (dict(ld_x=512), ARG),          # h is x, but the rows of h are dense
])
def test_norm_forward_refuses(lib, over, code):
    assert call(lib, "moe_norm_forward", NORM, over) == code


BWD = dict(ops=P, dtype=1, dy=P, dh=P, h=P, weight=P, rstd=P, T=4, d=256, dx=P, dw=P, workspace=P, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(ops=None), ARG), (dict(dtype=3), ARG), (dict(T=-1), ARG), (dict(dx=None, dw=None), ARG), (dict(d=12), UNSUP),
    (dict(dy=None), ARG), (dict(h=None), ARG), (dict(weight=None), ARG), (dict(rstd=None), ARG),
    (dict(dh=P + 4), UNSUP), (dict(workspace=None), WS), (dict(workspace=P + 8), WS),
])
def test_norm_backward_refuses(lib, over, code):
    assert call(lib, "moe_norm_backward", BWD, over) == code


def cfg(**over):
    base = dict(E=64, k=6, router=1, renorm=1, route_scale=2.5, n_groups=8, topk_groups=4)
    base.update(over)
    return mops.moe_gate_config(*base.values())


@pytest.mark.parametrize("over,code", [
    (dict(E=0), ARG), (dict(k=0), ARG), (dict(E=4, k=5, n_groups=1, topk_groups=1), ARG), (dict(router=2), ARG),
    (dict(route_scale=float("inf")), ARG), (dict(E=264), UNSUP), (dict(k=9), UNSUP), (dict(n_groups=7), ARG),
    (dict(n_groups=0), ARG), (dict(topk_groups=0), ARG), (dict(topk_groups=9), ARG),
    (dict(n_groups=64, topk_groups=6), UNSUP), (dict(n_groups=16, topk_groups=1), ARG),   # 4 experts left for k = 6
])
def test_gate_refuses_configurations(lib, over, code):
    c = cfg(**over)
    assert lib.moe_gate_forward(P, ctypes.byref(c), P, None, 4, P, P, P, P, P, P, P, None) == code


GATE = dict(ops=P, cfg=None, logits=P, bias=None, T=4, idx=P, gate=P, cnt=P, off=P, perm=P, inv=P, workspace=P,
            stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(ops=None), ARG), (dict(T=-1), ARG), (dict(T=1 << 28), UNSUP), (dict(logits=None), ARG),
    (dict(idx=None), ARG), (dict(gate=None), ARG), (dict(cnt=None), ARG), (dict(inv=None), ARG),
    (dict(T=65, workspace=None), WS), (dict(T=65, workspace=P + 4), WS),
])
def test_gate_refuses_arguments(lib, over, code):
    c = cfg()
    assert call(lib, "moe_gate_forward", {**GATE, "cfg": ctypes.byref(c)}, over) == code
    assert lib.moe_gate_forward(P, None, P, None, 4, P, P, P, P, P, P, P, None) == ARG
    assert lib.moe_gate_backward(P, ctypes.byref(c), P, P, None, 4, P, None) == ARG


MM = dict(ops=P, a=P, sa=P, a_rows=64, row_index=None, M=64, b=P, sb=P, off=None, G=1, N=128, K=256, c=P, out=1,
          workspace=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(ops=None), ARG), (dict(M=-1), ARG), (dict(N=0), ARG), (dict(K=0), ARG), (dict(G=0), ARG), (dict(G=2), ARG),
    (dict(a_rows=63), ARG), (dict(out=2), ARG), (dict(G=257, off=P), UNSUP), (dict(K=264), UNSUP),
    (dict(a=None), ARG), (dict(sa=None), ARG), (dict(b=None), ARG), (dict(sb=None), ARG), (dict(c=None), ARG),
    (dict(a=P + 8), UNSUP), (dict(b=P + 8), UNSUP), (dict(c=P + 8), UNSUP),
    (dict(G=256, off=P, N=1 << 24), UNSUP),
    (dict(M=200, row_index=P), WS), (dict(M=200, row_index=P, workspace=P + 8), WS),
])
def test_matmul_refuses(lib, over, code):
    assert call(lib, "moe_fp8_matmul", MM, over) == code


def test_matmul_of_no_rows_does_nothing(lib):
    assert call(lib, "moe_fp8_matmul", MM, dict(M=0, a=None, c=None, a_rows=0)) == OK


WG = dict(ops=P, dct=P, sd=P, xt=P, sx=P, T=64, off=None, G=1, N=128, K=256, c=P, out=1, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(ops=None), ARG), (dict(T=-1), ARG), (dict(c=None), ARG), (dict(dct=None), ARG), (dict(sx=None), ARG),
    (dict(G=3), ARG), (dict(G=300, off=P), UNSUP), (dict(T=(1 << 22) + 1), UNSUP), (dict(xt=P + 4), UNSUP),
    (dict(out=5), ARG), (dict(N=132), UNSUP), (dict(K=252), UNSUP), (dict(sd=P + 4), UNSUP),
])
def test_wgrad_refuses(lib, over, code):
    assert call(lib, "moe_fp8_wgrad", WG, over) == code


@pytest.mark.parametrize("name,args,code", [
    ("moe_quant_rows", (P, None, 64, 4, 64, 0, P, P, None), ARG),
    ("moe_quant_rows", (P, P, 64, -1, 64, 0, P, P, None), ARG),
    ("moe_quant_rows", (P, P, 64, 4, 64, 1, P, P, None), ARG),        # swiglu reads 2C values of a row
    ("moe_quant_rows", (P, P, 68, 4, 64, 0, P, P, None), UNSUP),
    ("moe_quant_rows", (P, P, 64, 4, 60, 0, P, P, None), UNSUP),
    ("moe_quant_cols", (P, P, 64, 4, 4, 60, None, 1, None, P, P, None), UNSUP),
    ("moe_quant_cols", (P, P, 64, 3, 4, 64, None, 1, None, P, P, None), ARG),     # fewer rows than tokens
    ("moe_quant_cols", (P, P, 64, 4, 4, 64, None, 2, None, P, P, None), ARG),     # segments without offsets
    ("moe_quant_cols", (P, P, 64, 4, 4, 64, P, 257, None, P, P, None), ARG),
    ("moe_quant_blocks", (P, P, 1, 128, 128, P, P, P, None, None), ARG),
    ("moe_quant_blocks", (P, P, 1, 124, 128, P, P, None, None, None), UNSUP),
    ("moe_quant_blocks", (P, P, 0, 128, 128, P, P, None, None, None), ARG),
])
def test_quantisers_refuse(lib, name, args, code):
    assert getattr(lib, name)(*args) == code


@pytest.mark.parametrize("make", [mops.default_ops, mops.MoeOps])
def test_handles_of_other_devices_are_refused(make):
    with pytest.raises(ValueError):
        make("cpu")


def test_padded_rows_of_the_token_axis(lib):
    n = ctypes.c_int()
    for T, G, want in [(0, 1, 0), (1, 1, 128), (128, 1, 128), (129, 1, 256), (129, 4, 256 + 4 * 128)]:
        assert lib.moe_quant_cols_rows(T, G, ctypes.byref(n)) == OK
        assert n.value == want
    # every split of T tokens over G segments fits
    rng = np.random.default_rng(0)
    for _ in range(200):
        G, T = int(rng.integers(2, 9)), int(rng.integers(0, 700))
        cnt = rng.multinomial(T, rng.dirichlet(np.ones(G) * 0.3))
        assert lib.moe_quant_cols_rows(T, G, ctypes.byref(n)) == OK
        assert sum(-(-c // 128) * 128 for c in cnt) <= n.value


# ------------------------------------------------- the 64-bit restatements

def test_e4m3_rounding_against_torch():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    codes = codes[torch.isfinite(codes)].double().numpy()
    assert np.array_equal(oo.e4m3(codes), codes)
    grid = np.sort(codes)
    mid = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([mid, mid * (1 + 1e-6), mid * (1 - 1e-6), np.linspace(-448, 448, 4001)])
    want = torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy()
    v32 = torch.from_numpy(v).float().double().numpy()
    assert np.array_equal(oo.e4m3(v32), want)


def _numeric(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    h, w, dy, dh = rng.normal(size=(3, 16)), rng.normal(size=16), rng.normal(size=(3, 16)), rng.normal(size=(3, 16))
    dx, dw, _, _ = oo.rms_norm_backward(dy, h, w, oo.rms_norm(h, w, 1e-6)[1], dh)
    assert np.allclose(dx, _numeric(lambda z: (oo.rms_norm(z, w, 1e-6)[0] * dy).sum() + (z * dh).sum(), h), atol=1e-7)
    assert np.allclose(dw, _numeric(lambda z: (oo.rms_norm(h, z, 1e-6)[0] * dy).sum(), w), atol=1e-7)


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_against_differences(router, renorm):
    rng = np.random.default_rng(2)
    l, b, dg = rng.normal(size=(4, 12)), 0.3 * rng.normal(size=12), rng.normal(size=(4, 3))
    kw = dict(k=3, router=router, renorm=renorm, scale=2.5, n_groups=4, topk_groups=2)
    idx, _ = oo.gate(l, b, **kw)
    f = lambda z: (oo.gate(z, b, **kw)[1] * dg).sum()  # noqa: E731  (the selection does not move)
    got, _ = oo.gate_backward(l, idx, dg, router, renorm, 2.5)
    assert np.allclose(got, _numeric(f, l), atol=1e-7)
