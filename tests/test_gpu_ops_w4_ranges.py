"""4-bit weights over the range that the calls accept (GPU): weights at the ends of bf16, products and layers whose CTAs
take many units and whose warps go several times round their rings, h's precision for fp32 outputs.

References are torch in 64 bits on the device. A product's sum: a value of x times a code less its zero point is exact
in fp32; a group's sum passes through at most 8 MMAs, each of which adds two partial sums (16 additions); a warp adds its
groups, and up to 15 warps are joined: 30 + groups additions in a row at most, each off by at most 2^-23 (a truncated
addition) of the sum of magnitudes. Then half a step of the output's type.
"""
import numpy as np
import pytest
import torch

import __graft_entry__
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def ops():
    __graft_entry__.build()
    import mixture_experts_layer_routing_gb300 as moe
    return moe.default_ops()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def weights(g, n, N, K, group, zero):
    KG = -(-K // group)
    scale = torch.rand(n, KG, N, generator=g, device="cuda") * torch.exp2(torch.randint(-9, -4, (n, KG, N), generator=g, device="cuda").float())
    scale = torch.where(torch.rand(n, KG, N, generator=g, device="cuda") < 0.05, -scale, scale).to(torch.bfloat16)
    w = dict(codes=torch.randint(-2 ** 31, 2 ** 31, (n, N, K // 8), generator=g, device="cuda").to(torch.int32), scale=scale, group=group)
    if zero:
        w["zero"] = torch.randint(0, 16, (n, KG, N), generator=g, device="cuda").to(torch.uint8)
    return w


def dense(w, e):
    """Matrix e in 64 bits."""
    words = w["codes"][e]
    at = torch.from_numpy(oo.W4_SHIFT).to("cuda", torch.int32)
    c = ((words[:, :, None] >> at) & 15).flatten(1).double()
    wide = lambda v: v[e].double().t().repeat_interleave(w["group"], 1)[:, :c.shape[1]]  # noqa: E731
    return (c - (wide(w["zero"]) if "zero" in w else 8.0)) * wide(w["scale"])


def first(w):
    return {n: v[0].contiguous() if torch.is_tensor(v) else v for n, v in w.items()}


def near(got, want, size, groups):
    tol = (30 + groups) * 2.0 ** -23 * size + HALF[got.dtype] * want.abs()
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), (err - tol).max().item()


def test_the_reference_reads_words_as_the_oracle_does():
    w = weights(gen(1), 2, 24, 96, 32, True)
    for e in range(2):
        want = oo.w4_values(w["codes"][e].cpu().numpy(), w["scale"][e].double().cpu().numpy(), w["zero"][e].double().cpu().numpy(), 32)
        assert np.array_equal(dense(w, e).cpu().numpy(), want)


# ------------------------------------------------ weights at the ends of bf16

@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
def test_finite_weights_read_finite(ops, group, zero):
    """Whatever a group spans: only a NaN or an infinity may read NaN. A value is off by half a step, by the scale's
    rounding (2^-9 of 15 steps) and with zero points by half a step more."""
    top = torch.finfo(torch.bfloat16).max
    w = rnd(gen(2), 16, 256).float()
    w[0, 3], w[0, 9] = 3e38, -1e38
    w[1, 3], w[1, 9] = top, -top
    w[2] = torch.where(w[2] > 0, top, -top)
    w[3] = top
    w[4] = -top
    w[5, 200], w[5, 201] = -top, 2e37
    w = w.to(torch.bfloat16)
    q = ops.quant_w4(w, group, zero)
    codes, scale, zeros = oo.quant_w4(w.double().cpu().numpy(), group, zero)
    assert np.array_equal(oo.w4_unpack(q["codes"].cpu().numpy()), codes)
    assert np.array_equal(q["scale"].double().cpu().numpy(), scale)
    if zero:
        assert np.array_equal(q["zero"].double().cpu().numpy(), zeros)
    back = dense({n: v[None] if torch.is_tensor(v) else v for n, v in q.items()}, 0)
    step = q["scale"].double().t().repeat_interleave(group, 1)
    assert bool(torch.isfinite(step).all())
    assert bool(((back - w.double()).abs() <= step * (0.5 + 15 * 2.0 ** -9 + (0.5 if zero else 0.0))).all())
