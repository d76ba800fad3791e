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


# -------------------------------------------------------------- long products

@pytest.mark.parametrize("M,N,K,group,zero", [
    (1, 20008, 7200, 128, False), (4, 12008, 7200, 32, True), (8, 12008, 7200, 64, False), (8, 20008, 7200, 128, True),
    (1, 194568, 96, 32, True), (3, 194568, 96, 64, False), (8, 194568, 288, 32, False), (2, 97288, 1312, 128, False),
    (21, 40008, 544, 64, True)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_products_of_many_units(ops, M, N, K, group, zero, out):
    """Several units a CTA and several chunks a warp; the last block of rows ends within it; K ends within a chunk."""
    g = gen(N + K)
    w, x = weights(g, 1, N, K, group, zero), rnd(g, M, K)
    c = ops.w4_matmul(x, first(w), out_dtype=out)
    v = dense(w, 0)
    near(c, x.double() @ v.t(), x.double().abs() @ v.abs().t(), -(-K // group))
    assert ops.status() == 0


@pytest.mark.parametrize("N,K,group,zero", [(4008, 2080, 32, True), (12008, 1056, 128, False), (4008, 7200, 64, False),
                                            (40008, 96, 32, False)])
def test_segments_that_grow_and_shrink(ops, N, K, group, zero):
    """A warp of these products meets tiles of one row, of eight and of none in between, in several chunks each."""
    cnt = [1, 8, 0, 3, 17, 1, 1, 9, 0, 0, 25, 2, 7]
    ends = [0] + list(np.cumsum(cnt))
    g = gen(N)
    w, x = weights(g, len(cnt), N, K, group, zero), rnd(g, 19, K)
    index = torch.randint(0, 19, (ends[-1],), generator=g, device="cuda", dtype=torch.int32)
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    c = ops.w4_matmul(x, w, off=off, row_index=index, out_dtype=torch.float32)
    a = x.double()[index.long()]
    for e, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        if hi > lo:
            v = dense(w, e)
            near(c[lo:hi], a[lo:hi] @ v.t(), a[lo:hi].abs() @ v.abs().t(), -(-K // group))
    assert ops.status() == 0


# ---------------------------------------------------------------- long layers

def layer(ops, T, d, f, E, k, shared, group, zero, out, idx=None, seed=0):
    """The layer against 64 bits. Its bound: the sums of both products, SwiGLU, h to 16 (fp32 outputs: 24) bits."""
    g = gen(seed + T + d + f)
    x, w13, wd = rnd(g, T, d), weights(g, E + shared, 2 * f, d, group, zero), weights(g, E + shared, d, f, group, zero)
    if idx is None:
        idx = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    gate = torch.rand(T, k, generator=g, device="cuda") - 0.2
    y = ops.w4_experts(x, idx, gate, w13, wd, n_shared=shared, out_dtype=out)
    add = (30 + max(-(-d // group), (k + shared) * -(-f // group))) * 2.0 ** -23
    kept = 2.0 ** -18 + 2.0 ** (-24 if out == torch.float32 else -16)
    want, bound = torch.zeros(T, d, dtype=torch.float64, device="cuda"), torch.zeros(T, d, dtype=torch.float64, device="cuda")
    per = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    per.scatter_add_(1, idx.long().clamp(0, E - 1), torch.where((idx >= 0) & (idx < E), gate, 0.0).double())
    for e in range(E + shared):
        t = (idx == e).any(1).nonzero().flatten() if e < E else torch.arange(T, device="cuda")
        if t.numel() == 0:
            continue
        v, xe, ge = dense(w13, e), x[t].double(), per[t, e, None] if e < E else 1.0
        (a, u), (sa, su) = (xe @ v.t()).chunk(2, 1), (xe.abs() @ v.abs().t()).chunk(2, 1)
        s = a * torch.special.expit(a)
        h = ge * s * u
        off = (ge.abs() if e < E else 1.0) * add * (1.1 * u.abs() * sa + s.abs() * su) + kept * h.abs()
        v = dense(wd, e)
        want.index_add_(0, t, h @ v.t())
        bound.index_add_(0, t, (off + add * h.abs()) @ v.abs().t())
    err = (y.double() - want).abs()
    tol = bound + HALF[out] * (want.abs() + bound)
    assert bool((err <= tol).all()), (err - tol).max().item()
    return (y.double() - want).norm() / want.norm()


@pytest.mark.parametrize("T,d,f,E,k,shared,group,zero", [
    (1, 7200, 96, 6, 3, 1, 128, False), (1, 14368, 544, 4, 2, 0, 32, True), (3, 7200, 288, 9, 4, 0, 64, True),
    (16, 7200, 160, 12, 6, 1, 32, False), (16, 14368, 96, 8, 3, 0, 128, True), (64, 14368, 96, 12, 4, 1, 64, False),
    (64, 7200, 544, 5, 2, 0, 128, True), (16, 2080, 2080, 12, 4, 1, 32, True), (40, 1056, 2080, 12, 8, 0, 128, False),
    (2, 2080, 4128, 6, 4, 1, 64, False)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_layers_of_many_units(ops, T, d, f, E, k, shared, group, zero, out):
    """Several units a CTA of either kernel: rings that wrap, pointers that step from rows to rows, sums taken over."""
    layer(ops, T, d, f, E, k, shared, group, zero, out)
    assert ops.status() == 0


@pytest.mark.parametrize("rows", [2, 3, 8, 16, 17, 64])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_layers_whose_tiles_grow_and_shrink(ops, rows, out):
    """One, then all, then a few tokens an expert, over and over, in several units a CTA and several chunks a warp: a
    warp of either kernel meets tiles with more rows than the one in front, and with fewer."""
    E, k = 60, 8
    idx = torch.full((rows, k), -1, dtype=torch.int32)
    idx[:, 0], idx[:, 1], idx[:, 2] = 1, 30, 58
    for t in range(rows):
        idx[t, 3:] = torch.tensor([2 + (5 * t + j) % 28 if j < 3 else 31 + (3 * t + j) % 27 for j in range(5)])
    layer(ops, rows, 4128, 1056, E, k, 0, 32, False, out, idx=idx.cuda())
    layer(ops, rows, 7200, 288, E, k, 1, 128, True, out, idx=idx.cuda(), seed=3)
    assert ops.status() == 0


# ---------------------------------------------------- h's precision, fp32 outputs

def one_code(n, N, K, at):
    """Matrices of which row r holds one 1 (code 9, scale 1), at column at[r]."""
    codes = torch.full((n, N, K), 8, dtype=torch.int64)
    codes[:, torch.arange(N), at] = 9
    words = torch.from_numpy(oo.w4_pack(codes.numpy())).cuda()
    return dict(codes=words, scale=torch.ones(n, K // 32, N, dtype=torch.bfloat16, device="cuda"), group=32)


@pytest.mark.parametrize("T", [1, 2, 16, 33])
def test_fp32_outputs_carry_24_bits_of_h(ops, T):
    """Each y is one h, and g and u are values of x, so that nothing but h's own rounding counts: the exponential (2^-23),
    1 + e, the quotient and the products with u and with the gate (2^-24 each), h's three parts (2^-26) and their sum
    (2^-24 twice): below 2^-23 + 7 * 2^-24 = 4.5 * 2^-23."""
    d, f, E = 128, 64, 3
    g = gen(T)
    x = (torch.rand(T, d, generator=g, device="cuda") * 80 - 40).to(torch.bfloat16)
    w13, wd = one_code(E, 2 * f, d, torch.arange(2 * f)), one_code(E, d, f, torch.arange(d) % f)
    idx = torch.randint(0, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    gate = torch.rand(T, 1, generator=g, device="cuda") + 0.5
    y = ops.w4_experts(x, idx, gate, w13, wd, out_dtype=torch.float32).double()
    a, u = x.double().chunk(2, 1)
    want = (a * torch.special.expit(a) * u * gate.double()).repeat(1, 2)
    off = ((y - want).abs() / want.abs()).max().item()
    assert off <= 4.5 * 2.0 ** -23, off * 2 ** 23
