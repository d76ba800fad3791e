"""Routing operators against the 64-bit restatement (GPU): selections and dispatch equal, gates and gradients near.

Gates: a score is within 14 units in the last place of the largest score (see the kernel), a renormalised gate
within three times that: 2^-18 of the sum's share. Gradients likewise, relative to the magnitudes that cancel.
"""
import numpy as np
import pytest
import torch

import __graft_entry__
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
NEAR = 2.0 ** -18


@pytest.fixture(scope="module")
def ops():
    __graft_entry__.build()
    import mixture_experts_layer_routing_gb300 as moe
    return moe.default_ops()


def check(ops, logits, bias, k, router="sigmoid", renorm=True, scale=1.0, n_groups=1, topk_groups=1):
    T, E = logits.shape
    kw = dict(router=router, renorm=renorm, n_groups=n_groups, topk_groups=topk_groups)
    out = ops.gate(logits.cuda(), k, bias=None if bias is None else bias.cuda(), route_scale=scale, **kw)
    idx, gate = oo.gate(logits.double().numpy(), None if bias is None else bias.double().numpy(), k, scale=scale, **kw)
    assert ops.status() == 0
    got = {n: t.cpu().numpy() for n, t in out.items()}
    assert np.array_equal(got["idx"], idx)
    for n, want in zip(("cnt", "off", "perm", "inv"), oo.dispatch(idx, E)):
        assert np.array_equal(got[n], want), n
    fine = np.isfinite(gate)
    assert np.array_equal(np.isnan(got["gate"]), np.isnan(gate))
    # softmax scores: relative to the row's largest
    top = oo.scores(logits.double().numpy(), router).max(1, keepdims=True) * scale if not renorm else gate
    assert np.all(np.abs(got["gate"] - gate)[fine] <= NEAR * np.maximum(np.abs(gate), np.broadcast_to(top, gate.shape))[fine])
    return out


CASES = [
    # T, E, k, router, renorm, groups, kept, bias
    (1, 1, 1, "softmax", True, 1, 1, False), (1, 256, 8, "sigmoid", True, 8, 4, True),
    (4, 256, 8, "sigmoid", True, 8, 4, True), (64, 64, 6, "softmax", True, 1, 1, False),
    (65, 64, 6, "softmax", False, 1, 1, True), (129, 60, 4, "softmax", False, 1, 1, True),
    (200, 96, 3, "sigmoid", False, 4, 1, True), (77, 160, 8, "softmax", True, 8, 3, True),
    (1000, 128, 2, "sigmoid", True, 32, 7, True), (33, 32, 5, "sigmoid", True, 32, 9, True),
    (500, 8, 2, "softmax", True, 2, 1, False), (300, 255, 7, "sigmoid", True, 5, 2, True),
    (40, 17, 8, "sigmoid", True, 1, 1, True), (9, 200, 1, "softmax", True, 8, 8, True),
]


@pytest.mark.parametrize("T,E,k,router,renorm,groups,kept,bias", CASES)
def test_forward(ops, T, E, k, router, renorm, groups, kept, bias):
    g = torch.Generator().manual_seed(T * 7 + E)
    check(ops, 1.5 * torch.randn(T, E, generator=g), 0.1 * torch.randn(E, generator=g) if bias else None, k, router,
          renorm, 2.5, groups, kept)


def test_many_chunks(ops):
    """More than 64 tokens a chunk, the last one short (the selection is checked on a sample)."""
    g = torch.Generator().manual_seed(3)
    T, E, k = 20011, 48, 5
    logits = torch.randn(T, E, generator=g)
    out = ops.gate(logits.cuda(), k, router="softmax")
    idx = out["idx"].cpu().numpy()
    assert np.array_equal(idx[::97], oo.gate(logits.double().numpy()[::97], None, k, "softmax", True, 1.0)[0])
    for n, want in zip(("cnt", "off", "perm", "inv"), oo.dispatch(idx, E)):
        assert np.array_equal(out[n].cpu().numpy(), want), n


@pytest.mark.parametrize("T", [16, 17, 24, 40, 63, 64, 65, 511, 513, 1030, 2049])
@pytest.mark.parametrize("E,k", [(64, 6), (256, 8)])
def test_chunks_of_several_sizes(ops, T, E, k):
    g = torch.Generator().manual_seed(T + E)
    check(ops, 1.5 * torch.randn(T, E, generator=g), None, k)


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
def test_equal_and_nearly_equal_keys(ops, router):
    """Ties go to the lower index; keys closer than 32 bits can tell are decided as in 64."""
    g = torch.Generator().manual_seed(4)
    base = torch.randn(300, 4, generator=g).repeat(1, 16)                   # each value 16 times
    near = base + torch.randint(-2, 3, base.shape, generator=g) * 1e-7      # or a few last places apart
    bias = torch.randint(-3, 4, (64,), generator=g) * 2.0 ** -24
    check(ops, base, None, 6, router)
    check(ops, near, None, 6, router)
    check(ops, near, bias, 8, router, n_groups=8, topk_groups=3)
    check(ops, torch.zeros(5, 64), None, 4, router, n_groups=4, topk_groups=2)
    check(ops, 30 + near, bias, 6, router)                                   # saturated sigmoids


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
def test_masked_experts(ops, router, groups, kept):
    """-inf takes an expert out; a row without any selects the lowest indexes with gates of 0; the lowest finite
    value is a number like others."""
    g = torch.Generator().manual_seed(5)
    l = torch.randn(64, 32, generator=g)
    l[torch.rand(64, 32, generator=g) < 0.5] = -float("inf")
    l[3], l[4, 1:], l[5, :-1] = -float("inf"), -float("inf"), -float("inf")
    l[6] = torch.finfo(torch.float32).min
    l[7, ::2] = torch.finfo(torch.float32).min
    bias = 0.2 * torch.randn(32, generator=g)
    for b in (None, bias):
        out = check(ops, l, b, 4, router, n_groups=groups, topk_groups=kept)
        assert torch.equal(out["gate"][3].cpu(), torch.zeros(4))
        assert torch.isfinite(out["gate"]).all()


def test_nan_logits_come_last(ops):
    g = torch.Generator().manual_seed(6)
    l = torch.randn(16, 40, generator=g)
    l[2, 7], l[3, :], l[4, 5] = float("nan"), float("nan"), float("inf")
    out = check(ops, l, None, 3, "sigmoid")
    assert torch.isnan(out["gate"][3]).all() and 7 not in out["idx"][2].tolist()
    out = ops.gate(l.cuda(), 3, router="softmax")       # a NaN makes every score of its row NaN
    assert torch.isnan(out["gate"][2:5]).all() and out["idx"][2].tolist() == [0, 1, 2]
    assert torch.isfinite(out["gate"][5:]).all()


def test_without_dispatch_and_without_tokens(ops):
    g = torch.Generator().manual_seed(7)
    l = torch.randn(100, 64, generator=g).cuda()
    a, b = ops.gate(l, 6), ops.gate(l, 6, dispatch=False)
    assert set(b) == {"idx", "gate"} and torch.equal(a["idx"], b["idx"]) and torch.equal(a["gate"], b["gate"])
    out = ops.gate(l[:0], 6)
    assert out["off"].tolist() == [0] * 65 and out["cnt"].tolist() == [0] * 64
    assert ops.gate_backward(l[:0], out["idx"], out["gate"])["dlogits"].shape == (0, 64)


@pytest.mark.parametrize("T,E,k,router,renorm", [(1, 256, 8, "sigmoid", True), (77, 64, 6, "softmax", True),
                                                 (130, 60, 4, "softmax", False), (33, 100, 3, "sigmoid", False),
                                                 (500, 8, 2, "softmax", True), (5, 1, 1, "softmax", False),
                                                 (9, 17, 8, "sigmoid", True)])
def test_backward(ops, T, E, k, router, renorm):
    g = torch.Generator().manual_seed(T + E)
    l, dg = 2 * torch.randn(T, E, generator=g), torch.randn(T, k, generator=g)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    got = ops.gate_backward(l.cuda(), idx.cuda(), dg.cuda(), router=router, renorm=renorm, route_scale=2.5)["dlogits"]
    want, size = oo.gate_backward(l.double().numpy(), idx.numpy().astype(np.int64), dg.double().numpy(), router,
                                  renorm, 2.5)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= NEAR * size), (err / np.maximum(size, 1e-30)).max()
    if renorm or router == "sigmoid":
        assert np.all(got.cpu().numpy()[want == 0] == 0)
    assert ops.status() == 0


def test_backward_of_masked_rows_and_bad_indexes(ops):
    import mixture_experts_layer_routing_gb300 as moe
    l = torch.randn(8, 16)
    l[1] = -float("inf")
    l[2, 3] = -float("inf")
    idx = torch.tensor([[3, 5]] * 8, dtype=torch.int32)
    for router in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d = ops.gate_backward(l.cuda(), idx.cuda(), torch.ones(8, 2).cuda(), router=router, renorm=renorm)["dlogits"]
            assert torch.isfinite(d).all() and not d[1].any()
    assert ops.status() == 0
    idx[4, 0], idx[5, 1] = 16, -1                      # out of range: recorded, their gradient left out
    d = ops.gate_backward(l.cuda(), idx.cuda(), torch.ones(8, 2).cuda(), router="sigmoid", renorm=False)["dlogits"]
    assert ops.status() == moe.MOE_ERR_DEVICE_INDEX and ops.status() == 0
    assert d[4].nonzero().flatten().tolist() == [5] and d[5].nonzero().flatten().tolist() == [3]


def test_gradient_against_differences(ops):
    g = torch.Generator().manual_seed(8)
    l, dg = torch.randn(3, 24, generator=g).double(), torch.randn(3, 4, generator=g)
    out = ops.gate(l.float().cuda(), 4, router="sigmoid", n_groups=4, topk_groups=2, route_scale=2.5)
    idx = out["idx"].cpu().numpy()
    d = ops.gate_backward(l.float().cuda(), out["idx"], dg.cuda(), router="sigmoid", route_scale=2.5)["dlogits"].cpu()
    def loss(z):
        p = oo.scores(z, "sigmoid")[np.arange(3)[:, None], idx]
        return (2.5 * p / p.sum(1, keepdims=True) * dg.double().numpy()).sum()
    l = l.float().double().numpy()
    for t in range(3):
        for e in range(24):
            a, b = l.copy(), l.copy()
            a[t, e] += 1e-5
            b[t, e] -= 1e-5
            assert abs((loss(a) - loss(b)) / 2e-5 - d[t, e].item()) <= 1e-5


def test_another_stream_graph_and_repeats(ops):
    g = torch.Generator().manual_seed(9)
    l, b = torch.randn(3000, 256, generator=g).cuda(), (0.1 * torch.randn(256, generator=g)).cuda()
    kw = dict(bias=b, router="sigmoid", n_groups=8, topk_groups=4)
    want = ops.gate(l, 8, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.gate(l, 8, stream=s, **kw)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = ops.gate(l, 8, **kw)
    graph.replay()
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(want[n], got[n]) and torch.equal(want[n], cap[n]), n


def test_python_refusals(ops):
    l = torch.randn(4, 64).cuda()
    with pytest.raises(TypeError):
        ops.gate(l.double(), 4)
    with pytest.raises(ValueError):
        ops.gate(l.t(), 4)
    with pytest.raises(KeyError):
        ops.gate(l, 4, router="relu")
    with pytest.raises(RuntimeError):
        ops.gate(l, 9)
    with pytest.raises(RuntimeError):
        ops.gate(l, 4, n_groups=7)
    with pytest.raises(ValueError):
        ops.gate_backward(l, torch.zeros(4, 2, dtype=torch.int32).cuda(), torch.zeros(4, 3).cuda())


BIASES = {
    "one +inf": lambda b: b.index_fill_(0, torch.tensor([37]), float("inf")),
    "three +inf": lambda b: b.index_fill_(0, torch.tensor([2, 37, 38]), float("inf")),
    "all +inf": lambda b: b.fill_(float("inf")),
    "one -inf": lambda b: b.index_fill_(0, torch.tensor([5]), -float("inf")),
    "few left of -inf": lambda b: b[:-3].fill_(-float("inf")),
    "all -inf": lambda b: b.fill_(-float("inf")),
    "+inf and -inf": lambda b: (b[::2].fill_(-float("inf")), b[9:10].fill_(float("inf"))),
    "masks of -1e9": lambda b: b[1::3].fill_(-1e9),
    "few left of -1e9": lambda b: b[4:].fill_(-1e9),
    "one of 1e9": lambda b: b[11:12].fill_(1e9),
    "lowest value": lambda b: b[::5].fill_(torch.finfo(torch.float32).min),
    "largest value": lambda b: b[7:9].fill_(torch.finfo(torch.float32).max),
}


@pytest.mark.parametrize("name", BIASES)
@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept", [(40, 1, 1), (64, 8, 3), (256, 1, 1), (256, 8, 4), (60, 5, 2)])
@pytest.mark.parametrize("k", [1, 2, 8])
def test_infinite_and_masking_biases(ops, name, router, E, groups, kept, k):
    """A bias of +inf puts an expert first, one of -inf (or the masks' usual numbers) behind the others."""
    g = torch.Generator().manual_seed(E + k)
    logits, bias = 1.5 * torch.randn(37, E, generator=g), 0.05 * torch.randn(E, generator=g)
    BIASES[name](bias)
    out = check(ops, logits, bias, k, router, n_groups=groups, topk_groups=kept)
    assert 0 <= out["idx"].min().item() and out["idx"].max().item() < E


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,kept", [(2, 2, 1, 1), (4, 4, 1, 1), (8, 8, 1, 1), (8, 4, 2, 1), (32, 8, 8, 2),
                                             (256, 8, 32, 1)])
def test_as_many_experts_as_are_selected(ops, router, E, k, groups, kept):
    """Every expert (of the groups kept) is selected, in the order of its key; equal keys, masked ones among them, by
    index."""
    g = torch.Generator().manual_seed(E)
    logits = torch.randint(-2, 3, (200, E), generator=g).float()
    logits[100:150][torch.rand(50, E, generator=g) < 0.4] = -float("inf")
    logits[0, :4] = torch.tensor([0.0, 1.0, 1.0, 0.0])[:E]
    out = check(ops, logits, None, k, router, n_groups=groups, topk_groups=kept)
    assert all(len(set(row)) == k for row in out["idx"].tolist())


def test_masks_and_peaked_scores_cost_what_others_do(ops):
    """Selections that 32 bits decide stay with them when one bias is far from the others or one score far above: less
    than twice the ordinary time (21 us; in 64 bits 183)."""
    g = torch.Generator().manual_seed(10)
    l, b = torch.randn(8192, 256, generator=g).cuda(), (0.05 * torch.randn(256, generator=g)).cuda()
    def masked(v):
        return b.index_fill(0, torch.tensor([3, 90], device="cuda"), v)
    def us(logits, **kw):
        out = ops.gate(logits, 8, **kw)
        best = []
        for _ in range(7):
            t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            t[0].record()
            for _ in range(20):
                ops.gate(logits, 8, out=out, **kw)
            t[1].record()
            torch.cuda.synchronize()
            best.append(t[0].elapsed_time(t[1]) * 50)
        return min(best)
    kw = dict(router="sigmoid", n_groups=8, topk_groups=4)
    usual = us(l, bias=b, **kw)
    for v in (-float("inf"), -1e9, float("inf")):
        assert us(l, bias=masked(v), **kw) < 2 * usual, v
    assert us(1.5 * l - 10, bias=0.01 * b, **kw) < 2 * usual
    assert us(8 * l, router="softmax") < 2 * us(l, router="softmax")


@pytest.mark.parametrize("E,k,scale", [(24, 1, 1.0), (24, 2, 1.0), (200, 8, 2.5), (64, 6, 1.0)])
def test_backward_of_selected_scores_far_below_the_largest(ops, E, k, scale):
    """Renormalised softmax gates whose scores' sum is near or below the 1e-20 that is added to it: the other logits
    have a gradient there.

    A score e^x of the row's largest, x = -30 .. -130, is off by |x| 2^-24 of itself through its rounded argument, and
    enters a gradient four times (its own, the sum, twice the mean); below 2^-126 it may be lost whole, over 1e-20."""
    g = torch.Generator().manual_seed(E + k)
    T = 101
    l, dg = torch.randn(T, E, generator=g), torch.randn(T, k, generator=g)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    down = torch.linspace(30, 130, T)[:, None]
    l.scatter_add_(1, idx, -down.expand(T, k) + torch.rand(T, k, generator=g))
    got = ops.gate_backward(l.cuda(), idx.int().cuda(), dg.cuda(), router="softmax", route_scale=scale)["dlogits"]
    want, size = oo.gate_backward(l.double().numpy(), idx.numpy(), dg.double().numpy(), "softmax", True, scale)
    lost = 2.0 ** -126 * 1e20 * 2 * k * scale * np.abs(dg.numpy()).max(1, keepdims=True)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= (NEAR + 4 * 2.0 ** -24 * (down.numpy() + 8)) * size + lost), (err / (size + lost)).max()
    # the stated example: gates 0.253 and 0.093, and a gradient of -0.105 at the largest logit
    d = ops.gate_backward(torch.tensor([[0.0, -47, -48, -49]]).cuda(), torch.tensor([[1, 2]], dtype=torch.int32).cuda(),
                          torch.tensor([[1.0, -1]]).cuda(), router="softmax")["dlogits"][0].tolist()
    assert np.allclose(d, [-0.105, 0.213, -0.108, 0], atol=1e-3)


def test_forward_and_backward_agree_near_the_added_constant(ops):
    """The gradient against differences of the forward pass's formula, D between 1e-24 and 1e-16."""
    l = torch.tensor([[0.0, -37, -38, 1], [0, -46, -45.5, -1], [0, -55, -54, 0.5]])
    dg = torch.tensor([[1.0, -1], [0.5, 2], [-1, 1]])
    idx = torch.tensor([[1, 2]] * 3)
    d = ops.gate_backward(l.cuda(), idx.int().cuda(), dg.cuda(), router="softmax")["dlogits"].double().cpu().numpy()
    def loss(z):
        p = oo.scores(z, "softmax")[np.arange(3)[:, None], idx.numpy()]
        return (p / (p.sum(1, keepdims=True) + 1e-20) * dg.double().numpy()).sum()
    z = l.double().numpy()
    for t in range(3):
        for e in range(4):
            a, b = z.copy(), z.copy()
            a[t, e] += 1e-5
            b[t, e] -= 1e-5
            assert abs((loss(a) - loss(b)) / 2e-5 - d[t, e]) <= 1e-4


@pytest.mark.parametrize("names", [("cnt",), ("cnt", "off"), ("inv",), ("perm",)])
def test_any_output_of_the_dispatch_is_written(ops, names):
    l = torch.randn(50, 16, generator=torch.Generator().manual_seed(11)).cuda()
    want = ops.gate(l, 3)
    out = {n: torch.full_like(want[n], -7) for n in names}
    got = ops.gate(l, 3, out=dict(out))
    for n in names:
        assert got[n] is out[n]
    for n in want:
        assert torch.equal(got[n], want[n]), n
    assert set(ops.gate(l, 3, out=dict(idx=None, gate=None))) == {"idx", "gate"}
