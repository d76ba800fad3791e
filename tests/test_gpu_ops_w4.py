"""4-bit weights against the 64-bit restatement (GPU): their quantiser, products of few rows, the experts' layer.

Quantiser: codes, scales and zero points equal (every step is rounded once, as the definition says).
Products: a value of x times a code less its zero point is exact in fp32. A group's sum passes through at most 8 MMAs,
each of which adds two partial sums (16 additions), then ceil(K / group) groups and 8 warps are added: under
(24 + groups) additions in a row, each off by at most 2^-23 (a truncated addition) of the sum of magnitudes. Then the
rounding to the output's type.
Layer: oracle.ops_oracle.w4_experts carries those errors through SwiGLU and the second product.
"""
import numpy as np
import pytest
import torch

import __graft_entry__
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
GROUPS = [(32, False), (32, True), (64, False), (64, True), (128, False), (128, True)]


@pytest.fixture(scope="module")
def ops():
    __graft_entry__.build()
    import mixture_experts_layer_routing_gb300 as moe
    return moe.default_ops()


def f64(t):
    return t.float().double().cpu().numpy()


def rnd(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def weights(G, N, K, group, zero, seed=0):
    """Random codes and scales on the GPU, and their values as G matrices."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 16, (G, N, K), generator=g).numpy()
    KG = -(-K // group)
    scale = (torch.rand(G, KG, N, generator=g) * torch.exp2(torch.randint(-9, -4, (G, KG, N), generator=g).float())).to(torch.bfloat16)
    scale[torch.rand(G, KG, N, generator=g) < 0.05] *= -1
    w = dict(codes=torch.from_numpy(oo.w4_pack(codes)).cuda(), scale=scale.cuda(), group=group)
    z = None
    if zero:
        z = torch.randint(0, 16, (G, KG, N), generator=g).to(torch.uint8)
        w["zero"] = z.cuda()
    values = [oo.w4_values(oo.w4_pack(codes[i]), f64(scale[i]), None if z is None else z[i].numpy().astype(float), group)
              for i in range(G)]
    return w, values


def first(w):
    return {n: v[0].contiguous() if torch.is_tensor(v) else v for n, v in w.items()}


def near(got, want, size, groups):
    err = np.abs(f64(got) - want)
    tol = (24 + groups) * 2.0 ** -23 * size + HALF[got.dtype] * np.abs(want)
    assert np.all(err <= tol), (np.unravel_index(np.argmax(err - tol), err.shape), err.max())


# --------------------------------------------------------------- quantiser

@pytest.mark.parametrize("group,zero", GROUPS)
@pytest.mark.parametrize("N,K", [(8, 32), (24, 96), (136, 416), (1000, 1056)])
def test_quant_w4(ops, group, zero, N, K):
    w = rnd(2, N, K, seed=N + K)
    w[0, 0] = 0
    w[0, 1] = w[0, 1].abs()
    w[0, 2] = -w[0, 2].abs()
    w[1, 3] *= 1e-30
    w[1, 4] *= 1e30
    w[1, 5] = (w[1, 5].float() * 2.0 ** -128).to(torch.bfloat16)       # scales that are subnormal in bf16
    out = ops.quant_w4(w.cuda(), group, zero)
    for g in range(2):
        codes, scale, zeros = oo.quant_w4(f64(w[g]), group, zero)
        assert np.array_equal(oo.w4_unpack(out["codes"][g].cpu().numpy()), codes)
        assert np.array_equal(f64(out["scale"][g]), scale)
        if zero:
            assert np.array_equal(f64(out["zero"][g]), zeros)
    flat = ops.quant_w4(w[1].contiguous().cuda(), group, zero)
    assert all(torch.equal(flat[n], out[n][1]) for n in flat if n != "group")
    assert flat["group"] == group


@pytest.mark.parametrize("zero", [False, True])
def test_groups_that_are_not_finite_read_nan(ops, zero):
    w = rnd(16, 256, seed=7)
    w[1, 3], w[2, 100], w[3, 255] = float("nan"), float("inf"), -float("inf")
    q = ops.quant_w4(w.cuda(), 64, zero)
    back = oo.w4_values(q["codes"].cpu().numpy(), f64(q["scale"]), f64(q["zero"]) if zero else None, 64)
    bad = np.zeros((16, 4), bool)
    bad[1, 0] = bad[2, 1] = bad[3, 3] = True
    assert np.array_equal(np.isnan(back), np.repeat(bad, 64, 1))


# ---------------------------------------------------------------- products

@pytest.mark.parametrize("group,zero", GROUPS)
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 40, 96), (2, 136, 416), (7, 1000, 1056), (8, 64, 2048), (9, 72, 160),
                                   (16, 264, 544), (33, 88, 1312), (100, 48, 128)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_w4_matmul(ops, group, zero, M, N, K, out):
    x = rnd(M, K, seed=M + K)
    w, v = weights(1, N, K, group, zero, seed=N)
    c = ops.w4_matmul(x.cuda(), first(w), out_dtype=out)
    near(c, f64(x) @ v[0].T, np.abs(f64(x)) @ np.abs(v[0]).T, -(-K // group))


@pytest.mark.parametrize("group,zero", [(32, True), (64, False), (128, False), (128, True)])
@pytest.mark.parametrize("cnt", [[1], [0, 3, 0], [5, 0, 8, 9, 1, 0, 17], [0, 0], [40, 1]])
@pytest.mark.parametrize("gather", [False, True])
def test_w4_matmul_of_segments(ops, group, zero, cnt, gather):
    N, K, M = 72, 288, sum(cnt)
    rows = 13 if gather else max(M, 1)
    x = rnd(rows, K, seed=M)
    w, v = weights(len(cnt), N, K, group, zero, seed=len(cnt))
    off = torch.tensor(np.concatenate([[0], np.cumsum(cnt)]), dtype=torch.int32).cuda()
    index = torch.randint(0, rows, (M,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    c = ops.w4_matmul(x.cuda() if gather else x[:M].cuda(), w, off=off, row_index=index.cuda() if gather else None,
                      out_dtype=torch.float32)
    assert c.shape == (M, N)
    a = f64(x)[index.long().numpy()] if gather else f64(x[:M])
    if M:
        want, size = oo.matmul(a, np.stack(v), np.concatenate([[0], np.cumsum(cnt)]))
        near(c, want, size, -(-K // group))
    assert ops.status() == 0


def test_as_many_segments_as_there_may_be(ops):
    G, N, K = 256, 40, 96
    cnt = [(7 * i) % 4 for i in range(G)]
    M = sum(cnt)
    w, v = weights(G, N, K, 32, False, seed=9)
    x = rnd(M, K, seed=10)
    off = torch.tensor(np.concatenate([[0], np.cumsum(cnt)]), dtype=torch.int32).cuda()
    c = ops.w4_matmul(x.cuda(), w, off=off, out_dtype=torch.float32)
    want, size = oo.matmul(f64(x), np.stack(v), np.concatenate([[0], np.cumsum(cnt)]))
    near(c, want, size, 3)
    assert ops.status() == 0


def test_rows_of_no_segment_stay_as_they_were(ops):
    import mixture_experts_layer_routing_gb300 as moe
    w, v = weights(2, 40, 64, 32, False, seed=1)
    x = rnd(6, 64, seed=2)
    off = torch.tensor([1, 3, 4], dtype=torch.int32).cuda()
    index = torch.tensor([99, 0, 5, 2, -7, 1 << 30], dtype=torch.int32).cuda()    # not read where there is no segment
    out = torch.full((6, 40), 7.0, device="cuda")
    ops.w4_matmul(x.cuda(), w, off=off, row_index=index, out=out)
    a = f64(x)
    near(out[1:3], a[[0, 5]] @ v[0].T, np.abs(a[[0, 5]]) @ np.abs(v[0]).T, 2)
    near(out[3:4], a[[2]] @ v[1].T, np.abs(a[[2]]) @ np.abs(v[1]).T, 2)
    assert (out[[0, 4, 5]] == 7).all()
    assert ops.status() == 0
    # an index out of range in a segment: a row of zeros, recorded
    ops.w4_matmul(x.cuda(), w, off=torch.tensor([0, 3, 4], dtype=torch.int32).cuda(), row_index=index, out=out)
    assert (out[0] == 0).all() and ops.status() == moe.MOE_ERR_DEVICE_INDEX
    # offsets that are not ascending within 0 .. M: nothing is written, recorded
    out.fill_(7.0)
    for bad in ([0, 4, 2], [-1, 2, 3], [0, 2, 7]):
        ops.w4_matmul(x.cuda(), w, off=torch.tensor(bad, dtype=torch.int32).cuda(), out=out)
        assert (out == 7).all() and ops.status() == moe.MOE_ERR_DEVICE_INDEX


def test_strided_rows_and_one_row_of_a_wider_array(ops):
    w, v = weights(1, 64, 160, 64, True, seed=3)
    wide = rnd(9, 1024, seed=4).cuda()
    for x in (wide[:, 64:224], wide[::2, 8:168], wide[3:4, 16:176]):
        near(ops.w4_matmul(x, first(w), out_dtype=torch.float32), f64(x) @ v[0].T, np.abs(f64(x)) @ np.abs(v[0]).T, 3)


def test_infinities_and_nan_of_x_stay_in_their_rows(ops):
    w, v = weights(1, 48, 96, 32, False, seed=5)
    codes = oo.w4_unpack(w["codes"][0].cpu().numpy())
    x = rnd(5, 96, seed=6)
    x[1, 7], x[3, 40], x[4, 95] = float("inf"), float("nan"), -float("inf")
    c = f64(ops.w4_matmul(x.cuda(), first(w), out_dtype=torch.float32))
    assert np.isfinite(c[[0, 2]]).all() and np.isnan(c[3]).all()
    for r, k, s in ((1, 7, 1), (4, 95, -1)):
        for n in range(48):       # code 8 stands for 0, and 0 times an infinity is a NaN
            assert np.isnan(c[r, n]) if codes[n, k] == 8 else c[r, n] == s * np.sign(v[0][n, k]) * np.inf


def test_scales_that_are_not_finite_stay_in_their_rows(ops):
    w, v = weights(1, 40, 416, 32, False, seed=5)
    w["scale"][0, 12, 5], w["scale"][0, 0, 9] = float("nan"), float("inf")
    c = f64(ops.w4_matmul(rnd(2, 416, seed=8).cuda(), first(w)))
    assert np.array_equal(~np.isfinite(c).all(0), np.isin(np.arange(40), (5, 9)))


# ------------------------------------------------------------------- layer

def layer(ops, T, d, f, E, k, shared, group, zero, out=torch.float32, seed=0, idx=None):
    x = rnd(T, d, seed=seed + 1)
    w13, v13 = weights(E + shared, 2 * f, d, group, zero, seed + 2)
    wd, vd = weights(E + shared, d, f, group, zero, seed + 3)
    g = torch.Generator().manual_seed(seed)
    if idx is None:
        idx = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32)
    gate = torch.rand(T, idx.shape[1], generator=g) - 0.2
    y = ops.w4_experts(x.cuda(), idx.cuda(), gate.cuda(), w13, wd, n_shared=shared, out_dtype=out)
    add = (24 + max(-(-d // group), (idx.shape[1] + shared) * -(-f // group))) * 2.0 ** -23
    want, bound = oo.w4_experts(f64(x), idx.numpy(), f64(gate), v13, vd, shared, add, 24 if out == torch.float32 else 16)
    err = np.abs(f64(y) - want)
    tol = bound + HALF[out] * (np.abs(want) + bound)
    assert np.all(err <= tol), (np.unravel_index(np.argmax(err - tol), err.shape), err.max())
    return y, (x.cuda(), idx.cuda(), gate.cuda(), w13, wd)


@pytest.mark.parametrize("group,zero", GROUPS)
@pytest.mark.parametrize("T,d,f,E,k,shared", [(1, 32, 32, 1, 1, 0), (1, 256, 160, 8, 3, 1), (3, 96, 288, 5, 2, 0),
                                              (8, 416, 64, 4, 4, 2), (9, 160, 544, 3, 2, 1), (16, 1056, 96, 32, 8, 1),
                                              (64, 128, 96, 6, 3, 1)])
def test_w4_experts(ops, group, zero, T, d, f, E, k, shared):
    layer(ops, T, d, f, E, k, shared, group, zero)
    assert ops.status() == 0


def test_w4_experts_bf16_and_many_experts(ops):
    layer(ops, 4, 256, 96, 256, 8, 1, 128, False, torch.bfloat16)
    layer(ops, 33, 256, 96, 250, 8, 8, 64, True, torch.bfloat16, seed=5)


@pytest.mark.parametrize("rows", [4, 5, 8, 9, 16, 17, 33, 64])
def test_w4_experts_all_tokens_on_one_expert(ops, rows):
    layer(ops, rows, 96, 64, 3, 1, 0, 32, False, idx=torch.full((rows, 1), 2, dtype=torch.int32))


@pytest.mark.parametrize("rows", [2, 3, 4, 8, 16, 24, 64])
def test_w4_experts_whose_tokens_grow_and_shrink(ops, rows):
    """One, then all, then two tokens an expert, over and over: each warp meets tiles with more rows than the one in front."""
    E, k = 60, 8
    idx = torch.full((rows, k), -1, dtype=torch.int32)
    idx[:, 0], idx[:, 1], idx[:, 2] = 1, 30, 58
    for t in range(rows):
        idx[t, 3:] = torch.tensor([2 + (5 * t + j) % 28 if j < 3 else 31 + (3 * t + j) % 27 for j in range(5)])
    layer(ops, rows, 256, 96, E, k, 0, 32, False, idx=idx)
    layer(ops, rows, 96, 288, E, k, 1, 128, True, idx=idx, seed=3)
    assert ops.status() == 0


def test_w4_experts_named_twice_and_out_of_range(ops):
    import mixture_experts_layer_routing_gb300 as moe
    idx = torch.tensor([[1, 1, 1], [0, 2, 0], [2, 3, 3]], dtype=torch.int32)
    layer(ops, 3, 96, 64, 4, 3, 1, 32, False, idx=idx)
    assert ops.status() == 0
    idx = torch.tensor([[1, -1, 4], [7, 1 << 30, -5], [0, 2, 3]], dtype=torch.int32)   # (4 is the shared expert's slot)
    y, _ = layer(ops, 3, 96, 64, 4, 3, 1, 32, False, idx=idx)
    assert ops.status() == moe.MOE_ERR_DEVICE_INDEX
    y, _ = layer(ops, 3, 96, 64, 4, 3, 0, 32, False, idx=torch.full((3, 3), -1, dtype=torch.int32))
    assert ops.status() == moe.MOE_ERR_DEVICE_INDEX and (y == 0).all()


def test_a_token_that_is_not_finite_leaves_the_others(ops):
    y, (x, idx, gate, w13, wd) = layer(ops, 12, 96, 64, 4, 2, 1, 64, False)
    x2 = x.clone()
    x2[5, 3] = float("nan")
    y2 = ops.w4_experts(x2, idx, gate, w13, wd, n_shared=1, out_dtype=torch.float32)
    assert torch.isnan(y2[5]).all()
    keep = [t for t in range(12) if t != 5]
    assert torch.equal(y2[keep], y[keep])


def test_no_tokens(ops):
    _, (x, idx, gate, w13, wd) = layer(ops, 2, 96, 64, 4, 2, 1, 64, False)
    assert ops.w4_experts(x[:0], idx[:0], gate[:0], w13, wd, n_shared=1).shape == (0, 96)
    assert ops.w4_matmul(x[:0], first(w13)).shape == (0, 128)


# ---------------------------------------------- repeats, streams and graphs

def test_repeats_streams_and_graphs_give_the_same_bits(ops):
    y, args = layer(ops, 5, 416, 288, 8, 3, 1, 32, True)
    x, idx, gate, w13, wd = args
    c = ops.w4_matmul(x, first(w13), out_dtype=torch.float32)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        s = streams[i % 3]
        got.append((ops.w4_experts(*args, n_shared=1, out_dtype=torch.float32, stream=s),
                    ops.w4_matmul(x, first(w13), out_dtype=torch.float32, stream=s)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, y) and torch.equal(b, c)
    # two captured graphs, replayed at once
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(ops.w4_experts(*args, n_shared=1, out_dtype=torch.float32))
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, y) for o in outs)
    # other inputs, through the same graph
    x.copy_(rnd(5, 416, seed=77))
    idx.copy_((idx + 1) % 8)
    graphs[0].replay()
    assert torch.equal(outs[0], ops.w4_experts(*args, n_shared=1, out_dtype=torch.float32))
    assert ops.status() == 0


def test_the_layer_behind_the_gate_and_its_two_products(ops):
    """gate() in front, and the same layer from w4_matmul and torch: gate/up by experts' rows, SwiGLU, down, sum."""
    T, d, f, E, k = 6, 256, 160, 8, 3
    W13, Wd = rnd(E, 2 * f, d, seed=1).cuda() / 16, rnd(E, d, f, seed=2).cuda() / 16
    x, logits = rnd(T, d, seed=3).cuda(), torch.randn(T, E, generator=torch.Generator().manual_seed(4)).cuda()
    w13, wd = ops.quant_w4(W13, 64, True), ops.quant_w4(Wd, 64, True)
    r = ops.gate(logits, k, router="sigmoid", route_scale=2.5)
    y = ops.w4_experts(x, r["idx"], r["gate"], w13, wd, out_dtype=torch.float32)
    gu = ops.w4_matmul(x, w13, off=r["off"], row_index=r["perm"] // k, out_dtype=torch.float32)
    h = (torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]).bfloat16()
    o = ops.w4_matmul(h, wd, off=r["off"], out_dtype=torch.float32)
    want = (o[r["inv"].view(T, k).long()] * r["gate"][:, :, None]).sum(1)
    # h is rounded to bf16 here: 2^-8 of a value, summed up in the root mean square
    assert ((y - want).norm() / want.norm()).item() < 2.0 ** -8
    # the weights' rounding: half a step of a fifteenth of a group's range, some 5% of the values
    dense = torch.einsum("tkf,tkdf->tkd", h.float()[r["inv"].view(T, k).long()], Wd.float()[r["idx"].long()])
    assert ((o[r["inv"].view(T, k).long()] - dense).norm() / dense.norm()).item() < 0.15
    assert ops.status() == 0


def test_host_threads_with_other_numbers_of_tokens(ops):
    """One kernel's shared memory differs with the number of tokens: host threads that share the handle and launch at
    once (a ctypes call lets other threads run) get their launches and their results."""
    import ctypes
    import threading

    from mixture_experts_layer_routing_gb300 import ops as mops
    d, f, E, k = 256, 96, 8, 3
    _, (x, idx, gate, w13, wd) = layer(ops, 16, d, f, E, k, 0, 32, False)
    pack = lambda w: mops.moe_w4(w["codes"].data_ptr(), w["scale"].data_ptr(), None, 32)  # noqa: E731
    a, b, cfg = pack(w13), pack(wd), mops.moe_w4_config(E, 0, k, d, f)
    counts = [3, 16, 5, 12]
    want = [ops.w4_experts(x[:T], idx[:T], gate[:T], w13, wd, out_dtype=torch.float32) for T in counts]
    out = [torch.zeros_like(w) for w in want]
    ws = [torch.empty(T * k * 3 * f * 2, dtype=torch.uint8, device="cuda") for T in counts]
    streams, bad = [torch.cuda.Stream() for _ in counts], []
    torch.cuda.synchronize()

    def work(i):
        for _ in range(2000):
            bad.append(ops._lib.moe_w4_experts(ops.h, ctypes.byref(cfg), x.data_ptr(), d, counts[i], idx.data_ptr(),
                                               gate.data_ptr(), ctypes.byref(a), ctypes.byref(b), out[i].data_ptr(), 0,
                                               ws[i].data_ptr(), ctypes.c_void_p(streams[i].cuda_stream)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not any(bad) and ops.status() == 0
    assert all(torch.equal(o, w) for o, w in zip(out, want))
