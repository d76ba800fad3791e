"""Quantisers and products of e4m3 operands against the 64-bit restatement (GPU).

Quantisers: codes and scales equal (bf16 values: every step of the definition is exact or rounded once).
Products: fp32 sums. Within a block of 128 the tensor core adds four partial sums, each block's sum is then added
to the total: under (8 + blocks) additions in a row, each off by at most 2^-23 (a truncated addition) of the sum of
magnitudes; then the rounding to the output's type.
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


def rnd(*shape, seed=0, spread=False):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(*shape, generator=g)
    if spread:   # block maxima of very different sizes
        v = v * torch.exp2(torch.randint(-12, 12, (shape[0], 1), generator=g).float())
    return v.to(torch.bfloat16)


def f64(t):
    return t.float().double().cpu().numpy()


def near(got, want, size, blocks):
    err = np.abs(f64(got) - want)
    tol = (8 + blocks) * 2.0 ** -23 * size + HALF[got.dtype] * np.abs(want)
    assert np.all(err <= tol), (np.unravel_index(np.argmax(err - tol), err.shape), err.max())


def make_off(cnt):
    return torch.tensor(np.concatenate([[0], np.cumsum(cnt)]), dtype=torch.int32)


# -------------------------------------------------------------- quantisers

@pytest.mark.parametrize("T,C", [(1, 8), (3, 128), (5, 136), (2, 7168), (300, 1408), (129, 2048)])
def test_quant_rows(ops, T, C):
    x = rnd(T, C, seed=T + C, spread=True)
    x[0, :min(C, 128)] = 0
    q, s = ops.quant_rows(x.cuda())
    wq, ws = oo.quantise(f64(x), 1)
    assert np.array_equal(f64(q), wq) and np.array_equal(f64(s), ws)


def test_quant_rows_strided_and_not_finite(ops):
    wide = rnd(17, 1024, seed=1).cuda()
    x = wide[:, 64:64 + 400]
    q, s = ops.quant_rows(x)
    wq, ws = oo.quantise(f64(x), 1)
    assert np.array_equal(f64(q), wq) and np.array_equal(f64(s), ws)
    y = rnd(4, 256, seed=2)
    y[0, 3], y[1, 200], y[2, 0] = float("nan"), float("inf"), -float("inf")
    q, s = ops.quant_rows(y.cuda())
    back = f64(q) * np.repeat(f64(s), 128, 1)
    for t, b in [(0, 0), (1, 1), (2, 0)]:
        assert np.isnan(back[t, b * 128:(b + 1) * 128]).all()
        assert np.isfinite(back[t, (1 - b) * 128:(2 - b) * 128]).all()
    assert np.isfinite(back[3]).all()


def test_quant_rows_swiglu(ops):
    x = rnd(40, 2 * 264, seed=3).cuda()
    q, s = ops.quant_rows(x, swiglu=True)
    g, u = f64(x)[:, :264], f64(x)[:, 264:]
    h = g / (1 + np.exp(-g)) * u
    wide = np.repeat(f64(s), 128, 1)[:, :264]
    # silu in fp32 with fast exp and division: within 2^-20
    assert np.all(np.abs(f64(q) * wide - h) <= (2.0 ** -4 + 2.0 ** -18) * np.abs(h) + 2.0 ** -10 * wide)


@pytest.mark.parametrize("T,C,cnt", [(1, 8, None), (128, 64, None), (129, 72, None), (300, 200, None),
                                     (300, 136, [0, 1, 127, 128, 0, 44, 0]), (257, 64, [129, 0, 128])])
@pytest.mark.parametrize("gather", [False, True])
def test_quant_cols(ops, T, C, cnt, gather):
    src = rnd(90 if gather else T, C, seed=T + C, spread=True)
    index = torch.randint(0, 90, (T,), generator=torch.Generator().manual_seed(4), dtype=torch.int32)
    off = None if cnt is None else make_off(cnt)
    q, s = ops.quant_cols(src.cuda(), off=None if off is None else off.cuda(), row_index=index.cuda() if gather else None)
    x = f64(src)[index.long().numpy()] if gather else f64(src)
    at = 0
    ends = [0, T] if off is None else off.tolist()
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


@pytest.mark.parametrize("N,K,G", [(128, 128, 1), (8, 16, 1), (200, 136, 2), (264, 400, 3), (1408, 256, 1)])
def test_quant_blocks(ops, N, K, G):
    w = rnd(G, N, K, seed=N + K)
    w[0, :8] *= 64
    out = ops.quant_blocks(w.cuda(), transpose=True)
    for g in range(G):
        wq, ws = oo.quantise_blocks(f64(w[g]))
        assert np.array_equal(f64(out["q"][g]), wq) and np.array_equal(f64(out["scale"][g]), ws)
        assert np.array_equal(f64(out["qt"][g]), wq.T) and np.array_equal(f64(out["scale_t"][g]), ws.T)
    flat = ops.quant_blocks(w[0].contiguous().cuda())
    assert torch.equal(flat["q"].float(), out["q"][0].float()) and torch.equal(flat["scale"], out["scale"][0])


# ---------------------------------------------------------------- products

def operands(ops, rows, N, K, G, seed):
    a, b = rnd(rows, K, seed=seed, spread=True), rnd(max(G, 1), N, K, seed=seed + 1)
    q, s = ops.quant_rows(a.cuda())
    w = ops.quant_blocks(b.cuda() if G else b[0].cuda().contiguous())
    A = oo.values(f64(q), f64(s))
    B = oo.values(f64(w["q"]), f64(w["scale"]), (-2, -1))
    return q, s, w, A, B


@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (1, 8, 16), (2, 264, 400), (13, 72, 144), (16, 128, 1024),
                                   (17, 200, 256), (40, 384, 528), (64, 136, 2048), (65, 264, 128), (100, 512, 272),
                                   (128, 256, 1024), (129, 520, 640), (300, 77, 256), (333, 1000, 1408), (3, 4096, 7168),
                                   (16, 520, 17408)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matmul(ops, M, N, K, dtype):
    a = rnd(M, K, seed=M + N, spread=True)
    b = rnd(N, K, seed=K)
    q, s = ops.quant_rows(a.cuda())
    wq, ws = oo.quantise_blocks(f64(b))
    bq = torch.from_numpy(wq).float().to(torch.float8_e4m3fn).cuda()
    bs = torch.from_numpy(ws).float().cuda()
    got = ops.fp8_matmul(q, s, bq, bs, out_dtype=dtype)
    want, size = oo.matmul(oo.values(f64(q), f64(s)), oo.values(wq, ws, (0, 1)))
    near(got, want, size, -(-K // 128))
    assert ops.status() == 0


COUNTS = [[5], [0, 3, 0, 0, 9, 1, 16, 0], [17, 0, 40, 33], [64, 65, 0, 1], [200, 0, 129, 128, 1, 0], [0, 0, 300, 0]]


@pytest.mark.parametrize("cnt", COUNTS)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(264, 400), (512, 1024)])
def test_matmul_by_experts(ops, cnt, gather, N, K):
    M, G = sum(cnt), len(cnt)
    rows = 50 if gather else M
    q, s, w, A, B = operands(ops, rows, N, K, G, seed=M + N)
    off = make_off(cnt)
    index = torch.randint(0, rows, (M,), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    got = ops.fp8_matmul(q, s, w["q"], w["scale"], off=off.cuda(), row_index=index.cuda() if gather else None)
    want, size = oo.matmul(A, B, off.tolist(), index.long().numpy() if gather else None)
    near(got, want, size, -(-K // 128))
    assert ops.status() == 0


@pytest.mark.parametrize("per", [3, 100])
def test_many_experts(ops, per):
    rng = np.random.default_rng(6)
    cnt = rng.integers(0, 2 * per, 256)
    M = int(cnt.sum())
    q, s, w, A, B = operands(ops, M, 136, 256, 256, seed=7)
    off = make_off(cnt)
    got = ops.fp8_matmul(q, s, w["q"], w["scale"], off=off.cuda(), out_dtype=torch.float32)
    want, size = oo.matmul(A, B, off.tolist())
    near(got, want, size, 2)
    assert ops.status() == 0


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("G,most,N,K", [(40, 33, 1100, 272), (160, 24, 72, 400), (20, 130, 2056, 144)])
def test_few_rows_of_many_tiles(ops, G, most, N, K, gather):
    """Short segments whose weights alone fill the GPU with tiles of the wide kernel."""
    cnt = np.random.default_rng(G).integers(0, most, G).tolist()
    M = sum(cnt)
    rows = 50 if gather else M
    b = rnd(G, N, K, seed=51)
    q, s = ops.quant_rows(rnd(rows, K, seed=50, spread=True).cuda())
    wq, ws = map(np.stack, zip(*(oo.quantise_blocks(f64(b[g])) for g in range(G))))   # (widths that 8 does not divide)
    w = dict(q=torch.from_numpy(wq).float().to(torch.float8_e4m3fn).cuda(), scale=torch.from_numpy(ws).float().cuda())
    A, B = oo.values(f64(q), f64(s)), oo.values(wq, ws, (-2, -1))
    off = make_off(cnt)
    index = torch.randint(0, rows, (M,), generator=torch.Generator().manual_seed(6), dtype=torch.int32)
    got = ops.fp8_matmul(q, s, w["q"], w["scale"], off=off.cuda(), row_index=index.cuda() if gather else None)
    want, size = oo.matmul(A, B, off.tolist(), index.long().numpy() if gather else None)
    near(got, want, size, -(-K // 128))
    assert ops.status() == 0


@pytest.mark.parametrize("M", [8, 32, 33, 64])
@pytest.mark.parametrize("gather", [False, True])
def test_few_rows_of_one_wide_matrix(ops, M, gather):
    rows = 50 if gather else M
    q, s, w, A, B = operands(ops, rows, 10016, 272, 0, seed=51)
    index = torch.randint(0, rows, (M,), generator=torch.Generator().manual_seed(7), dtype=torch.int32)
    got = ops.fp8_matmul(q, s, w["q"], w["scale"], row_index=index.cuda() if gather else None)
    want, size = oo.matmul(A[index.long().numpy()] if gather else A, B)
    near(got, want, size, 3)
    assert ops.status() == 0


@pytest.mark.parametrize("M,N,K,cnt", [(100, 40000, 2048, None), (700, 16384, 2176, None),
                                       (1500, 8192, 1536, [200, 0, 700, 130, 470])])
def test_many_tiles_a_cta(ops, M, N, K, cnt):
    """Several tiles for every CTA of the wide kernel, each of many blocks of the reduction (rows sampled)."""
    q, s, w, A, B = operands(ops, M, N, K, len(cnt) if cnt else 0, seed=30)
    off = make_off(cnt).tolist() if cnt else [0, M]
    got = ops.fp8_matmul(q, s, w["q"], w["scale"], off=make_off(cnt).cuda() if cnt else None)
    assert ops.status() == 0
    for g, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        rows = np.unique(np.linspace(lo, hi - 1, 7).astype(int)) if hi > lo else []
        if len(rows):
            b = B[g] if cnt else B
            near(got[torch.from_numpy(rows).cuda()], A[rows] @ b.T, np.abs(A[rows]) @ np.abs(b).T, -(-K // 128))


def test_many_tiles_of_weight_gradients(ops):
    cnt, N, K = [900, 0, 300, 1500], 1024, 4096
    off = make_off(cnt)
    dc, x = rnd(2700, N, seed=31), rnd(2700, K, seed=32)
    dq, ds = ops.quant_cols(dc.cuda(), off=off.cuda())
    xq, xs = ops.quant_cols(x.cuda(), off=off.cuda())
    got = ops.fp8_wgrad(dq, ds, xq, xs, off=off.cuda(), tokens=2700)
    assert ops.status() == 0
    rows = np.arange(0, N, 37)
    for g, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        if lo == hi:
            assert not got[g].any()
            continue
        d = oo.values(*oo.quantise(f64(dc)[lo:hi][:, rows], 0), 0)
        v = oo.values(*oo.quantise(f64(x)[lo:hi], 0), 0)
        near(got[g][torch.from_numpy(rows).cuda()], d.T @ v, np.abs(d).T @ np.abs(v), -(-(hi - lo) // 128))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [77, 264, 1000])
@pytest.mark.parametrize("cnt", [None, [700, 3, 1300, 37]])
def test_long_segments(ops, dtype, N, cnt):
    """Pairs of CTAs: 512 rows a segment and more, with ends inside a tile and inside a warp's 32 rows, and widths that
    its 128-byte stores divide, that they do not, and that cannot be stored 16 bytes at a time."""
    K, G = 400, len(cnt) if cnt else 1
    M = sum(cnt) if cnt else 1111
    a = rnd(M, K, seed=40, spread=True)
    b = rnd(G, N, K, seed=41)
    q, s = ops.quant_rows(a.cuda())
    wq, ws = map(np.stack, zip(*(oo.quantise_blocks(f64(b[g])) for g in range(G))))
    bq, bs = torch.from_numpy(wq).float().to(torch.float8_e4m3fn).cuda(), torch.from_numpy(ws).float().cuda()
    off = make_off(cnt) if cnt else None
    out = torch.full((M + 8, N), 7.0, dtype=dtype, device="cuda")
    got = ops.fp8_matmul(q, s, bq if cnt else bq[0], bs if cnt else bs[0], off=None if off is None else off.cuda(),
                         out=out[:M])
    A, B = oo.values(f64(q), f64(s)), oo.values(wq, ws, (-2, -1))
    want, size = oo.matmul(A, B if cnt else B[0], None if off is None else off.tolist())
    near(got, want, size, 4)
    assert torch.equal(out[M:], torch.full_like(out[M:], 7.0)) and ops.status() == 0


def test_outputs_past_32_bits(ops):
    """70,000 x 32,768 values: the last rows' offsets pass 2^31."""
    M, N, K = 70000, 32768, 128
    q, s, w, _, B = operands(ops, 600, N, K, 0, seed=42)
    index = torch.arange(M, dtype=torch.int32) % 600
    got = ops.fp8_matmul(q, s, w["q"], w["scale"], row_index=index.cuda())
    A = oo.values(f64(q), f64(s))
    for m in (0, 40000, 65535, 65536, 69999):
        near(got[m:m + 1], A[m % 600][None] @ B.T, np.abs(A[m % 600][None]) @ np.abs(B).T, 1)
    del got
    assert ops.status() == 0


def test_rows_of_no_segment_stay(ops):
    q, s, w, A, B = operands(ops, 300, 128, 256, 3, seed=8)
    for off in ([0, 10, 12, 40], [0, 100, 230, 260]):
        out = torch.full((300, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        ops.fp8_matmul(q, s, w["q"], w["scale"], off=torch.tensor(off, dtype=torch.int32).cuda(), out=out)
        want, size = oo.matmul(A, B, off)
        near(out[:off[-1]], want, size, 2)
        assert torch.equal(out[off[-1]:], torch.full_like(out[off[-1]:], 7.0))


@pytest.mark.parametrize("M", [20, 300])
def test_bad_offsets_and_indexes_are_recorded(ops, M):
    """The kernels' own checks: offsets that do not ascend within the rows write nothing, a row index out of range
    reads zeros."""
    import mixture_experts_layer_routing_gb300 as moe
    q, s, w, A, B = operands(ops, M, 128, 256, 2, seed=9)
    for off in ([0, M + 1, M], [0, 8, M + 5], [-4, 8, M], [0, 9, 8]):
        out = torch.full((M, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        ops.fp8_matmul(q, s, w["q"], w["scale"], off=torch.tensor(off, dtype=torch.int32).cuda(), out=out)
        assert ops.status() == moe.MOE_ERR_DEVICE_INDEX
        assert torch.equal(out, torch.full_like(out, 7.0))
    index = torch.arange(M, dtype=torch.int32)
    index[3], index[7] = M, -1
    off = torch.tensor([0, 5, M], dtype=torch.int32)
    got = ops.fp8_matmul(q, s, w["q"], w["scale"], off=off.cuda(), row_index=index.cuda())
    assert ops.status() == moe.MOE_ERR_DEVICE_INDEX
    A[3], A[7] = 0, 0
    want, size = oo.matmul(A, B, off.tolist())
    near(got, want, size, 2)


def test_a_nan_stays_in_its_row(ops):
    for M in (8, 200):
        a = rnd(M, 256, seed=10)
        a[5, 9] = float("nan")
        q, s = ops.quant_rows(a.cuda())
        w = ops.quant_blocks(rnd(128, 256, seed=11).cuda())
        got = ops.fp8_matmul(q, s, w["q"], w["scale"])
        assert torch.isnan(got[5]).all() and torch.isfinite(got[:5]).all() and torch.isfinite(got[6:]).all()


@pytest.mark.parametrize("T,N,K,cnt", [(1, 8, 16, None), (130, 136, 264, None), (700, 256, 512, None),
                                       (300, 200, 72, [0, 1, 127, 128, 0, 44, 0]), (900, 264, 520, [400, 0, 500]),
                                       (64, 128, 256, [64])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wgrad(ops, T, N, K, cnt, dtype):
    dc, x = rnd(T, N, seed=12, spread=True), rnd(90, K, seed=13)
    index = torch.randint(0, 90, (T,), generator=torch.Generator().manual_seed(14), dtype=torch.int32)
    off = None if cnt is None else make_off(cnt).cuda()
    dq, ds = ops.quant_cols(dc.cuda(), off=off)
    xq, xs = ops.quant_cols(x.cuda(), off=off, row_index=index.cuda())
    got = ops.fp8_wgrad(dq, ds, xq, xs, off=off, tokens=T, out_dtype=dtype)
    xr = f64(x)[index.long().numpy()]
    ends = [0, T] if cnt is None else off.tolist()
    for g, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        one = got if cnt is None else got[g]
        if lo == hi:
            assert not one.any()
            continue
        d, v = oo.values(*oo.quantise(f64(dc)[lo:hi], 0), 0), oo.values(*oo.quantise(xr[lo:hi], 0), 0)
        near(one, d.T @ v, np.abs(d).T @ np.abs(v), -(-(hi - lo) // 128))
    assert ops.status() == 0


def test_gradients_against_differences(ops):
    """dX and dW of sum(dc * c), c = a b^T of unquantised values, up to the operands' own rounding to e4m3."""
    a, b, dc = rnd(200, 256, seed=15), rnd(128, 256, seed=16), rnd(200, 128, seed=17)
    w = ops.quant_blocks(b.cuda(), transpose=True)
    dx = ops.fp8_matmul(*ops.quant_rows(dc.cuda()), w["qt"], w["scale_t"], out_dtype=torch.float32)
    dw = ops.fp8_wgrad(*ops.quant_cols(dc.cuda()), *ops.quant_cols(a.cuda()), out_dtype=torch.float32)
    A, B, D = f64(a), f64(b), f64(dc)
    loss = lambda p, q: (p @ q.T * D).sum()  # noqa: E731
    rng = np.random.default_rng(18)
    for _ in range(20):
        i, j, n = rng.integers(200), rng.integers(256), rng.integers(128)
        up, dn = A.copy(), A.copy()
        up[i, j] += 0.5
        dn[i, j] -= 0.5
        size = np.abs(D[i]) @ np.abs(B[:, j])
        assert abs(loss(up, B) - loss(dn, B) - f64(dx)[i, j]) <= (2 * 2.0 ** -4 + 2.0 ** -7) * size
        up, dn = B.copy(), B.copy()
        up[n, j] += 0.5
        dn[n, j] -= 0.5
        size = np.abs(D[:, n]) @ np.abs(A[:, j])
        assert abs(loss(A, up) - loss(A, dn) - f64(dw)[n, j]) <= (2 * 2.0 ** -4 + 2.0 ** -7) * size


def test_another_stream_graph_and_repeats(ops):
    cnt = [30, 0, 200, 70]
    off = make_off(cnt).cuda()
    x, dc, w = rnd(300, 512, seed=19).cuda(), rnd(300, 256, seed=20).cuda(), rnd(4, 256, 512, seed=21).cuda()
    def step():
        k = ops.quant_blocks(w, transpose=True)
        y = ops.fp8_matmul(*ops.quant_rows(x), k["q"], k["scale"], off=off)
        dx = ops.fp8_matmul(*ops.quant_rows(dc), k["qt"], k["scale_t"], off=off)
        dw = ops.fp8_wgrad(*ops.quant_cols(dc, off=off), *ops.quant_cols(x, off=off), off=off)
        return y, dx, dw
    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, cap):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert ops.status() == 0


def test_python_refusals(ops):
    q, s, w, _, _ = operands(ops, 8, 128, 256, 2, seed=22)
    off = torch.tensor([0, 4, 8], dtype=torch.int32).cuda()
    with pytest.raises(TypeError):
        ops.fp8_matmul(q.float(), s, w["q"], w["scale"], off=off)
    with pytest.raises(ValueError):
        ops.fp8_matmul(q, s, w["q"], w["scale"])                       # three dimensions without off
    with pytest.raises(ValueError):
        ops.fp8_matmul(q, s[:, :1].contiguous(), w["q"], w["scale"], off=off)
    with pytest.raises(ValueError):
        ops.fp8_matmul(q, s, w["q"], w["scale"], off=off[:2])
    with pytest.raises(TypeError):
        ops.fp8_matmul(q, s, w["q"], w["scale"], off=off.long())
    with pytest.raises(TypeError):
        ops.fp8_matmul(q, s, w["q"], w["scale"], off=off, out=torch.empty(8, 128, dtype=torch.float16, device="cuda"))
    with pytest.raises(TypeError):
        ops.quant_rows(torch.randn(4, 64).cuda())
    with pytest.raises(RuntimeError):
        ops.quant_rows(rnd(4, 60).cuda())


@pytest.mark.parametrize("M,G,N", [(24, 3, 128), (300, 2, 128), (1500, 2, 264), (200, 40, 1100)])
def test_indexes_of_rows_of_no_segment_are_not_read(ops, M, G, N):
    """An index list of fixed length, -1 where it holds no row: before the first segment and behind the last, whichever
    kernel takes the product."""
    K, rows = 256, 50
    b = rnd(G, N, K, seed=61)
    q, s = ops.quant_rows(rnd(rows, K, seed=60, spread=True).cuda())
    wq, ws = map(np.stack, zip(*(oo.quantise_blocks(f64(b[g])) for g in range(G))))
    bq, bs = torch.from_numpy(wq).float().to(torch.float8_e4m3fn).cuda(), torch.from_numpy(ws).float().cuda()
    A, B = oo.values(f64(q), f64(s)), oo.values(wq, ws, (-2, -1))
    lo, hi = 3, M - 5
    off = torch.linspace(lo, hi, G + 1).int()
    index = torch.full((M,), -1, dtype=torch.int32)
    index[lo:hi] = torch.randint(0, rows, (hi - lo,), generator=torch.Generator().manual_seed(8), dtype=torch.int32)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.fp8_matmul(q, s, bq, bs, off=off.cuda(), row_index=index.cuda(), out=out)
    assert ops.status() == 0
    for g, (a, z) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        r = A[index[a:z].long().numpy()]
        near(out[a:z], r @ B[g].T, np.abs(r) @ np.abs(B[g]).T, 2)
    for part in (out[:lo], out[hi:]):
        assert torch.equal(part, torch.full_like(part, 7.0))
    x = rnd(rows, 136, seed=62).cuda()
    q1, s1 = ops.quant_cols(x, off=off.cuda(), row_index=index.cuda())
    assert ops.status() == 0
