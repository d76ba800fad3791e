"""Cases, plain forms and 64-bit values of the operators around the expert layer.

Three operators (include/moe_ops.h):
  norm    RMS norm with the residual's addition and an e4m3 output with one fp32
          scale for each 128 values of a row; forward and backward
  route   routing from router logits: softmax or sigmoid scores, a balance bias,
          groups, top-k, renormalised gates, and the dispatch (counts, offsets,
          permutation); forward and backward
  matmul  e4m3 x e4m3 product with a scale for each 1 x 128 block of the rows and
          each 128 x 128 block of the weights, dense and by experts' rows; forward
          and backward (dX from the transposed weight, dW along the token axis)

own selects what run() does: the plain form (torch operations in 32 bits, 64
where a selection is decided) or the library's calls.
"""
import math

import torch

own = False

BLOCK = 128     # values that share a scale
E4M3_MAX = 448.0
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token in front of a d=7168 expert layer: pure latency
        dict(name="norm_decode_T1_d7168", op="norm", dir="fwd", T=1, d=7168, dtype="bf16", residual=True, quant=True),
        # a prefill batch in front of the same layer, keeping what the backward pass needs
        dict(name="norm_prefill_T8192_d7168", op="norm", dir="fwd", T=8192, d=7168, dtype="bf16", residual=True,
             quant=True),
        # the training step of one 2368-token chunk: gradients of the input and the weight
        dict(name="norm_backward_T2368_d7168", op="norm", dir="bwd", T=2368, d=7168, dtype="bf16", residual=True,
             quant=False),
        # the small fp32 layer, no 8-bit output
        dict(name="norm_fp32_T64_d256", op="norm", dir="fwd", T=64, d=256, dtype="fp32", residual=False, quant=False),
        # four decoded tokens, 256 experts in 8 groups of which 4 are kept
        dict(name="route_decode_T4_E256", op="route", dir="fwd", T=4, E=256, k=8, router="sigmoid", renorm=True,
             scale=2.5, groups=8, kept=4, bias=True),
        # a prefill batch of the same router
        dict(name="route_prefill_T8192_E256", op="route", dir="fwd", T=8192, E=256, k=8, router="sigmoid",
             renorm=True, scale=2.5, groups=8, kept=4, bias=True),
        # the training step of the 64-expert softmax router
        dict(name="route_backward_T2048_E64", op="route", dir="bwd", T=2048, E=64, k=6, router="softmax",
             renorm=True, scale=1.0, groups=1, kept=1, bias=False),
        # one decoded token through the shared expert's gate/up weight: reads 29 MB of weights
        dict(name="matmul_decode_M1_N4096_K7168", op="matmul", dir="fwd", M=1, N=4096, K=7168, E=0, k=1, skew=0.0,
             out="bf16"),
        # the shared expert's gate/up product of a prefill batch
        dict(name="matmul_prefill_M8192_N4096_K7168", op="matmul", dir="fwd", M=8192, N=4096, K=7168, E=0, k=1,
             skew=0.0, out="bf16"),
        # 16 decoded tokens, top-8 of 32 experts: about four rows an expert, 0.94 GB of weights
        dict(name="experts_decode_T16_E32", op="matmul", dir="fwd", M=16, N=4096, K=7168, E=32, k=8, skew=0.0,
             out="bf16"),
        # the gate/up product of the 2048-token layer, 64 experts with uneven loads
        dict(name="experts_prefill_T2048_E64", op="matmul", dir="fwd", M=2048, N=2816, K=2048, E=64, k=6, skew=1.0,
             out="bf16"),
        # its backward pass: row gradients and every expert's weight gradient
        dict(name="experts_backward_T2048_E64", op="matmul", dir="bwd", M=2048, N=2816, K=2048, E=64, k=6, skew=1.0,
             out="bf16"),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in lo..hi, spread over the logarithm."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        if lo <= v <= hi and v != 3072:
            return v


def draw(rng):
    op = rng.choice(["norm", "route", "matmul"])
    direction = rng.choice(["fwd", "fwd", "bwd"])
    if op == "norm":
        return dict(op=op, dir=direction, T=_spread(rng, 1, 8192), d=_spread(rng, 64, 7168, 8),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), residual=rng.random() < 0.7,
                    quant=direction == "fwd" and rng.random() < 0.7)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _spread(rng, 4, 256 // groups)
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(8, kept * (E // groups)))
        return dict(op=op, dir=direction, T=_spread(rng, 1, 8192), E=E, k=k,
                    router=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), groups=groups, kept=kept, bias=rng.random() < 0.6)
    E = rng.choice([0, 0, 8, 16, 32, 60])
    few = E > 0 and direction == "bwd"      # every expert's weight gradient is written whole
    N, K = _spread(rng, 64, 2048 if few else 4096, 16), _spread(rng, 128, 2048 if few else 4096 if E else 7168, 16)
    M = _spread(rng, 1, 8192 if E == 0 else 1024)
    return dict(op=op, dir=direction, M=M, N=N, K=K, E=E, k=rng.randint(1, 6) if E else 1,
                skew=rng.choice([0.0, 0.5, 1.0]) if E else 0.0, out=rng.choice(["bf16", "bf16", "fp32"]))


# ------------------------------------------------------------------ inputs

def _quantise(v, dim):
    """(codes, scales) of v (fp32) in blocks of 128 along the dims of the tuple `dim`, the last block shorter."""
    n = [v.shape[i] for i in dim]
    blocks = [-(-m // BLOCK) for m in n]
    pad = [0, 0] * v.dim()
    for i, m, b in zip(dim, n, blocks):
        pad[2 * (v.dim() - 1 - i) + 1] = b * BLOCK - m
    p = torch.nn.functional.pad(v, pad)
    whole, shape, over = p.shape, [], []
    for i in range(p.dim()):
        if i in dim:
            over.append(len(shape) + 1)
            shape += [p.shape[i] // BLOCK, BLOCK]
        else:
            shape.append(p.shape[i])
    p = p.view(shape)
    amax = p.abs().amax(over, keepdim=True)
    # 448 v is exact for bf16 v and a quotient is rounded once, so a value half way between two codes stays there
    q = torch.where(amax > 0, p * E4M3_MAX / amax, 0 * p).reshape(whole)
    q = q[tuple(slice(0, m) for m in v.shape)].to(F8)
    return q.contiguous(), (amax / E4M3_MAX).reshape([s for i, s in enumerate(shape) if i not in over])


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    g, c = _gen(seed), case
    new = lambda dt, *shape: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    if c["op"] == "norm":
        dt, T, d = DTYPES[c["dtype"]], c["T"], c["d"]
        # a residual stream has a few channels far larger than the others
        chan = 1.0 + 20.0 * (torch.rand(d, generator=g, device="cuda") < 0.01).float()
        x, w = (_randn(g, T, d) * chan).to(dt), (1.0 + 0.1 * _randn(g, d)).to(dt)
        res = (3.0 * _randn(g, T, d) * chan).to(dt) if c["residual"] else None
        s = dict(case=c, x=x, w=w, res=res)
        if c["dir"] == "fwd":
            out = dict(y=new(dt, T, d), rstd=new(torch.float32, T))
            if c["residual"]:
                out["h"] = new(dt, T, d)
            if c["quant"]:
                out.update(q=new(F8, T, d), scale=new(torch.float32, T, -(-d // BLOCK)))
        else:
            s["h"] = (x.float() + res.float()).to(dt) if res is not None else x
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
            s["dy"] = _randn(g, T, d).to(dt)
            s["dh"] = _randn(g, T, d).to(dt) if c["residual"] else None
            out = dict(dx=new(dt, T, d), dw=new(torch.float32, d))
        s["out"] = out
        return s
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        logits = 1.5 * _randn(g, T, E)
        bias = 0.05 * _randn(g, E) if c["bias"] else None
        s = dict(case=c, logits=logits, bias=bias)
        if c["dir"] == "fwd":
            i32 = torch.int32
            s["out"] = dict(idx=new(i32, T, k), gate=new(torch.float32, T, k), cnt=new(i32, E), off=new(i32, E + 1),
                            perm=new(i32, T * k), inv=new(i32, T * k))
        else:
            s["idx"] = _select(logits, bias, c)[0]
            s["dgate"] = _randn(g, T, k)
            s["out"] = dict(dlogits=new(torch.float32, T, E))
        return s
    M, N, K, E, k, odt = c["M"], c["N"], c["K"], c["E"], c["k"], DTYPES[c["out"]]
    s = dict(case=c, off=None, row=None, cap=M)
    rows = M
    if E:
        # k distinct experts for each token, loads falling off as 1/rank^skew
        load = -c["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        u = torch.rand(M, E, generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
        pick = (load - torch.log(-torch.log(u))).topk(k, 1).indices.reshape(-1)
        order = torch.sort(pick, stable=True).indices
        cnt = torch.bincount(pick, minlength=E)
        s["off"] = torch.nn.functional.pad(cnt.cumsum(0), (1, 0)).to(torch.int32)
        s["row"] = (order // k).to(torch.int32)
        s["cap"] = int(cnt.max())
        rows = M * k
    w = (_randn(g, max(E, 1), N, K) / math.sqrt(K)).to(torch.bfloat16).float()
    w = w if E else w[0]
    if c["dir"] == "fwd":
        s["a"], s["sa"] = _quantise(_randn(g, M, K).to(torch.bfloat16).float(), (1,))
        s["b"], s["sb"] = _quantise(w, (w.dim() - 2, w.dim() - 1))
        s["out"] = new(odt, rows, N)
    else:
        # the weight laid out for dX: transposed once, with its scales
        q, sc = _quantise(w, (w.dim() - 2, w.dim() - 1))
        s["bt"], s["sbt"] = q.transpose(-1, -2).contiguous(), sc.transpose(-1, -2).contiguous()
        s["x"] = _randn(g, M, K).to(torch.bfloat16)
        s["dc"] = _randn(g, rows, N).to(torch.bfloat16)
        s["out"] = dict(dx=new(torch.bfloat16, rows, K), dw=new(odt, *((E, N, K) if E else (N, K))))
    return s


# -------------------------------------------------------------- plain form

def _select(logits, bias, c):
    """(idx, gate) of the routing, decided and computed in 64 bits: scores next to a border differ by less than
    32 bits hold. Ties go to the lower index; experts whose score is not a number or masked (-inf) come last."""
    T, E, k, G = logits.shape[0], c["E"], c["k"], c["groups"]
    l = logits.double()
    p = torch.softmax(l, 1) if c["router"] == "softmax" else torch.sigmoid(l)
    low = torch.finfo(torch.float64).min
    key = p if bias is None else p + bias.double()
    key = torch.where(torch.isnan(key) | (l == -math.inf), low, key).clamp_min(low)
    if c["kept"] < G:
        per = key.view(T, G, E // G)
        best = torch.sort(per, dim=2, descending=True).values[:, :, :min(2, E // G)].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        key = torch.where(keep[:, :, None], per, -math.inf).view(T, E)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    gate = p.gather(1, idx)
    if c["renorm"]:
        gate = gate / (gate.sum(1, keepdim=True) + 1e-20)
    return idx.to(torch.int32), (c["scale"] * gate).float()


def _plain_norm(s):
    c, w, dt = s["case"], s["w"].float(), s["x"].dtype
    if c["dir"] == "bwd":
        h, dy, r = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
        u, n = dy * w, h * r
        dx = r * (u - n * (u * n).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return dict(dx=dx.to(dt), dw=(dy * n).sum(0))
    out = {}
    h = s["x"]
    if s["res"] is not None:
        h = out["h"] = (h.float() + s["res"].float()).to(dt)
    h = h.float()
    rstd = out["rstd"] = torch.rsqrt(h.square().mean(1) + EPS)
    y = h * rstd[:, None] * w
    out["y"] = y.to(dt)
    if c["quant"]:
        out["q"], out["scale"] = _quantise(y, (1,))
    return out


def _plain_route(s):
    c, logits = s["case"], s["logits"]
    if c["dir"] == "fwd":
        idx, gate = _select(logits, s["bias"], c)
        flat = idx.reshape(-1).long()
        cnt = torch.zeros(c["E"], dtype=torch.int64, device=flat.device).index_add_(0, flat, torch.ones_like(flat))
        perm = torch.sort(flat, stable=True).indices
        inv = torch.empty_like(perm).scatter_(0, perm, torch.arange(flat.numel(), device=flat.device))
        off = torch.nn.functional.pad(cnt.cumsum(0), (1, 0))
        i32 = torch.int32
        return dict(idx=idx, gate=gate, cnt=cnt.to(i32), off=off.to(i32), perm=perm.to(i32), inv=inv.to(i32))
    idx, dg = s["idx"].long(), s["dgate"] * c["scale"]
    p = torch.softmax(logits, 1) if c["router"] == "softmax" else torch.sigmoid(logits)
    ps = p.gather(1, idx)
    if c["renorm"]:
        den = ps.sum(1, keepdim=True) + 1e-20
        dg = (dg - (dg * ps).sum(1, keepdim=True) / den) / den
    dp = torch.zeros_like(logits).scatter_(1, idx, dg)
    if c["router"] == "softmax":
        return dict(dlogits=p * (dp - (p * dp).sum(1, keepdim=True)))
    return dict(dlogits=p * (1 - p) * dp)


def _expand(scale, n):
    return scale.repeat_interleave(BLOCK, -1)[..., :n]


def _values(q, scale, rows=False):
    """fp32 values of codes with scales along the last dim (rows: and along the one before it)."""
    scale = _expand(scale, q.shape[-1])
    if rows:
        scale = scale.repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :]
    return q.float() * scale


def _padded(s):
    """For the rows of each expert, padded to the fullest expert's: their indexes [E, cap], and which are real."""
    off, cap = s["off"].long(), s["cap"]
    at = off[:-1, None] + torch.arange(cap, device=off.device)
    real = at < off[1:, None]
    return at.clamp_max(max(int(s["row"].numel()) - 1, 0)), real


def _plain_matmul(s):
    c, odt = s["case"], DTYPES[s["case"]["out"]]
    grouped = s["off"] is not None
    if grouped:
        at, real = _padded(s)
    if c["dir"] == "fwd":
        a, b = _values(s["a"], s["sa"]), _values(s["b"], s["sb"], rows=True)
        if not grouped:
            return (a @ b.t()).to(odt)
        y = torch.bmm(a[s["row"].long()][at], b.transpose(1, 2))
        return y[real].to(odt)      # row-major over (expert, row of it) is the sorted order
    bt, dc, x = _values(s["bt"], s["sbt"], rows=True), s["dc"].float(), s["x"].float()
    dcr = _values(*_quantise(dc, (1,)))
    if not grouped:
        dct, xt = _values(*_quantise(dc.t().contiguous(), (1,))), _values(*_quantise(x.t().contiguous(), (1,)))
        return dict(dx=(dcr @ bt.t()).to(torch.bfloat16), dw=(dct @ xt.t()).to(odt))
    dx = torch.bmm(dcr[at], bt.transpose(1, 2))[real].to(torch.bfloat16)
    live = real[:, :, None].float()
    dct = _values(*_quantise((dc[at] * live).transpose(1, 2).contiguous(), (2,)))
    xt = _values(*_quantise((x[s["row"].long()][at] * live).transpose(1, 2).contiguous(), (2,)))
    return dict(dx=dx, dw=torch.bmm(dct, xt.transpose(1, 2)).to(odt))


# ------------------------------------------------------------ library calls

def _library(s):
    import mixture_experts_layer_routing_gb300 as moe
    ops, c, out = moe.default_ops(), s["case"], s["out"]
    if c["op"] == "norm":
        if c["dir"] == "fwd":
            return ops.rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS, out=out)
        return ops.rms_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], dh=s["dh"], out=out)
    if c["op"] == "route":
        if c["dir"] == "fwd":
            return ops.gate(s["logits"], c["k"], bias=s["bias"], router=c["router"], renorm=c["renorm"],
                            route_scale=c["scale"], n_groups=c["groups"], topk_groups=c["kept"], out=out)
        return ops.gate_backward(s["logits"], s["idx"], s["dgate"], router=c["router"], renorm=c["renorm"],
                                 route_scale=c["scale"], out=out)
    if c["dir"] == "fwd":
        return ops.fp8_matmul(s["a"], s["sa"], s["b"], s["sb"], off=s["off"], row_index=s["row"], out=out)
    q, sc = ops.quant_rows(s["dc"])
    dx = ops.fp8_matmul(q, sc, s["bt"], s["sbt"], off=s["off"], out=out["dx"])
    dct, sdct = ops.quant_cols(s["dc"], off=s["off"])
    xt, sxt = ops.quant_cols(s["x"], off=s["off"], row_index=s["row"])
    return dict(dx=dx, dw=ops.fp8_wgrad(dct, sdct, xt, sxt, off=s["off"], out=out["dw"]))


def run(state):
    if own:
        return _library(state)
    return {"norm": _plain_norm, "route": _plain_route, "matmul": _plain_matmul}[state["case"]["op"]](state)


# ------------------------------------------------------------ work, 64 bits

def work(case):
    c = case
    if c["op"] == "norm":
        n, e = c["T"] * c["d"], 4 if c["dtype"] == "fp32" else 2
        if c["dir"] == "fwd":
            b = n * e * (2 + (2 if c["residual"] else 0)) + (n + 4 * c["T"] * -(-c["d"] // BLOCK) if c["quant"] else 0)
            return dict(bytes=b + 4 * c["T"] + e * c["d"], flops=6 * n)
        return dict(bytes=n * e * (3 + (1 if c["residual"] else 0)) + 4 * c["T"] + (e + 4) * c["d"], flops=10 * n)
    if c["op"] == "route":
        n, a = c["T"] * c["E"], c["T"] * c["k"]
        if c["dir"] == "fwd":
            return dict(bytes=4 * n + 16 * a + 8 * c["E"] + (4 * c["E"] if c["bias"] else 0), flops=8 * n)
        reads = 4 * n if c["router"] == "softmax" and not c["renorm"] else 4 * a
        return dict(bytes=reads + 4 * n + 8 * a, flops=4 * n)
    M, N, K, E = c["M"], c["N"], c["K"], c["E"]
    rows = M * c["k"] if E else M
    G = min(E, rows) if E else 1       # experts that hold a row, at most
    o = 4 if c["out"] == "fp32" else 2
    scales = lambda r, n: 4 * r * -(-n // BLOCK)  # noqa: E731
    if c["dir"] == "fwd":
        return dict(bytes=M * K + scales(M, K) + G * (N * K + scales(-(-N // BLOCK), K)) + rows * N * o,
                    flops=2 * rows * N * K)
    return dict(bytes=2 * rows * N + 2 * M * K + G * (N * K + scales(-(-K // BLOCK), N)) + 2 * rows * K
                + max(E, 1) * N * K * o, flops=4 * rows * N * K)


def _e4m3(v):
    """v (64 bits, |v| <= 448) rounded to the nearest e4m3 value, ties to even: 3 mantissa bits, exponents from -6."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -9))).clamp_min(-6)
    step = torch.exp2(e - 3)
    r = torch.round(v / step) * step       # torch.round takes ties to even
    return r.clamp(-E4M3_MAX, E4M3_MAX)


def _blocks64(v):
    """Values in 64 bits of v quantised in blocks of 128 along the last dim, with (codes, scales)."""
    codes, scales = [], []
    for part in torch.split(v, BLOCK, -1):
        amax = part.abs().amax(-1, keepdim=True)
        codes.append(_e4m3(torch.where(amax > 0, part * E4M3_MAX / amax, 0.0 * part)))
        scales.append(amax / E4M3_MAX)
    q, sc = torch.cat(codes, -1), torch.cat(scales, -1)
    wide = torch.cat([c * m for c, m in zip(codes, scales)], -1)
    return wide, q, sc


def _weights64(q, scale):
    """[N, K] codes and [ceil(N/128), ceil(K/128)] scales."""
    n, k = q.shape
    i = torch.arange(n, device=q.device) // BLOCK
    j = torch.arange(k, device=q.device) // BLOCK
    return q.double() * scale.double()[i][:, j]


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        w = s["w"].double()
        if c["dir"] == "bwd":
            h, dy = s["h"].double(), s["dy"].double()
            n = h * s["rstd"].double()[:, None]
            g = w * dy
            dx = s["rstd"].double()[:, None] * (g - n * ((g * n).sum(1, keepdim=True) / c["d"]))
            return dict(dx=dx + s["dh"].double() if s["dh"] is not None else dx, dw=torch.einsum("td,td->d", dy, n))
        h = s["x"].double()
        out = {}
        if s["res"] is not None:
            h = (h + s["res"].double()).to(s["x"].dtype).double()   # the stored sum is what is normalised
            out["h"] = h
        r = 1.0 / torch.sqrt((h * h).sum(1) / c["d"] + EPS)
        y = h * r[:, None] * w
        out.update(rstd=r, y=y)
        if c["quant"]:
            _, out["q"], out["scale"] = _blocks64(y)
        return out
    if c["op"] == "route":
        l = s["logits"].double()
        if c["router"] == "softmax":
            e = torch.exp(l - l.max(1, keepdim=True).values)
            p = e / e.sum(1, keepdim=True)
        else:
            p = 1.0 / (1.0 + torch.exp(-l))
        idx = (s["idx"] if c["dir"] == "bwd" else _select(s["logits"], s["bias"], c)[0]).long()
        hot = torch.zeros_like(p).scatter_(1, idx, 1.0)
        den = (p * hot).sum(1, keepdim=True) if c["renorm"] else torch.ones_like(p[:, :1])
        if c["dir"] == "fwd":
            return dict(idx=None, gate=c["scale"] * torch.gather(p / den, 1, idx), cnt=None, off=None, perm=None,
                        inv=None)
        g = torch.zeros_like(p).scatter_(1, idx, c["scale"] * s["dgate"].double())
        # sum_j dgate_j gate_j with gate_j = p_j / den
        dp = hot * (g - (g * p).sum(1, keepdim=True) / den) / den if c["renorm"] else g
        if c["router"] == "sigmoid":
            return dict(dlogits=dp * p * (1 - p))
        return dict(dlogits=p * dp - p * (p * dp).sum(1, keepdim=True))
    E = c["E"]
    off = s["off"].tolist() if E else [0, c["M"]]
    if c["dir"] == "fwd":
        a = torch.cat([p.double() * s["sa"][:, i:i + 1].double()
                       for i, p in enumerate(torch.split(s["a"].float(), BLOCK, 1))], 1)
        if E:
            a = a[s["row"].long()]
        parts = []
        for e in range(max(E, 1)):
            w = _weights64(s["b"][e] if E else s["b"], s["sb"][e] if E else s["sb"])
            parts.append(a[off[e]:off[e + 1]] @ w.t())
        return torch.cat(parts)
    dc, x = s["dc"].double(), s["x"].double()
    if E:
        x = x[s["row"].long()]
    dcr = _blocks64(dc)[0]
    dx, dw = [], torch.zeros(max(E, 1), c["N"], c["K"], dtype=torch.float64, device="cuda")
    for e in range(max(E, 1)):
        lo, hi = off[e], off[e + 1]
        w = _weights64(s["bt"][e] if E else s["bt"], s["sbt"][e] if E else s["sbt"])
        dx.append(dcr[lo:hi] @ w.t())
        if hi > lo:
            dw[e] = _blocks64(dc[lo:hi].t())[0] @ _blocks64(x[lo:hi].t())[0].t()
    return dict(dx=torch.cat(dx), dw=dw if E else dw[0])
