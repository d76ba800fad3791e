"""Cases, plain forms and 64-bit values of the expert FFN's operators on compact storage.

Three operators (include/moe_ops.h):
  w4       products of few rows with 4-bit weights and a scale (and zero point) for
           each group of 32, 64 or 128 values, dense and by experts' rows
  experts  the experts' layer of a few tokens on such weights, behind the routing:
           gate/up products, SwiGLU, down products and the weighted sum
  save     SwiGLU with an 8-bit checkpoint of its input, its backward pass from the
           checkpoint, and 8-bit rows quantised anew along the token axis

own selects what run() does: the plain form (torch operations in 32 bits) or the
library's calls.
"""
import math

import torch

own = False

BLOCK = 128     # values that share a scale of the 8-bit forms
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through the shared expert's gate/up weight: 15 MB of codes
        dict(name="w4_decode_M1_N4096_K7168", op="w4", M=1, N=4096, K=7168, E=0, k=1, skew=0.0, group=128, zero=False,
             out="bf16"),
        # eight sequences decoded together through its down weight, small groups with zero points
        dict(name="w4_decode_M8_N7168_K2048_zero", op="w4", M=8, N=7168, K=2048, E=0, k=1, skew=0.0, group=32, zero=True,
             out="bf16"),
        # a small odd layer, more rows than a tile, fp32 output
        dict(name="w4_M33_N1000_K1056_fp32", op="w4", M=33, N=1000, K=1056, E=0, k=1, skew=0.0, group=64, zero=False,
             out="fp32"),
        # 16 decoded tokens, top-8 of 32 experts, uneven loads: 0.47 GB of codes
        dict(name="w4_experts_T16_E32", op="w4", M=16, N=4096, K=7168, E=32, k=8, skew=0.5, group=128, zero=False,
             out="bf16"),
        # one decoded token through a d=7168 layer, 8 experts and the shared one: 198 MB of codes
        dict(name="layer_T1_d7168_E32+1", op="experts", T=1, d=7168, f=2048, E=32, shared=1, k=8, group=128, zero=False,
             out="bf16"),
        # 16 sequences decoded together, every expert in use
        dict(name="layer_T16_d7168_E32+1", op="experts", T=16, d=7168, f=2048, E=32, shared=1, k=8, group=32, zero=False,
             out="bf16"),
        # four tokens of the 64-expert d=2048 layer, zero points
        dict(name="layer_T4_d2048_E64", op="experts", T=4, d=2048, f=1408, E=64, shared=0, k=6, group=64, zero=True,
             out="bf16"),
        # the rows of a 2048-token step of that layer (top-6), forward: act's codes and the checkpoint
        dict(name="save_forward_R12288_f1408", op="save", dir="fwd", R=12288, f=1408, act=False, quant=True, E=0),
        # a few rows of an odd width, act in bf16
        dict(name="save_forward_R77_f200", op="save", dir="fwd", R=77, f=200, act=True, quant=False, E=0),
        # the same step's backward pass: gradients by rows and along tokens, act along tokens, the gates' gradient
        dict(name="save_backward_R12288_f1408_E64", op="save", dir="bwd", R=12288, f=1408, E=64, skew=1.0, dgu=False,
             rows=True, cols=True, gate=True),
        # a small batch whose products stay in bf16
        dict(name="save_backward_R301_f392", op="save", dir="bwd", R=301, f=392, E=0, skew=0.0, dgu=True, rows=False,
             cols=False, gate=True),
        # the norm's 8-bit rows of 2048 tokens, gathered by experts' rows, for the gate/up weights' gradient
        dict(name="save_columns_R12288_C2048_E64", op="save", dir="cols", R=12288, f=2048, tokens=2048, E=64, skew=1.0),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in lo..hi, spread over the logarithm."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        if lo <= v <= hi:
            return v


def draw(rng):
    op = rng.choice(["w4", "experts", "save"])
    group, zero = rng.choice([32, 64, 128]), rng.random() < 0.4
    out = rng.choice(["bf16", "bf16", "fp32"])
    if op == "w4":
        E = rng.choice([0, 0, 8, 16, 32, 60])
        wide = 4096 if E else 7168
        return dict(op=op, M=_spread(rng, 1, 64), N=_spread(rng, 64, wide, 8), K=_spread(rng, 64, wide, 32), E=E,
                    k=rng.randint(1, 6) if E else 1, skew=rng.choice([0.0, 0.5, 1.0]) if E else 0.0, group=group,
                    zero=zero, out=out)
    if op == "experts":
        E = _spread(rng, 8, 48)
        return dict(op=op, T=_spread(rng, 1, 64), d=_spread(rng, 256, 4096, 32), f=_spread(rng, 128, 2048, 32), E=E,
                    shared=rng.choice([0, 1]), k=rng.randint(1, 8), group=group, zero=zero, out=out)
    direction = rng.choice(["fwd", "bwd", "bwd", "cols"])
    R, f = _spread(rng, 1, 8192), _spread(rng, 64, 2048, 8)
    E = rng.choice([0, 8, 60])
    if direction == "fwd":
        act = rng.random() < 0.5
        return dict(op=op, dir=direction, R=R, f=f, act=act, quant=not act or rng.random() < 0.5, E=0)
    skew = rng.choice([0.0, 1.0])
    if direction == "cols":
        return dict(op=op, dir=direction, R=R, f=f, tokens=rng.randint(1, R) if rng.random() < 0.6 else 0, E=E, skew=skew)
    rows = rng.random() < 0.6
    if rows:
        f = _spread(rng, 128, 2048, 128)
    cols = rng.random() < 0.6
    return dict(op=op, dir=direction, R=R, f=f, E=E, skew=skew, dgu=not (rows or cols) or rng.random() < 0.3, rows=rows,
                cols=cols, gate=rng.random() < 0.6)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 23)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _pack(codes):
    """Codes 0..15 [..., K] as words of eight: value 2i in bits 4i.., value 2i + 1 in bits 16 + 4i.."""
    c = codes.to(torch.int64).unflatten(-1, (-1, 8))
    at = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=codes.device)
    w = (c << at).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _unpack(words):
    at = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=words.device, dtype=torch.int32)
    return ((words[..., None] >> at) & 15).flatten(-2)


def _weights4(g, n, N, K, group, zero):
    """n matrices [N, K] quantised to 4 bits: dict of codes, scale, zero and group."""
    codes, scales, zeros = [], [], []
    Kp = -(-K // group) * group
    for _ in range(n):
        # a few columns are larger than the others, as in trained weights
        w = _randn(g, N, K) / math.sqrt(K) * (1.0 + 2.0 * (torch.rand(K, generator=g, device="cuda") < 0.01).float())
        w = torch.nn.functional.pad(w, (0, Kp - K)).view(N, Kp // group, group)
        if zero:
            lo, hi = w.amin(2, keepdim=True).clamp_max(0), w.amax(2, keepdim=True).clamp_min(0)
            s = ((hi - lo) / 15).bfloat16().float()
            z = torch.round(-lo / s).clamp(0, 15)
            c = (torch.round(w / s) + z).clamp(0, 15)
            zeros.append(z[:, :, 0].t().to(torch.uint8).contiguous())
        else:
            s = (w.abs().amax(2, keepdim=True) / 7).bfloat16().float()
            c = (torch.round(w / s) + 8).clamp(0, 15)
        codes.append(_pack(c.view(N, Kp)[:, :K]))
        scales.append(s[:, :, 0].t().bfloat16().contiguous())
    one = (lambda v: torch.stack(v)) if n > 0 else None
    w = dict(codes=one(codes), scale=one(scales), group=group)
    if zero:
        w["zero"] = one(zeros)
    return w


def _first(w):
    return {n: v[0] if torch.is_tensor(v) else v for n, v in w.items()}


def _rows8(v):
    """(codes, scales) of fp32 rows in blocks of 128, the last block shorter."""
    T, C = v.shape
    nb = -(-C // BLOCK)
    p = torch.nn.functional.pad(v, (0, nb * BLOCK - C)).view(T, nb, BLOCK)
    amax = p.abs().amax(2, keepdim=True)
    q = torch.where(amax > 0, p * E4M3_MAX / amax, 0 * p).view(T, nb * BLOCK)[:, :C].to(F8)
    return q.contiguous(), (amax / E4M3_MAX).view(T, nb)


def _halves8(gu, f):
    """The checkpoint of gu [R, 2f]: blocks of 128 of each half."""
    (qg, sg), (qu, su) = _rows8(gu[:, :f]), _rows8(gu[:, f:])
    return torch.cat([qg.view(torch.uint8), qu.view(torch.uint8)], 1).view(F8), torch.cat([sg, su], 1)


def _split(g, E, R, skew):
    """Rows of each of E segments: offsets, loads falling off as 1 / rank^skew, a segment without rows among them."""
    load = torch.arange(1, E + 1, device="cuda", dtype=torch.float32) ** -skew
    load = load[torch.randperm(E, generator=g, device="cuda")]
    load[int(torch.randint(E, (1,), generator=g, device="cuda"))] = 0.0
    pick = torch.multinomial(load, R, replacement=True, generator=g)
    return torch.nn.functional.pad(torch.bincount(pick, minlength=E).cumsum(0), (1, 0)).to(torch.int32)


def _padded_rows(R, E):
    return (-(-R // BLOCK) + (E if E > 1 else 0)) * BLOCK


def prepare(case, seed):
    g, c = _gen(seed), case
    new = lambda dt, *shape: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    zeros = lambda dt, *shape: torch.zeros(shape, dtype=torch.uint8 if dt == F8 else dt, device="cuda").view(dt)  # noqa: E731
    if c["op"] == "w4":
        M, N, K, E, k = c["M"], c["N"], c["K"], c["E"], c["k"]
        s = dict(case=c, off=None, row=None)
        rows = M
        if E:
            load = -c["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
            u = torch.rand(M, E, generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
            pick = (load - torch.log(-torch.log(u))).topk(k, 1).indices.reshape(-1)
            s["off"] = torch.nn.functional.pad(torch.bincount(pick, minlength=E).cumsum(0), (1, 0)).to(torch.int32)
            s["row"] = (torch.sort(pick, stable=True).indices // k).to(torch.int32)
            rows = M * k
        w = _weights4(g, max(E, 1), N, K, c["group"], c["zero"])
        s["w"] = w if E else _first(w)
        s["x"] = _randn(g, M, K).to(torch.bfloat16)
        s["out"] = new(DTYPES[c["out"]], rows, N)
        return s
    if c["op"] == "experts":
        T, d, f, E, k = c["T"], c["d"], c["f"], c["E"], c["k"]
        n = E + c["shared"]
        # the router's sigmoid scores, renormalised
        p, idx = torch.sigmoid(1.5 * _randn(g, T, E)).topk(k, 1)
        return dict(case=c, x=_randn(g, T, d).to(torch.bfloat16), idx=idx.to(torch.int32).contiguous(),
                    gate=(2.5 * p / p.sum(1, keepdim=True)).contiguous(),
                    w13=_weights4(g, n, 2 * f, d, c["group"], c["zero"]),
                    wd=_weights4(g, n, d, f, c["group"], c["zero"]), out=new(DTYPES[c["out"]], T, d))
    R, f, E = c["R"], c["f"], c["E"]
    bf, f32 = torch.bfloat16, torch.float32
    s = dict(case=c)
    half = -(-f // BLOCK)
    if c["dir"] == "fwd":
        s["gu"] = _randn(g, R, 2 * f).to(bf)
        out = dict(save=new(F8, R, 2 * f), save_scale=new(f32, R, 2 * half))
        if c["act"]:
            out["act"] = new(bf, R, f)
        if c["quant"]:
            out.update(q=new(F8, R, f), scale=new(f32, R, half))
        s["out"] = out
        return s
    s["off"] = _split(g, E, R, c["skew"]) if E else None
    Tp = _padded_rows(R, E)
    if c["dir"] == "cols":
        n = c["tokens"] or R
        s["row"] = torch.randint(n, (R,), generator=g, device="cuda", dtype=torch.int32) if c["tokens"] else None
        s["q"], s["scale"] = _rows8(_randn(g, n, f) * (1.0 + 0.1 * _randn(g, f)))
        # behind the last segment nothing is written
        s["out"] = dict(q=zeros(F8, f, Tp), scale=zeros(f32, Tp // BLOCK, f))
        return s
    s["save"], s["save_scale"] = _halves8(_randn(g, R, 2 * f).to(bf).float(), f)
    s["dact"] = (_randn(g, R, f) * 0.02).to(bf)
    s["gate"] = torch.rand(R, generator=g, device="cuda") if c["gate"] else None
    out = {}
    if c["dgu"]:
        out["dgu"] = new(bf, R, 2 * f)
    if c["rows"]:
        out.update(dq=new(F8, R, 2 * f), dq_scale=new(f32, R, 2 * half))
    if c["cols"]:
        out.update(dqt=zeros(F8, 2 * f, Tp), dqt_scale=zeros(f32, Tp // BLOCK, 2 * f), actt=zeros(F8, f, Tp),
                   actt_scale=zeros(f32, Tp // BLOCK, f))
    if c["gate"]:
        out["dgate"] = new(f32, R)
    s["out"] = out
    return s


# -------------------------------------------------------------- plain form

def _values4(w, K):
    """fp32 values of packed weights [..., N, K]."""
    c = _unpack(w["codes"]).float()
    wide = lambda v: v.transpose(-1, -2).float().repeat_interleave(w["group"], -1)[..., :K]  # noqa: E731
    return (c - (wide(w["zero"]) if "zero" in w else 8.0)) * wide(w["scale"])


def _plain_w4(s):
    c = s["case"]
    x, w, odt = s["x"].float(), _values4(s["w"], c["K"]), DTYPES[c["out"]]
    if s["off"] is None:
        return (x @ w.t()).to(odt)
    # the rows of each expert, padded to as many as there are tokens
    off = s["off"].long()
    at = off[:-1, None] + torch.arange(c["M"], device="cuda")
    real = at < off[1:, None]
    rows = x[s["row"].long()][at.clamp_max(s["row"].numel() - 1)]
    return torch.bmm(rows, w.transpose(1, 2))[real].to(odt)


def _plain_experts(s):
    c, x = s["case"], s["x"].float()
    T, d, f, E = c["T"], c["d"], c["f"], c["E"]
    n = E + c["shared"]
    gate = torch.zeros(T, n, device="cuda").scatter_add_(1, s["idx"].long(), s["gate"])
    gate[:, E:] = 1.0
    gu = torch.bmm(x.expand(n, T, d), _values4(s["w13"], d).transpose(1, 2))
    g, u = gu[..., :f], gu[..., f:]
    y = torch.bmm(g / (1 + torch.exp(-g)) * u, _values4(s["wd"], f).transpose(1, 2))
    return (y * gate.t()[:, :, None]).sum(0).to(DTYPES[c["out"]])


def _from8(q, scale, C):
    return q.float() * scale.repeat_interleave(BLOCK, 1)[:, :C]


def _tiles(off, R, Tp):
    """For each padded position along the token axis its row, and whether there is one."""
    if off is None:
        at = torch.arange(Tp, device="cuda")
        return at.clamp_max(R - 1), at < R
    off = off.long()
    cnt = off[1:] - off[:-1]
    ends = ((cnt + BLOCK - 1) // BLOCK * BLOCK).cumsum(0)
    at = torch.arange(Tp, device="cuda")
    e = torch.searchsorted(ends, at, right=True).clamp_max(cnt.numel() - 1)
    start = ends - (cnt + BLOCK - 1) // BLOCK * BLOCK
    r = off[e] + at - start[e]
    live = (r < off[e + 1]) & (at < ends[-1])
    return r.clamp(0, R - 1), live


def _cols8(v, off):
    """fp32 rows quantised along the token axis, segments padded to 128 tokens: q [C, Tp], scale [Tp / 128, C]."""
    R, C = v.shape
    Tp = _padded_rows(R, 0 if off is None else off.numel() - 1)
    row, live = _tiles(off, R, Tp)
    q, scale = _rows8((v[row] * live[:, None]).t().contiguous())
    return q, scale.t().contiguous()


def _plain_save(s):
    c = s["case"]
    f = c["f"]
    if c["dir"] == "fwd":
        gu = s["gu"].float()
        g, u = gu[:, :f], gu[:, f:]
        a = g / (1 + torch.exp(-g)) * u
        save, save_scale = _halves8(gu, f)
        out = dict(save=save, save_scale=save_scale)
        if c["act"]:
            out["act"] = a.to(torch.bfloat16)
        if c["quant"]:
            out["q"], out["scale"] = _rows8(a)
        return out
    if c["dir"] == "cols":
        v = _from8(s["q"], s["scale"], f)
        q, scale = _cols8(v if s["row"] is None else v[s["row"].long()], s["off"])
        return dict(q=q, scale=scale)
    half = -(-f // BLOCK)
    g, u = _from8(s["save"][:, :f], s["save_scale"][:, :half], f), _from8(s["save"][:, f:], s["save_scale"][:, half:], f)
    dact = s["dact"].float()
    sg = 1 / (1 + torch.exp(-g))
    a = g * sg * u
    out = {}
    if c["gate"]:
        out["dgate"] = (a * dact).sum(1)
        dact, a = dact * s["gate"][:, None], a * s["gate"][:, None]
    dgu = torch.cat([dact * u * sg * (1 + g * (1 - sg)), dact * g * sg], 1)
    if c["dgu"]:
        out["dgu"] = dgu.to(torch.bfloat16)
    if c["rows"]:
        out["dq"], out["dq_scale"] = _rows8(dgu)
    if c["cols"]:
        out["dqt"], out["dqt_scale"] = _cols8(dgu, s["off"])
        out["actt"], out["actt_scale"] = _cols8(a, s["off"])
    return out


# ------------------------------------------------------------ library calls

def _library(s):
    import mixture_experts_layer_routing_gb300 as moe
    ops, c, out = moe.default_ops(), s["case"], s["out"]
    if c["op"] == "w4":
        return ops.w4_matmul(s["x"], s["w"], off=s["off"], row_index=s["row"], out=out)
    if c["op"] == "experts":
        return ops.w4_experts(s["x"], s["idx"], s["gate"], s["w13"], s["wd"], n_shared=c["shared"], out=out)
    if c["dir"] == "fwd":
        return ops.swiglu(s["gu"], out=out)
    if c["dir"] == "cols":
        q, scale = ops.requant_cols(s["q"], s["scale"], off=s["off"], row_index=s["row"], out=out)
        return dict(q=q, scale=scale)
    return ops.swiglu_backward(s["dact"], s["save"], s["save_scale"], gate=s["gate"], off=s["off"], out=out)


def run(state):
    if own:
        return _library(state)
    return {"w4": _plain_w4, "experts": _plain_experts, "save": _plain_save}[state["case"]["op"]](state)


# ------------------------------------------------------------ work, 64 bits

def _in_use(E, k, T):
    """Experts that hold a row of T tokens, on average over even routings."""
    return E * (1.0 - (1.0 - k / E) ** T)


def work(case):
    c = case
    if c["op"] == "w4" or c["op"] == "experts":
        per = 0.5 + (3 if c["zero"] else 2) / c["group"]      # bytes of a weight
        o = 4 if c["out"] == "fp32" else 2
        if c["op"] == "w4":
            M, N, K, E = c["M"], c["N"], c["K"], c["E"]
            rows = M * c["k"] if E else M
            n = _in_use(E, c["k"], M) if E else 1
            return dict(bytes=int(n * N * K * per) + 2 * M * K + rows * N * o, flops=2 * rows * N * K)
        T, d, f = c["T"], c["d"], c["f"]
        n = _in_use(c["E"], c["k"], T) + c["shared"]
        pairs = T * (c["k"] + c["shared"])
        return dict(bytes=int(n * 3 * d * f * per) + T * d * (2 + o) + 8 * T * c["k"], flops=6 * pairs * d * f)
    R, f = c["R"], c["f"]
    n, half = R * f, 4 * R * -(-f // BLOCK)
    if c["dir"] == "fwd":
        return dict(bytes=4 * n + 2 * n + 2 * half + (2 * n if c["act"] else 0) + (n + half if c["quant"] else 0), flops=12 * n)
    if c["dir"] == "cols":
        src = (c["tokens"] or R) * f
        return dict(bytes=src + n + 4 * (src + n) // BLOCK, flops=4 * n)
    b = 2 * n + 2 * n + 2 * half + (8 * R if c["gate"] else 0)
    b += (4 * n if c["dgu"] else 0) + (2 * n + 2 * half if c["rows"] else 0) + (3 * n + 12 * n // BLOCK if c["cols"] else 0)
    return dict(bytes=b, flops=25 * n)


def _e4m3(v):
    """v (64 bits, |v| <= 448) rounded to the nearest e4m3 value, ties to even: 3 mantissa bits, exponents from -6."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -9))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)       # torch.round takes ties to even


def _blocks64(v):
    """Codes and scales in 64 bits of v in blocks of 128 along the last dim."""
    codes, scales = [], []
    for part in torch.split(v, BLOCK, -1):
        m = part.abs().amax(-1, keepdim=True)
        codes.append(_e4m3(torch.where(m > 0, part * E4M3_MAX / m, 0.0 * part)))
        scales.append(m / E4M3_MAX)
    return torch.cat(codes, -1), torch.cat(scales, -1)


def _columns64(v, off):
    """Segment by segment: codes [C, Tp] and scales [Tp / 128, C], zeros where there is no token."""
    R, C = v.shape
    ends = [0, R] if off is None else off.tolist()
    Tp = _padded_rows(R, len(ends) - 1)
    q = torch.zeros(C, Tp, dtype=torch.float64, device="cuda")
    scale = torch.zeros(Tp // BLOCK, C, dtype=torch.float64, device="cuda")
    at = 0
    for lo, hi in zip(ends[:-1], ends[1:]):
        if hi == lo:
            continue
        cq, cs = _blocks64(v[lo:hi].t())
        q[:, at:at + hi - lo] = cq
        scale[at // BLOCK:at // BLOCK + cs.shape[1]] = cs.t()
        at += -(-(hi - lo) // BLOCK) * BLOCK
    return q, scale


def _dense64(w, e, K):
    """One matrix of packed weights in 64 bits, nibble by nibble."""
    words = (w["codes"] if e is None else w["codes"][e]).to(torch.int64) & 0xffffffff
    scale = (w["scale"] if e is None else w["scale"][e]).double()
    zero = None if "zero" not in w else (w["zero"] if e is None else w["zero"][e]).double()
    out = torch.empty(words.shape[0], K, dtype=torch.float64, device="cuda")
    for j in range(8):
        out[:, j::8] = ((words >> (4 * (j // 2) + 16 * (j % 2))) & 15).double()
    for i in range(scale.shape[0]):
        part = out[:, i * w["group"]:(i + 1) * w["group"]]
        part -= 8.0 if zero is None else zero[i][:, None]
        part *= scale[i][:, None]
    return out


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "w4":
        x = s["x"].double()
        if s["off"] is None:
            return torch.einsum("mk,nk->mn", x, _dense64(s["w"], None, c["K"]))
        off, row = s["off"].tolist(), s["row"].long()
        return torch.cat([x[row[off[e]:off[e + 1]]] @ _dense64(s["w"], e, c["K"]).t() for e in range(c["E"])])
    if c["op"] == "experts":
        x, d, f = s["x"].double(), c["d"], c["f"]
        y = torch.zeros(c["T"], d, dtype=torch.float64, device="cuda")
        idx, gate = s["idx"].tolist(), s["gate"].double()
        for e in range(c["E"] + c["shared"]):
            use = [(t, j) for t in range(c["T"]) for j in range(c["k"]) if idx[t][j] == e]
            rows = [t for t, _ in use] if e < c["E"] else list(range(c["T"]))
            if not rows:
                continue
            gu = x[rows] @ _dense64(s["w13"], e, d).t()
            h = gu[:, :f] * torch.special.expit(gu[:, :f]) * gu[:, f:]
            o = h @ _dense64(s["wd"], e, f).t()
            if e < c["E"]:
                o = o * torch.stack([gate[t, j] for t, j in use])[:, None]
            y.index_add_(0, torch.tensor(rows, device="cuda"), o)
        return y
    f = c["f"]
    if c["dir"] == "fwd":
        gu = s["gu"].double()
        (qg, sg), (qu, su) = _blocks64(gu[:, :f]), _blocks64(gu[:, f:])
        a = gu[:, :f] * torch.special.expit(gu[:, :f]) * gu[:, f:]
        out = dict(save=torch.cat([qg, qu], 1), save_scale=torch.cat([sg, su], 1))
        if c["act"]:
            out["act"] = a
        if c["quant"]:
            out["q"], out["scale"] = _blocks64(a)
        return out
    wide = lambda q, sc: torch.cat([p.double() * sc[:, i:i + 1].double() for i, p in enumerate(torch.split(q.float(), BLOCK, 1))], 1)  # noqa: E731
    if c["dir"] == "cols":
        v = wide(s["q"], s["scale"])
        q, scale = _columns64(v if s["row"] is None else v[s["row"].long()], s["off"])
        return dict(q=q, scale=scale)
    half = -(-f // BLOCK)
    g, u = wide(s["save"][:, :f], s["save_scale"][:, :half]), wide(s["save"][:, f:], s["save_scale"][:, half:])
    da, sg = s["dact"].double(), torch.special.expit(g)
    silu = g * sg
    out, scaled = {}, da
    if c["gate"]:
        out["dgate"] = torch.einsum("rf,rf->r", silu * u, da)
        scaled = da * s["gate"].double()[:, None]
    dgu = torch.cat([scaled * u * (sg + silu * (1 - sg)), scaled * silu], 1)
    if c["dgu"]:
        out["dgu"] = dgu
    if c["rows"]:
        out["dq"], out["dq_scale"] = _blocks64(dgu)
    if c["cols"]:
        out["dqt"], out["dqt_scale"] = _columns64(dgu, s["off"])
        a = silu * u
        out["actt"], out["actt_scale"] = _columns64(a * s["gate"].double()[:, None] if c["gate"] else a, s["off"])
    return out
