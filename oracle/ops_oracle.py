"""Plain 64-bit restatements (numpy) of the operators of include/moe_ops.h.

Test infrastructure only: written from the formulas, sharing no code with the
CUDA path. Arrays are float64; values held in bf16 or e4m3 are passed as the
numbers they stand for.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0


def e4m3(v):
    """v rounded to the nearest e4m3 value (3 mantissa bits, exponents -6 .. 8, largest 448), ties to even."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    _, e = np.frexp(np.where(np.isfinite(a) & (a > 0), a, 1.0))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    r = np.where(np.isnan(v), np.nan, np.clip(np.rint(np.where(np.isfinite(v), v, 0.0) / step) * step, -E4M3_MAX, E4M3_MAX))
    return np.where(np.isinf(v), np.copysign(E4M3_MAX, v), r)


def quantise(v, axis):
    """(codes, scales) of v in blocks of 128 along `axis` (the last one shorter); scales fp32-rounded.

    The quotient 448 v / m is rounded to fp32 before the rounding to e4m3, as the header defines it.
    """
    v = np.moveaxis(np.asarray(v, np.float64), axis, -1)
    codes, scales = np.empty_like(v), []
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        for b in range(0, v.shape[-1], BLOCK):
            part = v[..., b:b + BLOCK]
            m = np.max(np.abs(part), axis=-1, keepdims=True)
            x = np.where(m > 0, (np.float32(E4M3_MAX) * part.astype(np.float32)) / m.astype(np.float32), 0.0 * part)
            codes[..., b:b + BLOCK] = e4m3(x)
            scales.append((m[..., 0].astype(np.float32) / np.float32(E4M3_MAX)).astype(np.float64))
    return np.moveaxis(codes, -1, axis), np.moveaxis(np.stack(scales, -1), -1, axis)


def quantise_blocks(w):
    """(codes, scales) of a matrix in 128 x 128 blocks."""
    N, K = w.shape
    codes = np.empty((N, K))
    scales = np.empty((-(-N // BLOCK), -(-K // BLOCK)))
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            m = np.abs(w[at]).max()
            scales[i, j] = np.float32(m) / np.float32(E4M3_MAX)
            codes[at] = e4m3((np.float32(E4M3_MAX) * w[at].astype(np.float32)) / np.float32(m)) if m > 0 else 0.0
    return codes, scales


def rms_norm(h, w, eps):
    """(y, rstd) of the stored sum h."""
    r = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * r[:, None] * w, r


def rms_norm_backward(dy, h, w, rstd, dh=None):
    """(dx, dw), and the sums of magnitudes that their rounding errors are relative to."""
    n, u = h * rstd[:, None], dy * w
    mean = (u * n).mean(1, keepdims=True)
    dx = rstd[:, None] * (u - n * mean)
    size = rstd[:, None] * (np.abs(u) + np.abs(n) * np.abs(u * n).mean(1, keepdims=True))
    if dh is not None:
        dx, size = dx + dh, size + np.abs(dh)
    return dx, (dy * n).sum(0), size, np.abs(dy * n).sum(0)


def scores(logits, router):
    l = np.asarray(logits, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        if router == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = np.max(l, 1, keepdims=True)
        m = np.where(m == -np.inf, 0.0, m)
        e = np.exp(l - m)
        s = e.sum(1, keepdims=True)
        return np.where(s == 0, 0.0, e / np.where(s == 0, 1.0, s))


def gate(logits, bias, k, router, renorm, scale, n_groups=1, topk_groups=1):
    """idx, gate and the dispatch, token by token and expert by expert."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    S = E // n_groups
    low = np.finfo(np.float64).min
    p = scores(logits, router)
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    idx, g = np.empty((T, k), np.int64), np.empty((T, k))
    with np.errstate(over="ignore"):
        for t in range(T):
            key = [low if logits[t, e] == -np.inf or np.isnan(p[t, e] + b[e]) else max(p[t, e] + b[e], low)
                   for e in range(E)]
            best = [sum(sorted(key[i * S:(i + 1) * S])[::-1][:2]) for i in range(n_groups)]
            kept = sorted(range(n_groups), key=lambda i: (-best[i], i))[:topk_groups]
            left = [e for i in sorted(kept) for e in range(i * S, (i + 1) * S)]
            idx[t] = sorted(left, key=lambda e: (-key[e], e))[:k]
            ps = p[t, idx[t]]
            g[t] = scale * (ps / (ps.sum() + 1e-20) if renorm else ps)
    return idx, g


def dispatch(idx, E):
    flat = idx.reshape(-1)
    perm = np.argsort(flat, kind="stable")
    inv = np.empty_like(perm)
    inv[perm] = np.arange(perm.size)
    cnt = np.bincount(flat, minlength=E)
    return cnt, np.concatenate([[0], np.cumsum(cnt)]), perm, inv


def gate_backward(logits, idx, dgate, router, renorm, scale):
    """dlogits by the chain rule through the k selected scores, and the magnitudes their errors are relative to."""
    p = scores(logits, router)
    T, k = idx.shape
    rows = np.arange(T)[:, None]
    ps, d = p[rows, idx], scale * np.asarray(dgate, np.float64)
    size = np.abs(d)
    if renorm:
        D = ps.sum(1, keepdims=True) + 1e-20
        size = (size + (size * ps).sum(1, keepdims=True) / D) / D
        d = (d - (d * ps).sum(1, keepdims=True) / D) / D
    dp, sp = np.zeros_like(p), np.zeros_like(p)
    dp[rows, idx], sp[rows, idx] = d, size
    if router == "sigmoid":
        rest = 1.0 / (1.0 + np.exp(np.asarray(logits, np.float64)))
        return p * rest * dp, p * rest * sp
    return (p * (dp - (p * dp).sum(1, keepdims=True)), p * (sp + (p * sp).sum(1, keepdims=True)))


def values(codes, scale, axis=1):
    """Values of codes with a scale for each 128 along `axis` (a number of axes: each)."""
    s = scale
    for ax in (axis if isinstance(axis, tuple) else (axis,)):
        s = np.take(s, np.arange(codes.shape[ax]) // BLOCK, axis=ax)
    return codes * s


def matmul(a, b, off=None, row_index=None):
    """(c, sum of |a b|): a [rows, K], b [N, K] or [G, N, K] values."""
    if row_index is not None:
        a = a[row_index]
    if off is None:
        return a @ b.T, np.abs(a) @ np.abs(b).T
    c = [a[off[g]:off[g + 1]] @ b[g].T for g in range(len(off) - 1)]
    s = [np.abs(a[off[g]:off[g + 1]]) @ np.abs(b[g]).T for g in range(len(off) - 1)]
    return np.concatenate(c), np.concatenate(s)


# ---- 4-bit weights: code order of a word's eight values, (code - zero) * scale

W4_SHIFT = np.array([0, 16, 4, 20, 8, 24, 12, 28])


def bf16(v):
    """fp32 values rounded to bf16, to nearest, ties to even (finite values)."""
    u = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7fff + ((u >> 16) & 1)) >> 16 << 16
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def w4_pack(codes):
    c = np.asarray(codes, np.uint64).reshape(*codes.shape[:-1], -1, 8)
    return (c << W4_SHIFT.astype(np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


def w4_unpack(words):
    w = np.asarray(words).view(np.uint32)
    return ((w[..., None] >> W4_SHIFT.astype(np.uint32)) & 15).reshape(*w.shape[:-1], -1).astype(np.float64)


def w4_values(words, scale, zero, group):
    """Values [N, K] of one matrix: words [N, K/8], scale and zero [KG, N] (zero None: 8)."""
    c = w4_unpack(words)
    at = np.arange(c.shape[1]) // group
    return (c - (8.0 if zero is None else zero.T[:, at])) * scale.T[:, at]


def quant_w4(w, group, with_zero):
    """codes [N, K], scale and zero [KG, N] of w [N, K]: quotients in fp32, the scale rounded to bf16 first."""
    w = np.asarray(w, np.float32)
    N, K = w.shape
    KG = -(-K // group)
    codes, scale, zero = np.empty((N, K)), np.empty((KG, N)), np.empty((KG, N))
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        for i in range(KG):
            v = w[:, i * group:(i + 1) * group]
            lo, hi = np.minimum(v.min(1), 0), np.maximum(v.max(1), 0)
            # (half the span where the whole one is beyond fp32)
            span = np.where(np.isinf(hi - lo), (hi * np.float32(0.5) - lo * np.float32(0.5)) / np.float32(7.5), (hi - lo) / np.float32(15))
            s = bf16(span if with_zero else np.abs(v).max(1) / np.float32(7)).astype(np.float32)
            live = (s > 0) & np.isfinite(s)
            z = np.clip(np.rint(-lo / s), 0, 15) if with_zero else np.full(N, 8.0, np.float32)
            z = np.where(live, z, 0.0 if with_zero else 8.0)
            codes[:, i * group:(i + 1) * group] = np.where(live[:, None], np.clip(np.rint(v / s[:, None]) + z[:, None], 0, 15),
                                                           z[:, None])
            scale[i], zero[i] = s, z
    return codes, scale, zero


def w4_experts(x, idx, gate, w13, wd, n_shared, add, kept=16):
    """(y, bound) of the experts' layer: w13 and wd lists of [2f, d] and [d, f] values. `add` is what an fp32 sum over
    d or f may be off, relative to the sum of its terms' magnitudes; bound is what y may be off before it is rounded:
    the products' sums, SwiGLU with the fast exponential and division (2^-18), and h kept to
    2^-kept (16 for bf16 outputs, 24 for fp32 ones)."""
    T = x.shape[0]
    E = len(w13) - n_shared
    y, bound = np.zeros((T, wd[0].shape[0])), np.zeros((T, wd[0].shape[0]))
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(T):
            use = [(e, g) for e, g in zip(idx[t], gate[t]) if 0 <= e < E] + [(E + s, 1.0) for s in range(n_shared)]
            for e, g in use:
                f = wd[e].shape[1]
                gu, size = w13[e] @ x[t], np.abs(w13[e]) @ np.abs(x[t])
                a, u, sa, su = gu[:f], gu[f:], size[:f], size[f:]
                s = a / (1 + np.exp(-a))
                h = g * s * u
                off = np.abs(g) * add * (1.1 * np.abs(u) * sa + np.abs(s) * su) + (2.0 ** -18 + 2.0 ** -kept) * np.abs(h)
                y[t] += wd[e] @ h
                bound[t] += np.abs(wd[e]) @ (off + add * np.abs(h))
    return y, bound


# ---- SwiGLU, 8-bit checkpoints

def swiglu_save(gu):
    """Codes [T, 2f] and scales of the two halves of gu, blocks within each half."""
    f = gu.shape[1] // 2
    (qg, sg), (qu, su) = quantise(gu[:, :f], 1), quantise(gu[:, f:], 1)
    return np.concatenate([qg, qu], 1), np.concatenate([sg, su], 1)


def swiglu_saved(save, scale):
    """The values (g, u) of a checkpoint, rounded to fp32 as code * scale."""
    f, nb = save.shape[1] // 2, scale.shape[1] // 2
    at = np.arange(f) // BLOCK
    mul = lambda c, s: (c.astype(np.float32) * s.astype(np.float32)[:, at]).astype(np.float64)  # noqa: E731
    return mul(save[:, :f], scale[:, :nb]), mul(save[:, f:], scale[:, nb:])


def swiglu(g, u):
    return g / (1 + np.exp(-g)) * u


def swiglu_backward(g, u, dact, gate):
    """(dg, du, gated act, dgate) and what the first three may be off where the sigmoid is off by 2^-18 of itself."""
    s = 1 / (1 + np.exp(-g))
    da, act = dact * gate[:, None], g * s * u
    dg, du = da * u * s * (1 + g * (1 - s)), da * g * s
    off = 2.0 ** -17
    return (dg, du, act * gate[:, None], (act * dact).sum(1),
            off * np.abs(da * u) * s * (1 + 2 * np.abs(g)), off * np.abs(du), off * np.abs(act * gate[:, None]),
            np.abs(act * dact).sum(1))
