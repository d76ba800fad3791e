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
