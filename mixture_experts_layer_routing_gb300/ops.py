"""Python binding of the operators of include/moe_ops.h.

MoeOps holds one handle and takes torch tensors: it checks types, shapes and
layouts, allocates outputs that are not given (`out`) and scratch, and forwards
to the C ABI call named in each method's docstring, which documents formulas and
limits. Work is enqueued on `stream` (default: the current torch stream). All
compute runs in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes

import torch

from . import (MOE_BF16, MOE_FP32, MOE_ROUTER_SIGMOID, MOE_ROUTER_SOFTMAX, MoeError, _check, load_library)

OPS_EXPORTED = ("moe_ops_create", "moe_ops_destroy", "moe_ops_get_status", "moe_ops_launch_count",
                "moe_norm_forward", "moe_norm_workspace_size", "moe_norm_backward", "moe_gate_workspace_size",
                "moe_gate_forward", "moe_gate_backward", "moe_quant_rows", "moe_quant_cols_rows", "moe_quant_cols",
                "moe_quant_blocks", "moe_fp8_matmul", "moe_fp8_matmul_workspace_size", "moe_fp8_wgrad")

BLOCK = 128                     # values that share a scale
F8 = torch.float8_e4m3fn
_DTYPES = {torch.bfloat16: MOE_BF16, torch.float32: MOE_FP32}
_ROUTERS = {"softmax": MOE_ROUTER_SOFTMAX, "sigmoid": MOE_ROUTER_SIGMOID}
_CURRENT_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class moe_gate_config(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int), ("k", ctypes.c_int), ("router", ctypes.c_int), ("renorm", ctypes.c_int),
                ("route_scale", ctypes.c_float), ("n_groups", ctypes.c_int), ("topk_groups", ctypes.c_int)]


_bound = None


def _lib():
    global _bound
    if _bound is not None:
        return _bound
    lib = load_library()
    vp, i32, i64, f32, sz, P = (ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t,
                                ctypes.POINTER)
    cfg = P(moe_gate_config)
    lib.moe_ops_create.argtypes = [P(vp)]
    lib.moe_ops_destroy.argtypes = [vp]
    lib.moe_ops_get_status.argtypes = [vp, vp, P(i32)]
    lib.moe_ops_launch_count.argtypes = [vp, P(i64)]
    lib.moe_norm_forward.argtypes = [vp, i32, vp, i64, vp, i64, vp, i32, i32, f32] + [vp] * 6
    lib.moe_norm_workspace_size.argtypes = [i32, i32, P(sz)]
    lib.moe_norm_backward.argtypes = [vp, i32] + [vp] * 5 + [i32, i32] + [vp] * 4
    lib.moe_gate_workspace_size.argtypes = [cfg, i32, P(sz)]
    lib.moe_gate_forward.argtypes = [vp, cfg, vp, vp, i32] + [vp] * 8
    lib.moe_gate_backward.argtypes = [vp, cfg, vp, vp, vp, i32, vp, vp]
    lib.moe_quant_rows.argtypes = [vp, vp, i64, i32, i32, i32, vp, vp, vp]
    lib.moe_quant_cols_rows.argtypes = [i32, i32, P(i32)]
    lib.moe_quant_cols.argtypes = [vp, vp, i64, i32, i32, i32, vp, i32, vp, vp, vp, vp]
    lib.moe_quant_blocks.argtypes = [vp, vp, i32, i32, i32] + [vp] * 5
    lib.moe_fp8_matmul.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, vp, i32, i32, i32, vp, i32, vp, vp]
    lib.moe_fp8_matmul_workspace_size.argtypes = [i32, i32, i32, i32, P(sz)]
    lib.moe_fp8_wgrad.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, i32, vp]
    for name in OPS_EXPORTED:
        getattr(lib, name).restype = i32
    _bound = lib
    return lib


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _want(t, what, dtype, shape, device):
    """t, checked: of this type and shape, dense, on the device."""
    if t.dtype != dtype:
        raise TypeError(f"{what}: {dtype} expected, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: has to be contiguous")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, not on {device}")
    return t


def _rows(t, what, device):
    """Row stride of a 2-D tensor whose rows are dense."""
    if t.dim() != 2:
        raise ValueError(f"{what}: two dimensions expected, got {t.dim()}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, not on {device}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the values of a row have to be neighbours")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0))


def _ptr(t):
    return None if t is None else t.data_ptr()


class MoeOps:
    """The operators around the expert layer on one device (include/moe_ops.h)."""

    def __init__(self, device=None):
        self.h = None
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"a CUDA device is needed, got {self.device}")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(_lib().moe_ops_create(ctypes.byref(h)), "moe_ops_create")
        self.h = h.value
        self._lib = _lib()

    def close(self):
        if self.h:
            _check(self._lib.moe_ops_destroy(self.h), "moe_ops_destroy")
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _stream(self, stream):
        if stream is None:
            return _CURRENT_STREAM(self.device.index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _scratch(self, nbytes, stream):
        """Scratch of one call; the allocator may hand it out again once the call's stream is past it."""
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=self.device)
        if stream is not None:
            ws.record_stream(torch.cuda.ExternalStream(stream, self.device) if isinstance(stream, int) else stream)
        return ws

    def _out(self, out, name, dtype, shape):
        t = out.get(name)
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=self.device)
            out[name] = t
            return t
        return _want(t, name, dtype, shape, self.device)

    def status(self, stream=None) -> int:
        """moe_ops_get_status: waits for the stream, reads and clears the device status word."""
        v = ctypes.c_int()
        _check(self._lib.moe_ops_get_status(self.h, self._stream(stream), ctypes.byref(v)), "moe_ops_get_status")
        return v.value

    def launch_count(self) -> int:
        v = ctypes.c_longlong()
        _check(self._lib.moe_ops_launch_count(self.h, ctypes.byref(v)), "moe_ops_launch_count")
        return v.value

    # ------------------------------------------------------------------ norm
    def rms_norm(self, x, weight, residual=None, eps=1e-6, want=None, out=None, stream=None) -> dict:
        """moe_norm_forward. x, residual [T, d] (rows may be strided), weight [d], all bf16 or all fp32.

        Returns a dict of the outputs named in `want` or, with `out`, of those that it holds (None values are
        allocated): "h" the sum, "y" the norm, "q" and "scale" its 8-bit form, "rstd". Default: y, and h with a
        residual.
        """
        if out is None:
            out = dict.fromkeys(want or (("h", "y") if residual is not None else ("y",)))
            if "q" in out or "scale" in out:
                out.update(q=None, scale=None)
        ld_x = _rows(x, "x", self.device)
        T, d = x.shape
        dt = x.dtype
        if dt not in _DTYPES:
            raise TypeError(f"x: bf16 or fp32 expected, got {dt}")
        ld_res = 0
        if residual is not None:
            ld_res = _rows(residual, "residual", self.device)
            if residual.dtype != dt or residual.shape != x.shape:
                raise ValueError("residual: type and shape of x expected")
        _want(weight, "weight", dt, (d,), self.device)
        unknown = set(out) - {"h", "y", "q", "scale", "rstd"}
        if unknown:
            raise ValueError(f"unknown outputs: {sorted(unknown)}")
        h = self._out(out, "h", dt, (T, d)) if "h" in out else None
        y = self._out(out, "y", dt, (T, d)) if "y" in out else None
        q = self._out(out, "q", F8, (T, d)) if "q" in out else None
        scale = self._out(out, "scale", torch.float32, (T, _blocks(d))) if "scale" in out else None
        rstd = self._out(out, "rstd", torch.float32, (T,)) if "rstd" in out else None
        _check(self._lib.moe_norm_forward(self.h, _DTYPES[dt], x.data_ptr(), ld_x, _ptr(residual), ld_res,
                                          weight.data_ptr(), T, d, eps, _ptr(h), _ptr(y), _ptr(q), _ptr(scale),
                                          _ptr(rstd), self._stream(stream)), "moe_norm_forward")
        return out

    def rms_norm_backward(self, dy, h, weight, rstd, dh=None, out=None, stream=None) -> dict:
        """moe_norm_backward. Returns {"dx", "dw"} (with `out`: those that it holds)."""
        if out is None:
            out = dict(dx=None, dw=None)
        if dy.dim() != 2 or dy.dtype not in _DTYPES:
            raise TypeError("dy: a bf16 or fp32 matrix expected")
        T, d = dy.shape
        dt = dy.dtype
        _want(dy, "dy", dt, (T, d), self.device)
        _want(h, "h", dt, (T, d), self.device)
        _want(weight, "weight", dt, (d,), self.device)
        _want(rstd, "rstd", torch.float32, (T,), self.device)
        if dh is not None:
            _want(dh, "dh", dt, (T, d), self.device)
        dx = self._out(out, "dx", dt, (T, d)) if "dx" in out else None
        dw = ws = None
        if "dw" in out:
            dw = self._out(out, "dw", torch.float32, (d,))
            n = ctypes.c_size_t()
            _check(self._lib.moe_norm_workspace_size(T, d, ctypes.byref(n)), "moe_norm_workspace_size")
            ws = self._scratch(n.value, stream)
        _check(self._lib.moe_norm_backward(self.h, _DTYPES[dt], dy.data_ptr(), _ptr(dh), h.data_ptr(),
                                           weight.data_ptr(), rstd.data_ptr(), T, d, _ptr(dx), _ptr(dw), _ptr(ws),
                                           self._stream(stream)), "moe_norm_backward")
        return out

    # --------------------------------------------------------------- routing
    def gate(self, logits, k, bias=None, router="softmax", renorm=True, route_scale=1.0, n_groups=1, topk_groups=1,
             dispatch=True, out=None, stream=None) -> dict:
        """moe_gate_forward. logits [T, E] fp32, bias [E] fp32. Returns idx, gate and (dispatch) cnt, off, perm, inv."""
        if logits.dim() != 2:
            raise ValueError("logits: two dimensions expected")
        T, E = logits.shape
        _want(logits, "logits", torch.float32, (T, E), self.device)
        if bias is not None:
            _want(bias, "bias", torch.float32, (E,), self.device)
        cfg = moe_gate_config(E, k, _ROUTERS[router], int(bool(renorm)), route_scale, n_groups, topk_groups)
        if out is None:
            out = {}
        else:
            dispatch = "perm" in out
        i32 = torch.int32
        idx, gate = self._out(out, "idx", i32, (T, k)), self._out(out, "gate", torch.float32, (T, k))
        cnt = off = perm = inv = ws = None
        if dispatch:
            cnt, off = self._out(out, "cnt", i32, (E,)), self._out(out, "off", i32, (E + 1,))
            perm, inv = self._out(out, "perm", i32, (T * k,)), self._out(out, "inv", i32, (T * k,))
            n = ctypes.c_size_t()
            _check(self._lib.moe_gate_workspace_size(ctypes.byref(cfg), T, ctypes.byref(n)),
                   "moe_gate_workspace_size")
            ws = self._scratch(n.value, stream)
        _check(self._lib.moe_gate_forward(self.h, ctypes.byref(cfg), logits.data_ptr(), _ptr(bias), T, idx.data_ptr(),
                                          gate.data_ptr(), _ptr(cnt), _ptr(off), _ptr(perm), _ptr(inv), _ptr(ws),
                                          self._stream(stream)), "moe_gate_forward")
        return out

    def gate_backward(self, logits, idx, dgate, router="softmax", renorm=True, route_scale=1.0, out=None,
                      stream=None) -> dict:
        """moe_gate_backward. Returns {"dlogits"} [T, E] fp32."""
        if logits.dim() != 2 or idx.dim() != 2:
            raise ValueError("logits, idx: two dimensions expected")
        T, E = logits.shape
        k = idx.shape[1]
        _want(logits, "logits", torch.float32, (T, E), self.device)
        _want(idx, "idx", torch.int32, (T, k), self.device)
        _want(dgate, "dgate", torch.float32, (T, k), self.device)
        out = {} if out is None else out
        dl = self._out(out, "dlogits", torch.float32, (T, E))
        cfg = moe_gate_config(E, k, _ROUTERS[router], int(bool(renorm)), route_scale, 1, 1)
        _check(self._lib.moe_gate_backward(self.h, ctypes.byref(cfg), logits.data_ptr(), idx.data_ptr(),
                                           dgate.data_ptr(), T, dl.data_ptr(), self._stream(stream)),
               "moe_gate_backward")
        return out

    # ------------------------------------------------------------ quantisers
    def quant_rows(self, src, swiglu=False, out=None, stream=None):
        """moe_quant_rows. src [T, C] bf16 (swiglu: [T, 2C], gate half then up half) -> (q [T, C], scale)."""
        ld = _rows(src, "src", self.device)
        if src.dtype != torch.bfloat16:
            raise TypeError(f"src: bf16 expected, got {src.dtype}")
        T, C = src.shape
        if swiglu:
            if C % 2:
                raise ValueError("src: an even number of columns expected")
            C //= 2
        out = {} if out is None else out
        q, s = self._out(out, "q", F8, (T, C)), self._out(out, "scale", torch.float32, (T, _blocks(C)))
        _check(self._lib.moe_quant_rows(self.h, src.data_ptr(), ld, T, C, int(bool(swiglu)), q.data_ptr(),
                                        s.data_ptr(), self._stream(stream)), "moe_quant_rows")
        return q, s

    def quant_cols(self, src, off=None, row_index=None, out=None, stream=None):
        """moe_quant_cols. src [rows, C] bf16 -> (q [C, Tp], scale [Tp / 128, C]), segments of tokens by off."""
        ld = _rows(src, "src", self.device)
        if src.dtype != torch.bfloat16:
            raise TypeError(f"src: bf16 expected, got {src.dtype}")
        rows, C = src.shape
        G = self._segments(off)
        T = rows if row_index is None else self._index(row_index)
        Tp = ctypes.c_int()
        _check(self._lib.moe_quant_cols_rows(T, G, ctypes.byref(Tp)), "moe_quant_cols_rows")
        Tp = Tp.value
        out = {} if out is None else out
        q, s = self._out(out, "q", F8, (C, Tp)), self._out(out, "scale", torch.float32, (Tp // BLOCK, C))
        _check(self._lib.moe_quant_cols(self.h, src.data_ptr(), ld, rows, T, C, _ptr(off), G, _ptr(row_index),
                                        q.data_ptr(), s.data_ptr(), self._stream(stream)), "moe_quant_cols")
        return q, s

    def quant_blocks(self, w, transpose=False, out=None, stream=None) -> dict:
        """moe_quant_blocks. w [N, K] or [G, N, K] bf16 -> {"q", "scale"} and, transpose, {"qt", "scale_t"}."""
        if w.dim() not in (2, 3) or w.dtype != torch.bfloat16:
            raise TypeError("w: a bf16 tensor of two or three dimensions expected")
        _want(w, "w", torch.bfloat16, w.shape, self.device)
        lead, (N, K) = tuple(w.shape[:-2]), w.shape[-2:]
        out = {} if out is None else out
        q = self._out(out, "q", F8, (*lead, N, K))
        s = self._out(out, "scale", torch.float32, (*lead, _blocks(N), _blocks(K)))
        qt = st = None
        if transpose:
            qt = self._out(out, "qt", F8, (*lead, K, N))
            st = self._out(out, "scale_t", torch.float32, (*lead, _blocks(K), _blocks(N)))
        _check(self._lib.moe_quant_blocks(self.h, w.data_ptr(), lead[0] if lead else 1, N, K, q.data_ptr(),
                                          s.data_ptr(), _ptr(qt), _ptr(st), self._stream(stream)), "moe_quant_blocks")
        return out

    # -------------------------------------------------------------- products
    def _segments(self, off):
        if off is None:
            return 1
        _want(off, "off", torch.int32, (off.numel(),), self.device)
        if off.numel() < 2:
            raise ValueError("off: one more value than segments expected")
        return off.numel() - 1

    def _index(self, row_index):
        _want(row_index, "row_index", torch.int32, (row_index.numel(),), self.device)
        return row_index.numel()

    def fp8_matmul(self, a, a_scale, b, b_scale, off=None, row_index=None, out=None, out_dtype=torch.bfloat16,
                   stream=None):
        """moe_fp8_matmul. a [rows, K], b [N, K] or (with off) [G, N, K], e4m3 with scales -> [M, N]."""
        if a.dim() != 2 or b.dim() != (2 if off is None else 3):
            raise ValueError("a: two dimensions, b: two, with off three, expected")
        rows, K = a.shape
        G = self._segments(off)
        lead, N = tuple(b.shape[:-2]), b.shape[-2]
        dev = self.device
        _want(a, "a", F8, (rows, K), dev)
        _want(a_scale, "a_scale", torch.float32, (rows, _blocks(K)), dev)
        _want(b, "b", F8, (*((G,) if off is not None else ()), N, K), dev)
        _want(b_scale, "b_scale", torch.float32, (*lead, _blocks(N), _blocks(K)), dev)
        M = rows if row_index is None else self._index(row_index)
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype, device=dev)
        if out.dtype not in _DTYPES:
            raise TypeError(f"out: bf16 or fp32 expected, got {out.dtype}")
        _want(out, "out", out.dtype, (M, N), dev)
        ws = None
        if row_index is not None:
            n = ctypes.c_size_t()
            _check(self._lib.moe_fp8_matmul_workspace_size(M, G, K, 1, ctypes.byref(n)),
                   "moe_fp8_matmul_workspace_size")
            ws = self._scratch(n.value, stream) if n.value else None
        _check(self._lib.moe_fp8_matmul(self.h, a.data_ptr(), a_scale.data_ptr(), rows, _ptr(row_index), M,
                                        b.data_ptr(), b_scale.data_ptr(), _ptr(off), G, N, K, out.data_ptr(),
                                        _DTYPES[out.dtype], _ptr(ws), self._stream(stream)), "moe_fp8_matmul")
        return out

    def fp8_wgrad(self, dct, dct_scale, xt, xt_scale, off=None, tokens=None, out=None, out_dtype=torch.bfloat16,
                  stream=None):
        """moe_fp8_wgrad, of quant_cols' results: dct [N, Tp], xt [K, Tp] -> [N, K] or (with off) [G, N, K].

        tokens: the number of tokens given to quant_cols (default: the most that Tp holds).
        """
        if dct.dim() != 2 or xt.dim() != 2:
            raise ValueError("dct, xt: two dimensions expected")
        N, Tp = dct.shape
        K = xt.shape[0]
        G = self._segments(off)
        dev = self.device
        T = Tp - (G * BLOCK if G > 1 else 0) if tokens is None else tokens
        n = ctypes.c_int()
        _check(self._lib.moe_quant_cols_rows(T, G, ctypes.byref(n)), "moe_quant_cols_rows")
        if n.value != Tp:
            raise ValueError(f"dct: {n.value} padded tokens expected, got {Tp}")
        _want(dct, "dct", F8, (N, Tp), dev)
        _want(dct_scale, "dct_scale", torch.float32, (Tp // BLOCK, N), dev)
        _want(xt, "xt", F8, (K, Tp), dev)
        _want(xt_scale, "xt_scale", torch.float32, (Tp // BLOCK, K), dev)
        shape = (N, K) if off is None else (G, N, K)
        if out is None:
            out = torch.empty(shape, dtype=out_dtype, device=dev)
        if out.dtype not in _DTYPES:
            raise TypeError(f"out: bf16 or fp32 expected, got {out.dtype}")
        _want(out, "out", out.dtype, shape, dev)
        _check(self._lib.moe_fp8_wgrad(self.h, dct.data_ptr(), dct_scale.data_ptr(), xt.data_ptr(),
                                       xt_scale.data_ptr(), T, _ptr(off), G, N, K, out.data_ptr(),
                                       _DTYPES[out.dtype], self._stream(stream)), "moe_fp8_wgrad")
        return out


_default = {}


def default_ops(device=None) -> MoeOps:
    """The process's handle for a device (default: the current one), created on first use."""
    index = torch.cuda.current_device() if device is None or torch.device(device).index is None \
        else torch.device(device).index
    ops = _default.get(index)
    if ops is None:
        ops = _default[index] = MoeOps(torch.device("cuda", index))
    return ops
