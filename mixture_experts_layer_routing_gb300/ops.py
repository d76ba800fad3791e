"""Python binding of the operators of include/moe_ops.h.

MoeOps holds one handle and takes torch tensors. Its methods forward to the
C ABI call named in each docstring, which documents formulas and limits, through
_ops_binding (csrc/ops_binding.cpp): that checks types, shapes and layouts and
allocates outputs that are not given (`out`) and scratch. Work is enqueued on
`stream` (default: the current torch stream). All compute runs in the library's
CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes

import torch

from . import MOE_ROUTER_SIGMOID, MOE_ROUTER_SOFTMAX, _check, load_library

OPS_EXPORTED = ("moe_ops_create", "moe_ops_destroy", "moe_ops_get_status", "moe_ops_launch_count",
                "moe_norm_forward", "moe_norm_workspace_size", "moe_norm_backward", "moe_gate_workspace_size",
                "moe_gate_forward", "moe_gate_backward", "moe_quant_rows", "moe_quant_cols_rows", "moe_quant_cols",
                "moe_quant_blocks", "moe_fp8_matmul", "moe_fp8_matmul_workspace_size", "moe_fp8_wgrad")

BLOCK = 128                     # values that share a scale
_ROUTERS = {"softmax": MOE_ROUTER_SOFTMAX, "sigmoid": MOE_ROUTER_SIGMOID}
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


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


_binding_module = None


def _binding():
    """The tensor binding, which links to the library (loaded first, from its own path)."""
    global _binding_module
    if _binding_module is None:
        load_library()
        try:
            from . import _ops_binding
        except ImportError as e:
            raise ImportError(f"{__package__}._ops_binding is missing or does not load ({e}): build it with "
                              f"{__package__}.build.build()") from e
        _binding_module = _ops_binding
    return _binding_module


class MoeOps:
    """The operators around the expert layer on one device (include/moe_ops.h)."""

    def __init__(self, device=None):
        self.h = None
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"a CUDA device is needed, got {self.device}")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self._lib, self._b = _lib(), _binding()
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            torch.cuda.current_stream()          # (initialises torch's context)
            _check(self._lib.moe_ops_create(ctypes.byref(h)), "moe_ops_create")
        self.h = h.value

    def close(self):
        if self.h:
            _check(self._lib.moe_ops_destroy(self.h), "moe_ops_destroy")
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _stream(self, stream=None):
        if stream is None:
            return _current_stream(self._index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _on(self, stream, method, *args, **kw):
        """The method with `stream` (a torch stream or a cudaStream_t) current, so that outputs and scratch that it
        allocates belong to that stream too."""
        s = torch.cuda.ExternalStream(stream, self.device) if isinstance(stream, int) else stream
        with torch.cuda.stream(s):
            return method(*args, **kw)

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
        if stream is not None:
            return self._on(stream, self.rms_norm, x, weight, residual, eps, want, out)
        if out is None:
            out = dict.fromkeys(want or (("h", "y") if residual is not None else ("y",)))
            if "q" in out or "scale" in out:
                out.update(q=None, scale=None)
        s = self._b.norm_forward(self.h, self._index, self._stream(), x, weight, residual, eps, out)
        if s:
            _check(s, "moe_norm_forward")
        return out

    def rms_norm_backward(self, dy, h, weight, rstd, dh=None, out=None, stream=None) -> dict:
        """moe_norm_backward. Returns {"dx", "dw"} (with `out`: those that it holds)."""
        if stream is not None:
            return self._on(stream, self.rms_norm_backward, dy, h, weight, rstd, dh, out)
        if out is None:
            out = dict(dx=None, dw=None)
        s = self._b.norm_backward(self.h, self._index, self._stream(), dy, h, weight, rstd, dh, out)
        if s:
            _check(s, "moe_norm_backward")
        return out

    # --------------------------------------------------------------- routing
    def gate(self, logits, k, bias=None, router="softmax", renorm=True, route_scale=1.0, n_groups=1, topk_groups=1,
             dispatch=True, out=None, stream=None) -> dict:
        """moe_gate_forward. logits [T, E] fp32, bias [E] fp32. Returns idx, gate and (dispatch) cnt, off, perm, inv.

        With `out` the dispatch is made where it holds any of its four outputs (the others are added)."""
        if stream is not None:
            return self._on(stream, self.gate, logits, k, bias, router, renorm, route_scale, n_groups, topk_groups, dispatch, out)
        kind = _ROUTERS[router]
        if out is None:
            out = {}
        else:
            dispatch = "perm" in out or "inv" in out or "off" in out or "cnt" in out
        s = self._b.gate(self.h, self._index, self._stream(), logits, k, bias, kind, renorm, route_scale,
                         n_groups, topk_groups, dispatch, out)
        if s:
            _check(s, "moe_gate_forward")
        return out

    def gate_backward(self, logits, idx, dgate, router="softmax", renorm=True, route_scale=1.0, out=None,
                      stream=None) -> dict:
        """moe_gate_backward. Returns {"dlogits"} [T, E] fp32."""
        if stream is not None:
            return self._on(stream, self.gate_backward, logits, idx, dgate, router, renorm, route_scale, out)
        if out is None:
            out = {}
        s = self._b.gate_backward(self.h, self._index, self._stream(), logits, idx, dgate, _ROUTERS[router],
                                  renorm, route_scale, out)
        if s:
            _check(s, "moe_gate_backward")
        return out

    # ------------------------------------------------------------ quantisers
    def quant_rows(self, src, swiglu=False, out=None, stream=None):
        """moe_quant_rows. src [T, C] bf16 (swiglu: [T, 2C], gate half then up half) -> (q [T, C], scale)."""
        if stream is not None:
            return self._on(stream, self.quant_rows, src, swiglu, out)
        if out is None:
            out = {}
        s = self._b.quant_rows(self.h, self._index, self._stream(), src, swiglu, out)
        if s:
            _check(s, "moe_quant_rows")
        return out["q"], out["scale"]

    def quant_cols(self, src, off=None, row_index=None, out=None, stream=None):
        """moe_quant_cols. src [rows, C] bf16 -> (q [C, Tp], scale [Tp / 128, C]), segments of tokens by off."""
        if stream is not None:
            return self._on(stream, self.quant_cols, src, off, row_index, out)
        if out is None:
            out = {}
        s = self._b.quant_cols(self.h, self._index, self._stream(), src, off, row_index, out)
        if s:
            _check(s, "moe_quant_cols")
        return out["q"], out["scale"]

    def quant_blocks(self, w, transpose=False, out=None, stream=None) -> dict:
        """moe_quant_blocks. w [N, K] or [G, N, K] bf16 -> {"q", "scale"} and, transpose, {"qt", "scale_t"}."""
        if stream is not None:
            return self._on(stream, self.quant_blocks, w, transpose, out)
        if out is None:
            out = {}
        s = self._b.quant_blocks(self.h, self._index, self._stream(), w, transpose, out)
        if s:
            _check(s, "moe_quant_blocks")
        return out

    # -------------------------------------------------------------- products
    def fp8_matmul(self, a, a_scale, b, b_scale, off=None, row_index=None, out=None, out_dtype=torch.bfloat16,
                   stream=None):
        """moe_fp8_matmul. a [rows, K], b [N, K] or (with off) [G, N, K], e4m3 with scales -> [M, N]."""
        if stream is not None:
            return self._on(stream, self.fp8_matmul, a, a_scale, b, b_scale, off, row_index, out, out_dtype)
        if out is None:
            rows = a.shape[0] if row_index is None else row_index.numel()
            out = torch.empty((rows, b.shape[-2]), dtype=out_dtype, device=self.device)
        s = self._b.fp8_matmul(self.h, self._index, self._stream(), a, a_scale, b, b_scale, off, row_index, out)
        if s:
            _check(s, "moe_fp8_matmul")
        return out

    def fp8_wgrad(self, dct, dct_scale, xt, xt_scale, off=None, tokens=None, out=None, out_dtype=torch.bfloat16,
                  stream=None):
        """moe_fp8_wgrad, of quant_cols' results: dct [N, Tp], xt [K, Tp] -> [N, K] or (with off) [G, N, K].

        tokens: the number of tokens given to quant_cols (default: the most that Tp holds).
        """
        if stream is not None:
            return self._on(stream, self.fp8_wgrad, dct, dct_scale, xt, xt_scale, off, tokens, out, out_dtype)
        if out is None:
            shape = (dct.shape[0], xt.shape[0])
            out = torch.empty(shape if off is None else (off.numel() - 1, *shape), dtype=out_dtype, device=self.device)
        s = self._b.fp8_wgrad(self.h, self._index, self._stream(), dct, dct_scale, xt, xt_scale, off, tokens,
                              out)
        if s:
            _check(s, "moe_fp8_wgrad")
        return out


_default = {}


def default_ops(device=None) -> MoeOps:
    """The process's handle for a device (default: the current one), created on first use."""
    if device is None and _default:
        index = _current_device()
    else:
        d = torch.device("cuda" if device is None else device)
        if d.type != "cuda":
            raise ValueError(f"a CUDA device is needed, got {d}")
        index = torch.cuda.current_device() if d.index is None else d.index
    ops = _default.get(index)
    if ops is None:
        ops = _default[index] = MoeOps(torch.device("cuda", index))
    return ops
