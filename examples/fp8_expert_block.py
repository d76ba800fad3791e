"""A pre-norm expert block on the operators of include/moe_ops.h, with 8-bit products, forward and backward.

    h = x + residual                         y = rms_norm(h) * w
    idx, gate = routing of y Wr^T            (scores + balance bias, groups, top-k)
    out_t = sum_j gate[t, j] * FFN_{idx[t, j]}(y_t),   FFN_e(y) = (silu(y Wg_e^T) * (y Wu_e^T)) Wd_e^T

The norm's 8-bit output feeds the gate/up product, whose rows are gathered by the routing's permutation; the SwiGLU
is quantised as it is computed and feeds the down product. The backward pass quantises each gradient along the two
axes that its products reduce. What has no operator of its own here (the router's small product, the weighted sum over
a token's experts, SwiGLU's gradient) is plain torch.

With save8 the forward pass keeps 8 bits of each activation (the norm's output as the first product read it, and the
gate/up product as codes of its halves) and no expert's output: SwiGLU's gradient, the gates' and the weights' operands
come from those. For decoding the experts may be held in 4 bits (quantise4, decode).

    python examples/fp8_expert_block.py [--tokens 2048]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_layer_routing_gb300 as moe  # noqa: E402


class Fp8ExpertBlock:
    """Weights are quantised once, in 128 x 128 blocks, and kept transposed as well for the row gradients."""

    def __init__(self, d, f, E, k, n_groups=1, topk_groups=1, router="sigmoid", route_scale=2.5, eps=1e-6, seed=0,
                 device="cuda", save8=False):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=device) / s[-1] ** 0.5  # noqa: E731
        self.ops = moe.default_ops(device)
        self.k, self.f, self.eps, self.save8 = k, f, eps, save8
        self.route = dict(router=router, route_scale=route_scale, n_groups=n_groups, topk_groups=topk_groups)
        self.norm_w = (1 + 0.1 * torch.randn(d, generator=g, device=device)).bfloat16()
        self.Wr, self.bias = rnd(E, d), 0.01 * torch.randn(E, generator=g, device=device)
        self.W13, self.Wd = rnd(E, 2 * f, d).bfloat16(), rnd(E, d, f).bfloat16()
        self.q13 = self.ops.quant_blocks(self.W13, transpose=True)
        self.qd = self.ops.quant_blocks(self.Wd, transpose=True)

    def forward(self, x, residual):
        """(h, out) and what the backward pass needs."""
        ops, k = self.ops, self.k
        n = ops.rms_norm(x, self.norm_w, residual, self.eps, want=("h", "y", "q", "rstd"))
        logits = n["y"].float() @ self.Wr.t()
        r = ops.gate(logits, k, bias=self.bias, **self.route)
        token = r["perm"] // k                                   # the token of each sorted row
        gu = ops.fp8_matmul(n["q"], n["scale"], self.q13["q"], self.q13["scale"], off=r["off"], row_index=token)
        act = ops.swiglu(gu, want=("q", "save")) if self.save8 else None
        a = (act["q"], act["scale"]) if self.save8 else ops.quant_rows(gu, swiglu=True)
        o = ops.fp8_matmul(*a, self.qd["q"], self.qd["scale"], off=r["off"])
        rows = r["inv"].view(-1, k).long()
        out = (o[rows].float() * r["gate"][:, :, None]).sum(1).bfloat16()
        if self.save8:
            return n["h"], out, dict(h=n["h"], rstd=n["rstd"], q=n["q"], scale=n["scale"], save=act["save"],
                                     save_scale=act["save_scale"], logits=logits, token=token, rows=rows, **r)
        return n["h"], out, dict(n, logits=logits, token=token, gu=gu, o=o, rows=rows, **r)

    def _backward8(self, dout, c):
        """(rows' gradient of y, dWd, dW13, dgate) from the 8-bit checkpoint."""
        ops, off, token = self.ops, c["off"], c["token"]
        gate = c["gate"].reshape(-1)[c["perm"].long()]
        # without the gates: they and their gradient belong to SwiGLU's rows
        dact = ops.fp8_matmul(*ops.quant_rows(dout[token.long()]), self.qd["qt"], self.qd["scale_t"], off=off)
        b = ops.swiglu_backward(dact, c["save"], c["save_scale"], gate=gate, off=off, want=("dq", "dqt", "dgate"))
        drows = ops.fp8_matmul(b["dq"], b["dq_scale"], self.q13["qt"], self.q13["scale_t"], off=off)
        tokens = token.numel()
        dWd = ops.fp8_wgrad(*ops.quant_cols(dout, off=off, row_index=token), b["actt"], b["actt_scale"], off=off, tokens=tokens)
        dW13 = ops.fp8_wgrad(b["dqt"], b["dqt_scale"], *ops.requant_cols(c["q"], c["scale"], off=off, row_index=token),
                             off=off, tokens=tokens)
        return drows, dWd, dW13, b["dgate"][c["rows"]]

    def quantise4(self, group=128, zero=False):
        """The experts in 4 bits, for decode()."""
        self.w13_4, self.wd_4 = (self.ops.quant_w4(w, group, zero) for w in (self.W13, self.Wd))

    def decode(self, x, residual):
        """(h, out) of a few tokens with the experts in 4 bits."""
        n = self.ops.rms_norm(x, self.norm_w, residual, self.eps, want=("h", "y"))
        r = self.ops.gate(n["y"].float() @ self.Wr.t(), self.k, bias=self.bias, dispatch=False, **self.route)
        return n["h"], self.ops.w4_experts(n["y"], r["idx"], r["gate"], self.w13_4, self.wd_4)

    def backward(self, dout, ctx, dh=None):
        """Gradients of x (and residual), and of every weight, for dL/dout (and dL/dh from elsewhere)."""
        ops, c, k, off = self.ops, ctx, self.k, ctx["off"]
        if "save" in c:                                          # kept by a forward pass with save8
            drows, dWd, dW13, dgate = self._backward8(dout, c)
            y = (c["h"].float() * c["rstd"][:, None] * self.norm_w.float()).bfloat16()
            return self._backward_router(c, y, drows, dWd, dW13, dgate, dh)
        gate = c["gate"].reshape(-1)[c["perm"].long()]
        up = dout[c["token"].long()]
        dgate = (dout.float()[:, None, :] * c["o"][c["rows"]].float()).sum(2)
        do = (up.float() * gate[:, None]).bfloat16()
        dact = ops.fp8_matmul(*ops.quant_rows(do), self.qd["qt"], self.qd["scale_t"], off=off).float()
        g, u = c["gu"][:, :self.f].float(), c["gu"][:, self.f:].float()
        s = torch.sigmoid(g)
        act = (g * s * u).bfloat16()
        dWd = ops.fp8_wgrad(*ops.quant_cols(do, off=off), *ops.quant_cols(act, off=off), off=off)
        dgu = torch.cat([dact * u * s * (1 + g * (1 - s)), dact * g * s], 1).bfloat16()
        drows = ops.fp8_matmul(*ops.quant_rows(dgu), self.q13["qt"], self.q13["scale_t"], off=off)
        dW13 = ops.fp8_wgrad(*ops.quant_cols(dgu, off=off), *ops.quant_cols(c["y"], off=off, row_index=c["token"]),
                             off=off)
        return self._backward_router(c, c["y"], drows, dWd, dW13, dgate, dh)

    def _backward_router(self, c, y, drows, dWd, dW13, dgate, dh):
        ops = self.ops
        dl = ops.gate_backward(c["logits"], c["idx"], dgate.contiguous(), router=self.route["router"],
                               route_scale=self.route["route_scale"])["dlogits"]
        dy = (drows[c["rows"]].float().sum(1) + dl @ self.Wr).bfloat16()
        b = ops.rms_norm_backward(dy, c["h"], self.norm_w, c["rstd"], dh=dh)
        return dict(dx=b["dx"], dnorm=b["dw"], dWr=dl.t() @ y.float(), dW13=dW13, dWd=dWd)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    d, f, E, k = 2048, 1408, 64, 6
    block = Fp8ExpertBlock(d, f, E, k, n_groups=8, topk_groups=4)
    x, res = (torch.randn(a.tokens, d, device="cuda").bfloat16() for _ in range(2))
    dout = torch.randn(a.tokens, d, device="cuda").bfloat16()

    def timed(fn, n=10):
        for _ in range(3):
            fn()
        t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        t[0].record()
        for _ in range(n):
            fn()
        t[1].record()
        torch.cuda.synchronize()
        return t[0].elapsed_time(t[1]) / n

    _, _, ctx = block.forward(x, res)
    print(f"d={d} f={f} experts={E} top-{k}, {a.tokens} tokens: forward {timed(lambda: block.forward(x, res)):.3f} ms, "
          f"backward {timed(lambda: block.backward(dout, ctx)):.3f} ms; one token forward "
          f"{timed(lambda: block.forward(x[:1], res[:1])):.3f} ms; device status {block.ops.status()}")
    block.save8 = True
    _, _, ctx8 = block.forward(x, res)
    kept = lambda c: sum(v.numel() * v.element_size() for v in c.values()) / 2 ** 20  # noqa: E731
    block.quantise4()
    print(f"with 8-bit checkpoints: forward {timed(lambda: block.forward(x, res)):.3f} ms, backward "
          f"{timed(lambda: block.backward(dout, ctx8)):.3f} ms, kept {kept(ctx8):.0f} MiB instead of {kept(ctx):.0f}; 4-bit "
          f"experts, one token {timed(lambda: block.decode(x[:1], res[:1])):.3f} ms, 16 tokens "
          f"{timed(lambda: block.decode(x[:16], res[:16])):.3f} ms")


if __name__ == "__main__":
    main()
