/*
 * moe_ops.h -- C ABI of the operators around the expert layer (moe.h), for callers
 * that compose their own blocks:
 *   moe_norm_*    RMS norm with the residual's addition and an 8-bit output
 *   moe_gate_*    routing from router logits: bias, groups, top-k, dispatch
 *   moe_quant_*   e4m3 codes with one fp32 scale for each 128 values
 *   moe_fp8_*     products of such operands, dense and by experts' rows
 *
 * Conventions are moe.h's: device pointers owned by the caller, row-major
 * layouts, every call only enqueues on `stream` and never synchronises, bad
 * arguments return an error code on the host and launch nothing, results are
 * bit-identical between runs, no floating-point atomics. None of the calls needs
 * a layer handle; they take a moe_ops handle, whose only device memory is its
 * status word. A wait that ran out (MOE_ERR_TIMEOUT) or an index out of range
 * that a kernel read on the device (MOE_ERR_DEVICE_INDEX; the access is left
 * out) is recorded there: read it with moe_ops_get_status. A handle may be used
 * from several streams and host threads. The device it was created on must be
 * current.
 *
 * 8-bit operands. A block of 128 values v (the last one of a row may be
 * shorter) with the largest magnitude m is held as
 *   scale = m / 448        codes = e4m3(448 v / m), to nearest, ties to even
 * (e4m3: 448 is its largest value; a block of zeros has scale 0 and codes 0), so
 * that code * scale stands for the value. 448 v is exact for bf16 values and the
 * quotient is rounded once before the rounding to e4m3, so ties stay ties. A NaN
 * or an infinity makes its whole block NaN when it is read back. Values of 2^119
 * and more saturate.
 */
#ifndef MOE_GB300_OPS_H
#define MOE_GB300_OPS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moe_ops_s* moe_ops;

moe_status moe_ops_create(moe_ops* out);
moe_status moe_ops_destroy(moe_ops ops);
/* Wait for `stream`, then read and clear the status word (in one step: an error that work on another stream records
 * meanwhile is returned by this call or by the next). */
moe_status moe_ops_get_status(moe_ops ops, void* stream, int* device_status);
/* Kernels that the operators launched since moe_ops_create (host counter). */
moe_status moe_ops_launch_count(moe_ops ops, long long* launches);

/* ---- RMS norm. dtype (MOE_BF16 or MOE_FP32) is the type of x, residual, weight,
 * h and y. Row t:
 *   h = round(x + residual)   (residual NULL: h = x, and output h is a copy)
 *   rstd = 1 / sqrt(mean(h^2) + eps)         y = h * rstd * weight
 * The norm is taken of h as it is stored, which is what the backward pass reads.
 * Outputs, each nullable (one at least): h [T, d], y [T, d] in dtype, q [T, d]
 * e4m3 with scale [T, ceil(d/128)] fp32 (both or neither; quantised from the
 * unrounded y), rstd [T] fp32. h may be x or residual itself. Rows of x and
 * residual start ld_x and ld_res elements apart (>= d); weight [d]; outputs are
 * dense. d is a multiple of 8 up to 16384; pointers and row starts 16-byte
 * aligned (q 8-byte). T = 0 does nothing. */
moe_status moe_norm_forward(moe_ops ops, int dtype, const void* x, long long ld_x, const void* residual,
                            long long ld_res, const void* weight, int T, int d, float eps, void* h, void* y,
                            void* q, float* scale, float* rstd, void* stream);
/* dy [T, d] = dL/dy (through an 8-bit output: the gradient of the values that it
 * stands for); dh (nullable) = the gradient that arrives at h from elsewhere.
 *   n = h rstd, u = dy weight:  dx = dh + rstd (u - n mean(u n)),  dw = sum_t dy n
 * dx [T, d] in dtype is the gradient of x and of residual alike (it may be dh or
 * dy itself); dw [d] fp32; either may be NULL. Sums over rows have a fixed order.
 * All arrays dense. workspace: moe_norm_workspace_size bytes, 16-byte aligned. */
moe_status moe_norm_workspace_size(int T, int d, size_t* bytes);
moe_status moe_norm_backward(moe_ops ops, int dtype, const void* dy, const void* dh, const void* h,
                             const void* weight, const float* rstd, int T, int d, void* dx, float* dw,
                             void* workspace, void* stream);

/* ---- Routing. */
typedef struct {
  int E;              /* experts, 1..256 */
  int k;              /* experts per token, 1..min(8, topk_groups * E / n_groups) */
  int router;         /* moe_router_kind: scores p = softmax(l) over all E, or sigmoid(l) */
  int renorm;         /* 1: gates divided by the sum of the selected scores (+ 1e-20) */
  float route_scale;  /* multiplies the gates */
  int n_groups;       /* groups of E / n_groups consecutive experts, 1..32, dividing E */
  int topk_groups;    /* groups that stay, 1..n_groups */
} moe_gate_config;

/* logits [T, E] fp32 -> key = p + bias (bias [E] fp32, NULL: zeros; selection
 * only). Groups are scored by the sum of their two largest keys (one, in groups of
 * one expert); the topk_groups best stay; of their experts the k with the largest
 * keys are selected, largest first. Equal groups and keys go to the lower index.
 * Selections are those of keys computed in 64 bits: keys of 32 bits decide where
 * their error cannot change the outcome, keys of 64 bits elsewhere. An expert
 * whose logit is -inf, or whose key is NaN or -inf, comes after all others (its
 * gate is 0 for a logit of -inf); one with a bias of +inf comes first, and so does
 * its group. A row with no expert left selects the lowest indexes with gates 0.
 * Outputs: idx [T, k] int32, gate [T, k] fp32 (required), and the dispatch of
 * moe_route, all four or none: cnt [E], off [E+1], perm [T*k], inv [T*k].
 * workspace (moe_gate_workspace_size bytes, 16-byte aligned; NULL without a
 * dispatch or where that is 0). T * k < 2^30. */
moe_status moe_gate_workspace_size(const moe_gate_config* cfg, int T, size_t* bytes);
moe_status moe_gate_forward(moe_ops ops, const moe_gate_config* cfg, const float* logits, const float* bias, int T,
                            int32_t* idx, float* gate, int32_t* cnt, int32_t* off, int32_t* perm, int32_t* inv,
                            void* workspace, void* stream);
/* dgate [T, k] = dL/dgate of the selection idx -> dlogits [T, E] fp32, written whole
 * (zeros where nothing flows; renormalised softmax gates reach the other logits
 * where the selected scores' sum is near the 1e-20 added to it). The bias and the selection get no gradient. Only
 * cfg's E, k, router, renorm and route_scale are read. */
moe_status moe_gate_backward(moe_ops ops, const moe_gate_config* cfg, const float* logits, const int32_t* idx,
                             const float* dgate, int T, float* dlogits, void* stream);

/* ---- Quantisers of bf16 arrays; src rows ld elements apart, 16-byte aligned, ld and C multiples of 8. */
/* Rows: src [T, C] -> q [T, C], scale [T, ceil(C/128)]. swiglu = 1: src is [T, 2C]
 * (gate half, up half) and silu(gate) * up (32 bits) is quantised. */
moe_status moe_quant_rows(moe_ops ops, const void* src, long long ld, int T, int C, int swiglu, void* q,
                          float* scale, void* stream);
/* Along the token axis, transposed: q [C, Tp], scale [Tp/128, C], Tp = moe_quant_cols_rows(T, G).
 * Row i of src is gathered at row_index[i] (nullable; of src_rows rows). Tokens
 * off[g] .. off[g+1] of segment g (off NULL: one segment of T, G = 1) start at
 * the next multiple of 128 after the segments before it and are padded with zeros up to one;
 * what lies behind the last segment is not written. C is a multiple of 8. */
moe_status moe_quant_cols_rows(int T, int G, int* Tp);
moe_status moe_quant_cols(moe_ops ops, const void* src, long long ld, int src_rows, int T, int C,
                          const int32_t* off, int G, const int32_t* row_index, void* q, float* scale, void* stream);
/* Weights w [G, N, K] dense, 128 x 128 blocks: q [G, N, K], scale [G, ceil(N/128), ceil(K/128)] and (both nullable)
 * the same codes transposed, qt [G, K, N], scale_t [G, ceil(K/128), ceil(N/128)], for gradients of the rows. */
moe_status moe_quant_blocks(moe_ops ops, const void* w, int G, int N, int K, void* q, float* scale, void* qt,
                            float* scale_t, void* stream);

/* ---- Products of 8-bit operands, sums in fp32, one rounding to out_dtype (MOE_BF16 or MOE_FP32) at the end.
 * K (the reduction's length) is a multiple of 16; code arrays 16-byte aligned. */
/* c[m, n] = sum over K of a[r(m), k] b[g(m), n, k], r(m) = row_index[m] or m:
 *   a [a_rows, K], a_scale [a_rows, ceil(K/128)]; b [G, N, K], b_scale [G, ceil(N/128), ceil(K/128)]; c [M, N].
 * off (nullable, device, G+1 ascending within 0 .. M): rows off[g] .. off[g+1] meet b[g], rows of no segment
 * are not written, whatever row_index holds there; NULL: G = 1. G is 1..256. A row_index out of range reads zeros and
 * records MOE_ERR_DEVICE_INDEX.
 * Forward: a = quantised rows, b = weights. Gradient of the rows: a = quantised dc, b = transposed weights. */
moe_status moe_fp8_matmul(moe_ops ops, const void* a, const float* a_scale, int a_rows, const int32_t* row_index,
                          int M, const void* b, const float* b_scale, const int32_t* off, int G, int N, int K,
                          void* c, int out_dtype, void* workspace, void* stream);
/* Bytes of workspace (16-byte aligned; 0: it may be NULL) of a call with these sizes, gathered = 1 with a row_index:
 * many gathered rows are put in order first. */
moe_status moe_fp8_matmul_workspace_size(int M, int G, int K, int gathered, size_t* bytes);
/* Gradient of the weights: c[g, n, k] = sum over the tokens t of segment g of dc[t, n] x[t, k], from moe_quant_cols
 * of both: dct [N, Tp], dct_scale [Tp/128, N], xt [K, Tp], xt_scale [Tp/128, K]; c [G, N, K], zeros for a segment
 * without tokens. T and off as they were given to moe_quant_cols; N and K multiples of 8, scales 16-byte aligned. */
moe_status moe_fp8_wgrad(moe_ops ops, const void* dct, const float* dct_scale, const void* xt, const float* xt_scale,
                         int T, const int32_t* off, int G, int N, int K, void* c, int out_dtype, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_OPS_H */
