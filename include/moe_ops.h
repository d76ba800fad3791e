/*
 * moe_ops.h -- C ABI of the operators around the expert layer (moe.h), for callers
 * that compose their own blocks:
 *   moe_norm_*    RMS norm with the residual's addition and an 8-bit output
 *   moe_gate_*    routing from router logits: bias, groups, top-k, dispatch
 *   moe_quant_*   e4m3 codes with one fp32 scale for each 128 values
 *   moe_fp8_*     products of such operands, dense and by experts' rows
 *   moe_swiglu_*, moe_requant_cols   SwiGLU with an 8-bit checkpoint, and its gradient from it
 *   moe_quant_w4, moe_w4_*   4-bit weights with a scale for a group of values: products of
 *                 few rows, and the experts' layer of a few tokens
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

/* ---- SwiGLU with an 8-bit checkpoint: gu = (g, u) halves of a row, act = silu(g) * u.
 * gu [T, 2f] bf16, rows ld elements apart; f (below 2^28) and ld multiples of 8, gu and act 16-byte aligned. The
 * exponential and the quotient are the fast ones: act is off by up to (5 + 1.2 |g|) 2^-23 of itself before it is rounded
 * or quantised, and 0 where g is below -87.3. Outputs (one at least): act [T, f] bf16; q [T, f] with scale
 * [T, ceil(f/128)], act's codes (of the unrounded values, as moe_quant_rows with swiglu); save [T, 2f] with save_scale
 * [T, 2 ceil(f/128)], the codes of g and of u, blocks of 128 within each half, the gate's scales first (what the
 * backward pass reads; with f a multiple of 128 they are moe_quant_rows of gu). Codes 8-byte aligned. */
moe_status moe_swiglu_forward(moe_ops ops, const void* gu, long long ld, int T, int f, void* act, void* q, float* scale,
                              void* save, float* save_scale, void* stream);
/* With g, u the values of save, s = sigmoid(g), dact [T, f] bf16 the gradient of act (rows ld elements apart, a multiple
 * of 8, 16-byte aligned) and gate [T] fp32 a factor of each row (NULL: 1):
 *   dg = gate dact u s (1 + g (1 - s))     du = gate dact g s     dgate[t] = sum_f act dact     act' = gate act
 * s is off by up to (4 + 0.7 |g|) 2^-23 of itself (0 where g is below -87.3), everything else is 32-bit arithmetic.
 * gate: where a row's product is weighted after the down product, out = sum gate (act Wd^T), dact is (dout Wd) without
 * the gate, dgate needs no output of that product, and dWd is act' along the tokens times dout.
 * Outputs, one at least, each pair both or neither, values quantised unrounded: dgu = (dg, du) [T, 2f] bf16; dq [T, 2f]
 * with dq_scale [T, 2f/128], its rows' codes (f a multiple of 128); dqt [2f, Tp] with dqt_scale [Tp/128, 2f], its codes
 * along the tokens, and with them actt [f, Tp], actt_scale [Tp/128, f], those of act', segments and padding as in
 * moe_quant_cols; dgate [T]. off (nullable, G+1 ascending within 0 .. T) tells the segments; rows of no segment are not
 * written. save is 8-byte aligned, dgu, dq, dqt and actt 16-byte. workspace: moe_swiglu_workspace_size bytes, 16-byte
 * aligned, for dgate where that is above 0; calls that may run at once need one each. */
moe_status moe_swiglu_workspace_size(int T, int f, size_t* bytes);
moe_status moe_swiglu_backward(moe_ops ops, const void* save, const float* save_scale, const void* dact, long long ld,
                               const float* gate, int T, int f, const int32_t* off, int G, void* dgu, void* dq,
                               float* dq_scale, void* dqt, float* dqt_scale, void* actt, float* actt_scale,
                               float* dgate, void* workspace, void* stream);
/* moe_quant_cols of rows that are held in 8 bits (q [src_rows, C], scale [src_rows, ceil(C/128)], as moe_quant_rows and
 * moe_norm_forward give them): the values code * scale, quantised along the tokens. C is a multiple of 8 below 2^28; q
 * 8-byte aligned, qt and scale_t 16-byte. */
moe_status moe_requant_cols(moe_ops ops, const void* q, const float* scale, int src_rows, int T, int C,
                            const int32_t* off, int G, const int32_t* row_index, void* qt, float* scale_t, void* stream);

/* ---- 4-bit weights. A group of `group` (32, 64 or 128; the last one of a row may be shorter) consecutive values along
 * K shares a scale and, where zero is given, a zero point:
 *   w = (code - zero) * scale      codes 0..15, zero 0..15 (8 without zero points)
 * codes [G, N, K/8] words of eight values, value 2i in bits 4i .. 4i+3 and value 2i+1 in bits 16+4i .. 16+4i+3;
 * scale [G, ceil(K/group), N] bf16; zero [G, ceil(K/group), N] bytes, or NULL. N is a multiple of 8, K of 32; codes and
 * scale 16-byte aligned, zero 8-byte. */
typedef struct {
  const uint32_t* codes;
  const void* scale;
  const uint8_t* zero;
  int group;
} moe_w4;

/* w [G, N, K] bf16, dense, to codes, scale and (nullable) zero. With m the largest magnitude of a group:
 *   scale = bf16(m / 7)              code = clamp(rint(w / scale) + 8)
 * with zero, lo and hi being the smallest and the largest of a group's values and 0:
 *   scale = bf16((hi - lo) / 15)     zero = clamp(rint(-lo / scale))     code = clamp(rint(w / scale) + zero)
 * clamped to 0..15, quotients in fp32 (that of a span hi - lo beyond fp32's largest value too). A group of zeros has
 * scale 0 and reads zeros; one that holds a NaN or an infinity reads NaN, no other one does. */
moe_status moe_quant_w4(moe_ops ops, const void* w, int G, int N, int K, int group, uint32_t* codes, void* scale,
                        uint8_t* zero, void* stream);
/* c[m, n] = sum over K of x[r(m), k] w[g(m), n, k], r(m) = row_index[m] or m: x [x_rows, K] bf16, rows ld_x elements
 * apart (a multiple of 8, 16-byte aligned); c [M, N] of out_dtype (MOE_BF16 or MOE_FP32); off, G, row_index and rows of
 * no segment as in moe_fp8_matmul; c 16-byte aligned. The values of x and code - zero meet on the tensor cores
 * unrounded, sums are fp32 (a group's before its scale: |x| up to 2^116 cannot overflow), one rounding at the end. Made
 * for few rows: the weights are decoded once for every 8 rows of a segment, so past some 32 rows the 8-bit products are
 * the faster ones. */
moe_status moe_w4_matmul(moe_ops ops, const void* x, long long ld_x, int x_rows, const int32_t* row_index, int M,
                         const moe_w4* w, const int32_t* off, int G, int N, int K, void* c, int out_dtype, void* stream);

typedef struct {
  int E;              /* routed experts, 1..256 */
  int n_shared;       /* experts E .. E+n_shared-1 that every token takes with a gate of 1, 0..8 */
  int k;              /* routed experts of a token, 1..8 */
  int d;              /* a multiple of 32 up to 2^20 */
  int f;              /* likewise */
} moe_w4_config;
/* The experts' layer of T = 0..64 tokens, behind the routing, in two kernels:
 *   y_t = sum_j gate[t, j] FFN_idx[t, j](x_t) + sum of the shared experts' FFN(x_t)
 *   FFN_e(x) = (silu(x Wg[e]^T) * (x Wu[e]^T)) Wd[e]^T
 * x [T, d] bf16, rows ld_x elements apart (a multiple of 8, 16-byte aligned); idx [T, k], gate [T, k] fp32 as
 * moe_gate_forward gives them (an expert may be named twice by a token: its gates add up); w13 of [E+n_shared, 2f, d]
 * (gate half, up half), wd of [E+n_shared, d, f], with one group size and both with zero points or neither; y [T, d]
 * of out_dtype, 16-byte aligned. An index outside 0..E-1 is left out and records MOE_ERR_DEVICE_INDEX. h, with the gate
 * in it, is kept to 16 bits of mantissa (24 for fp32 outputs), the other sums in fp32; one rounding at the end. Only
 * experts in use are read. workspace: moe_w4_experts_workspace_size bytes, 16-byte aligned; calls that may run at once
 * need one each. */
moe_status moe_w4_experts_workspace_size(const moe_w4_config* cfg, int T, size_t* bytes);
moe_status moe_w4_experts(moe_ops ops, const moe_w4_config* cfg, const void* x, long long ld_x, int T,
                          const int32_t* idx, const float* gate, const moe_w4* w13, const moe_w4* wd, void* y,
                          int out_dtype, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_OPS_H */
