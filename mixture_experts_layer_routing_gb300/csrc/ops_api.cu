// Host side of include/moe_ops.h: argument checks and launches. Every call only enqueues on the caller's stream.
#include <cmath>
#include <new>

#include "ops.h"

using namespace moe;

namespace {

inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// The handle's device has to be current: its status word lives there, and the kernels' attributes were set there.
moe_status check_handle(moe_ops o) {
  int dev = -1;
  if (!o) return MOE_ERR_INVALID_ARG;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  return dev == o->device ? MOE_OK : MOE_ERR_INVALID_ARG;
}

#define CHECK(cond, code)      \
  do {                         \
    if (!(cond)) return code;  \
  } while (0)
#define HANDLE(o)                                \
  do {                                           \
    const moe_status st_ = check_handle(o);      \
    if (st_ != MOE_OK) return st_;               \
  } while (0)
// A launch's result, with the kernels it launched counted.
#define DONE(call)                                                           \
  do {                                                                       \
    long long n_ = 0;                                                        \
    const cudaError_t e_ = (call);                                           \
    ops->launches += n_;                                                     \
    if (e_ != cudaSuccess) cudaGetLastError();                               \
    return e_ == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;                        \
  } while (0)

// Reads and clears in one step: what a kernel on another stream records meanwhile is read here or stays.
__global__ void take_status_kernel(int* status, int* out) { *out = atomicExch(status, 0); }

moe_status check_gate(const moe_gate_config* c, int T) {
  CHECK(c && c->E >= 1 && c->k >= 1 && T >= 0, MOE_ERR_INVALID_ARG);
  CHECK(c->router == MOE_ROUTER_SOFTMAX || c->router == MOE_ROUTER_SIGMOID, MOE_ERR_INVALID_ARG);
  CHECK(std::isfinite(c->route_scale), MOE_ERR_INVALID_ARG);
  CHECK(c->E <= 256 && c->k <= 8, MOE_ERR_UNSUPPORTED);
  CHECK(c->k <= c->E, MOE_ERR_INVALID_ARG);
  CHECK((long long)T * c->k < (1 << 30) && T < (1 << 30), MOE_ERR_UNSUPPORTED);
  return MOE_OK;
}

// 4-bit weights [G, N, K].
moe_status check_w4(const moe_w4* w, int N, int K) {
  CHECK(w && w->codes && w->scale, MOE_ERR_INVALID_ARG);
  CHECK(w->group == 32 || w->group == 64 || w->group == 128, MOE_ERR_UNSUPPORTED);
  CHECK(N % 8 == 0 && K % 32 == 0 && N < (1 << 28) && K < (1 << 28), MOE_ERR_UNSUPPORTED);
  CHECK(aligned(w->codes, 16) && aligned(w->scale, 16) && aligned(w->zero, 8), MOE_ERR_UNSUPPORTED);
  return MOE_OK;
}

moe_status check_w4_experts(const moe_w4_config* c, int T) {
  CHECK(c && c->E >= 1 && c->k >= 1 && c->n_shared >= 0 && c->d >= 1 && c->f >= 1 && T >= 0, MOE_ERR_INVALID_ARG);
  CHECK(c->E <= 256 && c->k <= 8 && c->n_shared <= 8 && T <= 64, MOE_ERR_UNSUPPORTED);
  CHECK(c->d % 32 == 0 && c->f % 32 == 0 && c->d <= (1 << 20) && c->f <= (1 << 20), MOE_ERR_UNSUPPORTED);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_ops_create(moe_ops* out) {
  CHECK(out, MOE_ERR_INVALID_ARG);
  *out = nullptr;
  moe_ops_s* o = new (std::nothrow) moe_ops_s();
  CHECK(o, MOE_ERR_CUDA);
  if (cudaGetDevice(&o->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&o->sms, cudaDevAttrMultiProcessorCount, o->device) != cudaSuccess ||
      fp8_init(&o->pairs) != cudaSuccess || o->pairs < 1 || cudaMalloc(&o->status, sizeof(int)) != cudaSuccess) {
    cudaGetLastError();
    delete o;
    return MOE_ERR_CUDA;
  }
  if (cudaMemset(o->status, 0, sizeof(int)) != cudaSuccess) {
    cudaFree(o->status);
    delete o;
    return MOE_ERR_CUDA;
  }
  *out = o;
  return MOE_OK;
}

moe_status moe_ops_destroy(moe_ops ops) {
  CHECK(ops, MOE_ERR_INVALID_ARG);
  const cudaError_t e = cudaFree(ops->status);
  delete ops;
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_ops_get_status(moe_ops ops, void* stream, int* device_status) {
  HANDLE(ops);
  CHECK(device_status, MOE_ERR_INVALID_ARG);
  cudaStream_t s = (cudaStream_t)stream;
  int v = 0;
  int* word = nullptr;   // the call's own: another one may be taking the status on another stream
  cudaError_t e = cudaMallocAsync(&word, sizeof(int), s);
  if (e == cudaSuccess) {
    take_status_kernel<<<1, 1, 0, s>>>(ops->status, word);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaMemcpyAsync(&v, word, sizeof(int), cudaMemcpyDeviceToHost, s);
    const cudaError_t freed = cudaFreeAsync(word, s);
    if (e == cudaSuccess) e = freed;
  }
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  *device_status = v;
  return MOE_OK;
}

moe_status moe_ops_launch_count(moe_ops ops, long long* launches) {
  CHECK(ops && launches, MOE_ERR_INVALID_ARG);
  *launches = ops->launches.load();
  return MOE_OK;
}

moe_status moe_norm_forward(moe_ops ops, int dtype, const void* x, long long ld_x, const void* residual,
                            long long ld_res, const void* weight, int T, int d, float eps, void* h, void* y, void* q,
                            float* scale, float* rstd, void* stream) {
  CHECK(ops, MOE_ERR_INVALID_ARG);
  CHECK(dtype == MOE_BF16 || dtype == MOE_FP32, MOE_ERR_INVALID_ARG);
  CHECK(T >= 0 && d >= 1 && eps >= 0.f && std::isfinite(eps), MOE_ERR_INVALID_ARG);
  CHECK(d % 8 == 0 && d <= 16384, MOE_ERR_UNSUPPORTED);
  if (T == 0) return MOE_OK;   // arrays without rows may have no address
  CHECK(h || y || q || rstd, MOE_ERR_INVALID_ARG);
  CHECK((q != nullptr) == (scale != nullptr), MOE_ERR_INVALID_ARG);
  CHECK(ld_x >= d && (!residual || ld_res >= d), MOE_ERR_INVALID_ARG);
  CHECK(x && weight, MOE_ERR_INVALID_ARG);
  const int unit = dtype == MOE_BF16 ? 8 : 4;   // values in 16 bytes
  CHECK(ld_x % unit == 0 && (!residual || ld_res % unit == 0), MOE_ERR_UNSUPPORTED);
  CHECK(aligned(x, 16) && aligned(residual, 16) && aligned(weight, 16) && aligned(h, 16) && aligned(y, 16) &&
            aligned(q, 8) && aligned(scale, 4) && aligned(rstd, 4),
        MOE_ERR_UNSUPPORTED);
  // in place only row by row
  CHECK((h != x || ld_x == d) && (!h || h != residual || ld_res == d), MOE_ERR_INVALID_ARG);
  HANDLE(ops);
  DONE(norm_forward(ops, dtype, x, ld_x, residual, ld_res, weight, T, d, eps, h, y, q, scale, rstd,
                    (cudaStream_t)stream, &n_));
}

moe_status moe_norm_workspace_size(int T, int d, size_t* bytes) {
  CHECK(T >= 0 && d >= 1 && bytes, MOE_ERR_INVALID_ARG);
  *bytes = sizeof(float) * (size_t)norm_partials(T, d) * d;
  return MOE_OK;
}

moe_status moe_norm_backward(moe_ops ops, int dtype, const void* dy, const void* dh, const void* h,
                             const void* weight, const float* rstd, int T, int d, void* dx, float* dw,
                             void* workspace, void* stream) {
  CHECK(ops, MOE_ERR_INVALID_ARG);
  CHECK(dtype == MOE_BF16 || dtype == MOE_FP32, MOE_ERR_INVALID_ARG);
  CHECK(T >= 0 && d >= 1, MOE_ERR_INVALID_ARG);
  CHECK(d % 8 == 0 && d <= 16384, MOE_ERR_UNSUPPORTED);
  if (T == 0) {
    if (!dw) return MOE_OK;
    HANDLE(ops);
    return cudaMemsetAsync(dw, 0, sizeof(float) * d, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  CHECK(dy && h && weight && rstd && (dx || dw), MOE_ERR_INVALID_ARG);
  CHECK(aligned(dy, 16) && aligned(dh, 16) && aligned(h, 16) && aligned(weight, 16) && aligned(dx, 16) &&
            aligned(rstd, 4) && aligned(dw, 4),
        MOE_ERR_UNSUPPORTED);
  CHECK(!dw || (workspace && aligned(workspace, 16)), MOE_ERR_WORKSPACE);
  HANDLE(ops);
  DONE(norm_backward(ops, dtype, dy, dh, h, weight, rstd, T, d, dx, dw, (float*)workspace, (cudaStream_t)stream, &n_));
}

moe_status moe_gate_workspace_size(const moe_gate_config* cfg, int T, size_t* bytes) {
  const moe_status st = check_gate(cfg, T);
  if (st != MOE_OK) return st;
  CHECK(bytes, MOE_ERR_INVALID_ARG);
  *bytes = gate_workspace(*cfg, T);
  return MOE_OK;
}

moe_status moe_gate_forward(moe_ops ops, const moe_gate_config* cfg, const float* logits, const float* bias, int T,
                            int32_t* idx, float* gate, int32_t* cnt, int32_t* off, int32_t* perm, int32_t* inv,
                            void* workspace, void* stream) {
  CHECK(ops, MOE_ERR_INVALID_ARG);
  const moe_status st = check_gate(cfg, T);
  if (st != MOE_OK) return st;
  CHECK(cfg->n_groups >= 1 && cfg->topk_groups >= 1 && cfg->topk_groups <= cfg->n_groups &&
            cfg->E % cfg->n_groups == 0 && cfg->k <= cfg->topk_groups * (cfg->E / cfg->n_groups),
        MOE_ERR_INVALID_ARG);
  CHECK(cfg->n_groups <= kMaxGroups, MOE_ERR_UNSUPPORTED);
  const int given = (cnt != nullptr) + (off != nullptr) + (perm != nullptr) + (inv != nullptr);
  if (T > 0) {
    CHECK(logits && idx && gate && (given == 0 || given == 4), MOE_ERR_INVALID_ARG);
    CHECK(given == 0 || gate_workspace(*cfg, T) == 0 || (workspace && aligned(workspace, 16)), MOE_ERR_WORKSPACE);
  }
  HANDLE(ops);
  if (T == 0) {   // perm and inv have no entries
    if (!cnt || !off) return MOE_OK;
    const bool ok = cudaMemsetAsync(cnt, 0, sizeof(int) * cfg->E, (cudaStream_t)stream) == cudaSuccess &&
                    cudaMemsetAsync(off, 0, sizeof(int) * (cfg->E + 1), (cudaStream_t)stream) == cudaSuccess;
    return ok ? MOE_OK : MOE_ERR_CUDA;
  }
  DONE(gate_forward(ops, *cfg, logits, bias, T, idx, gate, cnt, off, perm, inv, workspace, (cudaStream_t)stream, &n_));
}

moe_status moe_gate_backward(moe_ops ops, const moe_gate_config* cfg, const float* logits, const int32_t* idx,
                             const float* dgate, int T, float* dlogits, void* stream) {
  CHECK(ops, MOE_ERR_INVALID_ARG);
  const moe_status st = check_gate(cfg, T);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  CHECK(logits && idx && dgate && dlogits, MOE_ERR_INVALID_ARG);
  HANDLE(ops);
  DONE(gate_backward(ops, *cfg, logits, idx, dgate, T, dlogits, (cudaStream_t)stream, &n_));
}

moe_status moe_quant_rows(moe_ops ops, const void* src, long long ld, int T, int C, int swiglu, void* q, float* scale,
                          void* stream) {
  CHECK(ops, MOE_ERR_INVALID_ARG);
  if (T == 0) return MOE_OK;
  CHECK(src && q && scale, MOE_ERR_INVALID_ARG);
  CHECK(T >= 0 && C >= 1 && ld >= (swiglu ? 2ll : 1ll) * C, MOE_ERR_INVALID_ARG);
  CHECK(C % 8 == 0 && ld % 8 == 0 && aligned(src, 16) && aligned(q, 8), MOE_ERR_UNSUPPORTED);
  CHECK((long long)T * ceil_div(C, kScaleBlock) < (1ll << 31), MOE_ERR_UNSUPPORTED);
  HANDLE(ops);
  DONE(quant_rows(ops, src, ld, T, C, swiglu, q, scale, (cudaStream_t)stream, &n_));
}

moe_status moe_quant_cols_rows(int T, int G, int* Tp) {
  CHECK(Tp && T >= 0 && G >= 1 && G <= kMaxSegs, MOE_ERR_INVALID_ARG);
  CHECK(T <= (1 << 22), MOE_ERR_UNSUPPORTED);
  *Tp = quant_cols_rows(T, G);
  return MOE_OK;
}

moe_status moe_quant_cols(moe_ops ops, const void* src, long long ld, int src_rows, int T, int C, const int32_t* off,
                          int G, const int32_t* row_index, void* q, float* scale, void* stream) {
  CHECK(ops && T >= 0 && C >= 1 && ld >= C && src_rows >= 0, MOE_ERR_INVALID_ARG);
  CHECK(G >= 1 && G <= kMaxSegs && (off || G == 1), MOE_ERR_INVALID_ARG);
  CHECK(row_index || src_rows >= T, MOE_ERR_INVALID_ARG);
  CHECK(T <= (1 << 22) && C % 8 == 0 && ld % 8 == 0 && aligned(src, 16) && aligned(q, 16), MOE_ERR_UNSUPPORTED);
  CHECK(T == 0 || (src && q && scale), MOE_ERR_INVALID_ARG);
  if (T == 0) return MOE_OK;
  HANDLE(ops);
  DONE(quant_cols(ops, src, ld, src_rows, T, C, off, G, row_index, q, scale, (cudaStream_t)stream, &n_));
}

moe_status moe_quant_blocks(moe_ops ops, const void* w, int G, int N, int K, void* q, float* scale, void* qt,
                            float* scale_t, void* stream) {
  CHECK(ops && w && q && scale, MOE_ERR_INVALID_ARG);
  CHECK(G >= 1 && N >= 1 && K >= 1 && (qt != nullptr) == (scale_t != nullptr), MOE_ERR_INVALID_ARG);
  CHECK(G <= 65535 && ceil_div(N, 128) <= 65535 && N % 8 == 0 && K % 8 == 0 && aligned(w, 16) && aligned(q, 8) &&
            aligned(qt, 8),
        MOE_ERR_UNSUPPORTED);
  HANDLE(ops);
  DONE(quant_blocks(ops, w, G, N, K, q, scale, qt, scale_t, (cudaStream_t)stream, &n_));
}

moe_status moe_fp8_matmul_workspace_size(int M, int G, int K, int gathered, size_t* bytes) {
  CHECK(M >= 0 && G >= 1 && K >= 1 && bytes, MOE_ERR_INVALID_ARG);
  *bytes = fp8_matmul_workspace(M, G, K, gathered != 0);
  return MOE_OK;
}

moe_status moe_fp8_matmul(moe_ops ops, const void* a, const float* a_scale, int a_rows, const int32_t* row_index,
                          int M, const void* b, const float* b_scale, const int32_t* off, int G, int N, int K, void* c,
                          int out_dtype, void* workspace, void* stream) {
  CHECK(ops && M >= 0 && a_rows >= 0 && N >= 1 && K >= 1 && G >= 1, MOE_ERR_INVALID_ARG);
  CHECK(off || G == 1, MOE_ERR_INVALID_ARG);
  CHECK(row_index || a_rows >= M, MOE_ERR_INVALID_ARG);
  CHECK(out_dtype == MOE_BF16 || out_dtype == MOE_FP32, MOE_ERR_INVALID_ARG);
  CHECK(G <= kMaxSegs && K % 16 == 0, MOE_ERR_UNSUPPORTED);
  CHECK(M < (1 << 30) && (long long)G * N < (1ll << 31) && N < (1 << 28) && K < (1 << 28), MOE_ERR_UNSUPPORTED);
  CHECK((ceil_div(M, 128) + (long long)G) * ceil_div(N, 128) < (1ll << 27), MOE_ERR_UNSUPPORTED);   // tiles
  if (M == 0) return MOE_OK;
  CHECK(a && a_scale && a_rows >= 1 && b && b_scale && c, MOE_ERR_INVALID_ARG);
  CHECK(aligned(a, 16) && aligned(b, 16) && aligned(c, 16) && aligned(a_scale, 4) && aligned(b_scale, 4),
        MOE_ERR_UNSUPPORTED);
  CHECK(fp8_matmul_workspace(M, G, K, row_index != nullptr) == 0 || (workspace && aligned(workspace, 16)),
        MOE_ERR_WORKSPACE);
  HANDLE(ops);
  DONE(fp8_matmul(ops, a, a_scale, a_rows, row_index, M, b, b_scale, off, G, N, K, c, out_dtype == MOE_FP32, workspace,
                  (cudaStream_t)stream, &n_));
}

moe_status moe_fp8_wgrad(moe_ops ops, const void* dct, const float* dct_scale, const void* xt, const float* xt_scale,
                         int T, const int32_t* off, int G, int N, int K, void* c, int out_dtype, void* stream) {
  CHECK(ops && c && T >= 0 && N >= 1 && K >= 1 && G >= 1, MOE_ERR_INVALID_ARG);
  CHECK(off || G == 1, MOE_ERR_INVALID_ARG);
  CHECK(out_dtype == MOE_BF16 || out_dtype == MOE_FP32, MOE_ERR_INVALID_ARG);
  CHECK(G <= kMaxSegs && T <= (1 << 22) && N < (1 << 28) && K < (1 << 28), MOE_ERR_UNSUPPORTED);
  CHECK(N % 8 == 0 && K % 8 == 0 && aligned(dct, 16) && aligned(xt, 16) && aligned(dct_scale, 16) &&
            aligned(xt_scale, 16) && aligned(c, 16),
        MOE_ERR_UNSUPPORTED);
  CHECK((long long)ceil_div(N, 128) * ceil_div(K, 128) < (1ll << 27) / G, MOE_ERR_UNSUPPORTED);
  CHECK(T == 0 || (dct && dct_scale && xt && xt_scale), MOE_ERR_INVALID_ARG);
  HANDLE(ops);
  if (T == 0) {
    const size_t bytes = (size_t)G * N * K * (out_dtype == MOE_FP32 ? 4 : 2);
    return cudaMemsetAsync(c, 0, bytes, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  DONE(fp8_wgrad(ops, dct, dct_scale, xt, xt_scale, T, off, G, N, K, c, out_dtype == MOE_FP32, (cudaStream_t)stream,
                 &n_));
}

moe_status moe_swiglu_forward(moe_ops ops, const void* gu, long long ld, int T, int f, void* act, void* q, float* scale,
                              void* save, float* save_scale, void* stream) {
  CHECK(ops && T >= 0 && f >= 1 && ld >= 2ll * f, MOE_ERR_INVALID_ARG);
  CHECK(f % 8 == 0 && ld % 8 == 0 && f < (1 << 28), MOE_ERR_UNSUPPORTED);
  if (T == 0) return MOE_OK;
  CHECK(gu && (act || q || save) && (q != nullptr) == (scale != nullptr) && (save != nullptr) == (save_scale != nullptr),
        MOE_ERR_INVALID_ARG);
  CHECK(aligned(gu, 16) && aligned(act, 16) && aligned(q, 8) && aligned(save, 8), MOE_ERR_UNSUPPORTED);
  CHECK((long long)T * ceil_div(f, kScaleBlock) < (1ll << 31), MOE_ERR_UNSUPPORTED);
  HANDLE(ops);
  DONE(swiglu_forward(ops, gu, ld, T, f, act, q, scale, save, save_scale, (cudaStream_t)stream, &n_));
}

moe_status moe_swiglu_workspace_size(int T, int f, size_t* bytes) {
  CHECK(T >= 0 && f >= 1 && bytes, MOE_ERR_INVALID_ARG);
  CHECK(f < (1 << 28), MOE_ERR_UNSUPPORTED);
  *bytes = swiglu_workspace(T, f);
  return MOE_OK;
}

moe_status moe_swiglu_backward(moe_ops ops, const void* save, const float* save_scale, const void* dact, long long ld,
                               const float* gate, int T, int f, const int32_t* off, int G, void* dgu, void* dq,
                               float* dq_scale, void* dqt, float* dqt_scale, void* actt, float* actt_scale,
                               float* dgate, void* workspace, void* stream) {
  CHECK(ops && T >= 0 && f >= 1 && ld >= f && G >= 1 && G <= kMaxSegs && (off || G == 1), MOE_ERR_INVALID_ARG);
  CHECK((dq != nullptr) == (dq_scale != nullptr) && (dqt != nullptr) == (dqt_scale != nullptr) &&
            (actt != nullptr) == (actt_scale != nullptr) && (dqt != nullptr) == (actt != nullptr),
        MOE_ERR_INVALID_ARG);
  CHECK(f % 8 == 0 && ld % 8 == 0 && f < (1 << 28) && T <= (1 << 22) && (!dq || f % kScaleBlock == 0), MOE_ERR_UNSUPPORTED);
  if (T == 0) return MOE_OK;
  CHECK(save && save_scale && dact && (dgu || dq || dqt || dgate), MOE_ERR_INVALID_ARG);
  CHECK(aligned(save, 8) && aligned(dact, 16) && aligned(dgu, 16) && aligned(dq, 16) && aligned(dqt, 16) && aligned(actt, 16),
        MOE_ERR_UNSUPPORTED);
  CHECK(!dgate || swiglu_workspace(T, f) == 0 || (workspace && aligned(workspace, 16)), MOE_ERR_WORKSPACE);
  HANDLE(ops);
  DONE(swiglu_backward(ops, save, save_scale, dact, ld, gate, T, f, off, G, dgu, dq, dq_scale, dqt, dqt_scale, actt,
                       actt_scale, dgate, (float*)workspace, (cudaStream_t)stream, &n_));
}

moe_status moe_requant_cols(moe_ops ops, const void* q, const float* scale, int src_rows, int T, int C,
                            const int32_t* off, int G, const int32_t* row_index, void* qt, float* scale_t,
                            void* stream) {
  CHECK(ops && T >= 0 && C >= 1 && src_rows >= 0, MOE_ERR_INVALID_ARG);
  CHECK(G >= 1 && G <= kMaxSegs && (off || G == 1), MOE_ERR_INVALID_ARG);
  CHECK(row_index || src_rows >= T, MOE_ERR_INVALID_ARG);
  CHECK(T <= (1 << 22) && C % 8 == 0 && C < (1 << 28), MOE_ERR_UNSUPPORTED);
  if (T == 0) return MOE_OK;
  CHECK(q && scale && qt && scale_t, MOE_ERR_INVALID_ARG);
  CHECK(aligned(q, 8) && aligned(qt, 16) && aligned(scale_t, 16), MOE_ERR_UNSUPPORTED);
  HANDLE(ops);
  DONE(requant_cols(ops, q, scale, src_rows, T, C, off, G, row_index, qt, scale_t, (cudaStream_t)stream, &n_));
}

moe_status moe_quant_w4(moe_ops ops, const void* w, int G, int N, int K, int group, uint32_t* codes, void* scale,
                        uint8_t* zero, void* stream) {
  CHECK(ops && w && codes && scale && G >= 1 && N >= 1 && K >= 1, MOE_ERR_INVALID_ARG);
  const moe_w4 out = {codes, scale, zero, group};
  const moe_status st = check_w4(&out, N, K);
  if (st != MOE_OK) return st;
  CHECK(aligned(w, 16) && (long long)G * N < (1ll << 31) / ceil_div(K, group), MOE_ERR_UNSUPPORTED);
  HANDLE(ops);
  DONE(quant_w4(ops, w, G, N, K, group, codes, scale, zero, (cudaStream_t)stream, &n_));
}

moe_status moe_w4_matmul(moe_ops ops, const void* x, long long ld_x, int x_rows, const int32_t* row_index, int M,
                         const moe_w4* w, const int32_t* off, int G, int N, int K, void* c, int out_dtype,
                         void* stream) {
  CHECK(ops && M >= 0 && x_rows >= 0 && N >= 1 && K >= 1 && G >= 1, MOE_ERR_INVALID_ARG);
  CHECK(off || G == 1, MOE_ERR_INVALID_ARG);
  CHECK(row_index || x_rows >= M, MOE_ERR_INVALID_ARG);
  CHECK(out_dtype == MOE_BF16 || out_dtype == MOE_FP32, MOE_ERR_INVALID_ARG);
  const moe_status st = check_w4(w, N, K);
  if (st != MOE_OK) return st;
  CHECK(G <= kMaxSegs && M < (1 << 30), MOE_ERR_UNSUPPORTED);
  CHECK((ceil_div(M, 8) + (long long)G) * ceil_div(N, 16) < (1ll << 30), MOE_ERR_UNSUPPORTED);   // units
  if (M == 0) return MOE_OK;
  CHECK(x && c && x_rows >= 1 && ld_x >= K, MOE_ERR_INVALID_ARG);
  CHECK(ld_x % 8 == 0 && aligned(x, 16) && aligned(c, 16), MOE_ERR_UNSUPPORTED);
  CHECK((long long)x_rows <= 0xffffffffll / (ld_x / 8), MOE_ERR_UNSUPPORTED);   // row starts in units of 16 bytes
  HANDLE(ops);
  DONE(w4_matmul(ops, x, ld_x, x_rows, row_index, M, *w, off, G, N, K, c, out_dtype == MOE_FP32, (cudaStream_t)stream,
                 &n_));
}

moe_status moe_w4_experts_workspace_size(const moe_w4_config* cfg, int T, size_t* bytes) {
  const moe_status st = check_w4_experts(cfg, T);
  if (st != MOE_OK) return st;
  CHECK(bytes, MOE_ERR_INVALID_ARG);
  *bytes = w4_experts_workspace(*cfg, T);
  return MOE_OK;
}

moe_status moe_w4_experts(moe_ops ops, const moe_w4_config* cfg, const void* x, long long ld_x, int T,
                          const int32_t* idx, const float* gate, const moe_w4* w13, const moe_w4* wd, void* y,
                          int out_dtype, void* workspace, void* stream) {
  CHECK(ops, MOE_ERR_INVALID_ARG);
  moe_status st = check_w4_experts(cfg, T);
  if (st == MOE_OK) st = check_w4(w13, 2 * cfg->f, cfg->d);
  if (st == MOE_OK) st = check_w4(wd, cfg->d, cfg->f);
  if (st != MOE_OK) return st;
  CHECK(out_dtype == MOE_BF16 || out_dtype == MOE_FP32, MOE_ERR_INVALID_ARG);
  CHECK(w13->group == wd->group && (w13->zero != nullptr) == (wd->zero != nullptr), MOE_ERR_UNSUPPORTED);
  if (T == 0) return MOE_OK;
  CHECK(x && idx && gate && y && ld_x >= cfg->d, MOE_ERR_INVALID_ARG);
  CHECK(ld_x % 8 == 0 && ld_x < (1ll << 28) && aligned(x, 16) && aligned(y, 16), MOE_ERR_UNSUPPORTED);
  CHECK(workspace && aligned(workspace, 16), MOE_ERR_WORKSPACE);
  HANDLE(ops);
  DONE(w4_experts(ops, *cfg, x, ld_x, T, idx, gate, *w13, *wd, y, out_dtype == MOE_FP32, workspace,
                  (cudaStream_t)stream, &n_));
}

}  // extern "C"
