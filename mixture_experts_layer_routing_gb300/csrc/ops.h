// Internal interface of the operators of include/moe_ops.h (host entry points in ops_api.cu).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/moe_ops.h"

struct moe_ops_s {
  int device;
  int sms;
  int pairs;              // two-CTA clusters of the wide products that run at once
  int* status;            // device word: the first device-side error
  std::atomic<long long> launches;   // (host threads share a handle)
};

namespace moe {

constexpr int kScaleBlock = 128;     // values that share a scale
constexpr int kMaxGroups = 32;       // expert groups of the gate
constexpr int kMaxSegs = 256;        // segments (experts) of the 8-bit products

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Each returns cudaSuccess or the launch's error, and adds the kernels it launched to *n.
cudaError_t norm_forward(const moe_ops_s* o, int dtype, const void* x, long long ld_x, const void* res,
                         long long ld_res, const void* w, int T, int d, float eps, void* h, void* y, void* q,
                         float* scale, float* rstd, cudaStream_t s, long long* n);
int norm_partials(int T, int d);     // rows of the backward's weight-gradient partials
cudaError_t norm_backward(const moe_ops_s* o, int dtype, const void* dy, const void* dh, const void* h,
                          const void* w, const float* rstd, int T, int d, void* dx, float* dw, float* part,
                          cudaStream_t s, long long* n);

size_t gate_workspace(const moe_gate_config& c, int T);
cudaError_t gate_forward(const moe_ops_s* o, const moe_gate_config& c, const float* logits, const float* bias, int T,
                         int* idx, float* gate, int* cnt, int* off, int* perm, int* inv, void* ws, cudaStream_t s,
                         long long* n);
cudaError_t gate_backward(const moe_ops_s* o, const moe_gate_config& c, const float* logits, const int* idx,
                          const float* dgate, int T, float* dlogits, cudaStream_t s, long long* n);

int quant_cols_rows(int T, int G);
cudaError_t quant_rows(const moe_ops_s* o, const void* src, long long ld, int T, int C, int swiglu, void* q,
                       float* scale, cudaStream_t s, long long* n);
cudaError_t quant_cols(const moe_ops_s* o, const void* src, long long ld, int src_rows, int T, int C, const int* off,
                       int G, const int* row_index, void* q, float* scale, cudaStream_t s, long long* n);
cudaError_t quant_blocks(const moe_ops_s* o, const void* w, int G, int N, int K, void* q, float* scale, void* qt,
                         float* scale_t, cudaStream_t s, long long* n);

cudaError_t fp8_init(int* pairs);   // kernel attributes on the current device
size_t fp8_matmul_workspace(int M, int G, int K, bool gathered);
cudaError_t fp8_matmul(const moe_ops_s* o, const void* a, const float* sa, int a_rows, const int* row_index, int M,
                       const void* b, const float* sb, const int* off, int G, int N, int K, void* c, int out_fp32,
                       void* ws, cudaStream_t s, long long* n);
cudaError_t fp8_wgrad(const moe_ops_s* o, const void* dct, const float* sdct, const void* xt, const float* sxt, int T,
                      const int* off, int G, int N, int K, void* c, int out_fp32, cudaStream_t s, long long* n);

}  // namespace moe
