// RMS norm with the residual's addition and an e4m3 output, and its backward pass (include/moe_ops.h).
//
// Forward, one row a CTA: the row is read once, h = x + residual stays in registers (8 values a thread and step)
// through the one reduction (sum of squares), and every output leaves from there. A 128-value scale block is 16
// neighbouring lanes, so its maximum takes four shuffles. Bound by HBM at many rows, by latency at few: 8192 x 7168
// with residual, h and codes in 79 us (98% of the copy rate; 121 with rows unpacked to fp32 in registers, which left
// fewer CTAs a SM), one row in 2.7 us.
//
// Backward: one to four CTAs a SM walk the rows with stride gridDim, each with its part of dw in registers, and
// make one reduction a row (mean(u n); rstd comes from the forward pass). The parts are summed in a fixed order by a
// second kernel, so dw does not depend on timing.
#include "fp8_quant.cuh"
#include "launch.cuh"
#include "ops.h"

namespace moe {
namespace {

constexpr int kNormParts = 640;   // CTAs of the backward pass, at most

// Sum over the block; red holds one word a warp and is free for reuse after the next barrier.
__device__ __forceinline__ float block_sum(float v, float* red) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = warp_sum(v);
  if (lane == 0) red[w] = v;
  __syncthreads();
  return warp_sum(lane < nw ? red[lane] : 0.f);
}

template <typename T, int VPT>
__global__ void __launch_bounds__(VPT == 4 ? 512 : 1024, 1) norm_fwd_kernel(const T* x, long long ld_x, const T* res,
                                                        long long ld_res, const T* __restrict__ w, int d, float eps,
                                                        T* h, T* y, uint8_t* q, float* scale, float* rstd) {
  __shared__ float red[32];
  griddep_wait();
  griddep_launch();
  const long long t = blockIdx.x;
  const int nv = d >> 3;
  Raw8<T> v[VPT], e[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * blockDim.x + threadIdx.x;
    if (c < nv) v[i].load(x + t * ld_x + 8 * c);
  }
  if (res) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * blockDim.x + threadIdx.x;
      if (c < nv) e[i].load(res + t * ld_res + 8 * c);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * blockDim.x + threadIdx.x;
    if (c < nv) {
      float f[8];
      v[i].get(f);
      if (res) {
        float g[8];
        e[i].get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += g[j];
        v[i].set(f);     // the sum as it is stored
        v[i].get(f);
      }
      if (h) v[i].store(h + t * d + 8 * c);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += f[j] * f[j];
    }
  }
  const float r = __frsqrt_rn(block_sum(ss, red) / (float)d + eps);
  if (rstd && threadIdx.x == 0) rstd[t] = r;
  if (!y && !q) return;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * blockDim.x + threadIdx.x;
    float f[8];
    if (c < nv) {
      float g[8];
      v[i].get(f);
      load8(w + 8 * c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * r * g[j];
      if (y) store8(y + t * d + 8 * c, f);
    }
    if (q) {   // every lane takes part in the shuffles
      const float m = half_warp_max(c < nv ? amax8(f) : 0.f);
      if (c < nv) {
        *reinterpret_cast<uint2*>(q + t * d + 8 * c) = codes8(f, m);
        if ((c & 15) == 0) scale[t * ((d + kScaleBlock - 1) / kScaleBlock) + (c >> 4)] = block_scale(m);
      }
    }
  }
}

// A row is held as it is stored (12 registers of bf16 a thread) and unpacked twice, before and after its reduction, so
// that there is room for the next row, which is loaded a whole row ahead. (Unpacked values in registers and loads just
// before the reduction, two CTAs a SM in turn: 32.5 us for 2,368 x 7,168 with the sum of the parts, now 28.8.)
template <typename T, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) norm_bwd_kernel(const T* dy, const T* dh, const T* __restrict__ h,
                                                           const T* __restrict__ w, const float* __restrict__ rstd,
                                                           int rows, int d, T* dx, float* part) {
  __shared__ float red[2][32];
  griddep_wait();
  griddep_launch();
  const int nv = d >> 3;
  uint64_t acc[VPT][4];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0;
  const float inv_d = 1.0f / (float)d;
  struct Row {
    Raw8<T> y[VPT], h[VPT], e[VPT];
    float r;
  };
  const auto fetch = [&](Row& p, int t) {
    if (t >= rows) return;
    p.r = rstd[t];
    const long long at = (long long)t * d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * blockDim.x + threadIdx.x;
      if (c < nv) {
        p.y[i].load(dy + at + 8 * c);
        p.h[i].load(h + at + 8 * c);
        if (dh) p.e[i].load(dh + at + 8 * c);
      }
    }
  };
  const auto take = [&](Row& p, int t, float* words) {
    const uint64_t r2 = f32x2(p.r, p.r);
    uint64_t s2 = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * blockDim.x + threadIdx.x;
      if (c < nv) {
        uint64_t a[4], n[4], g[4];
        Raw8<T> wr;
        wr.load(w + 8 * c);
        p.y[i].pairs(a);
        p.h[i].pairs(n);
        wr.pairs(g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          n[j] = f32x2_mul(n[j], r2);
          acc[i][j] = f32x2_fma(a[j], n[j], acc[i][j]);
          s2 = f32x2_fma(f32x2_mul(a[j], g[j]), n[j], s2);
        }
      }
    }
    if (!dx) return;
    float s, s1;
    f32x2_get(s2, s, s1);
    const float mean = block_sum(s + s1, words) * inv_d;
    const uint64_t m2 = f32x2(-mean * p.r, -mean * p.r);      // n mean = h (rstd mean)
    const long long at = (long long)t * d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * blockDim.x + threadIdx.x;
      if (c < nv) {
        uint64_t a[4], n[4], g[4], o[4] = {0, 0, 0, 0};
        Raw8<T> wr;
        wr.load(w + 8 * c);
        p.y[i].pairs(a);
        p.h[i].pairs(n);
        wr.pairs(g);
        if (dh) p.e[i].pairs(o);
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f32x2_get(f32x2_fma(r2, f32x2_fma(n[j], m2, f32x2_mul(a[j], g[j])), o[j]), f[2 * j], f[2 * j + 1]);
        store8(dx + at + 8 * c, f);
      }
    }
  };
  Row a, b;
  int t = blockIdx.x;
  const int step = gridDim.x;
  fetch(a, t);
  while (t < rows) {      // (two buffers of words: one barrier a row)
    fetch(b, t + step);
    take(a, t, red[0]);
    t += step;
    if (t >= rows) break;
    fetch(a, t + step);
    take(b, t, red[1]);
    t += step;
  }
  if (part) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * blockDim.x + threadIdx.x;
      if (c < nv) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) f32x2_get(acc[i][j], f[2 * j], f[2 * j + 1]);
        store8(part + (long long)blockIdx.x * d + 8 * c, f);
      }
    }
  }
}

// dw[c] = sum over the parts: a CTA takes 32 columns, each of its 32 warps every 32nd part.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int parts, int d, float* dw) {
  __shared__ float red[32][33];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < d) {
#pragma unroll
    for (int i = 0; i < (kNormParts + 31) / 32; ++i)
      if (w + 32 * i < parts) s += part[(long long)(w + 32 * i) * d + c];
  }
  red[w][lane] = s;
  __syncthreads();
  s = warp_sum(red[lane][w]);
  if (lane == 0 && blockIdx.x * 32 + w < d) dw[blockIdx.x * 32 + w] = s;
}

template <typename T, int VPT>
cudaError_t fwd(const void* x, long long ld_x, const void* res, long long ld_res, const void* w, int rows, int d,
                float eps, void* h, void* y, void* q, float* scale, float* rstd, cudaStream_t s) {
  const int threads = ceil_div(ceil_div(d / 8, VPT), 32) * 32;
  return launch_pdl(norm_fwd_kernel<T, VPT>, dim3(rows), dim3(threads), 0, s, (const T*)x, ld_x, (const T*)res, ld_res,
                    (const T*)w, d, eps, (T*)h, (T*)y, (uint8_t*)q, scale, rstd);
}
template <typename T, int VPT, int MAXT>
cudaError_t bwd(const void* dy, const void* dh, const void* h, const void* w, const float* rstd, int rows, int d,
                void* dx, float* part, int parts, cudaStream_t s) {
  const int threads = ceil_div(ceil_div(d / 8, VPT), 32) * 32;
  return launch_pdl(norm_bwd_kernel<T, VPT, MAXT>, dim3(parts), dim3(threads), 0, s, (const T*)dy, (const T*)dh,
                    (const T*)h, (const T*)w, rstd, rows, d, (T*)dx, part);
}

// Steps of 8 values a thread. Few rows: as many threads as there are (one step up to d = 8192).
inline int steps(int d, bool wide) {
  const int nv = d / 8;
  if (wide) return nv <= 1024 ? 1 : 2;
  return nv <= 256 ? 1 : nv <= 1024 ? 2 : 4;
}

}  // namespace

// CTAs of the backward pass: about 1,024 threads a SM (its rows in flight are registers), of 152 SMs, as the size of the
// workspace is asked for without a handle. Above d = 4096 all of them run at once, one a SM. Below, a thread's 72
// registers (fp32: 88) let 28 (20) warps run: of d = 2048's 608 CTAs 456 (304) at once, of d = 4096's 304 152. Measured,
// 2,368 rows of 2,048, 4,096 and 7,168: 12, 18 and 29 us (bf16; their bytes take 6, 11 and 20), 16, 34 and 61 (fp32).
int norm_partials(int T, int d) {
  const int threads = ceil_div(ceil_div(d / 8, d > 8192 ? 2 : 1), 32) * 32;
  const int most = 152 * (threads > 512 ? 1 : threads > 256 ? 2 : 4);
  return T < most ? T : most;
}

cudaError_t norm_forward(const moe_ops_s* o, int dtype, const void* x, long long ld_x, const void* res,
                         long long ld_res, const void* w, int T, int d, float eps, void* h, void* y, void* q,
                         float* scale, float* rstd, cudaStream_t s, long long* n) {
  // 304 rows of 7,168 in 3.7 us with one step and 4.5 with two; 456 in 5.4 and 4.7.
  const int vpt = steps(d, T <= 2 * o->sms);
  const bool b = dtype == MOE_BF16;
  const auto call = vpt == 1 ? (b ? fwd<bf16, 1> : fwd<float, 1>) : vpt == 2 ? (b ? fwd<bf16, 2> : fwd<float, 2>)
                                                                            : (b ? fwd<bf16, 4> : fwd<float, 4>);
  *n += 1;
  return call(x, ld_x, res, ld_res, w, T, d, eps, h, y, q, scale, rstd, s);
}

cudaError_t norm_backward(const moe_ops_s* o, int dtype, const void* dy, const void* dh, const void* h,
                          const void* w, const float* rstd, int T, int d, void* dx, float* dw, float* part,
                          cudaStream_t s, long long* n) {
  const int parts = norm_partials(T, d);
  const bool b = dtype == MOE_BF16;
  // Threads an instance is compiled for. Fewer leave a thread more registers: fp32 spills 16 bytes in 72 registers at
  // 896 threads and 124 in 64 at 1,024 (2,368 x 7,168 in 61.0 and 70.4 us), bf16 takes 62 at either (29.3 and 29.4).
  // Past d = 8192 both types spill (232 and 640 bytes: 2,368 x 16,384 in 87 and 235 us, 46 and 92 of them bytes).
  const auto call = d > 8192 ? (b ? bwd<bf16, 2, 1024> : bwd<float, 2, 1024>)
                    : d > 4096 ? (b ? bwd<bf16, 1, 1024> : d > 7168 ? bwd<float, 1, 1024> : bwd<float, 1, 896>)
                               : (b ? bwd<bf16, 1, 512> : bwd<float, 1, 512>);
  *n += 1;
  MOE_TRY(call(dy, dh, h, w, rstd, T, d, dx, dw ? part : nullptr, parts, s));
  if (!dw) return cudaSuccess;
  *n += 1;
  return launch_pdl(norm_dw_kernel, dim3(ceil_div(d, 32)), dim3(1024), 0, s, (const float*)part, parts, d, dw);
}

}  // namespace moe
