// e4m3 codes with one fp32 scale for a block of 128 values (include/moe_ops.h):
// m = max |v|, scale = m / 448, code = e4m3(448 v / m).
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.0f;

// The larger of two magnitudes; NaN if one is (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float amax8(const float* v) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
  return m;
}
// 448 v is exact where v is a bf16 value, and the quotient is the one rounding before e4m3's, so a value half way
// between two codes is still there when it is rounded to even. A block of zeros (or with a NaN) keeps 0 * v.
__device__ __forceinline__ float code_value(float v, float m) { return m > 0.f ? __fdiv_rn(v * kE4m3Max, m) : 0.f * v; }
__device__ __forceinline__ float block_scale(float m) { return __fdiv_rn(m, kE4m3Max); }
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float m) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(code_value(a, m), code_value(b, m)), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(code_value(c, m), code_value(d, m)), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ uint2 codes8(const float* v, float m) {
  return make_uint2(codes4(v[0], v[1], v[2], v[3], m), codes4(v[4], v[5], v[6], v[7], m));
}
// Largest of the 16 lanes that hold a block (8 values each).
__device__ __forceinline__ float half_warp_max(float m) {
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// 8 consecutive values of either storage type as fp32, and back.
__device__ __forceinline__ void load8(const bf16* p, float* f) { unpack8(*reinterpret_cast<const uint4*>(p), f); }
__device__ __forceinline__ void load8(const float* p, float* f) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void store8(bf16* p, const float* f) { *reinterpret_cast<uint4*>(p) = pack8(f); }
__device__ __forceinline__ void store8(float* p, const float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

}  // namespace
}  // namespace moe
