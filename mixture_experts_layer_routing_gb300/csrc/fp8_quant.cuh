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
__device__ __forceinline__ uint32_t pack_codes4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// A block's divisor. Where neither 448 v nor a remainder can leave the range of normal numbers the quotient takes
// three operations, with one reciprocal a block: q = a r, then q + (a - q m) r, which is the correctly rounded a / m
// when r is the correctly rounded 1 / m (Markstein, IBM J. Res. Dev. 34, 1990). Elsewhere it is a division.
struct Divisor {
  float m, r;
  bool plain;
  __device__ __forceinline__ explicit Divisor(float amax) : m(amax) {
    plain = m >= 0x1p-100f && m < 0x1p118f;
    r = plain ? __frcp_rn(m) : 0.f;
  }
  __device__ __forceinline__ float code(float v) const {
    const float a = v * kE4m3Max, q = a * r;
    return fmaf(fmaf(-q, m, a), r, q);
  }
};
// The codes of N (a multiple of 4) values of a block with the largest magnitude m.
template <int N>
__device__ __forceinline__ void codes(const float* v, float m, uint32_t* out) {
  const Divisor d(m);
  if (d.plain) {
#pragma unroll
    for (int i = 0; i < N; i += 4) out[i / 4] = pack_codes4(d.code(v[i]), d.code(v[i + 1]), d.code(v[i + 2]), d.code(v[i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      out[i / 4] = pack_codes4(code_value(v[i], m), code_value(v[i + 1], m), code_value(v[i + 2], m),
                               code_value(v[i + 3], m));
  }
}
__device__ __forceinline__ uint2 codes8(const float* v, float m) {
  uint32_t w[2];
  codes<8>(v, m, w);
  return make_uint2(w[0], w[1]);
}
// Pairs of fp32 values, for the two-wide operations.
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f32x2_get(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Two values over two divisors' m and r at once (Divisor::code; -m in neg_m).
__device__ __forceinline__ uint64_t code2(uint64_t v, uint64_t r, uint64_t neg_m) {
  const uint64_t a = f32x2_mul(v, f32x2(kE4m3Max, kE4m3Max)), q = f32x2_mul(a, r);
  return f32x2_fma(f32x2_fma(q, neg_m, a), r, q);
}
// The larger magnitudes of bf16 pairs: without their signs they compare as integers, and a NaN is above all others.
__device__ __forceinline__ uint32_t bf16x2_amax(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }

// Largest of the 16 lanes that hold a block (8 values each).
__device__ __forceinline__ float half_warp_max(float m) {
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// 8 consecutive values of either storage type, as they are stored and as fp32.
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(bf16* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ __forceinline__ void get(float* f) const { unpack8(u, f); }
  __device__ __forceinline__ void set(const float* f) { u = pack8(f); }
  __device__ __forceinline__ void pairs(uint64_t* p) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void pairs(uint64_t* p) const {
    p[0] = f32x2(a.x, a.y);
    p[1] = f32x2(a.z, a.w);
    p[2] = f32x2(b.x, b.y);
    p[3] = f32x2(b.z, b.w);
  }
  __device__ __forceinline__ void set(const float* f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <typename T> __device__ __forceinline__ void load8(const T* p, float* f) {
  Raw8<T> r;
  r.load(p);
  r.get(f);
}
template <typename T> __device__ __forceinline__ void store8(T* p, const float* f) {
  Raw8<T> r;
  r.set(f);
  r.store(p);
}

}  // namespace
}  // namespace moe
