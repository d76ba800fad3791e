// SwiGLU with an 8-bit checkpoint of its input, its gradient from the checkpoint, and 8-bit rows quantised anew along the
// token axis (moe_swiglu_*, moe_requant_cols).
#include "fp8_quant.cuh"
#include "launch.cuh"
#include "segs.cuh"

namespace moe {
namespace {

// Two e4m3 codes as fp32.
__device__ __forceinline__ float2 from_codes2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)c));
  float2 f;
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

// Codes of 16 bf16 values (8 words) of a block with the largest magnitude m.
__device__ __forceinline__ uint4 codes16(const uint4 (&w)[2], float m) {
  uint32_t o[4];
  const Divisor d(m);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float f[8];
    if (d.plain) {
      const uint64_t rr = f32x2(d.r, d.r), nm = f32x2(-m, -m);
      const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f32x2_get(code2(f32x2(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xffff0000u)), rr, nm), f[2 * j], f[2 * j + 1]);
    } else {
      unpack8(w[k], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = code_value(f[j], m);
    }
    o[2 * k] = pack_codes4(f[0], f[1], f[2], f[3]);
    o[2 * k + 1] = pack_codes4(f[4], f[5], f[6], f[7]);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// 16 bytes of which the second half may be behind a row's end; 8-byte aligned.
__device__ __forceinline__ void store16(uint8_t* dst, const uint4& v, bool two) {
  if (two && ((uintptr_t)dst & 15) == 0) {
    *reinterpret_cast<uint4*>(dst) = v;
  } else {
    *reinterpret_cast<uint2*>(dst) = make_uint2(v.x, v.y);
    if (two) *reinterpret_cast<uint2*>(dst + 8) = make_uint2(v.z, v.w);
  }
}
__device__ __forceinline__ uint4 load16(const uint8_t* src, bool one, bool two) {
  uint2 a = make_uint2(0u, 0u), b = make_uint2(0u, 0u);
  if (one) a = *reinterpret_cast<const uint2*>(src);
  if (two) b = *reinterpret_cast<const uint2*>(src + 8);
  return make_uint4(a.x, a.y, b.x, b.y);
}

// Eight lanes a block of 128 gate values and the 128 up values beside them, 16 of each a lane. Each value is read once;
// both halves' codes, act and its codes leave in the same pass.
__global__ void __launch_bounds__(256) swiglu_fwd_kernel(const bf16* __restrict__ gu, long long ld, unsigned items, int nb,
                                                         int f, bf16* __restrict__ act, uint8_t* __restrict__ q,
                                                         float* __restrict__ scale, uint8_t* __restrict__ save,
                                                         float* __restrict__ save_scale) {
  griddep_wait();
  griddep_launch();
  const unsigned i = blockIdx.x * 32 + (threadIdx.x >> 3), r = i / (unsigned)nb;
  const int b = (int)(i - r * nb), c = b * kScaleBlock + (threadIdx.x & 7) * 16;
  const long long row = r;
  const bool in = i < items && c < f, two = c + 8 < f, first = (threadIdx.x & 7) == 0;
  uint4 g[2] = {}, u[2] = {};
  if (in) {
    const uint4* p = reinterpret_cast<const uint4*>(gu + row * ld + c);
    const uint4* v = reinterpret_cast<const uint4*>(gu + row * ld + f + c);
    g[0] = p[0];
    u[0] = v[0];
    if (two) g[1] = p[1], u[1] = v[1];
  }
  if (save) {
    uint32_t mg = 0u, mu = 0u;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      mg = bf16x2_amax(bf16x2_amax(bf16x2_amax(bf16x2_amax(mg, g[k].x), g[k].y), g[k].z), g[k].w);
      mu = bf16x2_amax(bf16x2_amax(bf16x2_amax(bf16x2_amax(mu, u[k].x), u[k].y), u[k].z), u[k].w);
    }
    // both maxima in one word: the gate's in the low half
    uint32_t m = max(mg & 0xffffu, mg >> 16) | max(mu & 0xffffu, mu >> 16) << 16;
#pragma unroll
    for (int o = 4; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (in) {
      const float a = __uint_as_float(m << 16), e = __uint_as_float(m & 0xffff0000u);
      store16(save + row * 2 * f + c, codes16(g, a), two);
      store16(save + row * 2 * f + f + c, codes16(u, e), two);
      if (first) {
        save_scale[row * 2 * nb + b] = block_scale(a);
        save_scale[row * 2 * nb + nb + b] = block_scale(e);
      }
    }
  }
  if (!act && !q) return;
  float a[16];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float y[8];
    unpack8(g[k], &a[8 * k]);
    unpack8(u[k], y);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[8 * k + j] = silu_f(a[8 * k + j]) * y[j];
  }
  if (act && in) {
    bf16* dst = act + row * f + c;
    *reinterpret_cast<uint4*>(dst) = pack8(a);
    if (two) *reinterpret_cast<uint4*>(dst + 8) = pack8(a + 8);
  }
  if (!q) return;
  float m = max_nan(amax8(a), amax8(a + 8));
#pragma unroll
  for (int o = 4; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!in) return;
  uint32_t w[4];
  codes<16>(a, m, w);
  store16(q + row * f + c, make_uint4(w[0], w[1], w[2], w[3]), two);
  if (first) scale[i] = block_scale(m);
}

// SwiGLU's gradient from g, u and what arrives at act (da): of the gate half, of the up half, and act itself (not gated).
struct Grad { float dg, du, a; };
__device__ __forceinline__ Grad swiglu_grad(float g, float u, float da) {
  const float s = sigmoid_f(g), gs = g * s;
  Grad r;
  r.a = gs * u;
  r.du = da * gs;
  r.dg = da * u * (s + gs * (1.f - s));
  return r;
}

struct SaveBwdParams {
  const uint8_t* save;
  const float* save_scale;
  const bf16* dact;
  long long ld;
  const float* gate;
  const int* off;
  int G, T, f, nb;
  bf16* dgu;
  uint8_t* dq;
  float* dq_scale;
  uint8_t *dqt, *actt;
  float *dqt_scale, *actt_scale;
  float* part;             // [nb][T]: the gates' gradient by column blocks
  long long Tp;
  int* status;
};

constexpr int kOutPitch = 144;     // bytes of a column's 128 codes, 16 apart in the banks

// CTA per 128 tokens of a segment and 128 columns of f. Rows first: eight lanes a row, 16 columns each, whose maxima by
// rows are shuffles and by columns stay in registers until the last row. Then (COLS) columns: a warp takes 16 tokens, a
// lane two neighbouring columns, and the values are computed again from the tile in shared memory, which costs less than
// keeping three fp32 values of each.
template <bool COLS>
__global__ void __launch_bounds__(256, 2) swiglu_bwd_kernel(SaveBwdParams P) {
  __shared__ SegSmem seg;
  __shared__ float4 row_of[128];          // scales of g and u, gate
  extern __shared__ __align__(16) uint8_t smem[];
  uint4(*sd)[16] = reinterpret_cast<uint4(*)[16]>(smem);                     // dact: [token][128 columns]
  uint4(*sg)[8] = reinterpret_cast<uint4(*)[8]>(smem + 32768);               // codes of g, u
  uint4(*su)[8] = reinterpret_cast<uint4(*)[8]>(smem + 49152);
  float(*red)[3][128] = reinterpret_cast<float(*)[3][128]>(smem + 65536);    // [warp]: maxima of columns
  uint8_t(*out)[64][kOutPitch] = reinterpret_cast<uint8_t(*)[64][kOutPitch]>(smem + 65536);   // after them: dg, du, act
  griddep_wait();
  griddep_launch();
  load_segments(seg, P.off, P.G, P.T, kScaleBlock, P.status);
  const int t = blockIdx.y;
  if (t >= seg.tile[P.G]) return;
  const int sgm = segment_of(seg, P.G, t);
  const int row0 = seg.off[sgm] + (t - seg.tile[sgm]) * kScaleBlock, row1 = seg.off[sgm + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  const int c = b * kScaleBlock + (tid & 7) * 16;
  const bool one = c < P.f, two = c + 8 < P.f;
  float cm[COLS ? 3 : 1][16];
  if (COLS) {
#pragma unroll
    for (int j = 0; j < 16; ++j) cm[0][j] = cm[COLS ? 1 : 0][j] = cm[COLS ? 2 : 0][j] = 0.f;
  }
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int lr = i * 32 + (tid >> 3);
    const long long row = row0 + lr;
    const bool in = row < row1;
    uint4 d[2] = {}, g = {}, u = {};
    float zg = 0.f, zu = 0.f, gate = 1.f;
    if (in) {
      const bf16* p = P.dact + row * P.ld + c;
      if (one) d[0] = *reinterpret_cast<const uint4*>(p);
      if (two) d[1] = *reinterpret_cast<const uint4*>(p + 8);
      g = load16(P.save + row * 2 * P.f + c, one, two);
      u = load16(P.save + row * 2 * P.f + P.f + c, one, two);
      zg = P.save_scale[row * 2 * P.nb + b];
      zu = P.save_scale[row * 2 * P.nb + P.nb + b];
      if (P.gate) gate = P.gate[row];
    }
    if (COLS) {
      sd[lr][(tid & 7) * 2] = d[0];
      sd[lr][(tid & 7) * 2 + 1] = d[1];
      sg[lr][tid & 7] = g;
      su[lr][tid & 7] = u;
      if ((tid & 7) == 0) row_of[lr] = make_float4(zg, zu, gate, 0.f);
    }
    const uint32_t wd[8] = {d[0].x, d[0].y, d[0].z, d[0].w, d[1].x, d[1].y, d[1].z, d[1].w};
    const uint32_t wg[4] = {g.x, g.y, g.z, g.w}, wu[4] = {u.x, u.y, u.z, u.w};
    float dg[16], du[16], mg = 0.f, mu = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 gv = from_codes2(wg[j >> 1] >> (16 * (j & 1))), uv = from_codes2(wu[j >> 1] >> (16 * (j & 1)));
      const float d0 = __uint_as_float(wd[j] << 16), d1 = __uint_as_float(wd[j] & 0xffff0000u);
      const Grad r0 = swiglu_grad(gv.x * zg, uv.x * zu, d0 * gate), r1 = swiglu_grad(gv.y * zg, uv.y * zu, d1 * gate);
      dg[2 * j] = r0.dg, dg[2 * j + 1] = r1.dg;
      du[2 * j] = r0.du, du[2 * j + 1] = r1.du;
      mg = max_nan(max_nan(mg, fabsf(r0.dg)), fabsf(r1.dg));
      mu = max_nan(max_nan(mu, fabsf(r0.du)), fabsf(r1.du));
      dot = fmaf(r1.a, d1, fmaf(r0.a, d0, dot));
      if (COLS) {
        cm[0][2 * j] = max_nan(cm[0][2 * j], fabsf(r0.dg)), cm[0][2 * j + 1] = max_nan(cm[0][2 * j + 1], fabsf(r1.dg));
        cm[COLS ? 1 : 0][2 * j] = max_nan(cm[COLS ? 1 : 0][2 * j], fabsf(r0.du));
        cm[COLS ? 1 : 0][2 * j + 1] = max_nan(cm[COLS ? 1 : 0][2 * j + 1], fabsf(r1.du));
        cm[COLS ? 2 : 0][2 * j] = max_nan(cm[COLS ? 2 : 0][2 * j], fabsf(r0.a * gate));
        cm[COLS ? 2 : 0][2 * j + 1] = max_nan(cm[COLS ? 2 : 0][2 * j + 1], fabsf(r1.a * gate));
      }
    }
    if (P.dgu && in) {
      bf16* dst = P.dgu + row * 2 * P.f + c;
      if (one) {
        *reinterpret_cast<uint4*>(dst) = pack8(dg);
        *reinterpret_cast<uint4*>(dst + P.f) = pack8(du);
      }
      if (two) {
        *reinterpret_cast<uint4*>(dst + 8) = pack8(dg + 8);
        *reinterpret_cast<uint4*>(dst + P.f + 8) = pack8(du + 8);
      }
    }
    if (P.dq) {              // (f is a multiple of 128)
#pragma unroll
      for (int o = 4; o; o >>= 1) {
        mg = max_nan(mg, __shfl_xor_sync(0xffffffffu, mg, o));
        mu = max_nan(mu, __shfl_xor_sync(0xffffffffu, mu, o));
      }
      if (in) {
        uint32_t w[4];
        codes<16>(dg, mg, w);
        *reinterpret_cast<uint4*>(P.dq + row * 2 * P.f + c) = make_uint4(w[0], w[1], w[2], w[3]);
        codes<16>(du, mu, w);
        *reinterpret_cast<uint4*>(P.dq + row * 2 * P.f + P.f + c) = make_uint4(w[0], w[1], w[2], w[3]);
        if ((tid & 7) == 0) {
          P.dq_scale[row * 2 * P.nb + b] = block_scale(mg);
          P.dq_scale[row * 2 * P.nb + P.nb + b] = block_scale(mu);
        }
      }
    }
    if (P.part) {
#pragma unroll
      for (int o = 4; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (in && (tid & 7) == 0) P.part[(long long)b * P.T + row] = dot;
    }
  }
  if (!COLS) return;
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float m = cm[COLS ? k : 0][j];
      m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 8));
      m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
      if (lane < 8) red[warp][k][lane * 16 + j] = m;
    }
  __syncthreads();
  float mx[2][3][2];         // [half of the columns][output][column of the pair]
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      float2 m = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(&red[w][k][h * 64 + 2 * lane]);
        m.x = max_nan(m.x, v.x);
        m.y = max_nan(m.y, v.y);
      }
      mx[h][k][0] = m.x, mx[h][k][1] = m.y;
    }
  __syncthreads();           // (out lies where the maxima were)
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c0 = b * kScaleBlock + h * 64;
    if (c0 >= P.f) break;
    uint64_t rr[3], nm[3];
    bool plain = true;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const Divisor x(mx[h][k][0]), y(mx[h][k][1]);
      plain = plain && x.plain && y.plain;
      rr[k] = f32x2(x.r, y.r);
      nm[k] = f32x2(-mx[h][k][0], -mx[h][k][1]);
    }
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      float v[3][2][4];      // codes' values of four tokens
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int lr = warp * 16 + q * 4 + i;
        const float4 z = row_of[lr];
        const uint32_t wd = reinterpret_cast<const uint32_t*>(&sd[lr][0])[h * 32 + lane];
        const float2 gv = from_codes2(reinterpret_cast<const uint16_t*>(&sg[lr][0])[h * 32 + lane]);
        const float2 uv = from_codes2(reinterpret_cast<const uint16_t*>(&su[lr][0])[h * 32 + lane]);
        const Grad r0 = swiglu_grad(gv.x * z.x, uv.x * z.y, __uint_as_float(wd << 16) * z.z);
        const Grad r1 = swiglu_grad(gv.y * z.x, uv.y * z.y, __uint_as_float(wd & 0xffff0000u) * z.z);
        const float p[3][2] = {{r0.dg, r1.dg}, {r0.du, r1.du}, {r0.a * z.z, r1.a * z.z}};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          if (plain) {
            f32x2_get(code2(f32x2(p[k][0], p[k][1]), rr[k], nm[k]), v[k][0][i], v[k][1][i]);
          } else {
            v[k][0][i] = code_value(p[k][0], mx[h][k][0]);
            v[k][1][i] = code_value(p[k][1], mx[h][k][1]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<uint32_t*>(&out[k][e * 32 + lane][warp * 16 + q * 4]) =
              pack_codes4(v[k][e][0], v[k][e][1], v[k][e][2], v[k][e][3]);
    }
    const int cl = c0 + 2 * lane;
    if (warp < 3 && cl < P.f) {     // f is even
      float* s = warp == 2 ? P.actt_scale + (long long)t * P.f + cl : P.dqt_scale + (long long)t * 2 * P.f + warp * P.f + cl;
      const float x = warp == 0 ? mx[h][0][0] : warp == 1 ? mx[h][1][0] : mx[h][2][0];
      const float y = warp == 0 ? mx[h][0][1] : warp == 1 ? mx[h][1][1] : mx[h][2][1];
      s[0] = block_scale(x);
      s[1] = block_scale(y);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int k = i >> 1, e = i & 1, r = e * 32 + (tid >> 3), col = c0 + 2 * (r & 31) + e;
      if (col < P.f) {
        uint8_t* dst = k == 2 ? P.actt + (long long)col * P.Tp : P.dqt + (long long)(k * P.f + col) * P.Tp;
        *reinterpret_cast<uint4*>(dst + (long long)t * kScaleBlock + (tid & 7) * 16) =
            *reinterpret_cast<const uint4*>(&out[k][r][(tid & 7) * 16]);
      }
    }
    __syncthreads();
  }
}

// The gates' gradient: column blocks added up in their order.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ part, int nb, int T,
                                                        const int* __restrict__ off, int G, float* __restrict__ dgate,
                                                        int* status) {
  __shared__ SegSmem seg;
  griddep_wait();
  griddep_launch();
  load_segments(seg, off, G, T, kScaleBlock, status);
  const int r = seg.off[0] + blockIdx.x * 256 + threadIdx.x;       // (rows of no segment stay as they were)
  if (r >= seg.off[G]) return;
  float v = 0.f;
  for (int b = 0; b < nb; ++b) v += part[(long long)b * T + r];
  dgate[r] = v;
}

// CTA per 128 tokens and 128 columns: 8-bit rows to 8-bit columns, of the values code * scale. A warp takes 16 tokens, a
// lane four neighbouring columns; its 16 words of codes are decoded twice, for the maxima and for the codes.
__global__ void __launch_bounds__(256) requant_cols_kernel(const uint8_t* __restrict__ q, const float* __restrict__ scale,
                                                           int src_rows, int T, int C, int nb, const int* __restrict__ off,
                                                           int G, const int* __restrict__ row_index, uint8_t* __restrict__ qt,
                                                           float* __restrict__ scale_t, long long Tp, int* status) {
  __shared__ SegSmem seg;
  __shared__ float4 red[8][32];
  __shared__ __align__(16) uint8_t out[128][kOutPitch];       // [column of four, four columns][token]
  griddep_wait();
  griddep_launch();
  load_segments(seg, off, G, T, kScaleBlock, status);
  const int t = blockIdx.y;
  if (t >= seg.tile[G]) return;
  const int g = segment_of(seg, G, t);
  const int row0 = seg.off[g] + (t - seg.tile[g]) * kScaleBlock, row1 = seg.off[g + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x, c = b * kScaleBlock + lane * 4;
  // lane i < 16 looks token i of the warp up
  int src = -1;
  float z = 0.f;
  if (lane < 16 && row0 + warp * 16 + lane < row1) {
    src = row0 + warp * 16 + lane;
    if (row_index) src = row_index[src];
    if ((unsigned)src >= (unsigned)src_rows) {
      set_error(status, MOE_ERR_DEVICE_INDEX);
      src = -1;
    } else {
      z = scale[(long long)src * nb + b];
    }
  }
  uint32_t w[16];
  float s[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = __shfl_sync(0xffffffffu, src, i);
    s[i] = __shfl_sync(0xffffffffu, z, i);
    w[i] = r >= 0 && c < C ? *reinterpret_cast<const uint32_t*>(q + (long long)r * C + c) : 0u;
  }
  float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = from_codes2(w[i]), y = from_codes2(w[i] >> 16);
    m.x = max_nan(m.x, fabsf(x.x * s[i]));
    m.y = max_nan(m.y, fabsf(x.y * s[i]));
    m.z = max_nan(m.z, fabsf(y.x * s[i]));
    m.w = max_nan(m.w, fabsf(y.y * s[i]));
  }
  red[warp][lane] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 v = red[i][lane];
    m.x = max_nan(m.x, v.x), m.y = max_nan(m.y, v.y), m.z = max_nan(m.z, v.z), m.w = max_nan(m.w, v.w);
  }
  const Divisor dx(m.x), dy(m.y), dz(m.z), dw(m.w);
  const bool plain = dx.plain && dy.plain && dz.plain && dw.plain;
  const uint64_t r0 = f32x2(dx.r, dy.r), r1 = f32x2(dz.r, dw.r), n0 = f32x2(-m.x, -m.y), n1 = f32x2(-m.z, -m.w);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float v[4][4];           // [column][token]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = from_codes2(w[4 * k + i]), y = from_codes2(w[4 * k + i] >> 16);
      const float e = s[4 * k + i];
      if (plain) {
        f32x2_get(code2(f32x2(x.x * e, x.y * e), r0, n0), v[0][i], v[1][i]);
        f32x2_get(code2(f32x2(y.x * e, y.y * e), r1, n1), v[2][i], v[3][i]);
      } else {
        v[0][i] = code_value(x.x * e, m.x), v[1][i] = code_value(x.y * e, m.y);
        v[2][i] = code_value(y.x * e, m.z), v[3][i] = code_value(y.y * e, m.w);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint32_t*>(&out[j * 32 + lane][warp * 16 + k * 4]) = pack_codes4(v[j][0], v[j][1], v[j][2], v[j][3]);
  }
  if (warp == 0 && c < C)    // C is a multiple of 8
    *reinterpret_cast<float4*>(scale_t + (long long)t * C + c) =
        make_float4(block_scale(m.x), block_scale(m.y), block_scale(m.z), block_scale(m.w));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 32 + (tid >> 3), col = b * kScaleBlock + 4 * (r & 31) + i;
    if (col < C)
      *reinterpret_cast<uint4*>(qt + (long long)col * Tp + (long long)t * kScaleBlock + (tid & 7) * 16) =
          *reinterpret_cast<const uint4*>(&out[r][(tid & 7) * 16]);
  }
}

}  // namespace

cudaError_t swiglu_forward(const moe_ops_s*, const void* gu, long long ld, int T, int f, void* act, void* q, float* scale,
                           void* save, float* save_scale, cudaStream_t s, long long* n) {
  const int nb = ceil_div(f, kScaleBlock);
  const long long items = (long long)T * nb;
  *n += 1;
  return launch_pdl(swiglu_fwd_kernel, dim3((unsigned)((items + 31) / 32)), dim3(256), 0, s, (const bf16*)gu, ld,
                    (unsigned)items, nb, f, (bf16*)act, (uint8_t*)q, scale, (uint8_t*)save, save_scale);
}

cudaError_t swiglu_backward(const moe_ops_s* o, const void* save, const float* save_scale, const void* dact, long long ld,
                            const float* gate, int T, int f, const int* off, int G, void* dgu, void* dq, float* dq_scale,
                            void* dqt, float* dqt_scale, void* actt, float* actt_scale, float* dgate, float* ws,
                            cudaStream_t s, long long* n) {
  const int nb = ceil_div(f, kScaleBlock), Tp = quant_cols_rows(T, G);
  const SaveBwdParams P = {(const uint8_t*)save, save_scale, (const bf16*)dact, ld, gate, off, G, T, f, nb, (bf16*)dgu,
                           (uint8_t*)dq, dq_scale, (uint8_t*)dqt, (uint8_t*)actt, dqt_scale, actt_scale,
                           dgate ? ws : nullptr, Tp, o->status};
  const dim3 grid(nb, Tp / kScaleBlock);
  *n += 1;
  if (dqt) {
    constexpr int smem = 65536 + 3 * 64 * kOutPitch;
    static_assert(3 * 64 * kOutPitch >= 8 * 3 * 128 * 4, "the maxima fit where the codes go");
    MOE_TRY(cudaFuncSetAttribute(swiglu_bwd_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    MOE_TRY(launch_pdl(swiglu_bwd_kernel<true>, grid, dim3(256), smem, s, P));
  } else {
    MOE_TRY(launch_pdl(swiglu_bwd_kernel<false>, grid, dim3(256), 0, s, P));
  }
  if (!dgate) return cudaSuccess;
  *n += 1;
  return launch_pdl(sum_parts_kernel, dim3(ceil_div(T, 256)), dim3(256), 0, s, ws, nb, T, off, G, dgate, o->status);
}

cudaError_t requant_cols(const moe_ops_s* o, const void* q, const float* scale, int src_rows, int T, int C, const int* off,
                         int G, const int* row_index, void* qt, float* scale_t, cudaStream_t s, long long* n) {
  const int Tp = quant_cols_rows(T, G), nb = ceil_div(C, kScaleBlock);
  *n += 1;
  return launch_pdl(requant_cols_kernel, dim3(nb, Tp / kScaleBlock), dim3(256), 0, s, (const uint8_t*)q, scale, src_rows, T,
                    C, nb, off, G, row_index, (uint8_t*)qt, scale_t, (long long)Tp, o->status);
}

}  // namespace moe
