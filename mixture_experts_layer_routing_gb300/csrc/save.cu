// SwiGLU with an 8-bit checkpoint of its input, its gradient from the checkpoint, and 8-bit rows quantised anew along the
// token axis (moe_swiglu_*, moe_requant_cols).
#include <type_traits>

#include "fp8_quant.cuh"
#include "launch.cuh"
#include "segs.cuh"
#include "tc_ptx.cuh"

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

// The larger of m and two magnitudes; NaN if one is.
__device__ __forceinline__ float amax3(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// SwiGLU's gradient, two values at a time: from g, u and what arrives at act (da) that of the gate half and of the up
// half, and act itself (not gated).
//
// The exponential is exp2 of the rounded -g log2(e), and the reciprocal the approximate one. The full exponential is closer
// where the sigmoid is small: act, in units of 2^-23, is off by 2.6 at most for |g| < 4 (0.63 in the root mean square) and by
// 15 for g in -40 .. -10, there with 1.8 (0.54) and 2.0. In sums over a row and behind e4m3's or bf16's rounding that does
// not show (12,288 x 1408: dgate is off by 1.20e-7 of its norm, in plain 32-bit operations by 1.19e-7), but
// 12,288 x 1408 take 89.5 us with all 8-bit forms instead of 81.7, and 43.0 instead of 41.0 with bf16 rows.
struct Grad2 { uint64_t dg, du, a; };
__device__ __forceinline__ Grad2 swiglu_grad2(uint64_t g, uint64_t u, uint64_t da) {
  float x, y;
  f32x2_get(f32x2_mul(g, f32x2(-1.44269504f, -1.44269504f)), x, y);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(y));
  const uint64_t one = f32x2(1.f, 1.f);
  f32x2_get(f32x2_fma(f32x2(x, y), one, one), x, y);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(y));
  const uint64_t s = f32x2(x, y), gs = f32x2_mul(g, s), rest = f32x2_fma(s, f32x2(-1.f, -1.f), one);
  Grad2 r;
  r.a = f32x2_mul(gs, u);
  r.du = f32x2_mul(da, gs);
  r.dg = f32x2_mul(f32x2_mul(da, u), f32x2_fma(gs, rest, s));
  return r;
}
__device__ __forceinline__ uint64_t codes_f32x2(uint32_t c, uint64_t scale) {
  const float2 v = from_codes2(c);
  return f32x2_mul(f32x2(v.x, v.y), scale);
}
__device__ __forceinline__ uint64_t bf16_f32x2(uint32_t w) {
  return f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// Codes of 16 values (8 pairs) of a block with the largest magnitude m.
__device__ __forceinline__ uint4 codes_of_pairs(const uint64_t (&v)[8], float m) {
  const Divisor d(m);
  float f[16];
  if (d.plain) {
    const uint64_t rr = f32x2(d.r, d.r), nm = f32x2(-m, -m);
#pragma unroll
    for (int i = 0; i < 8; ++i) f32x2_get(code2(v[i], rr, nm), f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f32x2_get(v[i], f[2 * i], f[2 * i + 1]);
      f[2 * i] = code_value(f[2 * i], m);
      f[2 * i + 1] = code_value(f[2 * i + 1], m);
    }
  }
  return make_uint4(pack_codes4(f[0], f[1], f[2], f[3]), pack_codes4(f[4], f[5], f[6], f[7]),
                    pack_codes4(f[8], f[9], f[10], f[11]), pack_codes4(f[12], f[13], f[14], f[15]));
}

// Four neighbouring columns' divisors; codes of four tokens' values, PLAIN where no quotient needs a division.
struct Divisor4 {
  float m[4];
  uint64_t r0, r1, n0, n1;
  bool plain;
  // (not `there`: columns behind the last one, whose codes nobody reads, need no division; taken as columns of zeros they
  // brought it to the whole warp, 301 x 392 by columns 26 us instead of 13)
  __device__ __forceinline__ Divisor4(const float4& v, bool there)
      : m{there ? v.x : 1.f, there ? v.y : 1.f, there ? v.z : 1.f, there ? v.w : 1.f} {
    const Divisor a(m[0]), b(m[1]), c(m[2]), d(m[3]);
    plain = a.plain && b.plain && c.plain && d.plain;
    r0 = f32x2(a.r, b.r), r1 = f32x2(c.r, d.r), n0 = f32x2(-m[0], -m[1]), n1 = f32x2(-m[2], -m[3]);
  }
  // lo, hi: columns 0, 1 and 2, 3 -> the quotients, by column
  template <bool PLAIN> __device__ __forceinline__ void quotients(uint64_t lo, uint64_t hi, float (&q)[4]) const {
    if (PLAIN) {
      f32x2_get(code2(lo, r0, n0), q[0], q[1]);
      f32x2_get(code2(hi, r1, n1), q[2], q[3]);
    } else {
      f32x2_get(lo, q[0], q[1]);
      f32x2_get(hi, q[2], q[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = code_value(q[i], m[i]);
    }
  }
};

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
  float* dgate;            // written here by a cluster of all column blocks,
  float* part;             // else [nb][T]: by column blocks, for sum_parts_kernel
  long long Tp;
  int* status;
};

// The gates' gradient is added up by clusters of all column blocks (8 CTAs at most) where tiles are few: a launch
// less (301 x 392 with bf16 outputs 3.7 us a call among others instead of 6.3, in a graph 3.4 and 3.5, 512 x 1024 4.0 and
// 3.7). With more tiles the CTAs of a cluster wait for one another: 1024 x 1024 8.0 us instead of 7.1, 12,288 x 1024 34.6
// instead of 29.0.
constexpr int kClusterBlocks = 8, kClusterTiles = 32;
inline bool clustered(int T, int nb) { return nb <= kClusterBlocks && ceil_div(T, kScaleBlock) * nb <= kClusterTiles; }
constexpr int kOutPitch = 144;     // bytes of a column's 128 codes, 16 apart in the banks

// The tile in shared memory that the columns are computed from. Their codes are put where it was.
struct BwdTile {
  uint2 d[128][32];        // dact: [token][four columns a lane]
  uint32_t g[128][32], u[128][32];
};
static_assert(3 * 128 * kOutPitch <= sizeof(BwdTile), "the codes fit where the tile was");

// Codes of a warp's 16 tokens and a lane's four columns, of dg, du and act: [output][column][token / 4].
template <bool PLAIN>
__device__ __forceinline__ void column_codes(const BwdTile& tile, const float4* row_of, const Divisor4 (&div)[3], int warp,
                                             int lane, uint32_t (&w)[3][4][4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[3][4][4];      // [output][token][column]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lr = warp * 16 + q * 4 + i;
      const float4 z = row_of[lr];
      const uint2 d = tile.d[lr][lane];
      const uint32_t g = tile.g[lr][lane], u = tile.u[lr][lane];
      const uint64_t zg = f32x2(z.x, z.x), zu = f32x2(z.y, z.y), gate = f32x2(z.z, z.z);
      const Grad2 a = swiglu_grad2(codes_f32x2(g, zg), codes_f32x2(u, zu), f32x2_mul(bf16_f32x2(d.x), gate));
      const Grad2 b = swiglu_grad2(codes_f32x2(g >> 16, zg), codes_f32x2(u >> 16, zu), f32x2_mul(bf16_f32x2(d.y), gate));
      div[0].quotients<PLAIN>(a.dg, b.dg, v[0][i]);
      div[1].quotients<PLAIN>(a.du, b.du, v[1][i]);
      div[2].quotients<PLAIN>(f32x2_mul(a.a, gate), f32x2_mul(b.a, gate), v[2][i]);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) w[k][c][q] = pack_codes4(v[k][0][c], v[k][1][c], v[k][2][c], v[k][3][c]);
  }
}

// Copies to shared memory; nothing is read where `there` is not set, and zeros are written.
__device__ __forceinline__ void cp16_or_zeros(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp8_or_zeros(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp4_or_zeros(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 4 : 0) : "memory");
}

// CTA per 128 tokens of a segment and 128 columns of f. Rows first: eight lanes a row, 16 columns each, whose maxima by
// rows are shuffles and by columns stay in registers until the last row. Then (COLS) columns: a warp takes 16 tokens, a
// lane four neighbouring columns, and the values are computed again from the tile in shared memory, which costs less than
// keeping three fp32 values of each. 12,288 x 1408 with all 8-bit forms in 82 us (24 at the copy rate): its 46.6 M warp
// instructions are half of that, and the rest is latency at four warps a scheduler (128 registers): of 7.4 cycles between
// a warp's instructions 1.5 are their own, 0.9 each shared memory's and the barriers', 0.8 the exponentials' pipe.
template <bool COLS>
__global__ void __launch_bounds__(256, 2) swiglu_bwd_kernel(SaveBwdParams P) {
  __shared__ SegSmem seg;
  __shared__ float4 row_of[128];          // scales of g and u, gate
  __shared__ float dots[128];             // act dact of this column block
  extern __shared__ __align__(16) uint8_t smem[];
  BwdTile& tile = *reinterpret_cast<BwdTile*>(smem);
  uint8_t(*out)[128][kOutPitch] = reinterpret_cast<uint8_t(*)[128][kOutPitch]>(smem);       // dg, du, act
  float(*red)[3][128] = reinterpret_cast<float(*)[3][128]>(smem + sizeof(BwdTile));         // [16 groups of rows]: maxima
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
  // the whole tile is on its way before the first row is looked at
  if (COLS) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lr = i * 32 + (tid >> 3);
      const bool in = row0 + lr < row1;
      const long long row = in ? row0 + lr : row0;
      const bf16* p = P.dact + row * P.ld + (one ? c : 0);
      cp16_or_zeros(&tile.d[lr][(tid & 7) * 4], p, in && one);
      cp16_or_zeros(&tile.d[lr][(tid & 7) * 4 + 2], two ? p + 8 : p, in && two);
      const uint8_t* g = P.save + row * 2 * P.f + (one ? c : 0);
      cp8_or_zeros(&tile.g[lr][(tid & 7) * 4], g, in && one);
      cp8_or_zeros(&tile.g[lr][(tid & 7) * 4 + 2], two ? g + 8 : g, in && two);
      cp8_or_zeros(&tile.u[lr][(tid & 7) * 4], g + P.f, in && one);
      cp8_or_zeros(&tile.u[lr][(tid & 7) * 4 + 2], two ? g + P.f + 8 : g, in && two);
      const float* z = P.save_scale + row * 2 * P.nb + b;
      if ((tid & 7) == 0) cp4_or_zeros(&row_of[lr].x, z, in);
      if ((tid & 7) == 1) cp4_or_zeros(&row_of[lr].y, z + P.nb, in);
      if ((tid & 7) == 2) {
        if (P.gate) cp4_or_zeros(&row_of[lr].z, P.gate + row, in);
        else row_of[lr].z = 1.f;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  const int each = 4 / gridDim.z, i0 = blockIdx.z * each;      // (COLS: all four)
#pragma unroll 1
  for (int i = i0; i < i0 + each; ++i) {
    if (row0 + i * 32 >= row1) break;      // (a segment's last tile)
    const int lr = i * 32 + (tid >> 3);
    const long long row = row0 + lr;
    const bool in = row < row1;
    uint4 d[2] = {}, g = {}, u = {};
    float zg = 0.f, zu = 0.f, gate = 1.f;
    if (COLS) {              // a thread reads what it copied, and its eight lanes' scales
      if (i == 0) asm volatile("cp.async.wait_group 3;" ::: "memory");
      else if (i == 1) asm volatile("cp.async.wait_group 2;" ::: "memory");
      else if (i == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
      d[0] = reinterpret_cast<const uint4*>(tile.d[lr])[(tid & 7) * 2];
      d[1] = reinterpret_cast<const uint4*>(tile.d[lr])[(tid & 7) * 2 + 1];
      g = reinterpret_cast<const uint4*>(tile.g[lr])[tid & 7];
      u = reinterpret_cast<const uint4*>(tile.u[lr])[tid & 7];
      const float4 z = row_of[lr];
      zg = z.x, zu = z.y, gate = z.z;
    } else if (in) {
      const bf16* p = P.dact + row * P.ld + c;
      if (one) d[0] = *reinterpret_cast<const uint4*>(p);
      if (two) d[1] = *reinterpret_cast<const uint4*>(p + 8);
      g = load16(P.save + row * 2 * P.f + c, one, two);
      u = load16(P.save + row * 2 * P.f + P.f + c, one, two);
      zg = P.save_scale[row * 2 * P.nb + b];
      zu = P.save_scale[row * 2 * P.nb + P.nb + b];
      if (P.gate) gate = P.gate[row];
    }
    const uint32_t wd[8] = {d[0].x, d[0].y, d[0].z, d[0].w, d[1].x, d[1].y, d[1].z, d[1].w};
    const uint32_t wg[4] = {g.x, g.y, g.z, g.w}, wu[4] = {u.x, u.y, u.z, u.w};
    const uint64_t z2g = f32x2(zg, zg), z2u = f32x2(zu, zu), gate2 = f32x2(gate, gate);
    uint64_t dg[8], du[8], dot2 = 0;
    float mg = 0.f, mu = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t da = bf16_f32x2(wd[j]);
      const Grad2 r = swiglu_grad2(codes_f32x2(wg[j >> 1] >> (16 * (j & 1)), z2g), codes_f32x2(wu[j >> 1] >> (16 * (j & 1)), z2u),
                                   f32x2_mul(da, gate2));
      dg[j] = r.dg;
      du[j] = r.du;
      dot2 = f32x2_fma(r.a, da, dot2);
      float x, y;
      f32x2_get(r.dg, x, y);
      mg = amax3(mg, x, y);
      if (COLS) cm[0][2 * j] = max_nan(cm[0][2 * j], fabsf(x)), cm[0][2 * j + 1] = max_nan(cm[0][2 * j + 1], fabsf(y));
      f32x2_get(r.du, x, y);
      mu = amax3(mu, x, y);
      if (COLS) {
        cm[COLS ? 1 : 0][2 * j] = max_nan(cm[COLS ? 1 : 0][2 * j], fabsf(x));
        cm[COLS ? 1 : 0][2 * j + 1] = max_nan(cm[COLS ? 1 : 0][2 * j + 1], fabsf(y));
        f32x2_get(f32x2_mul(r.a, gate2), x, y);
        cm[COLS ? 2 : 0][2 * j] = max_nan(cm[COLS ? 2 : 0][2 * j], fabsf(x));
        cm[COLS ? 2 : 0][2 * j + 1] = max_nan(cm[COLS ? 2 : 0][2 * j + 1], fabsf(y));
      }
    }
    if (P.dgu && in) {
      bf16* dst = P.dgu + row * 2 * P.f + c;
      uint32_t x[8], y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float p, q;
        f32x2_get(dg[j], p, q);
        x[j] = pack2(p, q);
        f32x2_get(du[j], p, q);
        y[j] = pack2(p, q);
      }
      if (one) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<uint4*>(dst + P.f) = make_uint4(y[0], y[1], y[2], y[3]);
      }
      if (two) {
        *reinterpret_cast<uint4*>(dst + 8) = make_uint4(x[4], x[5], x[6], x[7]);
        *reinterpret_cast<uint4*>(dst + P.f + 8) = make_uint4(y[4], y[5], y[6], y[7]);
      }
    }
    if (P.dq) {              // (f is a multiple of 128)
#pragma unroll
      for (int o = 4; o; o >>= 1) {
        mg = max_nan(mg, __shfl_xor_sync(0xffffffffu, mg, o));
        mu = max_nan(mu, __shfl_xor_sync(0xffffffffu, mu, o));
      }
      if (in) {
        *reinterpret_cast<uint4*>(P.dq + row * 2 * P.f + c) = codes_of_pairs(dg, mg);
        *reinterpret_cast<uint4*>(P.dq + row * 2 * P.f + P.f + c) = codes_of_pairs(du, mu);
        if ((tid & 7) == 0) {
          P.dq_scale[row * 2 * P.nb + b] = block_scale(mg);
          P.dq_scale[row * 2 * P.nb + P.nb + b] = block_scale(mu);
        }
      }
    }
    if (P.part || P.dgate) {
      float x, y;
      f32x2_get(dot2, x, y);
      float dot = x + y;
#pragma unroll
      for (int o = 4; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (in && (tid & 7) == 0) {
        if (P.dgate) dots[lr] = dot;
        else P.part[(long long)b * P.T + row] = dot;
      }
    }
  }
  if (P.dgate) {             // column blocks in their order
    cluster_sync();
    const int lr = i0 * 32 + tid;
    if (b == 0 && tid < each * 32 && row0 + lr < row1) {
      const uint32_t at = smem_u32(&dots[lr]);
      float v = 0.f;
      for (int r = 0; r < P.nb; ++r) {
        float x;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(mapa_shared(at, r)) : "memory");
        v += x;
      }
      P.dgate[row0 + lr] = v;
    }
    cluster_sync();          // (a CTA's sums are read until here)
  }
  if (!COLS) return;
  asm volatile("cp.async.wait_group 0;" ::: "memory");     // (rows behind the segment's end: the codes go where they are)
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      float4 m;
      float* v = &cm[COLS ? k : 0][j];
      m.x = max_nan(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
      m.y = max_nan(v[1], __shfl_xor_sync(0xffffffffu, v[1], 16));
      m.z = max_nan(v[2], __shfl_xor_sync(0xffffffffu, v[2], 16));
      m.w = max_nan(v[3], __shfl_xor_sync(0xffffffffu, v[3], 16));
      if (lane < 16) *reinterpret_cast<float4*>(&red[warp * 2 + (lane >> 3)][k][(lane & 7) * 16 + j]) = m;
    }
  __syncthreads();
  // one warp an output, four columns a lane: the first three warps finish the maxima
  if (warp < 3) {
    float4 m = *reinterpret_cast<const float4*>(&red[0][warp][lane * 4]);
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(&red[i][warp][lane * 4]);
      m.x = max_nan(m.x, v.x), m.y = max_nan(m.y, v.y), m.z = max_nan(m.z, v.z), m.w = max_nan(m.w, v.w);
    }
    *reinterpret_cast<float4*>(&red[0][warp][lane * 4]) = m;
    const int cl = b * kScaleBlock + lane * 4;
    if (cl < P.f) {            // f is a multiple of 8
      float* s = warp == 2 ? P.actt_scale + (long long)t * P.f + cl : P.dqt_scale + (long long)t * 2 * P.f + warp * P.f + cl;
      s[0] = block_scale(m.x), s[1] = block_scale(m.y), s[2] = block_scale(m.z), s[3] = block_scale(m.w);
    }
  }
  __syncthreads();
  const bool there = b * kScaleBlock + lane * 4 < P.f;
  const Divisor4 div[3] = {Divisor4(*reinterpret_cast<const float4*>(&red[0][0][lane * 4]), there),
                           Divisor4(*reinterpret_cast<const float4*>(&red[0][1][lane * 4]), there),
                           Divisor4(*reinterpret_cast<const float4*>(&red[0][2][lane * 4]), there)};
  uint32_t w[3][4][4] = {};
  if (row0 + warp * 16 < row1) {
    if (div[0].plain && div[1].plain && div[2].plain) column_codes<true>(tile, row_of, div, warp, lane, w);
    else column_codes<false>(tile, row_of, div, warp, lane, w);
  }
  __syncthreads();           // (the codes go where the tile is)
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int c4 = 0; c4 < 4; ++c4)
      *reinterpret_cast<uint4*>(&out[k][c4 * 32 + lane][warp * 16]) = make_uint4(w[k][c4][0], w[k][c4][1], w[k][c4][2], w[k][c4][3]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 12; ++i) {
    const int k = i >> 2, e = i & 3, r = e * 32 + (tid >> 3), col = b * kScaleBlock + 4 * (r & 31) + e;
    if (col < P.f) {
      uint8_t* dst = k == 2 ? P.actt + (long long)col * P.Tp : P.dqt + (long long)(k * P.f + col) * P.Tp;
      *reinterpret_cast<uint4*>(dst + (long long)t * kScaleBlock + (tid & 7) * 16) =
          *reinterpret_cast<const uint4*>(&out[k][r][(tid & 7) * 16]);
    }
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
// lane four neighbouring columns; its 16 words of codes are decoded twice, for the maxima and for the codes. 12,288
// gathered rows x 2048 in 24 us (4.5 at the copy rate): its 15.3 M warp instructions, some 12 a value, are half of that;
// of 13.4 cycles between a warp's instructions 3.2 are spent at barriers and 2.1 on the gathered words' way. Runs of 2, 4
// or 8 column blocks a CTA with the next block's words on their way took 25, 26 and 27.
__global__ void __launch_bounds__(256, 4) requant_cols_kernel(const uint8_t* __restrict__ q, const float* __restrict__ scale,
                                                              int src_rows, int T, int C, int nb, const int* __restrict__ off,
                                                              int G, const int* __restrict__ row_index,
                                                              uint8_t* __restrict__ qt, float* __restrict__ scale_t,
                                                              long long Tp, int* status) {
  __shared__ SegSmem seg;
  __shared__ float4 red[8][32];
  __shared__ float row_scale[8][16];
  __shared__ __align__(16) uint8_t out[128][kOutPitch];       // [column of four, four columns][token]
  griddep_wait();
  griddep_launch();
  load_segments(seg, off, G, T, kScaleBlock, status);
  const int t = blockIdx.y;
  if (t >= seg.tile[G]) return;
  const int g = segment_of(seg, G, t);
  const int row0 = seg.off[g] + (t - seg.tile[g]) * kScaleBlock, row1 = seg.off[g + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x, c = b * kScaleBlock + lane * 4;
  const bool any = row0 + warp * 16 < row1;        // (else the warp's columns are zeros)
  // lane i < 16 looks token i of the warp up
  int src = -1;
  if (lane < 16 && row0 + warp * 16 + lane < row1) {
    src = row0 + warp * 16 + lane;
    if (row_index) src = row_index[src];
    if ((unsigned)src >= (unsigned)src_rows) {
      set_error(status, MOE_ERR_DEVICE_INDEX);
      src = -1;
    }
  }
  uint32_t x[16];
  float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
  if (any) {
    const float z = src >= 0 ? scale[(long long)src * nb + b] : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = __shfl_sync(0xffffffffu, src, i);
      x[i] = r >= 0 && c < C ? *reinterpret_cast<const uint32_t*>(q + (long long)r * C + c) : 0u;
    }
    if (lane < 16) row_scale[warp][lane] = z;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float s0 = row_scale[warp][i], s1 = row_scale[warp][i + 1];
      float a0, a1, a2, a3, c0, c1, c2, c3;
      f32x2_get(codes_f32x2(x[i], f32x2(s0, s0)), a0, a1);
      f32x2_get(codes_f32x2(x[i] >> 16, f32x2(s0, s0)), a2, a3);
      f32x2_get(codes_f32x2(x[i + 1], f32x2(s1, s1)), c0, c1);
      f32x2_get(codes_f32x2(x[i + 1] >> 16, f32x2(s1, s1)), c2, c3);
      m.x = amax3(m.x, a0, c0);
      m.y = amax3(m.y, a1, c1);
      m.z = amax3(m.z, a2, c2);
      m.w = amax3(m.w, a3, c3);
    }
  }
  red[warp][lane] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 v = red[i][lane];
    m.x = max_nan(m.x, v.x), m.y = max_nan(m.y, v.y), m.z = max_nan(m.z, v.z), m.w = max_nan(m.w, v.w);
  }
  const Divisor4 div(m, c < C);
  const auto codes_to = [&](auto plain) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v[4][4];         // [token][column]
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = row_scale[warp][4 * k + i];
        div.quotients<decltype(plain)::value>(codes_f32x2(x[4 * k + i], f32x2(s, s)), codes_f32x2(x[4 * k + i] >> 16, f32x2(s, s)),
                                              v[i]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint32_t*>(&out[j * 32 + lane][warp * 16 + k * 4]) = pack_codes4(v[0][j], v[1][j], v[2][j], v[3][j]);
    }
  };
  if (!any) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(&out[j * 32 + lane][warp * 16]) = make_uint4(0u, 0u, 0u, 0u);
  } else if (div.plain) {
    codes_to(std::true_type{});
  } else {
    codes_to(std::false_type{});
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

// launch_pdl with clusters of `cluster` CTAs along x.
cudaError_t launch_cluster(void (*kern)(SaveBwdParams), dim3 grid, unsigned cluster, size_t smem, cudaStream_t s,
                           const SaveBwdParams& P) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, P);
}

}  // namespace

size_t swiglu_workspace(int T, int f) {
  const int nb = ceil_div(f, kScaleBlock);
  return clustered(T, nb) ? 0 : sizeof(float) * (size_t)T * nb;
}

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
  const bool joined = dgate && clustered(T, nb);
  const unsigned cluster = joined ? nb : 1;
  const SaveBwdParams P = {(const uint8_t*)save, save_scale, (const bf16*)dact, ld, gate, off, G, T, f, nb, (bf16*)dgu,
                           (uint8_t*)dq, dq_scale, (uint8_t*)dqt, (uint8_t*)actt, dqt_scale, actt_scale,
                           joined ? dgate : nullptr, dgate && !joined ? ws : nullptr, Tp, o->status};
  const dim3 grid(nb, Tp / kScaleBlock);
  *n += 1;
  if (dqt) {
    constexpr int smem = sizeof(BwdTile) + 16 * 3 * 128 * sizeof(float);
    MOE_TRY(cudaFuncSetAttribute(swiglu_bwd_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    MOE_TRY(launch_cluster(swiglu_bwd_kernel<true>, grid, cluster, smem, s, P));
  } else {
    // Without columns a tile's rows may go to four CTAs: where tiles are no more than the CTAs that run at once (with the
    // gates' gradient 301 x 392 take 3.4 us instead of 6.1, 1024 x 2048 of 8 segments 9.5 and 9.7, 2048 x 2048 of them,
    // 384 tiles, 13.5 instead of 11.3).
    const bool split = (long long)grid.x * grid.y <= 2ll * o->sms;
    MOE_TRY(launch_cluster(swiglu_bwd_kernel<false>, dim3(grid.x, grid.y, split ? 4 : 1), cluster, 0, s, P));
  }
  if (!P.part) return cudaSuccess;
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
