// Quantisers of include/moe_ops.h: e4m3 codes with one fp32 scale for 128 values, along rows, along the token axis
// (transposed, for the weights' gradient) and in 128 x 128 blocks (weights, optionally transposed as well).
// All read each value once; along rows HBM bounds them, along the token axis the instructions.
#include "fp8_quant.cuh"
#include "launch.cuh"
#include "segs.cuh"

namespace moe {
namespace {

// SwiGLU, half a warp a block: item i is block i % nb of row i / nb. 12,288 x 1408 in 17 us (12.8 at the copy rate).
__global__ void __launch_bounds__(256) quant_swiglu_kernel(const bf16* __restrict__ src, long long ld, unsigned items,
                                                           int nb, int C, uint8_t* __restrict__ q,
                                                           float* __restrict__ scale) {
  griddep_wait();
  griddep_launch();
  const unsigned i = blockIdx.x * 16 + (threadIdx.x >> 4), r = i / (unsigned)nb;
  const long long row = r;
  const int c = (int)(i - r * nb) * kScaleBlock + (threadIdx.x & 15) * 8;
  const bool in = i < items && c < C;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (in) {
    float u[8];
    load8(src + row * ld + c, v);
    load8(src + row * ld + C + c, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = silu_f(v[j]) * u[j];
  }
  const float m = half_warp_max(amax8(v));
  if (in) {
    *reinterpret_cast<uint2*>(q + row * C + c) = codes8(v, m);
    if ((threadIdx.x & 15) == 0) scale[i] = block_scale(m);
  }
}

// Rows of bf16 values, eight lanes a block of 128 (16 values each, so that what a block needs once, its maximum, its
// reciprocal and its scale, is shared by more of them: with 8 values a lane the kernel was bound by its instructions).
// 12,288 x 2816 in 17.4 us, 104 MB at 6.0 TB/s.
__global__ void __launch_bounds__(256) quant_rows_kernel(const bf16* __restrict__ src, long long ld, unsigned items,
                                                         int nb, int C, uint8_t* __restrict__ q,
                                                         float* __restrict__ scale) {
  griddep_wait();
  griddep_launch();
  const unsigned i = blockIdx.x * 32 + (threadIdx.x >> 3), r = i / (unsigned)nb;
  const long long row = r;
  const int c = (int)(i - r * nb) * kScaleBlock + (threadIdx.x & 7) * 16;
  const bool in = i < items && c < C, two = c + 8 < C;   // C is a multiple of 8
  uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (in) {
    const uint4* p = reinterpret_cast<const uint4*>(src + row * ld + c);
    w[0] = p[0];
    if (two) w[1] = p[1];
  }
  uint32_t m2 = 0u;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    m2 = bf16x2_amax(bf16x2_amax(bf16x2_amax(bf16x2_amax(m2, w[k].x), w[k].y), w[k].z), w[k].w);
#pragma unroll
  for (int o = 4; o; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
  const float m = __uint_as_float(max(m2 << 16, m2 & 0xffff0000u));
  if (!in) return;
  const Divisor d(m);
  uint2 u[2];
  if (d.plain) {
    const uint64_t rr = f32x2(d.r, d.r), nm = f32x2(-m, -m);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f32x2_get(code2(f32x2(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xffff0000u)), rr, nm), f[2 * j], f[2 * j + 1]);
      u[k] = make_uint2(pack_codes4(f[0], f[1], f[2], f[3]), pack_codes4(f[4], f[5], f[6], f[7]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float f[8];
      unpack8(w[k], f);
      u[k] = codes8(f, m);
    }
  }
  uint2* dst = reinterpret_cast<uint2*>(q + row * C + c);
  if (two && ((uintptr_t)dst & 15) == 0) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(u[0].x, u[0].y, u[1].x, u[1].y);
  } else {
    dst[0] = u[0];
    if (two) dst[1] = u[1];
  }
  if ((threadIdx.x & 7) == 0) scale[i] = block_scale(m);
}

// Codes of 16 bf16 values (low halves) by division: blocks of zeros, of NaN, of magnitudes at the ends of the range.
__device__ __forceinline__ void slow_codes16(const uint32_t (&x)[16], float m, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack_codes4(code_value(__uint_as_float(x[4 * i] << 16), m), code_value(__uint_as_float(x[4 * i + 1] << 16), m),
                       code_value(__uint_as_float(x[4 * i + 2] << 16), m), code_value(__uint_as_float(x[4 * i + 3] << 16), m));
}

// CTA per 128 tokens and a run of 64-column blocks: rows are read 128 bytes wide into shared memory (the next block's
// while this one is worked on), a warp takes 16 tokens and a lane two neighbouring columns of them, and the codes go
// back through shared memory so that a column's 128 leave as one 128-byte line. Segments and row indexes are looked up
// once a CTA. 12,288 x 2816 of 64 segments in 29 us, 12,288 gathered rows x 2048 in 20 us: bound by instructions and the
// three barriers a block (58% of the issue slots), not by HBM (32%).
constexpr int kColBlocks = 4;        // column blocks of a CTA
__global__ void __launch_bounds__(256, 4) quant_cols_kernel(const bf16* __restrict__ src, long long ld, int src_rows,
                                                         int T, int C, const int* __restrict__ off, int G,
                                                         const int* __restrict__ row_index, uint8_t* __restrict__ q,
                                                         float* __restrict__ scale, long long Tp, int* status) {
  __shared__ SegSmem seg;
  __shared__ uint4 tile[128][8];                 // [token][64 columns]
  __shared__ uint32_t red[8][32];                // [warp][column pair]
  __shared__ __align__(16) uint8_t out[64][144]; // [column of a pair, pair][token], rows 16 bytes apart in the banks
  griddep_wait();
  griddep_launch();
  load_segments(seg, off, G, T, kScaleBlock, status);
  const int t = blockIdx.y;            // padded tile
  if (t >= seg.tile[G]) return;
  const int g = segment_of(seg, G, t);
  const int row0 = seg.off[g] + (t - seg.tile[g]) * kScaleBlock, row1 = seg.off[g + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int rows[4];                         // this thread's rows (-1: zeros)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 32 + (tid >> 3);
    rows[i] = -1;
    if (row0 + r < row1) {
      int s = row0 + r;
      if (row_index) s = row_index[s];
      if ((unsigned)s < (unsigned)src_rows) rows[i] = s;
      else set_error(status, MOE_ERR_DEVICE_INDEX);
    }
  }
  const int c_first = blockIdx.x * kColBlocks * 64, c_end = min(C, c_first + kColBlocks * 64);
  uint4 v4[4];
  const auto fetch = [&](int c0) {
    const int c = c0 + (tid & 7) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v4[i] = rows[i] >= 0 && c < c_end ? *reinterpret_cast<const uint4*>(src + rows[i] * ld + c) : make_uint4(0u, 0u, 0u, 0u);
  };
  fetch(c_first);
  for (int c0 = c_first; c0 < c_end; c0 += 64) {
#pragma unroll
    for (int i = 0; i < 4; ++i) tile[i * 32 + (tid >> 3)][tid & 7] = v4[i];
    __syncthreads();
    if (c0 + 64 < c_end) fetch(c0 + 64);
    const uint32_t* mine = reinterpret_cast<const uint32_t*>(&tile[warp * 16][0]) + lane;
    uint32_t x[16], m2 = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = mine[i * 32];
      m2 = bf16x2_amax(m2, x[i]);
    }
    red[warp][lane] = m2;
    __syncthreads();
    m2 = red[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) m2 = __vmaxu2(m2, red[i][lane]);
    const float ma = __uint_as_float(m2 << 16), mb = __uint_as_float(m2 & 0xffff0000u);
    const Divisor da(ma), db(mb);
    uint32_t wa[4], wb[4];
    if (da.plain && db.plain) {
      const uint64_t rr = f32x2(da.r, db.r), nm = f32x2(-ma, -mb);
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        float a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f32x2_get(code2(f32x2(__uint_as_float(x[i + j] << 16), __uint_as_float(x[i + j] & 0xffff0000u)), rr, nm), a[j], b[j]);
        wa[i / 4] = pack_codes4(a[0], a[1], a[2], a[3]);
        wb[i / 4] = pack_codes4(b[0], b[1], b[2], b[3]);
      }
    } else {
      slow_codes16(x, ma, wa);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] >>= 16;
      slow_codes16(x, mb, wb);
    }
    *reinterpret_cast<uint4*>(&out[lane][warp * 16]) = make_uint4(wa[0], wa[1], wa[2], wa[3]);
    *reinterpret_cast<uint4*>(&out[32 + lane][warp * 16]) = make_uint4(wb[0], wb[1], wb[2], wb[3]);
    const int cl = c0 + 2 * lane;
    if (warp == 0 && cl < c_end) {     // C is even
      float* s = scale + (long long)t * C + cl;
      s[0] = block_scale(ma);
      s[1] = block_scale(mb);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 32 + (tid >> 3), col = c0 + 2 * (r & 31) + i;
      if (col < c_end)
        *reinterpret_cast<uint4*>(q + (long long)col * Tp + (long long)t * kScaleBlock + (tid & 7) * 16) =
            *reinterpret_cast<const uint4*>(&out[r][(tid & 7) * 16]);
    }
  }
}

// CTA per 128 x 128 block of one matrix: weights, once for inference and every step in training. 64 x 2816 x 2048 in
// 230 us, with the transposed codes 340 (163 and 218 at the copy rate); 4,096 x 7,168 in 19 and 33.
__global__ void __launch_bounds__(256) quant_blocks_kernel(const bf16* __restrict__ w, int N, int K,
                                                           uint8_t* __restrict__ q, float* __restrict__ scale,
                                                           uint8_t* __restrict__ qt, float* __restrict__ scale_t) {
  __shared__ uint8_t codes[128][132];
  __shared__ float red[8];
  griddep_wait();
  griddep_launch();
  const int tid = threadIdx.x, kb = blockIdx.x, nb = blockIdx.y;
  const long long base = (long long)blockIdx.z * N * K;
  const int c = kb * 128 + (tid & 15) * 8;
  float v[8][8], m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = nb * 128 + i * 16 + (tid >> 4);
    if (r < N && c < K) {
      load8(w + base + (long long)r * K + c, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
    m = max_nan(m, amax8(v[i]));
  }
  m = half_warp_max(m);
  m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, red[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int lr = i * 16 + (tid >> 4), r = nb * 128 + lr;
    const uint2 u = codes8(v[i], m);
    if (r < N && c < K) *reinterpret_cast<uint2*>(q + base + (long long)r * K + c) = u;
    if (qt) {
      uint32_t* d = reinterpret_cast<uint32_t*>(&codes[lr][(tid & 15) * 8]);
      d[0] = u.x;
      d[1] = u.y;
    }
  }
  const int NB = (N + 127) / 128, KB = (K + 127) / 128;
  if (tid == 0) {
    scale[((long long)blockIdx.z * NB + nb) * KB + kb] = block_scale(m);
    if (scale_t) scale_t[((long long)blockIdx.z * KB + kb) * NB + nb] = block_scale(m);
  }
  if (!qt) return;
  __syncthreads();
  // row k of the transpose: 128 codes; a thread packs 8 of them, 8 times
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int lk = i * 16 + (tid >> 4), k = kb * 128 + lk, n = nb * 128 + (tid & 15) * 8;
    if (k >= K || n >= N) continue;
    uint32_t x[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j >> 2] |= (uint32_t)codes[(tid & 15) * 8 + j][lk] << (8 * (j & 3));
    *reinterpret_cast<uint2*>(qt + base + (long long)k * N + n) = make_uint2(x[0], x[1]);
  }
}

}  // namespace

int quant_cols_rows(int T, int G) { return (ceil_div(T, kScaleBlock) + (G > 1 ? G : 0)) * kScaleBlock; }

cudaError_t quant_rows(const moe_ops_s*, const void* src, long long ld, int T, int C, int swiglu, void* q,
                       float* scale, cudaStream_t s, long long* n) {
  const int nb = ceil_div(C, kScaleBlock);
  const long long items = (long long)T * nb;
  *n += 1;
  if (swiglu)
    return launch_pdl(quant_swiglu_kernel, dim3((unsigned)((items + 15) / 16)), dim3(256), 0, s, (const bf16*)src, ld,
                      (unsigned)items, nb, C, (uint8_t*)q, scale);
  return launch_pdl(quant_rows_kernel, dim3((unsigned)((items + 31) / 32)), dim3(256), 0, s, (const bf16*)src, ld,
                    (unsigned)items, nb, C, (uint8_t*)q, scale);
}

cudaError_t quant_cols(const moe_ops_s* o, const void* src, long long ld, int src_rows, int T, int C, const int* off,
                       int G, const int* row_index, void* q, float* scale, cudaStream_t s, long long* n) {
  const int Tp = quant_cols_rows(T, G);
  *n += 1;
  return launch_pdl(quant_cols_kernel, dim3(ceil_div(C, 64 * kColBlocks), Tp / kScaleBlock), dim3(256), 0, s, (const bf16*)src, ld,
                    src_rows, T, C, off, G, row_index, (uint8_t*)q, scale, (long long)Tp, o->status);
}

cudaError_t quant_blocks(const moe_ops_s*, const void* w, int G, int N, int K, void* q, float* scale, void* qt,
                         float* scale_t, cudaStream_t s, long long* n) {
  *n += 1;
  return launch_pdl(quant_blocks_kernel, dim3(ceil_div(K, 128), ceil_div(N, 128), G), dim3(256), 0, s, (const bf16*)w,
                    N, K, (uint8_t*)q, scale, (uint8_t*)qt, scale_t);
}

}  // namespace moe
