// Quantisers of include/moe_ops.h: e4m3 codes with one fp32 scale for 128 values, along rows, along the token axis
// (transposed, for the weights' gradient) and in 128 x 128 blocks (weights, optionally transposed as well).
// All read each value once; bound by HBM.
#include "fp8_quant.cuh"
#include "launch.cuh"
#include "segs.cuh"

namespace moe {
namespace {

// Half a warp a block: item i is block i % nb of row i / nb.
template <bool SWIGLU>
__global__ void __launch_bounds__(256) quant_rows_kernel(const bf16* __restrict__ src, long long ld, long long items,
                                                         int nb, int C, uint8_t* __restrict__ q,
                                                         float* __restrict__ scale) {
  griddep_wait();
  griddep_launch();
  const long long i = (long long)blockIdx.x * 16 + (threadIdx.x >> 4);
  const long long row = i / nb;
  const int b = (int)(i - row * nb), c = b * kScaleBlock + (threadIdx.x & 15) * 8;
  const bool in = i < items && c < C;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (in) {
    load8(src + row * ld + c, v);
    if (SWIGLU) {
      float u[8];
      load8(src + row * ld + C + c, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = silu_f(v[j]) * u[j];
    }
  }
  const float m = half_warp_max(amax8(v));
  if (in) {
    *reinterpret_cast<uint2*>(q + row * C + c) = codes8(v, m);
    if ((threadIdx.x & 15) == 0) scale[i] = block_scale(m);
  }
}

// CTA per 128 tokens and a run of 64-column blocks: rows are read 128 bytes wide into shared memory, then each thread
// takes a quarter (32 tokens) of one column and writes its 32 codes, so a column's 128 codes leave as one 128-byte
// line. The next block's rows are on their way meanwhile; segments and row indexes are looked up once a CTA (a CTA
// for every block spent most of its time on that: 12,288 x 2,816 gathered rows took 51 us).
constexpr int kColBlocks = 11;       // column blocks of a CTA
__global__ void __launch_bounds__(256) quant_cols_kernel(const bf16* __restrict__ src, long long ld, int src_rows,
                                                         int T, int C, const int* __restrict__ off, int G,
                                                         const int* __restrict__ row_index, uint8_t* __restrict__ q,
                                                         float* __restrict__ scale, long long Tp, int* status) {
  __shared__ SegSmem seg;
  __shared__ uint4 tile4[2][128][8];      // [block parity][token][64 columns]
  __shared__ float red[2][4][64];
  griddep_wait();
  griddep_launch();
  load_segments(seg, off, G, T, kScaleBlock, status);
  const int t = blockIdx.y;            // padded tile
  if (t >= seg.tile[G]) return;
  const int g = segment_of(seg, G, t);
  const int row0 = seg.off[g] + (t - seg.tile[g]) * kScaleBlock, row1 = seg.off[g + 1];
  const int tid = threadIdx.x;
  const bf16* rows[4];                 // this thread's rows (null: zeros)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 32 + (tid >> 3);
    rows[i] = nullptr;
    if (row0 + r < row1) {
      int s = row0 + r;
      if (row_index) s = row_index[s];
      if ((unsigned)s < (unsigned)src_rows) rows[i] = src + s * ld + (tid & 7) * 8;
      else set_error(status, MOE_ERR_DEVICE_INDEX);
    }
  }
  const int c_end = min(C, (int)(blockIdx.x + 1) * kColBlocks * 64);
  uint4 v4[4];
  const auto fetch = [&](int c0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v4[i] = rows[i] && c0 + (tid & 7) * 8 < c_end ? *reinterpret_cast<const uint4*>(rows[i] + c0) : make_uint4(0u, 0u, 0u, 0u);
  };
  const int col = tid & 63, part = tid >> 6;
  int b = 0;
  fetch(blockIdx.x * kColBlocks * 64);
  for (int c0 = blockIdx.x * kColBlocks * 64; c0 < c_end; c0 += 64, b ^= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) tile4[b][i * 32 + (tid >> 3)][tid & 7] = v4[i];
    __syncthreads();
    if (c0 + 64 < c_end) fetch(c0 + 64);
    const bf16* column = reinterpret_cast<const bf16*>(&tile4[b][0][0]) + part * 32 * 64 + col;
    float v[32], m = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      v[i] = to_f(column[i * 64]);
      m = max_nan(m, fabsf(v[i]));
    }
    red[b][part][col] = m;
    __syncthreads();
    m = max_nan(max_nan(red[b][0][col], red[b][1][col]), max_nan(red[b][2][col], red[b][3][col]));
    if (c0 + col < c_end) {
      uint32_t w[8];
      codes<32>(v, m, w);
      uint4* dst = reinterpret_cast<uint4*>(q + (long long)(c0 + col) * Tp + (long long)t * kScaleBlock + part * 32);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      if (part == 0) scale[(long long)t * C + c0 + col] = block_scale(m);
    }
  }
}

// CTA per 128 x 128 block of one matrix.
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
  return launch_pdl(swiglu ? quant_rows_kernel<true> : quant_rows_kernel<false>, dim3((unsigned)((items + 15) / 16)),
                    dim3(256), 0, s, (const bf16*)src, ld, items, nb, C, (uint8_t*)q, scale);
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
