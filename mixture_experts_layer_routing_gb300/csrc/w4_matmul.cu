// Products of few rows with 4-bit weights (moe_w4_matmul), dense and by segments of rows, and their quantiser.
#include "launch.cuh"
#include "segs.cuh"
#include "w4.cuh"

namespace moe {
namespace {

struct W4MatmulParams {
  const uint8_t* x;
  unsigned ld16;          // row of x in 16-byte units
  int x_rows, M;
  const int* row_index;
  W4 w;
  W4Shape s;
  const int* off;
  int G, out_fp32;
  void* c;
  int* status;
};

constexpr int kMmStages = 3;

template <int NT, int GROUP, bool ZERO> struct W4MatmulSmem {
  W4Stage<1, NT, GROUP, ZERO> stage[kW4Warps][kMmStages];
  float part[2][kW4Warps][NT * 8][20];      // [row of x][16 rows of w]
};

// A CTA takes units of 16 weight rows x up to 8 NT rows of one segment; its warps split K and add up in a fixed order.
template <int NT, int GROUP, bool ZERO>
__global__ void __launch_bounds__(kW4Warps * 32, 1) w4_matmul_kernel(W4MatmulParams P) {
  using Core = W4Core<1, NT, GROUP, ZERO>;
  constexpr int kRows = Core::kRows;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<W4MatmulSmem<NT, GROUP, ZERO>*>(smem_raw);
  __shared__ SegSmem seg;
  griddep_wait();
  griddep_launch();
  load_segments(seg, P.off, P.G, P.M, kRows, P.status);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int mtiles = (P.s.N + 15) / 16, units = seg.tile[P.G] * mtiles;
  const int C = (P.s.K + kChunk - 1) / kChunk, c0 = C * warp / kW4Warps, c1 = C * (warp + 1) / kW4Warps;
  Core core;
  core.px = P.x;
  int lu = blockIdx.x, lc = c0, tile_at = -1;
  const auto issue = [&](int slot) {
    if (lu < units && c0 < c1) {
      if (lc == c0) {
        const int tile = lu / mtiles, m = lu - tile * mtiles, g = segment_of(seg, P.G, tile);
        const int row0[1] = {m * 16}, end[1] = {P.s.N};
        core.set_weights(w4_matrix(P.w, P.s, g), P.s, row0, end, lane);
        if (tile != tile_at) {
          tile_at = tile;
          const int r0 = seg.off[g] + (tile - seg.tile[g]) * kRows, R = min(kRows, seg.off[g + 1] - r0);
          core.xn = (R + 1) / 2;
#pragma unroll
          for (int i = 0; i < NT * 4; ++i) {
            const int r = (lane >> 4) + 2 * i;
            core.xoff[i] = ~0u;
            if (r < R) {
              const int s = P.row_index ? P.row_index[r0 + r] : r0 + r;
              if ((unsigned)s < (unsigned)P.x_rows) core.xoff[i] = (unsigned)s * P.ld16;
              else set_error(P.status, MOE_ERR_DEVICE_INDEX);
            }
          }
        }
      }
      core.copy_weights(sm.stage[warp][slot], P.s, lc, lane);
      core.copy_x(sm.stage[warp][slot], P.s, lc, lane);
      if (++lc == c1) {
        lc = c0;
        lu += gridDim.x;
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kMmStages - 1; ++i) issue(i);
  int slot = 0, buf = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x, buf ^= 1) {
    const int tile = u / mtiles, m = u - tile * mtiles, g = segment_of(seg, P.G, tile);
    const int r0 = seg.off[g] + (tile - seg.tile[g]) * kRows, R = min(kRows, seg.off[g + 1] - r0);
    float acc[1][NT][4] = {};
    for (int c = c0; c < c1; ++c) {
      cp_wait<kMmStages - 2>();
      __syncwarp();
      issue(slot == 0 ? kMmStages - 1 : slot - 1);
      Core::multiply(sm.stage[warp][slot], acc, (R + 7) / 8, lane);
      slot = slot + 1 == kMmStages ? 0 : slot + 1;
    }
    const int quad = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float(*p)[20] = &sm.part[buf][warp][n * 8 + 2 * t];
      p[0][quad] = acc[0][n][0];
      p[1][quad] = acc[0][n][1];
      p[0][quad + 8] = acc[0][n][2];
      p[1][quad + 8] = acc[0][n][3];
    }
    __syncthreads();      // (the buffer before the last one has been read by all when they are here)
    for (int i = tid; i < R * 16; i += kW4Warps * 32) {
      const int r = i >> 4, j = i & 15, col = m * 16 + j;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kW4Warps; ++w) v += sm.part[buf][w][r][j];
      if (col < P.s.N) {
        const long long at = (long long)(r0 + r) * P.s.N + col;
        if (P.out_fp32) reinterpret_cast<float*>(P.c)[at] = v;
        else reinterpret_cast<bf16*>(P.c)[at] = __float2bfloat16_rn(v);
      }
    }
  }
}

// Eight values of a group a lane; lanes of a group are neighbours.
template <int GROUP, bool ZERO>
__global__ void __launch_bounds__(256) quant_w4_kernel(const bf16* __restrict__ w, long long items, int K, int N, int KG,
                                                       uint32_t* __restrict__ codes, bf16* __restrict__ scale,
                                                       uint8_t* __restrict__ zero) {
  constexpr int kLanes = GROUP / 8;
  griddep_wait();
  griddep_launch();
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) / kLanes;   // group: KG of a row
  const int l = threadIdx.x % kLanes;
  const long long row = i / KG;
  const int kg = (int)(i - row * KG), k = kg * GROUP + l * 8;
  const bool in = i < items && k < K;
  float v[8] = {};
  if (in) unpack8(*reinterpret_cast<const uint4*>(w + row * K + k), v);
  // largest magnitude, or smallest and largest value with 0 among them
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float p = ZERO ? v[j] : fabsf(v[j]);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(p));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(p));
  }
#pragma unroll
  for (int o = kLanes / 2; o; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, hi, o), m = __shfl_xor_sync(0xffffffffu, lo, o);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(h));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(m));
  }
  const bf16 sb = __float2bfloat16_rn(ZERO ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(hi, 7.f));
  const float s = __bfloat162float(sb);
  const bool plain = s > 0.f && s <= 3.3895314e38f;     // (else all codes are the zero point: 0, or NaN, times the scale)
  const float z = !ZERO ? 8.f : plain ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f) : 0.f;
  if (!in) return;
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float c = plain ? fminf(fmaxf(rintf(__fdiv_rn(v[j], s)) + z, 0.f), 15.f) : z;
    word |= (uint32_t)c << (4 * (j >> 1) + 16 * (j & 1));
  }
  codes[row * (K / 8) + k / 8] = word;
  if (l == 0) {
    const long long g = row / N, at = (g * KG + kg) * N + (row - g * N);
    scale[at] = sb;
    if (ZERO) zero[at] = (uint8_t)z;
  }
}

template <int NT, int GROUP, bool ZERO>
cudaError_t launch_matmul(const moe_ops_s* o, const W4MatmulParams& P, cudaStream_t s) {
  auto* kern = w4_matmul_kernel<NT, GROUP, ZERO>;
  const size_t smem = sizeof(W4MatmulSmem<NT, GROUP, ZERO>);
  MOE_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  const long long units = (long long)(ceil_div(P.M, NT * 8) + (P.off ? min(P.G, P.M) : 0)) * ceil_div(P.s.N, 16);
  const long long grid = min(units, (long long)o->sms * 2);
  return launch_pdl(kern, dim3((unsigned)grid), dim3(kW4Warps * 32), smem, s, P);
}
template <int NT> cudaError_t pick_matmul(const moe_ops_s* o, const W4MatmulParams& P, int group, cudaStream_t s) {
  const bool z = P.w.zero != nullptr;
  if (group == 32) return z ? launch_matmul<NT, 32, true>(o, P, s) : launch_matmul<NT, 32, false>(o, P, s);
  if (group == 64) return z ? launch_matmul<NT, 64, true>(o, P, s) : launch_matmul<NT, 64, false>(o, P, s);
  return z ? launch_matmul<NT, 128, true>(o, P, s) : launch_matmul<NT, 128, false>(o, P, s);
}

}  // namespace

cudaError_t w4_matmul(const moe_ops_s* o, const void* x, long long ld, int x_rows, const int* row_index, int M,
                      const moe_w4& w, const int* off, int G, int N, int K, void* c, int out_fp32, cudaStream_t s,
                      long long* n) {
  const W4MatmulParams P = {(const uint8_t*)x, (unsigned)(ld / 8), x_rows, M, row_index,
                            {w.codes, (const bf16*)w.scale, w.zero}, {N, K, ceil_div(K, w.group)}, off, G, out_fp32, c,
                            o->status};
  *n += 1;
  return M > 8 ? pick_matmul<2>(o, P, w.group, s) : pick_matmul<1>(o, P, w.group, s);
}

cudaError_t quant_w4(const moe_ops_s*, const void* w, int G, int N, int K, int group, uint32_t* codes, void* scale,
                     uint8_t* zero, cudaStream_t s, long long* n) {
  const int KG = ceil_div(K, group);
  const long long items = (long long)G * N * KG, blocks = (items * (group / 8) + 255) / 256;
  const auto go = [&](auto kern) {
    *n += 1;
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, s, (const bf16*)w, items, K, N, KG, codes, (bf16*)scale, zero);
  };
  if (group == 32) return zero ? go(quant_w4_kernel<32, true>) : go(quant_w4_kernel<32, false>);
  if (group == 64) return zero ? go(quant_w4_kernel<64, true>) : go(quant_w4_kernel<64, false>);
  return zero ? go(quant_w4_kernel<128, true>) : go(quant_w4_kernel<128, false>);
}

}  // namespace moe
