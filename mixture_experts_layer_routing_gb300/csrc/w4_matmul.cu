// Products of few rows with 4-bit weights (moe_w4_matmul), dense and by segments of rows, and their quantiser.
#include "launch.cuh"
#include "segs.cuh"
#include "w4.cuh"

namespace moe {
namespace {

struct W4MatmulParams {
  const bf16* x;
  unsigned ld16;          // row of x in units of 16 bytes
  int x_rows, M;
  const int* row_index;
  W4 w;
  W4Shape s;
  const int* off;
  int G, out_fp32;
  void* c;
  int* status;
};

// A CTA takes units of MT x 16 weight rows x up to XR rows of one segment. Their chunks are dealt to its warps in turn; the
// last warp adds up the others' sums, in a fixed order.
template <int MT, int XR, int GROUP, bool ZERO>
__global__ void __launch_bounds__(kW4Warps * 32, 1) w4_matmul_kernel(W4MatmulParams P) {
  using Core = W4Core<MT, XR, GROUP, ZERO>;
  constexpr int kCols = MT * 16, kPitch = Core::kPitch, kSums = XR * kPitch;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ SegSmem seg;
  __shared__ W4Handover<kSumBuffers> hand;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5), warps = (blockDim.x >> 5) - 1;
  if (tid == 0) hand.init(warps);
  griddep_wait();
  griddep_launch();
  load_segments(seg, P.off, P.G, P.M, XR, P.status);
  float* sums = reinterpret_cast<float*>(smem + warps * Core::kBytes);     // [kSumBuffers][warp][XR][kPitch]
  const int blocks = (P.s.N + kCols - 1) / kCols, tiles = uniform(seg.tile[P.G]), C = (P.s.K + kChunk - 1) / kChunk;
  const int units = tiles * blocks, u0 = (int)((long long)units * blockIdx.x / gridDim.x);      // this CTA's, in a row
  const int u1 = (int)((long long)units * (blockIdx.x + 1) / gridDim.x);
  int tile = u0 / blocks, m = u0 - tile * blocks, at = -1, r0 = 0, R = 0;
  const auto rows = [&](int tl) {
    at = tl;
    const int g = uniform(segment_of(seg, P.G, tl));
    r0 = uniform(seg.off[g] + (tl - seg.tile[g]) * XR);
    R = uniform(min(XR, seg.off[g + 1] - r0));
  };
  if (warp == warps) {
    for (int u = u0; u < u1; ++u) {
      if (tile != at) rows(tile);
      hand.wait_full(u - u0, P.status);
      const float* from = sums + (u - u0) % kSumBuffers * warps * kSums;
      for (int i = lane; i < R * (kCols / 4); i += 32) {
        const int r = i / (kCols / 4), j = i % (kCols / 4) * 4, col = m * kCols + j;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int w = 0; w < warps; ++w) {
          const float4 q = *reinterpret_cast<const float4*>(from + w * kSums + r * kPitch + j);
          v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
        }
        if (col < P.s.N) {      // (N is a multiple of 8)
          const long long to = (long long)(r0 + r) * P.s.N + col;
          if (P.out_fp32) *reinterpret_cast<float4*>(reinterpret_cast<float*>(P.c) + to) = v;
          else *reinterpret_cast<uint2*>(reinterpret_cast<bf16*>(P.c) + to) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
        }
      }
      hand.taken(u - u0, lane);
      if (++m == blocks) m = 0, ++tile;
    }
    return;
  }
  Core core;
  core.init(smem + warp * Core::kBytes, warps, lane);
  W4Cursor w(u0, tile, m, warp, C, blocks), x = w;      // the next chunks of the weights and of x to read
  int aimed = -1, xt = -1, xR = 0;
  unsigned there = 0;
  bool fresh = true;                                    // the first chunk of its unit
  const auto issue = [&](unsigned to) {
    if (w.u < u1) {
      if (w.tile != aimed || (fresh && w.m + 1 == blocks)) {       // (the last block's rows may end within it)
        aimed = w.tile;
        int row0[MT], up0[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) row0[i] = w.m * kCols + i * 16, up0[i] = row0[i] + 8;
        core.aim(w4_matrix(P.w, P.s, uniform(segment_of(seg, P.G, w.tile))), P.s, row0, up0, P.s.N, w.c, lane);
      }
      core.copy(P.s, to, lane);
      const int n = w.next(warps, C, blocks);
      fresh = n > 0;
      for (int i = 0; i < n; ++i) core.step(P.s, kCols, C);
    }
    cp_commit();
  };
  const auto read_x = [&]() {
    if (x.u >= u1) return;
    if (x.tile != xt) {
      xt = x.tile;
      const int g = uniform(segment_of(seg, P.G, xt)), first = uniform(seg.off[g] + (xt - seg.tile[g]) * XR);
      xR = uniform(min(XR, seg.off[g + 1] - first));
      there = 0;
#pragma unroll
      for (int r = 0; r < XR; ++r) {
        core.xoff[r] = 0;
        if (r < xR) {
          const int s = P.row_index ? P.row_index[first + r] : first + r;
          if ((unsigned)s < (unsigned)P.x_rows) core.xoff[r] = (unsigned)s * P.ld16, there |= 1u << r;
          else set_error(P.status, MOE_ERR_DEVICE_INDEX);
        }
      }
    }
    core.read_x(P.x, x.c, P.s.K, xR, there, lane);
    x.next(warps, C, blocks);
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i * Core::kStage);
  read_x();
  int c = warp;
  for (int u = u0; u < u1; ++u) {
    if (tile != at) rows(tile);
    float acc[MT][4] = {};
    for (; c < C; c += warps) {
      cp_wait<kStages - 2>();
      __syncwarp();
      issue(core.free_slot());
      core.store_x();
      read_x();
      __syncwarp();
      core.multiply(acc, P.s.K - c * kChunk, lane);
      core.next();
    }
    c -= C;
    hand.wait_empty(u - u0, P.status);
    core.put(acc, sums + ((u - u0) % kSumBuffers * warps + warp) * kSums, R, lane);
    hand.put(u - u0, lane);
    if (++m == blocks) m = 0, ++tile;
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
  // (finite values may span more than fp32 holds: half the span over half of 15 is the same quotient)
  const float span = hi - lo;
  const bf16 sb = __float2bfloat16_rn(!ZERO                 ? __fdiv_rn(hi, 7.f)
                                      : span > 3.4028235e38f ? __fdiv_rn(0.5f * hi - 0.5f * lo, 7.5f)
                                                             : __fdiv_rn(span, 15.f));
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

template <int MT, int XR, int GROUP, bool ZERO>
cudaError_t launch_matmul(const moe_ops_s* o, const W4MatmulParams& P, cudaStream_t s) {
  using Core = W4Core<MT, XR, GROUP, ZERO>;
  auto* kern = w4_matmul_kernel<MT, XR, GROUP, ZERO>;
  constexpr size_t per = Core::kBytes + kSumBuffers * XR * Core::kPitch * sizeof(float);
  const long long units = (long long)(ceil_div(P.M, XR) + (P.off ? min(P.G, P.M) : 0)) * ceil_div(P.s.N, MT * 16);
  constexpr size_t fixed = sizeof(SegSmem) + 128;
  constexpr int warps = w4_warps(fixed, per);
  static_assert((warps + 1) * 32 >= 256, "load_segments takes 256 threads");
  MOE_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)w4_smem(fixed)));
  return launch_pdl(kern, dim3((unsigned)min(units, (long long)o->sms)), dim3((warps + 1) * 32), warps * per, s, P);
}
template <int MT, int XR> cudaError_t pick_matmul(const moe_ops_s* o, const W4MatmulParams& P, int group, cudaStream_t s) {
  const bool z = P.w.zero != nullptr;
  if (group == 32) return z ? launch_matmul<MT, XR, 32, true>(o, P, s) : launch_matmul<MT, XR, 32, false>(o, P, s);
  if (group == 64) return z ? launch_matmul<MT, XR, 64, true>(o, P, s) : launch_matmul<MT, XR, 64, false>(o, P, s);
  return z ? launch_matmul<MT, XR, 128, true>(o, P, s) : launch_matmul<MT, XR, 128, false>(o, P, s);
}

}  // namespace

cudaError_t w4_matmul(const moe_ops_s* o, const void* x, long long ld, int x_rows, const int* row_index, int M,
                      const moe_w4& w, const int* off, int G, int N, int K, void* c, int out_fp32, cudaStream_t s,
                      long long* n) {
  const W4MatmulParams P = {(const bf16*)x, (unsigned)(ld / 8), x_rows, M, row_index,
                            {w.codes, (const bf16*)w.scale, w.zero}, {N, K, ceil_div(K, w.group)}, off, G, out_fp32, c, o->status};
  *n += 1;
  if (M <= 2) return pick_matmul<2, 2>(o, P, w.group, s);
  return M <= 4 ? pick_matmul<2, 4>(o, P, w.group, s) : pick_matmul<2, 8>(o, P, w.group, s);
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
