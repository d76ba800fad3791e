// The experts' layer of a few tokens on 4-bit weights (moe_w4_experts) in two kernels: gate/up products with SwiGLU, and
// down products with the weighted sum over a token's experts.
#include "launch.cuh"
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kMaxSlots = 264;               // experts, shared ones included
constexpr int kSlotsEach = 3;                // of a thread that counts, in CTAs of at least 4 warps

// The experts in use and their tokens, made by every CTA of both kernels from idx alone. Pairs (token, expert) are
// sorted by expert, then token; an expert that a token names twice is one pair with both gates. A tile is up to `rows`
// pairs of a slot. TMAX is 16 or 64: lists for 64 tokens take 6 KB of shared memory more.
template <int TMAX> struct LayerLists {
  static constexpr int kPairs = TMAX * 16, kWords = (TMAX + 31) / 32;
  unsigned mask[kMaxSlots][kWords];          // tokens of a slot
  uint16_t pair[kMaxSlots + 1], tile[kMaxSlots + 1];
  uint16_t slot_of_tile[kPairs];
  uint8_t token[kPairs];
  int tmp[kW4Warps];
};
template <int TMAX> struct LayerGates {
  int idx[TMAX * 8];
  float gate[TMAX * 8];
};

struct W4LayerParams {
  const bf16* x;
  unsigned ld16;          // row of x in units of 16 bytes
  int T, k, E, slots, d, f;
  const int* idx;
  const float* gate;
  W4 w13, wd;
  W4Shape s13, sd;
  bf16* h;                // [pairs][parts][f]: rounded, what the rounding left, and (3) what its rounding left
  int parts;
  void* y;
  int out_fp32;
  int* status;
};

template <int TMAX>
__device__ __forceinline__ void build_lists(LayerLists<TMAX>& L, LayerGates<TMAX>* gates, const W4LayerParams& P, int rows) {
  constexpr int kWords = LayerLists<TMAX>::kWords;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, kThreads = blockDim.x;
  for (int i = tid; i < P.slots * kWords; i += kThreads) {
    const int n = P.T - 32 * (i % kWords);   // tokens from this word on
    L.mask[i / kWords][i % kWords] = i / kWords < P.E || n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
  }
  __syncthreads();
  for (int i = tid; i < P.T * P.k; i += kThreads) {
    const int e = P.idx[i], t = i / P.k;
    if (gates) {
      gates->idx[i] = e;
      gates->gate[i] = P.gate[i];
    }
    if ((unsigned)e < (unsigned)P.E) atomicOr(&L.mask[e][t >> 5], 1u << (t & 31));
    else set_error(P.status, MOE_ERR_DEVICE_INDEX);
  }
  __syncthreads();
  int n[kSlotsEach], v = 0;                  // tiles in the high half
#pragma unroll
  for (int j = 0; j < kSlotsEach; ++j) {
    const int i = kSlotsEach * tid + j;
    int r = 0;
    if (i < P.slots)
      for (int h = 0; h < kWords; ++h) r += __popc(L.mask[i][h]);
    n[j] = ((r + rows - 1) / rows << 16) + r;
    v += n[j];
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) L.tmp[warp] = v;
  __syncthreads();
  for (int i = 0; i < warp; ++i) v += L.tmp[i];
  int before = v;
#pragma unroll
  for (int j = 0; j < kSlotsEach; ++j) before -= n[j];
#pragma unroll
  for (int j = 0; j < kSlotsEach; ++j) {
    const int i = kSlotsEach * tid + j;
    if (i <= P.slots) {
      L.pair[i] = (uint16_t)before;
      L.tile[i] = (uint16_t)(before >> 16);
    }
    if (i < P.slots) {
      int p = before & 0xffff;
      for (int h = 0; h < kWords; ++h)
        for (unsigned m = L.mask[i][h]; m; m &= m - 1) L.token[p++] = (uint8_t)(h * 32 + __ffs(m) - 1);
      for (int k = before >> 16; k < (before + n[j]) >> 16; ++k) L.slot_of_tile[k] = (uint16_t)i;
    }
    before += n[j];
  }
  __syncthreads();
}
// Slot of a tile, its first pair and how many (by a whole warp).
template <int TMAX>
__device__ __forceinline__ int find_tile(const LayerLists<TMAX>& L, int tile, int rows, int& pair0, int& R) {
  const int e = uniform(L.slot_of_tile[tile]);
  pair0 = uniform(L.pair[e] + (tile - L.tile[e]) * rows);
  R = uniform(min(rows, L.pair[e + 1] - pair0));
  return e;
}

// Gate and up rows of MT x 8 values of h, up to XR pairs of an expert, for each unit (a tile of 16 weight rows is 8 gate
// rows and the 8 up rows of the same values). A unit's chunks are dealt to the warps in turn; the last warp adds up the
// others' sums, in a fixed order, and applies SwiGLU and the gate.
template <int MT, int XR, int TMAX, int GROUP, bool ZERO>
__global__ void __launch_bounds__(kW4Warps * 32, 1) w4_up_kernel(W4LayerParams P) {
  using Core = W4Core<MT, XR, GROUP, ZERO>;
  constexpr int kCols = MT * 8, kPitch = Core::kPitch, kSums = XR * kPitch;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ LayerLists<TMAX> L;
  __shared__ LayerGates<TMAX> gates;
  __shared__ W4Handover<kSumBuffers> hand;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5), warps = (blockDim.x >> 5) - 1;
  if (tid == 0) hand.init(warps);
  griddep_wait();
  griddep_launch();
  build_lists(L, &gates, P, XR);
  float* sums = reinterpret_cast<float*>(smem + warps * Core::kBytes);     // [kSumBuffers][warp][XR][kPitch]
  const int blocks = P.f / kCols, tiles = uniform(L.tile[P.slots]), C = (P.d + kChunk - 1) / kChunk;
  const int units = tiles * blocks, u0 = (int)((long long)units * blockIdx.x / gridDim.x);      // this CTA's, in a row
  const int u1 = (int)((long long)units * (blockIdx.x + 1) / gridDim.x);
  int tile = u0 / blocks, m = u0 - tile * blocks, pair0 = 0, R = 0;
  if (warp == warps) {
    for (int u = u0; u < u1; ++u) {
      const int e = find_tile(L, tile, XR, pair0, R);
      hand.wait_full(u - u0, P.status);
      const float* from = sums + (u - u0) % kSumBuffers * warps * kSums;
      for (int i = lane; i < R * kCols; i += 32) {
        const int r = i / kCols, j = i % kCols, at = r * kPitch + (j / 8) * 16 + j % 8, t = L.token[pair0 + r];
        float g = 0.f, up = 0.f, gate = e < P.E ? 0.f : 1.f;
        if (e < P.E)
          for (int q = 0; q < P.k; ++q)
            if (gates.idx[t * P.k + q] == e) gate += gates.gate[t * P.k + q];
#pragma unroll 4
        for (int w = 0; w < warps; ++w) {
          g += from[w * kSums + at];
          up += from[w * kSums + at + 8];
        }
        // (The full exponential and quotient, with no difference in time: the fast ones were off by 14 units of 2^-23 where
        // |g| is 40, these by 4 at most.)
        const float h = g / (1.f + expf(-g)) * up * gate;
        // h as a sum of bf16 values, two (16 bits of mantissa) or for fp32 outputs three (24), so that the layer rounds
        // once, at its output. (Two for fp32 outputs were off by up to 3.2e-6 of y's norm, three are by 2.1e-7; 16 tokens
        // of 32 experts, d = 7168, take 273 us instead of 212, one token 49 instead of 47.)
        bf16* dst = P.h + (long long)(pair0 + r) * P.parts * P.f + m * kCols + j;
        const bf16 hi = __float2bfloat16_rn(h);
        float rest = h - __bfloat162float(hi);
        if (!(fabsf(rest) <= 3.3895314e38f)) rest = 0.f;        // (an infinity or a NaN has left nothing)
        const bf16 lo = __float2bfloat16_rn(rest);
        dst[0] = hi;
        dst[P.f] = lo;
        if (P.parts == 3) dst[2 * (long long)P.f] = __float2bfloat16_rn(rest - __bfloat162float(lo));
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
  const auto issue = [&](unsigned to) {
    if (w.u < u1) {
      if (w.tile != aimed) {
        aimed = w.tile;
        int row0[MT], up0[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) row0[i] = w.m * kCols + i * 8, up0[i] = P.f + row0[i];
        core.aim(w4_matrix(P.w13, P.s13, uniform(L.slot_of_tile[aimed])), P.s13, row0, up0, 2 * P.f, w.c, lane);
      }
      core.copy(P.s13, to, lane);
      for (int n = w.next(warps, C, blocks); n > 0; --n) core.step(P.s13, kCols, C);
    }
    cp_commit();
  };
  const auto read_x = [&]() {
    if (x.u >= u1) return;
    if (x.tile != xt) {
      xt = x.tile;
      int p0;
      find_tile(L, xt, XR, p0, xR);
#pragma unroll
      for (int r = 0; r < XR; ++r) core.xoff[r] = r < xR ? L.token[p0 + r] * P.ld16 : 0u;
    }
    core.read_x(P.x, x.c, P.d, xR, ~0u, lane);
    x.next(warps, C, blocks);
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i * Core::kStage);
  read_x();
  int c = warp, at = -1;
  for (int u = u0; u < u1; ++u) {
    if (tile != at) find_tile(L, at = tile, XR, pair0, R);
    float acc[MT][4] = {};
    for (; c < C; c += warps) {
      cp_wait<kStages - 2>();
      __syncwarp();
      issue(core.free_slot());
      core.store_x();
      read_x();
      __syncwarp();
      core.multiply(acc, P.d - c * kChunk, lane);
      core.next();
    }
    c -= C;
    hand.wait_empty(u - u0, P.status);
    core.put(acc, sums + ((u - u0) % kSumBuffers * warps + warp) * kSums, R, lane);
    hand.put(u - u0, lane);
    if (++m == blocks) m = 0, ++tile;
  }
}

constexpr int down_buffers(int tmax) { return tmax > 16 ? 1 : 2; }      // (of all tokens' sums, a warp)

// MT x 16 values of y for all tokens a unit. The chunks of all experts in use are dealt to the warps in runs; the rows of
// a tile are the parts of its pairs' h, 2 a pair, or 3 and a row of zeros, and a warp adds an expert's product to its own
// sums of the tokens, which the last warp adds up.
template <int MT, int XR, int PARTS, int TMAX, int GROUP, bool ZERO>
__global__ void __launch_bounds__(kW4Warps * 32, 1) w4_down_kernel(W4LayerParams P) {
  using Core = W4Core<MT, XR, GROUP, ZERO>;
  constexpr int kRows = PARTS == 3 ? 4 : 2, kPairs = XR / kRows, kCols = MT * 16, kPitch = Core::kPitch, kBufs = down_buffers(TMAX);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ LayerLists<TMAX> L;
  __shared__ W4Handover<kBufs> hand;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5), quad = lane >> 2, t = lane & 3;
  const int warps = (blockDim.x >> 5) - 1;
  if (tid == 0) hand.init(warps);
  // idx was written before the kernel in front of this one began; only h is that kernel's
  build_lists(L, (LayerGates<TMAX>*)nullptr, P, kPairs);
  float* sums = reinterpret_cast<float*>(smem + warps * Core::kBytes);     // [kBufs][warp][token][kPitch]
  const int units = (P.d + kCols - 1) / kCols, C = (P.f + kChunk - 1) / kChunk, items = uniform(L.tile[P.slots]) * C;
  if (warp == warps) {
    griddep_wait();
    griddep_launch();
    for (int u = blockIdx.x, i = 0; u < units; u += gridDim.x, ++i) {
      hand.wait_full(i, P.status);
      const float* from = sums + (i % kBufs) * warps * P.T * kPitch;
      for (int q = lane; q < P.T * (kCols / 4); q += 32) {
        const int r = q / (kCols / 4), j = q % (kCols / 4) * 4, col = u * kCols + j;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int w = 0; w < warps; ++w) {
          const float4 a = *reinterpret_cast<const float4*>(from + (w * P.T + r) * kPitch + j);
          v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
        }
        if (col < P.d) {       // (d is a multiple of 32)
          const long long to = (long long)r * P.d + col;
          if (P.out_fp32) *reinterpret_cast<float4*>(reinterpret_cast<float*>(P.y) + to) = v;
          else *reinterpret_cast<uint2*>(reinterpret_cast<bf16*>(P.y) + to) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
        }
      }
      hand.taken(i, lane);
    }
    return;
  }
  const int q0 = items * warp / warps, n = items * (warp + 1) / warps - q0;
  const int tile0 = q0 / C, c0 = q0 - tile0 * C;
  Core core;
  core.init(smem + warp * Core::kBytes, 1, lane);
  int lu = n ? blockIdx.x : units, left = 0, lc = 0, ltile = 0;
  const auto issue = [&](unsigned to) {
    if (lu < units) {
      if (left == 0 || lc == C) {
        if (left == 0) ltile = tile0, lc = c0, left = n;
        else ++ltile, lc = 0;
        int row0[MT], up0[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) row0[i] = lu * kCols + i * 16, up0[i] = row0[i] + 8;
        core.aim(w4_matrix(P.wd, P.sd, uniform(L.slot_of_tile[ltile])), P.sd, row0, up0, P.d, lc, lane);
      }
      core.copy(P.sd, to, lane);
      ++lc;
      if (--left == 0) lu += gridDim.x;
    }
    cp_commit();
  };
  int xu = n ? blockIdx.x : units, xleft = 0, xc = 0, xtile = 0, xR = 0;
  const auto read_h = [&]() {
    if (xu >= units) return;
    if (xleft == 0 || xc == C) {
      if (xleft == 0) xtile = tile0, xc = c0, xleft = n;
      else ++xtile, xc = 0;
      int p0;
      find_tile(L, xtile, kPairs, p0, xR);
#pragma unroll
      for (int r = 0; r < XR; ++r)
        core.xoff[r] = r / kRows < xR && r % kRows < PARTS ? (unsigned)((p0 + r / kRows) * PARTS + r % kRows) * (unsigned)(P.f / 8) : 0u;
    }
    core.read_x(P.h, xc, P.f, kRows * xR, PARTS == 3 ? 0x77u : 0xffu, lane);
    ++xc;
    if (--xleft == 0) xu += gridDim.x;
  };
  // the first weights do not wait for h
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i * Core::kStage);
  griddep_wait();
  griddep_launch();
  read_h();
  for (int u = blockIdx.x, i = 0; u < units; u += gridDim.x, ++i) {
    float* mine = sums + ((i % kBufs) * warps + warp) * P.T * kPitch;
    hand.wait_empty(i, P.status);
    for (int j = lane; j < P.T * kPitch; j += 32) mine[j] = 0.f;
    float acc[MT][4] = {};
    int tile = tile0, c = c0, pair0 = 0, R = 0;
    if (n) find_tile(L, tile, kPairs, pair0, R);
    for (int q = 1; q <= n; ++q) {
      cp_wait<kStages - 2>();
      __syncwarp();
      issue(core.free_slot());
      core.store_x();
      read_h();
      __syncwarp();
      core.multiply(acc, P.f - c * kChunk, lane);
      core.next();
      if (++c == C || q == n) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float lo = acc[mt][0] + acc[mt][1], hi = acc[mt][2] + acc[mt][3];
          if (PARTS == 3) {        // two lanes a pair
            lo += __shfl_xor_sync(0xffffffffu, lo, 1);
            hi += __shfl_xor_sync(0xffffffffu, hi, 1);
          }
          const int r = PARTS == 3 ? t >> 1 : t;
          if (r < R && (PARTS == 2 || !(t & 1))) {
            float* dst = mine + L.token[pair0 + r] * kPitch + mt * 16 + quad;
            dst[0] += lo;
            dst[8] += hi;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[mt][k] = 0.f;
        }
        __syncwarp();
        if (q < n) {
          c = 0;
          find_tile(L, ++tile, kPairs, pair0, R);
        }
      }
    }
    hand.put(i, lane);
  }
}

template <int MT, int XR, int TMAX, int GROUP, bool ZERO>
cudaError_t launch_up(const moe_ops_s* o, const W4LayerParams& P, cudaStream_t s) {
  using Core = W4Core<MT, XR, GROUP, ZERO>;
  auto* kern = w4_up_kernel<MT, XR, TMAX, GROUP, ZERO>;
  constexpr size_t per = Core::kBytes + kSumBuffers * XR * Core::kPitch * sizeof(float);
  const long long units = (long long)P.T * (P.k + P.slots - P.E) * (P.f / (MT * 8));
  constexpr size_t fixed = sizeof(LayerLists<TMAX>) + sizeof(LayerGates<TMAX>) + 128;
  constexpr int warps = w4_warps(fixed, per);
  static_assert((warps + 1) * 32 * kSlotsEach > kMaxSlots, "a place for every slot");
  MOE_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)w4_smem(fixed)));
  return launch_pdl(kern, dim3((unsigned)min(units, (long long)o->sms)), dim3((warps + 1) * 32), warps * per, s, P);
}
template <int MT, int XR, int PARTS, int TMAX, int GROUP, bool ZERO>
cudaError_t launch_down(const moe_ops_s* o, const W4LayerParams& P, cudaStream_t s) {
  using Core = W4Core<MT, XR, GROUP, ZERO>;
  auto* kern = w4_down_kernel<MT, XR, PARTS, TMAX, GROUP, ZERO>;
  constexpr size_t token = down_buffers(TMAX) * Core::kPitch * sizeof(float), fixed = sizeof(LayerLists<TMAX>) + 128;
  static_assert((w4_warps(fixed, Core::kBytes + TMAX * token) + 1) * 32 * kSlotsEach > kMaxSlots, "a place for every slot");
  const size_t per = Core::kBytes + P.T * token;
  const int units = ceil_div(P.d, MT * 16);
  const int warps = w4_warps(fixed, per);
  const size_t smem = warps * per;
  // (a constant: host threads with other numbers of tokens may be between this and their launch)
  MOE_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)w4_smem(fixed)));
  return launch_pdl(kern, dim3(min(units, o->sms)), dim3((warps + 1) * 32), smem, s, P);
}
template <int GROUP, bool ZERO> cudaError_t pick_layer(const moe_ops_s* o, const W4LayerParams& P, cudaStream_t s) {
  if (P.T > 16) {
    MOE_TRY((launch_up<2, 8, 64, GROUP, ZERO>(o, P, s)));
    return P.parts == 3 ? launch_down<2, 8, 3, 64, GROUP, ZERO>(o, P, s) : launch_down<2, 8, 2, 64, GROUP, ZERO>(o, P, s);
  }
  // (4 rows a tile instead of 8 for 3 or 4 tokens, or where experts have one pair on average, measured within 2% and up to
  // 7% slower at 8 tokens of 64 experts; 32 weight rows a unit of the down product instead of 16 takes 222 us instead of
  // 210 for 16 tokens of 32 experts at d = 7168, and 94 instead of 75 at d = 2048: fewer units than SMs)
  if (P.T <= 2) MOE_TRY((launch_up<2, 2, 16, GROUP, ZERO>(o, P, s)));
  else MOE_TRY((launch_up<2, 8, 16, GROUP, ZERO>(o, P, s)));
  if (P.parts == 3) return launch_down<1, 8, 3, 16, GROUP, ZERO>(o, P, s);
  return P.T <= 1 ? launch_down<1, 2, 2, 16, GROUP, ZERO>(o, P, s) : launch_down<1, 8, 2, 16, GROUP, ZERO>(o, P, s);
}

}  // namespace

size_t w4_experts_workspace(const moe_w4_config& c, int T) {
  return (size_t)T * (c.k + c.n_shared) * 3 * c.f * sizeof(bf16);
}

cudaError_t w4_experts(const moe_ops_s* o, const moe_w4_config& c, const void* x, long long ld, int T, const int* idx,
                       const float* gate, const moe_w4& w13, const moe_w4& wd, void* y, int out_fp32, void* ws,
                       cudaStream_t s, long long* n) {
  const auto weights = [](const moe_w4& w) { return W4{w.codes, (const bf16*)w.scale, w.zero}; };
  const W4LayerParams P = {(const bf16*)x, (unsigned)(ld / 8), T, c.k, c.E, c.E + c.n_shared, c.d, c.f, idx, gate,
                           weights(w13), weights(wd), {2 * c.f, c.d, ceil_div(c.d, w13.group)},
                           {c.d, c.f, ceil_div(c.f, w13.group)}, (bf16*)ws, out_fp32 ? 3 : 2, y, out_fp32, o->status};
  *n += 2;
  const bool z = w13.zero != nullptr;
  if (w13.group == 32) return z ? pick_layer<32, true>(o, P, s) : pick_layer<32, false>(o, P, s);
  if (w13.group == 64) return z ? pick_layer<64, true>(o, P, s) : pick_layer<64, false>(o, P, s);
  return z ? pick_layer<128, true>(o, P, s) : pick_layer<128, false>(o, P, s);
}

}  // namespace moe
