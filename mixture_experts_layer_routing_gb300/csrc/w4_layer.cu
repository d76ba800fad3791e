// The experts' layer of a few tokens on 4-bit weights (moe_w4_experts) in two kernels: gate/up products with SwiGLU, and
// down products with the weighted sum over a token's experts.
#include "launch.cuh"
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kMaxSlots = 264;               // experts, shared ones included
constexpr int kMaxPairs = 64 * 16;           // (token, expert) pairs
constexpr int kThreads = kW4Warps * 32;

// The experts in use and their tokens, made by every CTA of both kernels from idx alone. Pairs are sorted by expert,
// then token; an expert that a token names twice is one pair with both gates. A tile is up to `rows` pairs of a slot.
struct LayerLists {
  unsigned mask[kMaxSlots][2];               // tokens of a slot
  int pair[kMaxSlots + 1], tile[kMaxSlots + 1];
  uint16_t slot_of[kMaxPairs];
  uint8_t token[kMaxPairs];
  int tmp[kW4Warps];
};

struct W4LayerParams {
  const uint8_t* x;
  unsigned ld16;
  int T, k, E, slots, d, f;
  const int* idx;
  const float* gate;
  W4 w13, wd;
  W4Shape s13, sd;
  uint8_t* h;             // [pairs][2][f] bf16: rounded, and what the rounding left
  void* y;
  int out_fp32;
  int* status;
};

__device__ __forceinline__ void build_lists(LayerLists& L, const W4LayerParams& P, int rows) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned all[2] = {P.T >= 32 ? ~0u : (1u << P.T) - 1u, P.T >= 64 ? ~0u : P.T > 32 ? (1u << (P.T - 32)) - 1u : 0u};
  for (int i = tid; i < P.slots; i += kThreads) {
    L.mask[i][0] = i < P.E ? 0u : all[0];
    L.mask[i][1] = i < P.E ? 0u : all[1];
  }
  __syncthreads();
  for (int i = tid; i < P.T * P.k; i += kThreads) {
    const int e = P.idx[i], t = i / P.k;
    if ((unsigned)e < (unsigned)P.E) atomicOr(&L.mask[e][t >> 5], 1u << (t & 31));
    else set_error(P.status, MOE_ERR_DEVICE_INDEX);
  }
  __syncthreads();
  int n[2], v = 0;                           // two slots a thread; tiles in the high half
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * tid + j, r = i < P.slots ? __popc(L.mask[i][0]) + __popc(L.mask[i][1]) : 0;
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
  int before = v - n[0] - n[1];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * tid + j;
    if (i <= P.slots) {
      L.pair[i] = before & 0xffff;
      L.tile[i] = before >> 16;
    }
    if (i < P.slots) {
      int p = before & 0xffff;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        for (unsigned m = L.mask[i][h]; m; m &= m - 1) {
          L.token[p] = (uint8_t)(h * 32 + __ffs(m) - 1);
          L.slot_of[p++] = (uint16_t)i;
        }
    }
    before += n[j];
  }
  __syncthreads();
}
// Slot of a tile, its first pair and how many.
__device__ __forceinline__ int find_tile(const LayerLists& L, const W4LayerParams& P, int tile, int rows, int& pair0, int& R) {
  int lo = 0, hi = P.slots;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (L.tile[mid] <= tile) lo = mid; else hi = mid;
  }
  pair0 = L.pair[lo] + (tile - L.tile[lo]) * rows;
  R = min(rows, L.pair[lo + 1] - pair0);
  return lo;
}

constexpr int kUpStages = 3, kDownStages = 3;

template <int NT, int GROUP, bool ZERO> struct W4UpSmem {
  W4Stage<2, NT, GROUP, ZERO> stage[kW4Warps][kUpStages];
  float part[2][kW4Warps][NT * 8][36];       // [pair][16 gate rows, 16 up rows]
  LayerLists lists;
  float gate[kMaxPairs];
};

// Gate and up rows of 16 values of h, up to 8 NT pairs of an expert, for each unit; warps split K = d.
template <int NT, int GROUP, bool ZERO>
__global__ void __launch_bounds__(kThreads, 1) w4_up_kernel(W4LayerParams P) {
  using Core = W4Core<2, NT, GROUP, ZERO>;
  constexpr int kRows = Core::kRows;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<W4UpSmem<NT, GROUP, ZERO>*>(smem_raw);
  LayerLists& L = sm.lists;
  griddep_wait();
  griddep_launch();
  build_lists(L, P, kRows);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int p = tid; p < L.pair[P.slots]; p += kThreads) {
    const int t = L.token[p], e = L.slot_of[p];
    float g = e < P.E ? 0.f : 1.f;
    if (e < P.E)
      for (int j = 0; j < P.k; ++j)
        if (P.idx[t * P.k + j] == e) g += P.gate[t * P.k + j];
    sm.gate[p] = g;
  }
  const int blocks = P.f / 16, units = L.tile[P.slots] * blocks;
  const int C = (P.d + kChunk - 1) / kChunk, c0 = C * warp / kW4Warps, c1 = C * (warp + 1) / kW4Warps;
  Core core;
  core.px = P.x;
  int lu = blockIdx.x, lc = c0;
  const auto issue = [&](int slot) {
    if (lu < units && c0 < c1) {
      if (lc == c0) {
        int pair0, R;
        const int tile = lu / blocks, m = lu - tile * blocks, e = find_tile(L, P, tile, kRows, pair0, R);
        const int row0[2] = {m * 16, P.f + m * 16}, end[2] = {P.f, 2 * P.f};
        core.set_weights(w4_matrix(P.w13, P.s13, e), P.s13, row0, end, lane);
        core.xn = (R + 1) / 2;
#pragma unroll
        for (int i = 0; i < NT * 4; ++i) {
          const int r = (lane >> 4) + 2 * i;
          core.xoff[i] = r < R ? (unsigned)L.token[pair0 + r] * P.ld16 : ~0u;
        }
      }
      core.copy_weights(sm.stage[warp][slot], P.s13, lc, lane);
      core.copy_x(sm.stage[warp][slot], P.s13, lc, lane);
      if (++lc == c1) {
        lc = c0;
        lu += gridDim.x;
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kUpStages - 1; ++i) issue(i);
  __syncthreads();        // the gates
  int slot = 0, buf = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x, buf ^= 1) {
    int pair0, R;
    const int tile = u / blocks, m = u - tile * blocks;
    find_tile(L, P, tile, kRows, pair0, R);
    float acc[2][NT][4] = {};
    for (int c = c0; c < c1; ++c) {
      cp_wait<kUpStages - 2>();
      __syncwarp();
      issue(slot == 0 ? kUpStages - 1 : slot - 1);
      Core::multiply(sm.stage[warp][slot], acc, (R + 7) / 8, lane);
      slot = slot + 1 == kUpStages ? 0 : slot + 1;
    }
    const int quad = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        float(*p)[36] = &sm.part[buf][warp][n * 8 + 2 * t];
        p[0][mt * 16 + quad] = acc[mt][n][0];
        p[1][mt * 16 + quad] = acc[mt][n][1];
        p[0][mt * 16 + quad + 8] = acc[mt][n][2];
        p[1][mt * 16 + quad + 8] = acc[mt][n][3];
      }
    __syncthreads();      // (the buffer before the last one has been read by all when they are here)
    for (int i = tid; i < R * 16; i += kThreads) {
      const int r = i >> 4, j = i & 15;
      float g = 0.f, up = 0.f;
#pragma unroll
      for (int w = 0; w < kW4Warps; ++w) {
        g += sm.part[buf][w][r][j];
        up += sm.part[buf][w][r][16 + j];
      }
      const float h = silu_f(g) * up * sm.gate[pair0 + r];
      // h as a sum of two bf16 (16 bits of mantissa), so that the layer rounds once, at its output
      const bf16 hi = __float2bfloat16_rn(h);
      const float left = h - __bfloat162float(hi);
      const bf16 lo = __float2bfloat16_rn(fabsf(left) <= 3.3895314e38f ? left : 0.f);
      bf16* dst = reinterpret_cast<bf16*>(P.h) + (long long)(pair0 + r) * 2 * P.f + m * 16 + j;
      dst[0] = hi;
      dst[P.f] = lo;
    }
  }
}

template <int NT, int GROUP, bool ZERO> struct W4DownSmem {
  W4Stage<1, NT, GROUP, ZERO> stage[kW4Warps][kDownStages];
  LayerLists lists;
  // float sum[kW4Warps][T][20] follows: [token][16 rows]
};

// 16 values of y for all tokens a unit. The chunks of all experts in use are dealt to the warps; columns 2r and 2r + 1
// of a product are the two parts of pair r's h, and a warp adds an expert's product to its own sums of the tokens.
template <int NT, int GROUP, bool ZERO>
__global__ void __launch_bounds__(kThreads, 1) w4_down_kernel(W4LayerParams P) {
  using Core = W4Core<1, NT, GROUP, ZERO>;
  constexpr int kPairs = Core::kRows / 2;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<W4DownSmem<NT, GROUP, ZERO>*>(smem_raw);
  LayerLists& L = sm.lists;
  float(*sum)[20] = reinterpret_cast<float(*)[20]>(smem_raw + sizeof(W4DownSmem<NT, GROUP, ZERO>));
  // idx was written before the kernel in front of this one began; only h is that kernel's
  build_lists(L, P, kPairs);
  griddep_wait();
  griddep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = lane >> 2, t = lane & 3;
  const int units = (P.d + 15) / 16, C = (P.f + kChunk - 1) / kChunk, items = L.tile[P.slots] * C;
  const int q0 = (int)((long long)items * warp / kW4Warps), q1 = (int)((long long)items * (warp + 1) / kW4Warps);
  float(*mine)[20] = sum + warp * P.T;
  Core core;
  core.px = P.h;
  int lu = blockIdx.x, lq = q0, lc = 0, ltile = 0;
  const auto issue = [&](int slot) {
    if (lu < units && q0 < q1) {
      if (lq == q0 || lc == C) {
        if (lq == q0) ltile = q0 / C, lc = q0 - ltile * C;
        else ++ltile, lc = 0;
        int pair0, R;
        const int e = find_tile(L, P, ltile, kPairs, pair0, R);
        const int row0[1] = {lu * 16}, end[1] = {P.d};
        core.set_weights(w4_matrix(P.wd, P.sd, e), P.sd, row0, end, lane);
        core.xn = R;
#pragma unroll
        for (int i = 0; i < NT * 4; ++i) {
          const int r = (lane >> 4) + 2 * i;
          core.xoff[i] = r < 2 * R ? (unsigned)(2 * pair0 + r) * (unsigned)(P.f / 8) : ~0u;
        }
      }
      core.copy_weights(sm.stage[warp][slot], P.sd, lc, lane);
      core.copy_x(sm.stage[warp][slot], P.sd, lc, lane);
      ++lc;
      if (++lq == q1) {
        lq = q0;
        lu += gridDim.x;
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kDownStages - 1; ++i) issue(i);
  int slot = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    for (int i = lane; i < P.T * 20; i += 32) mine[0][i] = 0.f;
    float acc[1][NT][4] = {};
    int tile = q0 / C, c = q0 - tile * C, pair0 = 0, R = 0;
    if (q0 < q1) find_tile(L, P, tile, kPairs, pair0, R);
    for (int q = q0; q < q1; ++q) {
      cp_wait<kDownStages - 2>();
      __syncwarp();
      issue(slot == 0 ? kDownStages - 1 : slot - 1);
      Core::multiply(sm.stage[warp][slot], acc, (R + 3) / 4, lane);
      slot = slot + 1 == kDownStages ? 0 : slot + 1;
      if (++c == C || q + 1 == q1) {
        __syncwarp();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int r = n * 4 + t;
          if (r < R) {
            float* dst = mine[L.token[pair0 + r]];
            dst[quad] += acc[0][n][0] + acc[0][n][1];
            dst[quad + 8] += acc[0][n][2] + acc[0][n][3];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[0][n][j] = 0.f;
        }
        if (q + 1 < q1) {
          c = 0;
          find_tile(L, P, ++tile, kPairs, pair0, R);
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < P.T * 16; i += kThreads) {
      const int r = i >> 4, j = i & 15, col = u * 16 + j;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kW4Warps; ++w) v += sum[w * P.T + r][j];
      if (col < P.d) {
        const long long at = (long long)r * P.d + col;
        if (P.out_fp32) reinterpret_cast<float*>(P.y)[at] = v;
        else reinterpret_cast<bf16*>(P.y)[at] = __float2bfloat16_rn(v);
      }
    }
    __syncthreads();
  }
}

template <int NT, int GROUP, bool ZERO>
cudaError_t launch_layer(const moe_ops_s* o, const W4LayerParams& P, cudaStream_t s) {
  auto* up = w4_up_kernel<NT, GROUP, ZERO>;
  auto* down = w4_down_kernel<NT, GROUP, ZERO>;
  const size_t su = sizeof(W4UpSmem<NT, GROUP, ZERO>);
  const size_t sd = sizeof(W4DownSmem<NT, GROUP, ZERO>) + sizeof(float) * kW4Warps * P.T * 20;
  MOE_TRY(cudaFuncSetAttribute(up, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)su));
  MOE_TRY(cudaFuncSetAttribute(down, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sd));
  const int pairs = P.T * (P.k + P.slots - P.E);
  const long long units = (long long)pairs * (P.f / 16);
  MOE_TRY(launch_pdl(up, dim3((unsigned)min(units, (long long)o->sms * 2)), dim3(kThreads), su, s, P));
  return launch_pdl(down, dim3(min(ceil_div(P.d, 16), o->sms * 2)), dim3(kThreads), sd, s, P);
}
template <int NT> cudaError_t pick_layer(const moe_ops_s* o, const W4LayerParams& P, int group, cudaStream_t s) {
  const bool z = P.w13.zero != nullptr;
  if (group == 32) return z ? launch_layer<NT, 32, true>(o, P, s) : launch_layer<NT, 32, false>(o, P, s);
  if (group == 64) return z ? launch_layer<NT, 64, true>(o, P, s) : launch_layer<NT, 64, false>(o, P, s);
  return z ? launch_layer<NT, 128, true>(o, P, s) : launch_layer<NT, 128, false>(o, P, s);
}

}  // namespace

size_t w4_experts_workspace(const moe_w4_config& c, int T) {
  return (size_t)T * (c.k + c.n_shared) * 2 * c.f * sizeof(bf16);
}

cudaError_t w4_experts(const moe_ops_s* o, const moe_w4_config& c, const void* x, long long ld, int T, const int* idx,
                       const float* gate, const moe_w4& w13, const moe_w4& wd, void* y, int out_fp32, void* ws,
                       cudaStream_t s, long long* n) {
  const auto weights = [](const moe_w4& w) { return W4{w.codes, (const bf16*)w.scale, w.zero}; };
  const W4LayerParams P = {(const uint8_t*)x, (unsigned)(ld / 8), T, c.k, c.E, c.E + c.n_shared, c.d, c.f, idx, gate,
                           weights(w13), weights(wd), {2 * c.f, c.d, ceil_div(c.d, w13.group)},
                           {c.d, c.f, ceil_div(c.f, w13.group)}, (uint8_t*)ws, y, out_fp32, o->status};
  *n += 2;
  return T > 8 ? pick_layer<2>(o, P, w13.group, s) : pick_layer<1>(o, P, w13.group, s);
}

}  // namespace moe
