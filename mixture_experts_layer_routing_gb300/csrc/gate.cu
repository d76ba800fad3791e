// Routing from router logits (include/moe_ops.h): scores, balance bias, groups, top-k, gates and the dispatch
// (counts, offsets, stable permutation), and the gradient of the logits.
//
// One warp a token; lane i holds the PER consecutive experts i*PER .. (E <= 32 PER), so the lowest lane that holds
// a maximum also holds the lowest expert, and equal keys need no index comparison. Every round of the top-k is one
// redux over the lanes' own maxima. Keys are computed in 32 bits. Their error bound (tau) decides whether the
// outcome could differ from that of 64-bit keys: every gap that the selection rests on (between neighbours of the
// sorted selection, to the first expert left out, between the worst group kept and the best left out) has to exceed
// it; a token where one does not is selected again with 64-bit keys. Double precision is slow on this GPU (about
// 1/64 of the fp32 rate), and only a fraction of a percent of tokens takes that path.
//
// The dispatch: tokens are cut into chunks, one CTA each, at most one chunk a SM. The selecting CTA counts its
// chunk's experts. With one chunk it also writes offsets and permutation; otherwise a second kernel adds up the
// chunk counts before its own chunk and ranks the chunk's assignments. Integers only, the same in every run.
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"

namespace moe {
namespace {

constexpr int kGateThreads = 1024, kGateWarps = kGateThreads / 32;
constexpr int kGateTokens = 64;      // tokens of a chunk, at least
constexpr unsigned kFull = 0xffffffffu;

// Order-preserving map of floats (no NaN) to unsigned, so that redux finds the maximum in one instruction.
__device__ __forceinline__ unsigned order_of(float v) {
  const unsigned u = __float_as_uint(v);
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_order(unsigned u) {
  return __uint_as_float(u >> 31 ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ float lanes_max(float v) { return of_order(__reduce_max_sync(kFull, order_of(v))); }
__device__ __forceinline__ double lanes_max(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <typename F> __device__ __forceinline__ F lowest();
template <> __device__ __forceinline__ float lowest<float>() { return -FLT_MAX; }
template <> __device__ __forceinline__ double lowest<double>() { return -DBL_MAX; }
template <typename F> __device__ __forceinline__ F inf_of() { return (F)INFINITY; }

// Lane j < k returns the j-th selected expert. `sure` turns false where a gap that the outcome rests on is not
// above tau.
template <int PER, typename F>
__device__ __forceinline__ int select_experts(F (&key)[PER], const moe_gate_config& c, F tau, bool& sure) {
  const int lane = threadIdx.x & 31, e0 = lane * PER;
  if (c.topk_groups < c.n_groups) {
    const int S = c.E / c.n_groups;
    F score = -inf_of<F>();   // lane g: group g
    for (int g = 0; g < c.n_groups; ++g) {
      F a = -inf_of<F>(), b = -inf_of<F>();   // this lane's two best of group g
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        if (e0 + q >= g * S && e0 + q < (g + 1) * S) {
          if (key[q] > a) {
            b = a;
            a = key[q];
          } else if (key[q] > b) {
            b = key[q];
          }
        }
      }
      const F m = lanes_max(a);
      F sum = m;
      if (S > 1) {
        const int owner = __ffs(__ballot_sync(kFull, a == m)) - 1;
        sum += lanes_max(lane == owner ? b : a);
      }
      if (lane == g) score = sum;
    }
    int rank = 0;
    for (int g = 0; g < c.n_groups; ++g) {
      const F other = __shfl_sync(kFull, score, g);
      rank += other > score || (other == score && g < lane);
    }
    const bool kept = lane < c.n_groups && rank < c.topk_groups;
    const unsigned mask = __ballot_sync(kFull, kept);
    const F worst = -lanes_max(kept ? -score : -inf_of<F>());
    const F best = lanes_max(lane < c.n_groups && !kept ? score : -inf_of<F>());
    if (!(worst - best > 3 * tau)) sure = false;   // a score is a sum of two keys
    int g = e0 / S, r = e0 - g * S;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      if (!(mask >> g & 1u)) key[q] = -inf_of<F>();
      if (++r == S) {
        r = 0;
        ++g;
        if (g > 31) g = 31;   // (past the last expert: the key is -inf already)
      }
    }
  }
  int mine = 0, at = 0;
  F top = key[0];
#pragma unroll
  for (int q = 1; q < PER; ++q)
    if (key[q] > top) {
      top = key[q];
      at = q;
    }
  F last = 0;
  for (int j = 0; j <= c.k; ++j) {
    const F m = lanes_max(top);
    if (j > 0 && !(last - m > tau)) sure = false;
    if (j == c.k) break;
    last = m;
    const int owner = __ffs(__ballot_sync(kFull, top == m)) - 1;
    const int e = __shfl_sync(kFull, e0 + at, owner);
    if (lane == j) mine = e;
    if (lane == owner) {
      F best = -inf_of<F>();
      int b = 0;
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        if (q == at) key[q] = -inf_of<F>();
        if (key[q] > best) {
          best = key[q];
          b = q;
        }
      }
      top = best;
      at = b;
    }
  }
  return mine;
}

template <typename F>
__device__ __forceinline__ F key_of(F p, F b, float l) {
  const F k = p + b;
  return (l == -INFINITY || isnan(k)) ? lowest<F>() : fmax(k, lowest<F>());
}

// The selection with 64-bit keys.
template <int PER>
__device__ __noinline__ int select_exact(const float* __restrict__ logits, const float* __restrict__ bias, float m,
                                         const moe_gate_config& c) {
  const int e0 = (threadIdx.x & 31) * PER;
  double key[PER], sum = 0.0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    key[q] = 0.0;
    if (e0 + q < c.E) {
      const double l = (double)logits[e0 + q];
      key[q] = c.router == MOE_ROUTER_SOFTMAX ? exp(l - (double)m) : 1.0 / (1.0 + exp(-l));
      sum += key[q];
    }
  }
  if (c.router == MOE_ROUTER_SOFTMAX) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    if (e0 + q < c.E) {
      const double p = c.router == MOE_ROUTER_SOFTMAX ? (sum == 0.0 ? 0.0 : key[q] / sum) : key[q];
      key[q] = key_of<double>(p, bias ? (double)bias[e0 + q] : 0.0, logits[e0 + q]);
    } else {
      key[q] = -inf_of<double>();
    }
  }
  bool sure = true;
  return select_experts<PER, double>(key, c, 0.0, sure);
}

// One token: lane j < k returns expert j of the selection and its gate.
template <int PER>
__device__ __forceinline__ int gate_token(const float* __restrict__ logits, const float* __restrict__ bias,
                                          const moe_gate_config& c, float& gate) {
  const int lane = threadIdx.x & 31, e0 = lane * PER;
  float l[PER], p[PER], key[PER];
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    l[q] = e0 + q < c.E ? logits[e0 + q] : -INFINITY;
    m = fmaxf(m, l[q]);
  }
  float pmax = 1.f;
  if (c.router == MOE_ROUTER_SOFTMAX) {
    m = lanes_max(m);
    if (m == -INFINITY) m = 0.f;   // no expert left: every score 0
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      p[q] = expf(l[q] - m);
      sum += p[q];
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int q = 0; q < PER; ++q) p[q] = sum == 0.f ? 0.f : p[q] / sum;
    pmax = sum == 0.f ? 0.f : 1.f / sum;
  } else {
#pragma unroll
    for (int q = 0; q < PER; ++q) p[q] = 1.f / (1.f + expf(-l[q]));
  }
  float kmax = 0.f;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const bool in = e0 + q < c.E;
    key[q] = in ? key_of<float>(p[q], bias ? bias[e0 + q] : 0.f, l[q]) : -INFINITY;
    if (in && key[q] != -FLT_MAX) kmax = fmaxf(kmax, fabsf(key[q]));
  }
  kmax = lanes_max(kmax);
  // Error of a difference of two keys: scores within 14 units in the last place of the largest score (exp, the
  // argument's and the sum's rounding, the quotient; a sigmoid within 4), each key's addition half a unit.
  const float tau = (c.router == MOE_ROUTER_SOFTMAX ? 0x1p-18f : 0x1p-20f) * pmax + 0x1p-22f * kmax;
  bool sure = true;
  int e = select_experts<PER, float>(key, c, tau, sure);
  if (!sure) e = select_exact<PER>(logits, bias, m, c);
  float ps = 0.f;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const float v = __shfl_sync(kFull, p[q], e / PER);
    if (e % PER == q) ps = v;
  }
  if (lane >= c.k) ps = 0.f;
  gate = c.renorm ? c.route_scale * (ps / (warp_sum(ps) + 1e-20f)) : c.route_scale * ps;
  return e;
}

// Exclusive scan of v over threads 0..255 (others pass 0 and get no meaningful value). tmp: 8 words.
__device__ __forceinline__ int scan256(int v, int* tmp) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += u;
  }
  if (w < 8 && lane == 31) tmp[w] = s;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < (w < 8 ? w : 0); ++i) before += tmp[i];
  return before + s - v;
}

// Shared memory of the dispatch: run[e] = next sorted position of expert e, wcnt[w][e] = counts of a pass's warps.
struct DispatchSmem {
  int run[kMaxE], wcnt[kGateWarps][kMaxE], tmp[8];
};

// Sorted positions of the assignments a0 .. a1, in passes of the block's threads; run[] holds each expert's first.
__device__ __forceinline__ void rank_chunk(DispatchSmem& sm, const int* idx, int a0, int a1, int E,
                                           int* __restrict__ perm, int* __restrict__ inv) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  for (int p0 = a0; p0 < a1; p0 += kGateThreads) {
    const int nw = min(kGateWarps, (a1 - p0 + 31) / 32);
    for (int i = tid; i < nw * kMaxE; i += kGateThreads) (&sm.wcnt[0][0])[i] = 0;
    __syncthreads();
    const int a = p0 + tid;
    const int e = a < a1 ? idx[a] : -1;
    const unsigned same = __match_any_sync(kFull, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) sm.wcnt[w][e] = __popc(same);
    __syncthreads();
    if (tid < E) {   // counts -> first positions
      int r = sm.run[tid];
      for (int i = 0; i < nw; ++i) {
        const int n = sm.wcnt[i][tid];
        sm.wcnt[i][tid] = r;
        r += n;
      }
      sm.run[tid] = r;
    }
    __syncthreads();
    if (e >= 0) {
      const int pos = sm.wcnt[w][e] + rank;
      perm[pos] = a;
      inv[a] = pos;
    }
    __syncthreads();
  }
}

// Chunk = `tokens` tokens a CTA. hist (nullable): the chunk's expert counts. With one chunk (gridDim.x = 1) and
// cnt given, the whole dispatch.
template <int PER>
__global__ void __launch_bounds__(kGateThreads) gate_kernel(const float* __restrict__ logits,
                                                            const float* __restrict__ bias, int T, int tokens,
                                                            moe_gate_config c, int* idx, float* gate, int* hist,
                                                            int* cnt, int* off, int* perm, int* inv) {
  __shared__ DispatchSmem sm;
  griddep_wait();
  griddep_launch();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const bool counts = hist || cnt;
  if (counts && tid < kMaxE) sm.run[tid] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * tokens, t1 = min(T, t0 + tokens);
  for (int t = t0 + w; t < t1; t += kGateWarps) {
    float g;
    const int e = gate_token<PER>(logits + (size_t)t * c.E, bias, c, g);
    if (lane < c.k) {
      idx[(size_t)t * c.k + lane] = e;
      gate[(size_t)t * c.k + lane] = g;
      if (counts) atomicAdd(&sm.run[e], 1);
    }
  }
  if (!counts) return;
  __syncthreads();
  if (hist) {
    if (tid < c.E) hist[blockIdx.x * c.E + tid] = sm.run[tid];
    return;
  }
  const int n = tid < c.E ? sm.run[tid] : 0;
  const int first = scan256(n, sm.tmp);
  if (tid < c.E) {
    cnt[tid] = n;
    off[tid] = first;
    sm.run[tid] = first;
    if (tid == c.E - 1) off[c.E] = first + n;
  }
  __syncthreads();
  rank_chunk(sm, idx, 0, T * c.k, c.E, perm, inv);
}

// Second kernel of a dispatch of several chunks: CTA ch adds up every chunk's counts (and those before its own) and
// ranks its assignments.
__global__ void __launch_bounds__(kGateThreads) dispatch_kernel(const int* __restrict__ hist, int nch, int T,
                                                                int tokens, int E, int k, const int* __restrict__ idx,
                                                                int* cnt, int* off, int* perm, int* inv) {
  __shared__ DispatchSmem sm;
  griddep_wait();
  griddep_launch();
  const int tid = threadIdx.x, ch = blockIdx.x;
  // four threads an expert, each a quarter of the chunks
  const int e = tid & (kMaxE - 1), part = tid / kMaxE;
  int all = 0, before = 0;
  if (e < E) {
#pragma unroll 8
    for (int i = part; i < nch; i += kGateThreads / kMaxE) {
      const int n = hist[i * E + e];
      all += n;
      before += i < ch ? n : 0;
    }
  }
  sm.wcnt[part][e] = all;
  sm.wcnt[4 + part][e] = before;
  __syncthreads();
  int n = 0;
  before = 0;
  if (tid < E) {
#pragma unroll
    for (int i = 0; i < kGateThreads / kMaxE; ++i) {
      n += sm.wcnt[i][tid];
      before += sm.wcnt[4 + i][tid];
    }
  }
  const int first = scan256(n, sm.tmp);
  if (tid < E) {
    sm.run[tid] = first + before;
    if (ch == 0) {
      cnt[tid] = n;
      off[tid] = first;
      if (tid == E - 1) off[E] = first + n;
    }
  }
  __syncthreads();
  rank_chunk(sm, idx, ch * tokens * k, min(T, (ch + 1) * tokens) * k, E, perm, inv);
}

// One warp a token. With p the scores, ps those selected, D = sum ps + 1e-20:
//   dL/dps_j = scale (renorm ? (dgate_j - sum_i dgate_i ps_i / D) / D : dgate_j)
//   sigmoid: dl = p (1 - p) dp;   softmax: dl = p (dp - sum p dp)
// Renormalised softmax gates do not depend on the logits that were not selected (sum p dp is 0 up to 1e-20), and
// there p / D is the softmax over the selected alone, so neither router reads more than the selected logits; plain
// softmax gates need the row.
template <int PER>
__global__ void __launch_bounds__(256) gate_bwd_kernel(const float* __restrict__ logits, const int* __restrict__ idx,
                                                       const float* __restrict__ dgate, int T, moe_gate_config c,
                                                       float* __restrict__ dlogits, int* status) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, t = blockIdx.x * 8 + (threadIdx.x >> 5), e0 = lane * PER;
  if (t >= T) return;
  logits += (size_t)t * c.E;
  int e = -1;
  float dg = 0.f, l = -INFINITY;
  if (lane < c.k) {
    e = idx[(size_t)t * c.k + lane];
    if ((unsigned)e >= (unsigned)c.E) {
      set_error(status, MOE_ERR_DEVICE_INDEX);
      e = -1;
    } else {
      dg = c.route_scale * dgate[(size_t)t * c.k + lane];
      l = logits[e];
    }
  }
  float v;                        // dlogits of this lane's selected expert
  float row[PER], dot = 0.f;      // plain softmax: the row's scores
#pragma unroll
  for (int q = 0; q < PER; ++q) row[q] = 0.f;
  if (c.router == MOE_ROUTER_SOFTMAX) {
    float m = l;
    const bool whole = !c.renorm;
    if (whole) {
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        row[q] = e0 + q < c.E ? logits[e0 + q] : -INFINITY;
        m = fmaxf(m, row[q]);
      }
    }
    m = lanes_max(m);
    if (m == -INFINITY) m = 0.f;
    float ps = e >= 0 ? expf(l - m) : 0.f, sum = ps;
    if (whole) {
      sum = 0.f;
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        row[q] = expf(row[q] - m);
        sum += row[q];
      }
    }
    sum = warp_sum(sum);
    const float r = sum == 0.f ? 0.f : 1.f / sum;
    ps *= r;
    dot = warp_sum(ps * dg);
    v = ps * (dg - dot);
#pragma unroll
    for (int q = 0; q < PER; ++q) row[q] *= -r * dot;
  } else {
    const float ps = e >= 0 ? 1.f / (1.f + expf(-l)) : 0.f;
    // 1 - p without cancellation where p is near one
    const float rest = e >= 0 ? 1.f / (1.f + expf(l)) : 0.f;
    if (c.renorm) {
      const float D = warp_sum(ps) + 1e-20f;
      dg = (dg - warp_sum(dg * ps) / D) / D;
    }
    v = ps * rest * dg;
  }
  for (int j = 0; j < c.k; ++j) {
    const int ej = __shfl_sync(kFull, e, j);
    const float vj = __shfl_sync(kFull, v, j);
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (ej == e0 + q) row[q] = vj;
  }
#pragma unroll
  for (int q = 0; q < PER; ++q)
    if (e0 + q < c.E) dlogits[(size_t)t * c.E + e0 + q] = row[q];
}

inline int chunk_tokens(int T, int sms) {
  const int t = ceil_div(T, sms);
  return t < kGateTokens ? kGateTokens : t;
}

template <int PER>
cudaError_t fwd(const float* logits, const float* bias, int T, int tokens, const moe_gate_config& c, int* idx,
                float* gate, int* hist, int* cnt, int* off, int* perm, int* inv, cudaStream_t s) {
  return launch_pdl(gate_kernel<PER>, dim3(ceil_div(T, tokens)), dim3(kGateThreads), 0, s, logits, bias, T, tokens, c,
                    idx, gate, hist, cnt, off, perm, inv);
}
template <int PER>
cudaError_t bwd(const float* logits, const int* idx, const float* dgate, int T, const moe_gate_config& c,
                float* dlogits, int* status, cudaStream_t s) {
  return launch_pdl(gate_bwd_kernel<PER>, dim3(ceil_div(T, 8)), dim3(256), 0, s, logits, idx, dgate, T, c, dlogits,
                    status);
}

}  // namespace

// One count of every expert for each chunk; chunks number at most one for each 64 tokens.
size_t gate_workspace(const moe_gate_config& c, int T) { return sizeof(int) * (size_t)c.E * ceil_div(T, kGateTokens); }

cudaError_t gate_forward(const moe_ops_s* o, const moe_gate_config& c, const float* logits, const float* bias, int T,
                         int* idx, float* gate, int* cnt, int* off, int* perm, int* inv, void* ws, cudaStream_t s,
                         long long* n) {
  const int tokens = chunk_tokens(T, o->sms), nch = ceil_div(T, tokens);
  const bool two = cnt && nch > 1;
  const auto call = c.E <= 32 ? fwd<1> : c.E <= 64 ? fwd<2> : c.E <= 128 ? fwd<4> : fwd<8>;
  *n += 1;
  MOE_TRY(call(logits, bias, T, tokens, c, idx, gate, two ? (int*)ws : nullptr, two ? nullptr : cnt, off, perm, inv,
               s));
  if (!two) return cudaSuccess;
  *n += 1;
  return launch_pdl(dispatch_kernel, dim3(nch), dim3(kGateThreads), 0, s, (const int*)ws, nch, T, tokens, c.E, c.k,
                    (const int*)idx, cnt, off, perm, inv);
}

cudaError_t gate_backward(const moe_ops_s* o, const moe_gate_config& c, const float* logits, const int* idx,
                          const float* dgate, int T, float* dlogits, cudaStream_t s, long long* n) {
  const auto call = c.E <= 32 ? bwd<1> : c.E <= 64 ? bwd<2> : c.E <= 128 ? bwd<4> : bwd<8>;
  *n += 1;
  return call(logits, idx, dgate, T, c, dlogits, o->status, s);
}

}  // namespace moe
