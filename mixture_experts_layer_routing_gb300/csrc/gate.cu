// Routing from router logits (include/moe_ops.h): scores, balance bias, groups, top-k, gates and the dispatch
// (counts, offsets, stable permutation), and the gradient of the logits.
//
// One warp a token; lane i holds the PER consecutive experts i*PER .. (E <= 32 PER). Keys are computed in 32 bits
// with fast exponentials and kept as unsigned integers in the floats' order, so a round of the top-k is one redux
// over the lanes and a masked maximum over a lane's own keys. A bound of each key's error (KeyBound) decides whether
// the outcome could differ from that of 64-bit keys: the intervals of neighbours of the sorted selection, of its last
// and the first expert left out, and of the worst group kept and the best left out must not meet. Where two do, the
// experts that may belong to the selection get 64-bit keys, one a lane (double precision runs at about 1/64 of the fp32
// rate here, so not every expert's). The gates are computed from the selected logits with expf; a softmax's
// denominator is the sum of the fast exponentials, up to 20 units of 2^-24 off, which renormalised gates cancel.
//
// The dispatch: tokens are cut into chunks, one CTA each, at most one chunk a SM. The selecting CTA counts its
// chunk's experts. With one chunk it also writes offsets and permutation; otherwise a second kernel adds up the
// chunk counts before its own chunk and ranks the chunk's assignments. Integers only, the same in every run.
//
// Measured, 8192 tokens of 256 experts in 8 groups: 22 us, 16 of them the selection (63% of the issue slots, some 1,100
// instructions a token; its 8.4 MB would take 1.3) and the rest the dispatch. With 64-bit keys for all 183 us. The
// same with an expert or 32 masked by the bias, logits around -10, or peaked softmax rows: 18-22 us. Sigmoid logits
// around 10 without a bias need 64 bits in most rows, their scores being within some 2^-24 of 1 and each other: 58 us.
// Four tokens in 4.7 us (the bounds are 0.2 of it).
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"

namespace moe {
namespace {

constexpr int kGateThreads = 1024, kGateWarps = kGateThreads / 32;
// Tokens of a chunk: all of them up to 16 (then one kernel does it all), else 8 in up to 64 chunks and 32, a token a
// warp, before there are more. A warp with a second token, or many of them on one SM, cost more than a second launch
// and its reading of all chunks' counts: 64 tokens of 256 experts take 13.7 us in one chunk, 9.3 in chunks of 32 and
// 6.4 of 8, 512 tokens 17.0 in chunks of 32 and 14.0 of 8, but 2,048 tokens 17.4 and 18.2, of 64 experts 9.4 and 11.0.
constexpr int kOneChunk = 16, kChunkLeast = 8, kChunkTokens = 32, kFewChunks = 64;
constexpr unsigned kFull = 0xffffffffu;

// Order-preserving map of floats (no NaN) to unsigned; 0 is below every float's.
__device__ __forceinline__ unsigned order_of(float v) {
  const unsigned u = __float_as_uint(v);
  return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_order(unsigned u) {
  return __uint_as_float(u >> 31 ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ float lanes_max(float v) { return of_order(__reduce_max_sync(kFull, order_of(v))); }
// The same for doubles: compared as integers, in the integer pipe.
typedef unsigned long long u64;
__device__ __forceinline__ u64 order_of(double v) {
  const u64 u = (u64)__double_as_longlong(v);
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double of_order(u64 u) {
  return __longlong_as_double((long long)(u >> 63 ? u & 0x7fffffffffffffffull : ~u));
}
__device__ __forceinline__ u64 lanes_max(u64 v) {
  const unsigned hi = __reduce_max_sync(kFull, (unsigned)(v >> 32));
  const unsigned lo = __reduce_max_sync(kFull, (unsigned)(v >> 32) == hi ? (unsigned)v : 0u);
  return (u64)hi << 32 | lo;
}
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// The 64-bit path is rarely taken, so its instructions come from far: it is written for few of them (no unrolling, one
// copy of each double-precision function), not for speed once they are there.
__device__ __noinline__ double exact_exp(double x) { return exp(x); }
// The 64-bit key of an expert, in order. m, sum: the row's largest logit and sum of exponentials (softmax).
__device__ __noinline__ u64 exact_key(int softmax, float l, float b, float m, double sum) {
  const double t = exact_exp(softmax ? (double)l - (double)m : -(double)l);
  const double p = softmax && sum == 0.0 ? 0.0 : (softmax ? t : 1.0) / (softmax ? sum : 1.0 + t);
  const double k = p + (double)b;
  return order_of((l == -INFINITY || isnan(k)) ? -DBL_MAX : fmax(k, -DBL_MAX));
}
__device__ __forceinline__ double exact_sum(const moe_gate_config& c, const float* __restrict__ logits, float m) {
  double s = 0.0;
  if (c.router != MOE_ROUTER_SOFTMAX) return s;
#pragma unroll 1
  for (int e = threadIdx.x & 31; e < c.E; e += 32) s += exact_exp((double)logits[e] - (double)m);
  return lanes_sum(s);
}

// The whole selection with 64-bit keys: lane j < k returns its j-th expert. The lowest lane that holds a maximum also
// holds the lowest such expert, so ties need no comparison of indexes.
template <int PER>
__device__ __noinline__ int select_exact(const float* __restrict__ logits, const float* __restrict__ bias, float m,
                                         const moe_gate_config& c) {
  const int lane = threadIdx.x & 31, e0 = lane * PER;
  const double sum = exact_sum(c, logits, m);
  u64 key[PER];
#pragma unroll 1
  for (int q = 0; q < PER; ++q)
    key[q] = e0 + q < c.E ? exact_key(c.router == MOE_ROUTER_SOFTMAX, logits[e0 + q], bias ? bias[e0 + q] : 0.f, m, sum)
                          : 0ull;
  if (c.topk_groups < c.n_groups) {
    const int S = c.E / c.n_groups;
    u64 score = 0ull;   // lane g: group g
#pragma unroll 1
    for (int g = 0; g < c.n_groups; ++g) {
      u64 a = 0ull, b = 0ull;   // this lane's two best of group g
#pragma unroll 1
      for (int q = 0; q < PER; ++q) {
        if (e0 + q >= g * S && e0 + q < (g + 1) * S) {
          b = max(b, min(a, key[q]));
          a = max(a, key[q]);
        }
      }
      const u64 first = lanes_max(a);
      u64 s = first;
      if (S > 1) {
        const int owner = __ffs(__ballot_sync(kFull, a == first)) - 1;
        s = order_of(of_order(first) + of_order(lanes_max(lane == owner ? b : a)));
      }
      if (lane == g) score = s;
    }
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < c.n_groups; ++g) {
      const u64 other = __shfl_sync(kFull, score, g);
      rank += other > score || (other == score && g < lane);
    }
    const unsigned kept = __ballot_sync(kFull, lane < c.n_groups && rank < c.topk_groups);
#pragma unroll 1
    for (int q = 0; q < PER; ++q)
      if (e0 + q < c.E && !(kept >> ((e0 + q) / S) & 1u)) key[q] = 0ull;
  }
  int mine = 0;
#pragma unroll 1
  for (int j = 0; j < c.k; ++j) {
    u64 top = 0ull;
    int at = 0;
#pragma unroll 1
    for (int q = 0; q < PER; ++q) {
      if (key[q] > top) {
        top = key[q];
        at = q;
      }
    }
    const u64 best = lanes_max(top);
    const int owner = __ffs(__ballot_sync(kFull, top == best)) - 1;
    const int e = __shfl_sync(kFull, e0 + at, owner);
    if (lane == j) mine = e;
#pragma unroll 1
    for (int q = 0; q < PER; ++q)
      if (lane == owner && q == at) key[q] = 0ull;
  }
  return mine;
}

// Rank of lane i's expert e among those of the lanes with `in`, by 64-bit keys (equal ones: the lower expert first).
__device__ __noinline__ int rank_exact(const float* __restrict__ logits, const float* __restrict__ bias, float m,
                                       const moe_gate_config& c, int e, bool in) {
  const double sum = exact_sum(c, logits, m);
  const u64 key = in ? exact_key(c.router == MOE_ROUTER_SOFTMAX, logits[e], bias ? bias[e] : 0.f, m, sum) : 0ull;
  int rank = 0;
#pragma unroll 1
  for (unsigned left = __ballot_sync(kFull, in); left; left &= left - 1) {
    const int i = __ffs(left) - 1;
    const u64 other = __shfl_sync(kFull, key, i);
    const int oe = __shfl_sync(kFull, e, i);
    rank += other > key || (other == key && oe < e);
  }
  return rank;
}

// The groups that stay (a bit each), from the experts that can be one of their group's two best: lane i's e where `in`.
__device__ __noinline__ unsigned groups_exact(const float* __restrict__ logits, const float* __restrict__ bias,
                                              float m, const moe_gate_config& c, int e, bool in) {
  const int lane = threadIdx.x & 31, S = c.E / c.n_groups;
  const double sum = exact_sum(c, logits, m);
  const u64 key = in ? exact_key(c.router == MOE_ROUTER_SOFTMAX, logits[e], bias ? bias[e] : 0.f, m, sum) : 0ull;
  const int mine = in ? e / S : -1;
  u64 score = 0ull;   // lane g: group g
#pragma unroll 1
  for (int g = 0; g < c.n_groups; ++g) {
    const u64 k = mine == g ? key : 0ull, first = lanes_max(k);
    u64 s = first;
    if (S > 1) {
      const int owner = __ffs(__ballot_sync(kFull, k == first)) - 1;
      s = order_of(of_order(first) + of_order(lanes_max(lane == owner ? 0ull : k)));
    }
    if (lane == g) score = s;
  }
  int rank = 0;
#pragma unroll 1
  for (int g = 0; g < c.n_groups; ++g) {
    const u64 other = __shfl_sync(kFull, score, g);
    rank += other > score || (other == score && g < lane);
  }
  return __ballot_sync(kFull, lane < c.n_groups && rank < c.topk_groups);
}

// A lane's PER consecutive values of a row, in 16-byte loads where rows are made of them.
template <int PER>
__device__ __forceinline__ void load_lane(const float* __restrict__ row, int E, float fill, float (&v)[PER]) {
  const int e0 = (threadIdx.x & 31) * PER;
  if (PER >= 4 && (E & 3) == 0 && ((uintptr_t)row & 15) == 0) {
#pragma unroll
    for (int q = 0; q + 3 < PER; q += 4) {
      float4 u = make_float4(fill, fill, fill, fill);
      if (e0 + q < E) u = *reinterpret_cast<const float4*>(row + e0 + q);
      v[q] = u.x;
      v[q + 1] = u.y;
      v[q + 2] = u.z;
      v[q + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < PER; ++q) v[q] = e0 + q < E ? row[e0 + q] : fill;
  }
}

// 2^x and 1/x, approximate (2 units in the last place), without the steps that keep subnormal values.
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Where a lane's experts lie among the groups (integer divisions, once a warp).
struct Place {
  int S;          // experts of a group
  int step;       // lanes of a group where its experts fill a power of two of lanes, else 1
  bool fills;
  int g, left;    // group of the lane's first expert, and experts until the next group
  int mine;       // group that the lane speaks for
  __device__ __forceinline__ Place(const moe_gate_config& c, int per) {
    const int lane = threadIdx.x & 31, e0 = lane * per;
    S = c.E / c.n_groups;
    const int L = S / per;
    fills = L * per == S && (L & (L - 1)) == 0;
    step = fills ? L : 1;
    g = e0 / S;
    left = (g + 1) * S - e0;
    mine = fills ? g : lane;
  }
};

// How far a key may be from the one computed in 64 bits, with u = 2^-24. A softmax's score is off by its exponential
// (4 u, and 2.23 u |x| for the rounded argument x) and a product, a sigmoid's by (1 - p) (4 u + 1.25 u |x|), an addition
// and a reciprocal (3 u): with 2 u for the bound's own use both are under 8 u + 2 u log2(largest / score) of
// themselves. (A sigmoid's largest score is 1; the denominator that all scores of a softmax share does not move their
// order.) Without a bias the key is the score: the bound is the key's own, so that small scores beside a large one are
// told apart. With one, scores of any size can stand behind a key: base is the bound of the row's largest score (32 u of
// it with the softmax's denominator), and an addition and its comparison cost u |key| each. A key plus its bound grows
// with the key, so only neighbours need to be compared, whatever lies below them (a mask of -1e9, say). Infinite keys
// come from an infinite bias, and the lowest value stands for experts that are masked: they have no error.
struct KeyBound {
  float base, rel, per_doubling, top;     // top: log2 of the largest score
  __device__ __forceinline__ float operator()(float k) const {
    const float a = fabsf(k), doublings = fmaxf(top - __log2f(fmaxf(a, FLT_MIN)), 0.f);
    return a < FLT_MAX ? fmaf(a, fmaf(per_doubling, doublings, rel), base) : 0.f;
  }
};
constexpr float kScoreBase = 0x1p-125f, kScoreRel = 0x1p-21f, kScoreDoubling = 0x1p-23f;   // (below 2^-126: taken for 0)

// The groups that stay, a bit each. Where their choice rests on scores (sums of two keys) whose bounds meet, by 64-bit
// keys of the experts that can be one of their group's two best; sure turns false if these are more than a warp holds.
// scr: 32 words.
template <int PER>
__device__ __forceinline__ unsigned kept_groups(const unsigned (&key)[PER], const moe_gate_config& c,
                                                const Place& at_, const KeyBound& bound,
                                                const float* __restrict__ logits, const float* __restrict__ bias,
                                                float m, unsigned* scr, bool& sure) {
  const int lane = threadIdx.x & 31, e0 = lane * PER, S = at_.S, L = at_.step;
  // Groups that fill a power of two of lanes: all at once, every lane with its own group's. Others: group by group,
  // lane g with group g's.
  const bool fills = at_.fills;
  float first = -FLT_MAX, second = -FLT_MAX;
  if (fills) {
    unsigned a = 0u, b = 0u;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      b = max(b, min(a, key[q]));
      a = max(a, key[q]);
    }
    for (int o = 1; o < L; o <<= 1) {
      const unsigned oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
      b = max(min(a, oa), max(b, ob));
      a = max(a, oa);
    }
    if (e0 < c.E) {
      first = of_order(a);
      second = of_order(S > 1 ? b : a);
    }
  } else {
    for (int g = 0; g < c.n_groups; ++g) {
      unsigned a = 0u, b = 0u;
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        if (e0 + q >= g * S && e0 + q < (g + 1) * S) {
          b = max(b, min(a, key[q]));
          a = max(a, key[q]);
        }
      }
      const unsigned best = __reduce_max_sync(kFull, a);
      unsigned other = best;
      if (S > 1) {
        const int owner = __ffs(__ballot_sync(kFull, a == best)) - 1;
        other = __reduce_max_sync(kFull, lane == owner ? b : a);
      }
      if (lane == g) {
        first = of_order(best);
        second = of_order(other);
      }
    }
  }
  // (sums past the finite range are pulled back to its end, and the bounds there reach over it)
  const float score = S > 1 && first <= FLT_MAX ? fminf(fmaxf(first + second, -FLT_MAX), FLT_MAX) : first;
  const float off2 = bound(second);
  const float off = S > 1 && first <= FLT_MAX ? bound(first) + off2 + 0x1p-22f * fabsf(score) : bound(first);
  // a masked expert's 64-bit key is far below the lowest value
  const float low = second == -FLT_MAX ? -INFINITY : score - off, high = score + off;
  const int step = at_.step, g = at_.mine;
  int rank = 0;
  for (int i = 0; i < c.n_groups; ++i) {
    const float other = __shfl_sync(kFull, score, i * step);
    rank += other > score || (other == score && i < g);
  }
  const bool in = g < c.n_groups, kept = in && rank < c.topk_groups;
  const float worst = -lanes_max(kept ? -low : -INFINITY), best = lanes_max(in && !kept ? high : -INFINITY);
  if (worst > best) {
    // bit g of a ballot of the lanes that speak for the groups
    const unsigned mask = __ballot_sync(kFull, kept && lane == g * step);
    if (step == 1) return mask;
    unsigned bits = 0u;
    for (int i = 0; i < c.n_groups; ++i) bits |= (mask >> (i * step) & 1u) << i;
    return bits;
  }
  int n = 0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int mine = min((e0 + q) / S, c.n_groups - 1);
    const float limit = __shfl_sync(kFull, second - 2 * off2, mine * step);
    const bool cand = key[q] && !(of_order(key[q]) < limit);
    const unsigned mask = __ballot_sync(kFull, cand);
    const int at = n + __popc(mask & ((1u << lane) - 1u));
    if (cand && at < 32) scr[at] = e0 + q;
    n += __popc(mask);
  }
  __syncwarp();
  if (n > 32) {
    sure = false;
    return 0u;
  }
  const int e = lane < n ? (int)scr[lane] : 0;
  __syncwarp();
  return groups_exact(logits, bias, m, c, e, lane < n);
}

// One token: lane j < k returns expert j of the selection and its gate. scr: 64 words of the warp's own.
template <int PER>
__device__ __forceinline__ int gate_token(const float* __restrict__ logits, const float* __restrict__ bias,
                                          const moe_gate_config& c, const Place& place, unsigned* scr, float& gate) {
  const int lane = threadIdx.x & 31, e0 = lane * PER;
  float l[PER], p[PER], b[PER];
  load_lane<PER>(logits, c.E, -INFINITY, l);
#pragma unroll
  for (int q = 0; q < PER; ++q) b[q] = 0.f;
  if (bias) load_lane<PER>(bias, c.E, 0.f, b);
  float m = -INFINITY, sum = 1.f, pmax = 1.f;
  if (c.router == MOE_ROUTER_SOFTMAX) {
#pragma unroll
    for (int q = 0; q < PER; ++q) m = fmaxf(m, l[q]);
    m = lanes_max(m);
    if (m == -INFINITY) m = 0.f;   // no expert left: every score 0
    sum = 0.f;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      p[q] = fast_exp(l[q] - m);
      sum += p[q];
    }
    sum = warp_sum(sum);
    pmax = sum == 0.f ? 0.f : fast_rcp(sum);
#pragma unroll
    for (int q = 0; q < PER; ++q) p[q] *= pmax;
  } else {
#pragma unroll
    for (int q = 0; q < PER; ++q) p[q] = fast_rcp(1.f + fast_exp(-l[q]));
  }
  unsigned key[PER];               // 0: no expert, or of a group that is left out
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const float k = p[q] + b[q];
    const bool on = l[q] > -INFINITY && k == k;      // neither masked nor NaN
    key[q] = order_of(on ? fmaxf(k, -FLT_MAX) : -FLT_MAX);
  }
  if (e0 + PER > c.E) {
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (e0 + q >= c.E) key[q] = 0u;
  }
  KeyBound bound = {kScoreBase, kScoreRel, kScoreDoubling, c.router == MOE_ROUTER_SOFTMAX ? __log2f(pmax) : 0.f};
  if (bias) {
    float large = pmax;
    if (c.router == MOE_ROUTER_SIGMOID) {
      large = 0.f;
#pragma unroll
      for (int q = 0; q < PER; ++q) large = fmaxf(large, p[q]);
      large = bound(__uint_as_float(__reduce_max_sync(kFull, __float_as_uint(large))));
    } else {
      large *= 0x1p-19f;
    }
    bound = {large, 0x1p-23f, 0.f, 0.f};
  }
  bool groups_sure = true;
  if (c.topk_groups < c.n_groups) {
    const unsigned keep = kept_groups<PER>(key, c, place, bound, logits, bias, m, scr, groups_sure);
    int g = place.g, left = place.left;
    if (place.fills) {
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (!(keep >> (g & 31) & 1u)) key[q] = 0u;
    } else
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      if (!(keep >> (g & 31) & 1u)) key[q] = 0u;
      if (--left == 0) {
        left = place.S;
        g = min(g + 1, 31);                      // (past the last expert the key is 0 already)
      }
    }
  }
  // The k + 1 largest different keys; lane j keeps the j-th. (Equal ones are told by the candidates' number below.)
  unsigned mine = 0u, last = kFull;
  for (int j = 0; j <= c.k; ++j) {
    unsigned top = 0u;
#pragma unroll
    for (int q = 0; q < PER; ++q) top = max(top, key[q] < last ? key[q] : 0u);
    last = __reduce_max_sync(kFull, top);
    if (lane == j) mine = last;
  }
  const float value = of_order(mine), off = bound(value);
  const unsigned next = __shfl_down_sync(kFull, mine, 1);
  const float below = __shfl_down_sync(kFull, value + off, 1);
  const bool near = lane < c.k && next && !(value - off > below);
  const bool sure = !__any_sync(kFull, near);
  const unsigned kth = __shfl_sync(kFull, mine, c.k - 1);   // 0: fewer than k different keys
  // Candidates: the selection, or where it is not sure every expert whose key may reach it (its own bound is at most
  // that of the larger kth, up to what the bounds have to spare). An infinite kth has no bound and stays what it is.
  unsigned least = kth;
  if (!sure && kth) least = order_of(__shfl_sync(kFull, value - 2 * off, c.k - 1));
  int n = 0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const bool in = key[q] && key[q] >= least;
    const unsigned mask = __ballot_sync(kFull, in);
    const int at = n + __popc(mask & ((1u << lane) - 1u));
    if (in && at < 32) {
      scr[at] = e0 + q;
      scr[32 + at] = key[q];
    }
    n += __popc(mask);
  }
  __syncwarp();
  int e;
  if (!groups_sure || n > 32 || n < c.k) {   // (never fewer than k; a lane below takes only an index that was written)
    e = select_exact<PER>(logits, bias, m, c);
  } else {
    e = lane < n ? (int)scr[lane] : 0;
    int rank = 0;
    if (sure && kth && n == c.k) {   // k different keys (equal ones, also where just k experts are left, go by index)
      const unsigned k1 = lane < n ? scr[32 + lane] : 0u;
      for (int i = 0; i < n; ++i) rank += scr[32 + i] > k1;
    } else {
      rank = rank_exact(logits, bias, m, c, e, lane < n);
    }
    __syncwarp();
    if (lane < n) scr[rank] = e;
    __syncwarp();
    e = lane < c.k ? (int)scr[lane] : 0;
  }
  __syncwarp();   // scr is free for the next token
  float ps = 0.f;
  if (lane < c.k) {
    const float x = logits[e];
    ps = c.router == MOE_ROUTER_SIGMOID ? 1.f / (1.f + expf(-x)) : sum == 0.f ? 0.f : expf(x - m) / sum;
  }
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
  int run[kMaxE], wcnt[kGateWarps][kMaxE], tmp[8];   // (wcnt also: each warp's scratch while it selects)
};

// Sorted positions of the assignments a0 .. a1, in passes of the block's threads; run[] holds each expert's first.
// first: the expert of assignment a0 + threadIdx.x (-1 behind a1), which the caller may have loaded long before.
__device__ __forceinline__ void rank_chunk(DispatchSmem& sm, const int* idx, int a0, int a1, int E, int first,
                                           int* __restrict__ perm, int* __restrict__ inv) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  for (int p0 = a0; p0 < a1; p0 += kGateThreads) {
    const int nw = min(kGateWarps, (a1 - p0 + 31) / 32);
    for (int i = tid; i < nw * kMaxE; i += kGateThreads) (&sm.wcnt[0][0])[i] = 0;
    __syncthreads();
    const int a = p0 + tid;
    const int e = p0 == a0 ? first : a < a1 ? idx[a] : -1;
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
  const Place place(c, PER);
  for (int t = t0 + w; t < t1; t += kGateWarps) {
    float g;
    const int e = gate_token<PER>(logits + (size_t)t * c.E, bias, c, place, reinterpret_cast<unsigned*>(sm.wcnt[w]), g);
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
  rank_chunk(sm, idx, 0, T * c.k, c.E, tid < T * c.k ? idx[tid] : -1, perm, inv);
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
  const int a0 = ch * tokens * k, a1 = min(T, (ch + 1) * tokens) * k;
  const int mine = a0 + tid < a1 ? idx[a0 + tid] : -1;
  // four threads an expert, each a quarter of the chunks
  const int e = tid & (kMaxE - 1), part = tid / kMaxE;
  int all = 0, before = 0;
  if (e < E) {
#pragma unroll 16
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
  rank_chunk(sm, idx, a0, a1, E, mine, perm, inv);
}

// One warp a token. With p the scores, ps those selected, D = sum ps + 1e-20, G = sum dgate ps / D:
//   dL/dps_j = scale (renorm ? (dgate_j - G) / D : dgate_j)
//   sigmoid: dl = p (1 - p) dp;   softmax: dl = p (dp - sum p dp)
// Of renormalised softmax gates sum p dp is scale G 1e-20 / D, which reaches every logit of the row: nothing beside
// sums of selected scores as they usually are, the whole gradient of the others where a bias or a group limit selects
// scores that small. It is left out below half a step of the magnitudes that cancel in the selected logits' gradients
// (2^-24 G), so that rows without it hold zeros. Exponentials are taken of the row's largest logit, as in the forward
// pass, so softmax reads the row either way (8,192 x 256 in 8.0 us and 2,048 x 64 in 2.8; the selected logits alone took
// 7.8 and 2.6).
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
  float row[PER];                 // of every expert; softmax: the row's exponentials first
#pragma unroll
  for (int q = 0; q < PER; ++q) row[q] = 0.f;
  if (c.router == MOE_ROUTER_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      row[q] = e0 + q < c.E ? logits[e0 + q] : -INFINITY;
      m = fmaxf(m, row[q]);
    }
    m = lanes_max(m);
    if (m == -INFINITY) m = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      row[q] = expf(row[q] - m);
      sum += row[q];
    }
    sum = warp_sum(sum);
    const float r = sum == 0.f ? 0.f : 1.f / sum, es = e >= 0 ? expf(l - m) : 0.f;
    float dot;                    // sum p dp
    if (c.renorm) {               // numerator and denominator times sum: no score that is far below 1 is lost
      const float added = 1e-20f * sum, kept = warp_sum(es), D = kept + added, gate = D == 0.f ? 0.f : es / D;
      const float G = warp_sum(gate * dg);
      dot = added < 0x1p-24f * kept || D == 0.f ? 0.f : G * (added / D);
      v = gate * (dg - G) - es * r * dot;
    } else {
      dot = warp_sum(es * r * dg);
      v = es * r * (dg - dot);
    }
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

inline int least_tokens(int T) {
  const int t = ceil_div(T, kFewChunks);
  return t < kChunkLeast ? kChunkLeast : t < kChunkTokens ? t : kChunkTokens;
}
inline int chunk_tokens(int T, int sms) {
  if (T <= kOneChunk) return T;
  const int least = least_tokens(T), t = ceil_div(T, sms);
  return t < least ? least : t;
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

// One count of every expert for each chunk; a single chunk needs none.
size_t gate_workspace(const moe_gate_config& c, int T) {
  return T <= kOneChunk ? 0 : sizeof(int) * (size_t)c.E * ceil_div(T, least_tokens(T));
}

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
