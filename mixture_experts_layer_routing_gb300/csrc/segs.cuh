// Segments (experts) of token rows given by device offsets, as every kernel of the 8-bit products sees them:
// rows off[g] .. off[g+1] of segment g, cut into tiles of `tile` rows.
#pragma once
#include "common.cuh"
#include "ops.h"

namespace moe {
namespace {

struct SegSmem {
  int off[kMaxSegs + 1];    // first row of each segment
  int tile[kMaxSegs + 1];   // tiles of the segments before it
  int tmp[8];
};

// All threads of a block of at least 256. off null: one segment of M rows. Offsets that are not ascending within
// 0 .. M are recorded as MOE_ERR_DEVICE_INDEX and every segment is taken as empty, so no access follows them.
__device__ __forceinline__ void load_segments(SegSmem& s, const int* __restrict__ off, int G, int M, int tile,
                                              int* status) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (!off) {
    if (tid == 0) {
      s.off[0] = s.tile[0] = 0;
      s.off[1] = M;
      s.tile[1] = (M + tile - 1) / tile;
    }
    __syncthreads();
    return;
  }
  int lo = 0, hi = 0;
  if (tid < G) {
    lo = off[tid];
    hi = off[tid + 1];
  }
  const bool bad = __syncthreads_or(lo < 0 || lo > hi || hi > M);
  if (bad) {
    if (tid == 0) set_error(status, MOE_ERR_DEVICE_INDEX);
    lo = hi = 0;
  }
  const int n = (hi - lo + tile - 1) / tile;
  int v = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (w < 8 && lane == 31) s.tmp[w] = v;
  __syncthreads();
  if (tid < G) {
    for (int i = 0; i < w; ++i) v += s.tmp[i];
    s.off[tid] = lo;
    s.tile[tid] = v - n;
    if (tid == G - 1) {
      s.off[G] = hi;
      s.tile[G] = v;
    }
  }
  __syncthreads();
}

// Segment of tile t (< s.tile[G]): the last one whose first tile is not behind t (empty ones before it share it).
__device__ __forceinline__ int segment_of(const SegSmem& s, int G, int t) {
  int lo = 0, hi = G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.tile[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace
}  // namespace moe
