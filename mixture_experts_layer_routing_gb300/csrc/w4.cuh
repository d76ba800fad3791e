// Few rows times 4-bit weights: what the kernels of w4.cu share.
//
// A warp takes 128 values of K (a chunk) of MT x 16 weight rows at a time and multiplies them with up to NT x 8 rows of
// x on the legacy MMA (m16n8k16, weights as its 16 rows, x's rows as its columns): at one to eight rows the product is
// bound by the weights' bytes, and an MMA issued by the warp that decoded its operand needs no hand-over through shared
// or tensor memory. Chunks go through a ring of the warp's own in shared memory, filled by cp.async of 16 bytes, so no
// warp waits for another one inside a product.
//
// Decoding. A word holds eight values, the even ones in its low half, so (word >> 4i) & 0x000f000f is a pair of
// neighbours; moved to the top of a bf16 mantissa under the exponent of 16 a code c reads 16 + c, and one packed
// subtraction of 16 + zero makes it c - zero, exactly. The order of K inside an MMA is free as long as both operands
// agree: lane t of a quad takes GROUP/4 consecutive values of each group, which are whole words of the weights and
// whole 16-byte units of x. The group's scale multiplies the fp32 sum of its MMAs.
#pragma once
#include "common.cuh"
#include "ops.h"

namespace moe {
namespace {

constexpr int kChunk = 128;      // values of K
constexpr int kW4Warps = 8;      // warps of a CTA

__device__ __forceinline__ void cp16(void* dst, const void* src, bool ok) {   // zeros where !ok
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  const int n = ok ? 16 : 0;
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp8(void* dst, const void* src, bool ok) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  const int n = ok ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The four pairs of a word's codes as bf16 values c - zero; off = 16 + zero in both halves.
__device__ __forceinline__ void decode8(uint32_t v, uint32_t off, uint32_t (&p)[4]) {
  p[0] = bf16x2_sub(((v << 3) & 0x00780078u) | 0x41804180u, off);
  p[1] = bf16x2_sub(((v >> 1) & 0x00780078u) | 0x41804180u, off);
  p[2] = bf16x2_sub(((v >> 5) & 0x00780078u) | 0x41804180u, off);
  p[3] = bf16x2_sub(((v >> 9) & 0x00780078u) | 0x41804180u, off);
}

// A matrix of 4-bit weights: codes [N, K/8], scale [KG, N], zero [KG, N].
struct W4 {
  const uint32_t* codes;
  const bf16* scale;
  const uint8_t* zero;
};
struct W4Shape {
  int N, K, KG;      // KG = ceil(K / GROUP)
};
// Matrix g of an array of them.
__device__ __forceinline__ W4 w4_matrix(const W4& w, const W4Shape& s, int g) {
  return {w.codes + (long long)g * s.N * (s.K / 8), w.scale + (long long)g * s.KG * s.N,
          w.zero ? w.zero + (long long)g * s.KG * s.N : nullptr};
}

// One chunk in shared memory. Rows of codes are 64 bytes, rows of x 256; their 16-byte units are permuted so that the
// reads of a quarter (16-byte), half (8-byte) or whole warp (4-byte) meet 32 banks.
template <int MT, int NT, int GROUP, bool ZERO> struct W4Stage {
  static constexpr int kGroups = kChunk / GROUP;
  uint4 a[MT * 16][4];
  uint4 b[NT * 8][16];
  uint4 scale[kGroups][MT * 2];                // 16 rows x bf16 a tile
  uint2 zero[ZERO ? kGroups : 1][MT * 2];
};

template <int MT, int NT, int GROUP, bool ZERO> struct W4Core {
  using Stage = W4Stage<MT, NT, GROUP, ZERO>;
  static constexpr int kGroups = kChunk / GROUP;
  static constexpr int W = GROUP / 32;         // words of a lane in a group
  static constexpr int kRows = NT * 8;

  // ---- copies
  const uint8_t* pa[MT];   // this lane's 16 bytes of row `quad` of each tile, at chunk 0
  unsigned a_ok;           // bit 2 mt + h: row quad + 8 h of tile mt is there
  const bf16* ps;          // this lane's 8 scales at chunk 0
  const uint8_t* pz;
  bool s_ok;
  const uint8_t* px;       // x
  unsigned xoff[NT * 4];   // this lane's rows of x in 16-byte units (~0: zeros)
  int xn;                  // pairs of rows to copy

  // Rows row0[mt] .. +16 of the matrix w, of which those below `end[mt]` are there.
  __device__ __forceinline__ void set_weights(const W4& w, const W4Shape& s, const int (&row0)[MT], const int (&end)[MT], int lane) {
    const int quad = lane >> 2, t = lane & 3;
    a_ok = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      pa[mt] = reinterpret_cast<const uint8_t*>(w.codes) + (long long)(row0[mt] + quad) * (s.K / 2) + t * 16;
      a_ok |= (unsigned)(row0[mt] + quad < end[mt]) << (2 * mt) | (unsigned)(row0[mt] + quad + 8 < end[mt]) << (2 * mt + 1);
    }
    const int gi = lane / (MT * 2), j = lane % (MT * 2);
    int r = row0[0], e = end[0];
    if (MT > 1 && j >= 2) r = row0[MT - 1], e = end[MT - 1];
    r += 8 * (j & 1);
    s_ok = lane < kGroups * MT * 2 && r < e;
    const long long at = (long long)gi * s.N + r;
    ps = w.scale + at;
    pz = w.zero + at;
  }
  __device__ __forceinline__ void copy_weights(Stage& st, const W4Shape& s, int c, int lane) const {
    const int quad = lane >> 2, t = lane & 3;
    const int u = W == 4 ? t : W == 2 ? t ^ (((quad >> 1) & 1) << 1) : t ^ ((quad >> 1) & 3);
    const bool k_ok = c * kChunk + t * 32 < s.K;
    const long long step = (long long)c * (kChunk / 2);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (k_ok && (a_ok >> (2 * mt) & 1)) cp16(&st.a[mt * 16 + quad][u], pa[mt] + step, true);
      if (k_ok && (a_ok >> (2 * mt + 1) & 1)) cp16(&st.a[mt * 16 + quad + 8][u], pa[mt] + step + (long long)8 * (s.K / 2), true);
    }
    if (lane < kGroups * MT * 2) {     // (zeros for groups past the end: a stale scale could be a NaN)
      const int gi = lane / (MT * 2), j = lane % (MT * 2);
      const bool ok = s_ok && c * kGroups + gi < s.KG;
      const long long at = (long long)c * kGroups * s.N;
      cp16(&st.scale[gi][j], ok ? (const void*)(ps + at) : px, ok);
      if (ZERO) cp8(&st.zero[gi][j], ok ? (const void*)(pz + at) : px, ok);
    }
  }
  __device__ __forceinline__ void copy_x(Stage& st, const W4Shape& s, int c, int lane) const {
    const int v = lane & 15, h = lane >> 4;
    // unit v of a row: group, word and lane that read it
    const int p = W == 4 ? (v & 3) * 4 + (v >> 2) : W == 2 ? (v & 8) | ((v & 1) * 4 + ((v & 7) >> 1)) : v;
    const bool k_ok = c * kChunk + v * 8 < s.K;
    const uint8_t* base = px + ((long long)c * 16 + v) * 16;
#pragma unroll
    for (int i = 0; i < NT * 4; ++i) {
      if (i >= xn) break;
      const int r = h + 2 * i;
      const bool ok = k_ok && xoff[i] != ~0u;
      cp16(&st.b[r][p ^ ((r & 1) * 4)], ok ? base + (long long)xoff[i] * 16 : px, ok);
    }
  }

  // ---- product of a chunk; tiles of x's rows from `nt` on are left out
  __device__ __forceinline__ static void multiply(const Stage& st, float (&acc)[MT][NT][4], int nt, int lane) {
    const int quad = lane >> 2, t = lane & 3;
#pragma unroll
    for (int gi = 0; gi < kGroups; ++gi) {
      uint32_t wa[MT][2][W];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4* row = st.a[mt * 16 + h * 8 + quad];
          if (W == 4) {
            const uint4 v = row[t];
            wa[mt][h][0] = v.x, wa[mt][h][1 % W] = v.y, wa[mt][h][2 % W] = v.z, wa[mt][h][3 % W] = v.w;
          } else if (W == 2) {
            const uint2 v = reinterpret_cast<const uint2*>(row + ((gi ^ ((quad >> 1) & 1)) << 1))[t];
            wa[mt][h][0] = v.x, wa[mt][h][1 % W] = v.y;
          } else {
            wa[mt][h][0] = reinterpret_cast<const uint32_t*>(row + (gi ^ ((quad >> 1) & 3)))[t];
          }
        }
      uint32_t off[MT][2];
      float s[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s[mt][h] = __bfloat162float(reinterpret_cast<const bf16*>(&st.scale[gi][mt * 2 + h])[quad]);
          off[mt][h] = ZERO ? (uint32_t)reinterpret_cast<const uint8_t*>(&st.zero[gi][mt * 2 + h])[quad] * 0x00080008u | 0x41804180u
                            : 0x41c041c0u;     // 24
        }
      float sum[MT][NT][4] = {};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t p[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          decode8(wa[mt][0][w], off[mt][0], p[mt][0]);
          decode8(wa[mt][1][w], off[mt][1], p[mt][1]);
        }
        const int u = W == 4 ? w * 4 + t : W == 2 ? gi * 8 + w * 4 + t : gi * 4 + t;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n >= nt) break;
          const uint4 x = st.b[n * 8 + quad][u ^ ((quad & 1) * 4)];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816(sum[mt][n], p[mt][0][0], p[mt][1][0], p[mt][0][1], p[mt][1][1], x.x, x.y);
            mma16816(sum[mt][n], p[mt][0][2], p[mt][1][2], p[mt][0][3], p[mt][1][3], x.z, x.w);
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[mt][n][0] = fmaf(s[mt][0], sum[mt][n][0], acc[mt][n][0]);
          acc[mt][n][1] = fmaf(s[mt][0], sum[mt][n][1], acc[mt][n][1]);
          acc[mt][n][2] = fmaf(s[mt][1], sum[mt][n][2], acc[mt][n][2]);
          acc[mt][n][3] = fmaf(s[mt][1], sum[mt][n][3], acc[mt][n][3]);
        }
    }
  }
};

}  // namespace
}  // namespace moe
