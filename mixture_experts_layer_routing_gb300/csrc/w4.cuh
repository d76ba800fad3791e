// Few rows times 4-bit weights: what the kernels of w4_matmul.cu and w4_layer.cu share.
//
// A warp takes 256 values of K (a chunk) of MT x 16 weight rows at a time and multiplies them with up to 8 rows of x on
// the legacy MMA (m16n8k16, weights as its 16 rows, x's rows as its columns): at so few rows tensor throughput is no
// limit (20% of this MMA's), and one issued by the warp that decoded its operand needs no hand-over through shared or
// tensor memory. Chunks go through a ring of the warp's own in shared memory, filled by cp.async of 16 bytes, so no warp
// waits for another one inside a product.
//
// What bounds it. The floor is the weights' bytes. Copies alone reach 83% of the copy rate (three stages of 4 KB for each
// of 14 or 15 warps; with x in the same ring and two stages it was 55%). The products alone take longer: decoding 32 x 256
// codes is 224 shifts and LOP3s on a pipe that issues one in two cycles and 128 subtractions, of some 640 instructions in
// all, at 16 warps of 128 registers on an SM. 32,768 x 7168 by one row in 29.0 us (17.8 at the copy rate), by eight in
// 37.7: 17% more instructions (x goes through shared memory for each 32 weight rows), and as x and the sums take room 12
// warps multiply instead of 15, each of which waits nearly four times as long for shared memory. Shifts as multiplications
// on the other pipe (mul.hi) were slower, and so were 24 warps of 80 registers, bulk prefetches of the next units to L2,
// and two barriers a unit instead of a warp that joins.
//
// Decoding. A word holds eight values, the even ones in its low half, so (word >> 4i) & 0x000f000f is a pair of
// neighbours; in the last bits of a bf16 mantissa under the exponent of 128 a code c reads 128 + c, and one packed
// subtraction of 128 + zero makes it c - zero, exactly. The order of K inside an MMA is free as long as both operands
// agree: lane t of a quad takes GROUP/4 consecutive values of each group, which are whole words of the weights and
// whole 16-byte units of x. The group's scale multiplies the fp32 sum of its MMAs.
#pragma once
#include <stddef.h>

#include "common.cuh"
#include "ops.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kChunk = 256;      // values of K
constexpr int kStages = 3;       // of a warp's ring
constexpr int kW4Warps = 16;     // warps of a CTA, at most: the last one joins the others' sums

// Copies of 16 bytes to shared memory where left > need: rows r, r + 4 and r + 8, r + 12 of 128 bytes.
__device__ __forceinline__ void cp16_four(uint32_t d, uint32_t e, const void* s0, const void* s1, const void* s2,
                                          const void* s3, int left, int need) {
  asm volatile("{.reg .pred p; setp.gt.s32 p, %6, %7;\n"
               "@p cp.async.cg.shared.global.L2::128B [%0], [%2], 16;\n"
               "@p cp.async.cg.shared.global.L2::128B [%1 + 512], [%3], 16;\n"
               "@p cp.async.cg.shared.global.L2::128B [%0 + 1024], [%4], 16;\n"
               "@p cp.async.cg.shared.global.L2::128B [%1 + 1536], [%5], 16;}"
               ::"r"(d), "r"(e), "l"(s0), "l"(s1), "l"(s2), "l"(s3), "r"(left), "r"(need) : "memory");
}
// `size` bytes, the rest becomes zeros
__device__ __forceinline__ void cp16_if(uint32_t dst, const void* src, int size, int left, int need) {
  asm volatile("{.reg .pred p; setp.gt.s32 p, %3, %4; @p cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;}"
               ::"r"(dst), "l"(src), "r"(size), "r"(left), "r"(need) : "memory");
}
__device__ __forceinline__ void cp8_if(uint32_t dst, const void* src, int size, int left, int need) {
  asm volatile("{.reg .pred p; setp.gt.s32 p, %3, %4; @p cp.async.ca.shared.global [%0], [%1], 8, %2;}"
               ::"r"(dst), "l"(src), "r"(size), "r"(left), "r"(need) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with sums that start at zero
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A constant that stays in a register.
__device__ __forceinline__ uint32_t held(uint32_t v) {
  uint32_t r;
  asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// (v & 0x000f000f) | magic in one operation (of C's two operators the compiler made two: 176 instead of 112 for the
// words of 32 rows x 128 values, on the pipe that bounds these kernels).
__device__ __forceinline__ uint32_t pair_of(uint32_t v, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(r) : "r"(v), "r"(magic));
  return r;
}
// The four pairs of a word's codes as bf16 values c - zero; off = 128 + zero in both halves, magic = 128 in both.
__device__ __forceinline__ void decode8(uint32_t v, uint32_t off, uint32_t magic, uint32_t (&p)[4]) {
  p[0] = bf16x2_sub(pair_of(v, magic), off);
  p[1] = bf16x2_sub(pair_of(v >> 4, magic), off);
  p[2] = bf16x2_sub(pair_of(v >> 8, magic), off);
  p[3] = bf16x2_sub(pair_of(v >> 12, magic), off);
}

// A value that is the same in all lanes, told to the compiler: what depends on it runs in the uniform pipe, and branches
// on it need no reconvergence.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

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

// One chunk in shared memory. Rows of codes are 128 bytes, copied as whole lines; their 16-byte units are permuted so
// that the reads of a quarter (16-byte), half (8-byte) or whole warp (4-byte) meet 32 banks.
template <int MT, int GROUP, bool ZERO> struct alignas(128) W4Stage {
  static constexpr int kGroups = kChunk / GROUP;
  uint4 a[MT * 16][8];
  uint4 scale[kGroups][MT * 2];                // 16 rows x bf16 a tile
  uint2 zero[ZERO ? kGroups : 0][MT * 2];
};

// A warp's ring of chunks, its copies and its products with up to XR (2, 4 or 8) rows of x. Weights are copied two chunks
// ahead; a chunk of x is read one chunk ahead into registers, 16 bytes of each row a lane, and goes through shared memory.
template <int MT, int XR, int GROUP, bool ZERO> struct W4Core {
  using Stage = W4Stage<MT, GROUP, ZERO>;
  static constexpr int kPitch = MT * 16 + 4;
  static constexpr int kGroups = kChunk / GROUP;
  static constexpr int W = GROUP / 32;         // words of a lane in a group
  static constexpr unsigned kStage = sizeof(Stage), kX = kStages * kStage, kBytes = kX + XR * 512;    // of shared memory
  static constexpr unsigned kLast = (kStages - 1) * kStage;

  uint8_t* ring;           // this warp's, in shared memory
  uint32_t da, ds;         // addresses that this lane copies to, of the first stage
  unsigned ra, rs;         // offsets in a stage that it reads from
  uint32_t magic, eight;   // 128 and 136 as pairs of bf16
  unsigned slot;           // offset of the stage that is read next; the one before it is free
  // the next chunk to copy
  const uint8_t* pa[MT];  // this lane's 16 bytes of row lane / 8 of each tile
  unsigned long long row4, row8[MT];   // to the rows 4 and (where they are there) 8 further on
  const uint8_t* ps;       // its 8 scales
  const uint8_t* pz;
  int k_left, g_left;      // values and groups from the chunk on
  int every;               // chunks from one to the next
  // x
  uint4 x[XR];             // the next chunk
  int rows;                // of x that hold it
  unsigned xoff[XR];       // its rows, in units of 16 bytes
  unsigned wx, rx;         // offsets that this lane writes to and reads from

  __device__ __forceinline__ void init(uint8_t* ring_, int every_, int lane) {
    ring = ring_;
    every = every_;
    magic = held(0x43004300u);
    eight = held(0x43084308u);
    const int quad = lane >> 2, t = lane & 3;
    Stage& st = *reinterpret_cast<Stage*>(ring);
    // unit u of row r: u ^ 4 (r & 1), u ^ 2 (r & 3) or u ^ (r & 7); four rows a copy
    const int r = lane >> 3, u = lane & 7;
    da = smem_u32(&st.a[r][W == 4 ? u ^ (r & 1) * 4 : W == 2 ? u ^ (r & 3) * 2 : u ^ (r & 7)]);
    ds = smem_u32(&st.scale[0][0]) + lane * 16;
    ra = quad * 128 + (W == 4 ? (quad & 1) * 64 + t * 16 : W == 2 ? (quad & 3) * 32 + t * 8 : (quad & 7) * 16 + t * 4);
    rs = (unsigned)offsetof(Stage, scale) + quad * 2;
    // halves of x's rows [half][row][16 units]: unit v by the group, word and lane that read it; odd rows four further
    const int v = lane & 15, p = W == 4 ? (v & 3) * 4 + (v >> 2) : W == 2 ? (v & 8) | ((v & 1) * 4 + ((v & 7) >> 1)) : v;
    wx = kX + (lane >> 4) * (XR * 256) + p * 16;
    rx = kX + (quad & (XR - 1)) * 256 + (quad & 1) * 64 + t * 16;      // (columns from XR on repeat others, unused)
    slot = 0;
    // No register of this state is without a value. Without the zeros in x the layer's fp32 form gave wrong sums wherever a
    // warp's first tile has fewer rows than a later one, also with the rows' count carried beside them, while starting
    // values of 1 and of NaN give the right ones: no result reads them, but code made for undefined registers was wrong.
    rows = k_left = g_left = 0;
    row4 = 0ull;
    ps = pz = nullptr;
#pragma unroll
    for (int i = 0; i < MT; ++i) pa[i] = nullptr, row8[i] = 0ull;
#pragma unroll
    for (int i = 0; i < XR; ++i) x[i] = make_uint4(0u, 0u, 0u, 0u), xoff[i] = 0u;
  }
  // From chunk c on of rows row0[i] .. +8 and up0[i] .. +8 (i = 0 .. MT) of the matrix w, as far as they are below `end`
  // (a multiple of 8, above row0[0]); others repeat some and get scales of zero.
  __device__ __forceinline__ void aim(const W4& w, const W4Shape& s, const int (&row0)[MT], const int (&up0)[MT], int end,
                                      int c, int lane) {
    const unsigned pitch = s.K / 2;
    row4 = 4 * (unsigned long long)pitch;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = row0[mt] < end ? row0[mt] : row0[0];
      pa[mt] = reinterpret_cast<const uint8_t*>(w.codes) + (unsigned long long)(unsigned)(r + (lane >> 3)) * pitch + (unsigned)(c * (kChunk / 2) + (lane & 7) * 16);
      row8[mt] = up0[mt] < end ? (unsigned long long)(unsigned)(up0[mt] - r) * pitch : 0ull;
    }
    const int gi = lane / (MT * 2), j = lane % (MT * 2), mt = j / 2;
    int r = j & 1 ? up0[0] : row0[0];
#pragma unroll
    for (int i = 1; i < MT; ++i)
      if (mt == i) r = j & 1 ? up0[i] : row0[i];
    const bool there = r < end;
    const unsigned long long at = (unsigned long long)(unsigned)(c * kGroups + gi) * (unsigned)s.N + (unsigned)(there ? r : 0);
    ps = reinterpret_cast<const uint8_t*>(w.scale + at);
    if (ZERO) pz = w.zero + at;
    k_left = s.K - c * kChunk;
    g_left = there ? s.KG - c * kGroups - gi : 0;
  }
  // `rows` rows further on, all of them below the end, and n chunks back.
  __device__ __forceinline__ void step(const W4Shape& s, int rows, int n) {
    const long long by = (long long)((unsigned long long)(unsigned)rows * (unsigned)(s.K / 2)) - (long long)n * (kChunk / 2);
    const long long back = (long long)((unsigned long long)(unsigned)s.N * (unsigned)(n * kGroups));
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) pa[mt] += by;
    ps += 2 * (rows - back);
    if (ZERO) pz += rows - back;
    k_left += n * kChunk;
    g_left += n * kGroups;
  }
  // Copies the next chunk to the stage at offset `at` (codes past the end of K stay what they were: x is zero there, and
  // any code is finite. A stale scale might not be: zeros).
  __device__ __forceinline__ void copy(const W4Shape& s, unsigned at, int lane) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint8_t* up = pa[mt] + row8[mt];
      const uint32_t d = da + at + mt * 2048;      // (rows r and r + 4 are permuted alike but for W = 1)
      cp16_four(d, W == 1 ? d ^ 64 : d, pa[mt], pa[mt] + row4, up, up + row4, k_left, (lane & 7) * 32);
      pa[mt] += every * (kChunk / 2);
    }
    // (no address is followed for zeros)
    cp16_if(ds + at, ps, g_left > 0 ? 16 : 0, kGroups * MT * 2, lane);
    ps += (unsigned long long)(unsigned)s.N * (unsigned)(every * kGroups * 2);
    if (ZERO) {
      cp8_if(ds + at + kGroups * MT * 32 - lane * 8, pz, g_left > 0 ? 8 : 0, kGroups * MT * 2, lane);
      pz += (unsigned long long)(unsigned)s.N * (unsigned)(every * kGroups);
    }
    g_left -= every * kGroups;
    k_left -= every * kChunk;
  }
  // Reads chunk c of the first n rows of x (zeros past the end of K, and for the rows whose bit in `there` is not set).
  __device__ __forceinline__ void read_x(const bf16* x0, int c, int K, int n, unsigned there, int lane) {
    const int k = c * kChunk + lane * 8;
    const uint8_t* p = reinterpret_cast<const uint8_t*>(x0 + k);
    const unsigned in = k < K ? there : 0u;
    rows = n;
#pragma unroll
    for (int r = 0; r < XR; ++r) {
      if (r > 0 && r >= n) break;
      x[r] = make_uint4(0u, 0u, 0u, 0u);
      asm volatile("{.reg .pred p; setp.ne.b32 p, %5, 0; @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];}"
                   : "+r"(x[r].x), "+r"(x[r].y), "+r"(x[r].z), "+r"(x[r].w)
                   : "l"(p + (unsigned long long)xoff[r] * 16), "r"(in >> r & 1) : "memory");
    }
  }
  // and puts them where multiply() reads them; a __syncwarp before and after
  __device__ __forceinline__ void store_x() const {
#pragma unroll
    for (int r = 0; r < XR; ++r) {
      if (r > 0 && r >= rows) break;
      *reinterpret_cast<uint4*>(ring + (wx ^ (r & 1) * 64) + r * 256) = x[r];
    }
  }
  __device__ __forceinline__ unsigned free_slot() const { return slot == 0 ? kLast : slot - kStage; }
  __device__ __forceinline__ void next() { slot = slot == kLast ? 0 : slot + kStage; }

  // The product of the chunk in `slot`; k: values of it.
  __device__ __forceinline__ void multiply(float (&acc)[MT][4], int k, int lane) const {
    product<0>(acc, lane);
    if (k > kChunk / 2) product<1>(acc, lane);
  }
  template <int HALF> __device__ __forceinline__ void product(float (&acc)[MT][4], int lane) const {
    // unit j of a lane's half row of x is at 64 (j ^ (quad & 1)): even and odd ones from two addresses
    const uint8_t* sx[2] = {ring + rx, ring + (rx ^ 64)};
    const uint8_t *base = ring + slot, *ss = base + rs;
#pragma unroll
    for (int g = 0; g < kGroups / 2; ++g) {
      const int gi = HALF * (kGroups / 2) + g;
      const uint8_t* sa = base + (ra ^ (W == 4 ? gi * 64 : W == 2 ? gi * 32 : gi * 16));
      uint32_t wa[MT][2][W];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = (mt * 16 + h * 8) * 128;
          if (W == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(sa + r);
            wa[mt][h][0] = v.x, wa[mt][h][1 % W] = v.y, wa[mt][h][2 % W] = v.z, wa[mt][h][3 % W] = v.w;
          } else if (W == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(sa + r);
            wa[mt][h][0] = v.x, wa[mt][h][1 % W] = v.y;
          } else {
            wa[mt][h][0] = *reinterpret_cast<const uint32_t*>(sa + r);
          }
        }
      uint32_t off[MT][2];
      float s[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = gi * MT * 2 + mt * 2 + h;
          s[mt][h] = __bfloat162float(*reinterpret_cast<const bf16*>(ss + i * 16));
          off[mt][h] = ZERO ? (uint32_t)base[offsetof(Stage, zero) + i * 8 + (lane >> 2)] * 0x00010001u + magic : eight;
        }
      float sum[MT][4];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t p[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          decode8(wa[mt][0][w], off[mt][0], magic, p[mt][0]);
          decode8(wa[mt][1][w], off[mt][1], magic, p[mt][1]);
        }
        const int j = g * W + w;
        const uint4 x = *reinterpret_cast<const uint4*>(sx[j & 1] + (j >> 1) * 128 + HALF * (XR * 256));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (w == 0) mma16816_first(sum[mt], p[mt][0][0], p[mt][1][0], p[mt][0][1], p[mt][1][1], x.x, x.y);
          else mma16816(sum[mt], p[mt][0][0], p[mt][1][0], p[mt][0][1], p[mt][1][1], x.x, x.y);
          mma16816(sum[mt], p[mt][0][2], p[mt][1][2], p[mt][0][3], p[mt][1][3], x.z, x.w);
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        acc[mt][0] = fmaf(s[mt][0], sum[mt][0], acc[mt][0]);
        acc[mt][1] = fmaf(s[mt][0], sum[mt][1], acc[mt][1]);
        acc[mt][2] = fmaf(s[mt][1], sum[mt][2], acc[mt][2]);
        acc[mt][3] = fmaf(s[mt][1], sum[mt][3], acc[mt][3]);
      }
    }
  }
  // A unit's sums of the first R rows of x, [row of x][MT x 16 rows, 4 apart in the banks].
  __device__ __forceinline__ static void put(const float (&acc)[MT][4], float* dst, int R, int lane) {
    const int quad = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * t + i;
      if (r < R) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          dst[r * kPitch + mt * 16 + quad] = acc[mt][i];
          dst[r * kPitch + mt * 16 + quad + 8] = acc[mt][i + 2];
        }
      }
    }
  }
};

// A warp's place in a CTA's units: unit u is block m of tile `tile`, and the warp's next chunk of it is c.
struct W4Cursor {
  int u, tile, m, c;
  __device__ __forceinline__ W4Cursor(int u_, int tile_, int m_, int warp, int C, int blocks) : u(u_), tile(tile_), m(m_), c(warp) {
    next(0, C, blocks);
  }
  // every `by`-th chunk is the warp's; returns the units that were passed
  __device__ __forceinline__ int next(int by, int C, int blocks) {
    int n = 0;
    for (c += by; c >= C; c -= C, ++n) {
      ++u;
      if (++m == blocks) m = 0, ++tile;
    }
    return n;
  }
};
constexpr int kSumBuffers = 2;       // of a warp

// One CTA on an SM: the warps that multiply and, one more, the warp that joins; as many as its shared memory holds with
// `fixed` bytes of the CTA's own. (Two CTAs of 8 warps each took 34.7 us for 32,768 x 7168 and one row where one of 16 took
// 30.3, before the other steps: half as many ranges of units, so the longest is nearer to the average.)
constexpr size_t w4_smem(size_t fixed) { return 227 * 1024 - 1024 - fixed; }
constexpr int w4_warps(size_t fixed, size_t per_warp) {
  const size_t n = w4_smem(fixed) / per_warp;
  return n < kW4Warps - 1 ? (int)n : kW4Warps - 1;
}

// Sums of N units between the warps of a product and the warp that joins them, so that no product waits for another
// warp's or for the join.
template <int N> struct W4Handover {
  uint64_t full[N], empty[N];
  int abort;
  __device__ __forceinline__ void init(int warps) {      // one thread, before a barrier of the CTA
    for (int b = 0; b < N; ++b) {
      mbar_init(smem_u32(&full[b]), warps);
      mbar_init(smem_u32(&empty[b]), 1);
    }
    abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // unit i of the CTA: its buffer (i % N) is free / holds every warp's sums
  __device__ __forceinline__ void wait_empty(int i, int* status) {
    if (i >= N) mbar_wait(smem_u32(&empty[i % N]), (i / N - 1) & 1, &abort, status);
  }
  __device__ __forceinline__ void wait_full(int i, int* status) {
    mbar_wait(smem_u32(&full[i % N]), (i / N) & 1, &abort, status);
  }
  __device__ __forceinline__ void put(int i, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&full[i % N]));
  }
  __device__ __forceinline__ void taken(int i, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&empty[i % N]));
  }
};

}  // namespace
}  // namespace moe
