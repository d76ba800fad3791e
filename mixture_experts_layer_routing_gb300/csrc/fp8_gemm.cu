// Products of e4m3 operands with a scale for each 128 values (include/moe_ops.h) on tcgen05.mma kind::f8f6f4.
//
// The scales change every 128 values of the reduction, so a product of 128 is finished in TMEM by itself (four
// MMAs of K = 32 into one of several partial accumulators), read back, and added with its scales to sums that live
// in registers: c += (sa sb) * partial, in fp32. Two kernels:
//
// wide: many rows. 128 rows x 256 columns a CTA, one CTA a SM, persistent, two CTAs on one tile of 256 rows where
//   segments are long. TMEM holds two partials of 256 columns (all 512), so that the tensor core works on one while
//   eight epilogue warps (128 sums a thread) take in the other. Per K block the MMAs take 512 cycles, the 32,768 FMAs
//   of the sums 256 and the partial's way out of TMEM about as long as the MMAs.
// narrow: few rows a segment (decoding). The operands change places: 128 weight rows are the MMA's M and 16 to 64
//   token rows its N, so that the MMA's M is filled by weights and a weight byte is read once. The reduction is
//   split over the CTAs of a cluster where tiles alone would not fill the GPU; the parts are added through
//   distributed shared memory in rank order. Bound by the weights' bytes.
//
// Operands come by TMA (128-byte swizzle); gathered rows (row_index) by TMA gathers of four rows in the narrow kernel,
// and put in order by a kernel of their own before the wide one, which reads a row once a column tile. Every wait is
// bounded: a role that gives up sets the abort flag and the others leave their loops too.
#include "common.cuh"
#include "launch.cuh"
#include "segs.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int BK = 128;                      // bytes (values) of the reduction a stage holds: one scale block

// kind::f8f6f4: e4m3 A and B (both K-major), fp32 accumulator, M x N.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
template <int CG>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (CG == 1)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrival, in every CTA of the group, once this thread's MMAs so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if (CG == 1) mma_commit(bar);
  else mma_commit_pair_mc(bar, 0x3);
}
// Four rows r0 .. r3 of the map's matrix, 128 bytes from column c each (rows past the matrix: zeros).
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* tm, int c, int r0, int r1, int r2, int r3,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
      "%5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
template <int CG, int COLS> __device__ __forceinline__ void tmem_alloc(uint32_t slot) {
  if (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG, int COLS> __device__ __forceinline__ void tmem_free(uint32_t base) {
  if (CG == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(COLS) : "memory");
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(COLS) : "memory");
}
// Bounded wait that does not look at the abort flag: for what a role itself has in flight when it leaves.
__device__ __forceinline__ void wait_own(uint32_t bar, uint32_t parity, int* status) {
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_ns() - t0 > kWaitLimitNs) {
      set_error(status, MOE_ERR_TIMEOUT);
      break;
    }
  }
}

// As mbar_wait, without a call: inside the epilogue's loop a call would have to save its 128 sums.
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0) {
      if (*abort_flag) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        set_error(status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}
// A whole warp's wait. Every lane tests: one lane's test and a broadcast of its result measured slower, through the
// warp's divergence (a product of 8192 x 4096 x 7168 in 222 us instead of 139, its epilogue taken out).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return __all_sync(0xffffffffu, wait_inline(bar, parity, abort_flag, status));
}
// A single thread's wait by tests that do not suspend it (mbarrier.test_wait): it goes on sooner.
__device__ __forceinline__ bool spin_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 0xfff) == 0) {
      if (*abort_flag) return false;
      if (t0 == 0) t0 = global_ns();
      if (global_ns() - t0 > kWaitLimitNs) {
        set_error(status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}
// Arrival on a barrier that may be the other CTA's. What it hands over is tensor memory that was read (ordered by
// tcgen05.fence), so it needs no release of ordinary memory to the cluster, which costs over 1,000 cycles here.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// n / d for n < 2^31 by a multiplication (Granlund and Montgomery, PLDI 1994). A unit's place takes several divisions,
// which cost a warp some 500 cycles as divisions.
struct FastDiv {
  unsigned d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(unsigned by) : d(by), mul(0), shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = (unsigned)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ unsigned div(unsigned n) const { return (__umulhi(n, mul) + n) >> shift; }
};

struct GemmParams {
  const float* sa;        // scales of the rows: [a_rows][nkb], or (wgrad) [K blocks][M]
  const float* sb;        // of the columns: [G][ceil(N / 128)][nkb], or (wgrad) [K blocks][N]
  const int* row_index;
  const int* off;
  int G;
  int rows;               // rows of all segments (off's bound): M, or (wgrad) tokens
  int a_rows;             // rows of a (gathered from)
  int M;                  // wgrad: rows of c
  int N;
  int nkb;                // K blocks (wgrad: from the segment)
  int vec;                // widest aligned store to c: 32 or 16 bytes, or 0
  FastDiv nt, mnt, rnt;   // wide: column tiles; (wgrad) tiles of a segment; tiles of a group of kRasterM row tiles
  FastDiv last;           // (wgrad) row tiles of a segment's last such group
  void* c;
  int* status;
};

// Row of a that row m of c reads; past the segment, or with an index out of range, the first row behind a (zeros).
__device__ __forceinline__ int gather_row(const GemmParams& p, int m, int row_end) {
  const int r = m < row_end ? p.row_index[m] : p.a_rows;
  return (unsigned)r < (unsigned)p.a_rows ? r : p.a_rows;
}

// Pairs of fp32 values, for the two-wide multiply-add.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ void fma2(uint64_t& c, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Waits for this thread's TMEM loads; u is used after it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&u)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7]),
                 "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15])
               :
               : "memory");
}
// Scales of 16 columns as pairs: the row's s, times the columns' own v where they differ.
template <bool COLS>
__device__ __forceinline__ void pair_scales(uint64_t (&w)[8], float s, const float* v) {
  const uint64_t s2 = pair(s, s);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    w[i] = w[i + 1] = s2;
    if (COLS) {
      const float4 f = *reinterpret_cast<const float4*>(v + 2 * i);
      w[i] = mul2(s2, pair(f.x, f.y));
      w[i + 1] = mul2(s2, pair(f.z, f.w));
    }
  }
}

// The first `left` of 16 neighbouring values of a row of c, in the widest stores its alignment allows (32 bytes: a
// whole sector, so that no sector is written in two parts).
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
template <typename O>
__device__ __forceinline__ void store16(O* p, const float (&f)[16], int left, int vec) {
  constexpr bool F32 = sizeof(O) == 4;
  if (vec == 32) {            // rows are made of 32-byte pieces
    uint32_t w[8];
    if (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
      store32(p, w);
      if (left > 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[8 + i]);
        store32(p + 8, w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack2(f[2 * i], f[2 * i + 1]);
      store32(p, w);
    }
  } else if (vec == 16) {
#pragma unroll
    for (int i = 0; i < 16; i += F32 ? 4 : 8) {
      if (i < left) {
        uint4 w;
        if (F32) w = make_uint4(__float_as_uint(f[i]), __float_as_uint(f[i + 1]), __float_as_uint(f[i + 2]), __float_as_uint(f[i + 3]));
        else w = pack8(f + (i & 8));
        *reinterpret_cast<uint4*>(p + i) = w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) p[i] = from_f<O>(f[i]);
  }
}

// ------------------------------------------------------------------- wide
constexpr int WM = 128, WN = 256, WC = 128;            // rows a CTA, columns a tile, columns (sums) a thread
constexpr int kWBufs = 512 / WN;                       // partials in TMEM, and warps that issue MMAs
constexpr int kWEpi = 4 * WN / WC;                     // epilogue warps: four lane quadrants x column halves
constexpr int kWThreads = (4 + kWEpi) * 32;            // producer, MMA warps, scales, epilogue
constexpr int kWChunk = 8;                             // K blocks whose scales are fetched at a time
// CG CTAs work on one tile of CG x 128 rows; each holds its own rows and 1 / CG of the columns' operand.
template <int CG> constexpr int w_stage_bytes() { return (WM + WN / CG) * BK; }
template <int CG> constexpr int w_stages() { return 4; }
struct alignas(128) WideSmem {
  // Scales of the K blocks: of this CTA's rows, and of the columns. wgrad's come by TMA with the operands (slot it mod
  // 8, a scale for each column), the others by a warp of their own, in two chunks of 8 K blocks (a scale for each
  // half of the columns: sbh).
  float sa[2 * kWChunk][WM], sb[kWChunk][WN], sbh[2 * kWChunk][2];
  SegSmem seg;
  uint64_t full[6], empty[6], pfull[kWBufs], pempty[kWBufs], sfull[2], sempty[2], drain;
  uint32_t tmem;
  int abort;
};
// Output staging of a pair's CTA: each epilogue warp writes 32 rows x 128 bytes at a time (128-byte swizzle) and sends
// them by TMA. Rows stored directly, a row a lane, took 32 wavefronts an instruction and bound the weight gradients
// (89% of L1's throughput); single CTAs have no room for it.
constexpr int kWOutBufs = 2, kWOutBytes = 32 * 128;
template <int CG> constexpr int w_out_bytes() { return CG == 1 ? 0 : kWEpi * kWOutBufs * kWOutBytes; }
template <int CG> constexpr int w_smem() {
  return w_stages<CG>() * w_stage_bytes<CG>() + w_out_bytes<CG>() + 1024 + (int)sizeof(WideSmem);
}
// Registers: 384 threads are launched with 168 each, of which the epilogue's 256 take more and the other 128 give up
// some: the split at which neither side spills (a spill of eight registers in the loop cost 20% of the time).
constexpr int kWRegs = 168;
template <int CG> constexpr int w_regs_epi() { return 208; }
template <int CG> constexpr int w_regs_rest() { return 88; }
template <int CG> constexpr bool w_regs_fit() {
  return kWEpi * 32 * w_regs_epi<CG>() + 128 * w_regs_rest<CG>() <= kWThreads * kWRegs;
}
static_assert(w_regs_fit<1>() && w_regs_fit<2>(), "register split");

struct WTile {
  int g, row0, row_end, n0, kb0, nkb;
};

// Unit L of the schedule: row tiles in groups of 16, all column tiles of a group before the next (L2 reuse).
// row0: this CTA's rows.
template <int CG, bool WGRAD>
__device__ __forceinline__ WTile wide_tile(const GemmParams& p, const SegSmem& s, int L, int rank) {
  constexpr int TM = CG * WM;
  WTile t;
  int mt, local;
  if (WGRAD) {
    t.g = p.mnt.div(L);
    local = L - t.g * p.mnt.d;
    mt = (p.M + TM - 1) / TM;
  } else {
    int lo = 0, hi = p.G;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.tile[mid] * (int)p.nt.d <= L) lo = mid; else hi = mid;
    }
    t.g = lo;
    mt = s.tile[lo + 1] - s.tile[lo];
    local = L - s.tile[lo] * p.nt.d;
  }
  const int grp = p.rnt.div(local), within = local - grp * p.rnt.d, gm = mt - grp * kRasterM;
  const int n = gm >= kRasterM ? within / kRasterM : WGRAD ? (int)p.last.div(within) : within / gm;
  const int m = grp * kRasterM + within - n * min(gm, kRasterM);
  t.n0 = n * WN;
  if (WGRAD) {
    t.row0 = m * TM + rank * WM;
    t.row_end = p.M;
    t.kb0 = s.tile[t.g];
    t.nkb = s.tile[t.g + 1] - t.kb0;
  } else {
    t.row0 = s.off[t.g] + m * TM + rank * WM;
    t.row_end = s.off[t.g + 1];
    t.kb0 = 0;
    t.nkb = p.nkb;
  }
  return t;
}
template <int CG, bool WGRAD>
__device__ __forceinline__ int wide_units(const GemmParams& p, const SegSmem& s) {
  const int nt = (p.N + WN - 1) / WN;
  return (WGRAD ? p.G * ((p.M + CG * WM - 1) / (CG * WM)) : s.tile[p.G]) * nt;
}

// K block `it` of this CTA's run is stage it mod the ring and partial it mod 2. A warp of its own issues each
// partial's MMAs: the tensor pipe holds little more than one MMA of queued work, and a single thread that tests
// barriers between its MMAs leaves it idle for the tests (about 100 cycles each; 225 us became 210 with the second
// warp). A partial's uses have to come from one warp: barriers tell phases by parity, and a warp ahead of another
// would take an older release of the same partial for its own.
// Measured, 8192 x 4096 x 7168: 196 us (2.45 PFLOP/s) at 1.82 GHz under the power limit; 167 with the epilogue's
// loads and sums left out, 140 without the operands' copies either. Single CTAs instead of pairs: 220 us (48 KB of
// operands a K block of 512 MMA cycles is more than the 56 bytes a cycle that come from L2 into an SM, and shared
// memory's 128 bytes a cycle carry the copies and the MMAs' reads). Four partials of 128 columns: 198 us (twice the
// MMAs to issue). Sixteen epilogue warps of 64 columns: 216 us.
template <int CG, bool WGRAD, typename O>
__global__ void __launch_bounds__(kWThreads, 1)
    fp8_wide_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ CUtensorMap tmC, GemmParams p) {
  constexpr int ST = w_stages<CG>(), SB = w_stage_bytes<CG>();
  // wgrad's slots: the copies of K block i follow the MMAs of i - ST, which follow the epilogue's release of
  // i - ST - 2, so they cannot meet the reading of i - 8.
  static_assert(ST + 3 <= kWChunk, "scale slots");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* staging = ring + ST * SB;
  WideSmem& sm = *reinterpret_cast<WideSmem*>(staging + w_out_bytes<CG>());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)cluster_ctarank() : 0;
  volatile int* abort_flag = &sm.abort;
  const uint32_t full0 = smem_u32(sm.full), empty0 = smem_u32(sm.empty), pfull0 = smem_u32(sm.pfull),
                 pempty0 = smem_u32(sm.pempty), sfull0 = smem_u32(sm.sfull), sempty0 = smem_u32(sm.sempty),
                 drain = smem_u32(&sm.drain);
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < kWBufs; ++i) {
      mbar_init(pfull0 + 8 * i, 1);
      mbar_init(pempty0 + 8 * i, kWEpi * CG);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(sm.sfull + i), 32);
      mbar_init(smem_u32(sm.sempty + i), kWEpi);
    }
    mbar_init(drain, kWBufs);
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();     // before the allocation: no CTA holds TMEM while the predecessor may still want some
  griddep_launch();
  if (warp == 1) tmem_alloc<CG, 512>(smem_u32(&sm.tmem));
  load_segments(sm.seg, p.off, p.G, p.rows, WGRAD ? BK : CG * WM, p.status);
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();   // the other CTA's barriers are initialised
  tc_fence_after();
  // (each role reads what it needs of these itself: kept over the branch they cost the epilogue registers)
  const auto tmem_base = [&] { return *(volatile uint32_t*)&sm.tmem; };
  const auto unit_count = [&] { return wide_units<CG, WGRAD>(p, sm.seg); };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(w_regs_rest<CG>()));
    const uint32_t tmem = tmem_base();
    const int units = unit_count(), first = blockIdx.x / CG, step = gridDim.x / CG;
    if (warp == 0) {
      // ------------------------------------------------------- producer (lane 0)
      int it = 0;
      bool ok = true;
      const uint32_t lead = CG == 2 ? mapa_shared(full0, 0) : full0;   // both CTAs' copies count on rank 0's barrier
      for (int L = first; L < units && ok && lane == 0; L += step) {
        const WTile t = wide_tile<CG, WGRAD>(p, sm.seg, L, rank);
        const int brow = (WGRAD ? t.n0 : t.g * p.N + t.n0) + rank * (WN / CG);
        for (int kb = 0; kb < t.nkb; ++kb, ++it) {
          const int s = it % ST;
          ok = mbar_wait(empty0 + 8 * s, ((it / ST) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          const uint32_t a = smem_u32(ring + s * SB), b = a + WM * BK;
          const int k = (t.kb0 + kb) * BK;
          if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, CG * (SB + (WGRAD ? 4 * (WM + WN) : 0)));
          const auto load = [&](uint32_t dst, const CUtensorMap* tm, int c0, int c1) {
            if (CG == 1) tma_load_2d(dst, tm, c0, c1, lead + 8 * s);
            else tma_load_2d_pair(dst, tm, c0, c1, lead + 8 * s);
          };
          load(b, &tmB, k, brow);          // (a pair: this CTA's half of the columns)
          load(a, &tmA, k, t.row0);
          if (WGRAD) {
            load(smem_u32(sm.sa[it % kWChunk]), &tmSA, t.row0, t.kb0 + kb);
            load(smem_u32(sm.sb[it % kWChunk]), &tmSB, t.n0, t.kb0 + kb);
          }
        }
      }
      if (!ok && rank == 0) {   // the copies still in flight (lane 0)
        for (int i = max(0, it - ST); i < it; ++i) wait_own(full0 + 8 * (i % ST), (i / ST) & 1, p.status);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ------------------------------------------------------------- scales
      // A thread's row is a row of the scales too, so an epilogue that reads them itself touches a line a lane and K
      // block. This warp reads a chunk ahead.
      int ch = 0;
      bool ok = true;
      for (int L = first; L < units && ok && !WGRAD; L += step) {
        const WTile t = wide_tile<CG, WGRAD>(p, sm.seg, L, rank);
        const int nb = (p.N + 127) / 128;
        for (int k0 = 0; k0 < t.nkb; k0 += kWChunk, ++ch) {
          const int j = (ch & 1) * kWChunk, n = min(kWChunk, t.nkb - k0);
          ok = warp_wait(sempty0 + 8 * (ch & 1), ((ch >> 1) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
#pragma unroll
          for (int i = lane; i < WM; i += 32) {
            const float* row = p.sa + (size_t)min(t.row0 + i, max(t.row_end - 1, 0)) * p.nkb + k0;
            float v[kWChunk];
#pragma unroll
            for (int k = 0; k < kWChunk; ++k) v[k] = k < n ? __ldg(row + k) : 0.f;
#pragma unroll
            for (int k = 0; k < kWChunk; ++k) sm.sa[j + k][i] = v[k];
          }
          if (lane < 2 * kWChunk) {
            const int h = lane / kWChunk, k = lane % kWChunk;
            if (k < n) sm.sbh[j + k][h] = __ldg(p.sb + ((size_t)t.g * nb + min(t.n0 / 128 + h, nb - 1)) * p.nkb + k0 + k);
          }
          mbar_arrive(sfull0 + 8 * (ch & 1));
        }
      }
    } else {
      // --------------------------------------------- MMA (lane 0; rank 0 for a pair)
      if (lane == 0 && rank == 0 && warp <= kWBufs) {
        const int b = warp - 1;
        int it = 0;
        bool ok = true;
        for (int L = first; L < units && ok; L += step) {
          const WTile t = wide_tile<CG, WGRAD>(p, sm.seg, L, rank);
          for (int kb = 0; kb < t.nkb; ++kb, ++it) {
            if (it % kWBufs != b) continue;
            const int s = it % ST;
            ok = spin_wait(full0 + 8 * s, (it / ST) & 1, abort_flag, p.status) &&
                 spin_wait(pempty0 + 8 * b, ((it / kWBufs) & 1) ^ 1, abort_flag, p.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = smem_u32(ring + s * SB);
            const uint64_t da = desc_kmajor(a), db = desc_kmajor(a + WM * BK);
#pragma unroll
            for (int k = 0; k < BK / 32; ++k)
              mma_f8<CG>(tmem + b * WN, da + 2 * k, db + 2 * k, idesc_f8(CG * WM, WN), k > 0 ? 1u : 0u);
            commit<CG>(pfull0 + 8 * b);
            commit<CG>(empty0 + 8 * s);
          }
        }
        // nothing of this CTA's is in flight when its TMEM is given back
        if (CG == 1) mma_commit(drain);
        else mma_commit_pair(drain);
        wait_own(drain, 0, p.status);
      }
      __syncwarp();
    }
  } else {
    // ----------------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(w_regs_epi<CG>()));
    const uint32_t tmem = tmem_base();
    const int units = unit_count(), first = blockIdx.x / CG, step = gridDim.x / CG;
    const int quad = warp & 3, part = (warp - 4) >> 2;
    const int r = quad * 32 + lane;                           // row of the tile
    const uint32_t tq = tmem + part * WC + ((uint32_t)(quad * 32) << 16);
    const uint32_t back0 = CG == 2 ? mapa_shared(pempty0, 0) : pempty0;
    int it = 0, ch = 0;
    bool ok = true;   // after a failed wait: no more waiting or storing
    for (int L = first; L < units && ok; L += step) {
      uint64_t acc[WC / 2];    // pairs of neighbouring columns
#pragma unroll
      for (int i = 0; i < WC / 2; ++i) acc[i] = 0;
      const WTile t0 = wide_tile<CG, WGRAD>(p, sm.seg, L, rank);
      const bool some = WGRAD || t0.row0 + quad * 32 < t0.row_end;   // this warp's rows are not all behind the segment
      for (int left = t0.nkb; left > 0 && ok; left -= kWChunk, ++ch) {
        const int n = min(kWChunk, left);
        if (!WGRAD) ok = warp_wait(sfull0 + 8 * (ch & 1), (ch >> 1) & 1, abort_flag, p.status);
#pragma unroll 1
        for (int k = 0; k < n && ok; ++k, ++it) {
          const int b = it % kWBufs, slot = WGRAD ? it % kWChunk : (ch & 1) * kWChunk + k;
          ok = warp_wait(pfull0 + 8 * b, (it / kWBufs) & 1, abort_flag, p.status);
          if (!ok) break;
          const float* cs = &sm.sb[WGRAD ? slot : 0][part * WC];
          const float s = WGRAD ? sm.sa[slot][r] : sm.sa[slot][r] * sm.sbh[slot][part * WC / 128];
          tc_fence_after();
          if (!some) {
            __syncwarp();
            if (lane == 0) {
              if (CG == 1) mbar_arrive(back0 + 8 * b);
              else arrive_remote(back0 + 8 * b);
            }
            continue;
          }
#pragma unroll
          for (int c = 0; c < WC; c += 16) {
            uint32_t u[16];
            uint64_t w[8];
            tmem_ld16(tq + b * WN + c, u);
            if (WGRAD) pair_scales<true>(w, s, cs + c);   // while they come
            tmem_ld_wait_for(u);
            if (!WGRAD) pair_scales<false>(w, s, cs);
            if (c == WC - 16) {   // the partial is read: its MMAs may have it again
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if (CG == 1) mbar_arrive(back0 + 8 * b);
                else arrive_remote(back0 + 8 * b);
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              fma2(acc[c / 2 + i], pair(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), w[i]);
          }
        }
        __syncwarp();
        if (!WGRAD && lane == 0) mbar_arrive(sempty0 + 8 * (ch & 1));
      }
      const WTile t = wide_tile<CG, WGRAD>(p, sm.seg, L, rank);
      const int row = t.row0 + r, col0 = t.n0 + part * WC;
      // by TMA where it cannot reach rows of another segment (its map ends with c's rows, wgrad's with a segment's)
      if (CG == 2 && ok && p.vec && (WGRAD || t.row0 + quad * 32 + 32 <= t.row_end)) {
        constexpr int SC = 128 / sizeof(O);      // columns of a piece
        uint8_t* buf = staging + (warp - 4) * kWOutBufs * kWOutBytes;
#pragma unroll
        for (int i0 = 0; i0 < WC; i0 += kWOutBufs * SC) {
          if (col0 + i0 >= p.N || t.row0 + quad * 32 >= t.row_end) break;
          if (lane == 0) bulk_wait_read<0>();    // what was sent from here before
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kWOutBufs * SC; i += SC) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {        // 16 bytes each
              float f[8];
#pragma unroll
              for (int q = 0; q < 16 / (int)sizeof(O); q += 2)
                unpair(acc[(i0 + i + j * (SC / 8) + q) / 2], f[q], f[q + 1]);
              uint4 w;
              if (sizeof(O) == 4) w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
              else w = pack8(f);
              *reinterpret_cast<uint4*>(buf + i / SC * kWOutBytes + lane * 128 + ((j ^ (lane & 7)) << 4)) = w;
            }
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < kWOutBufs * SC; i += SC)
              if (col0 + i0 + i < p.N)
                tma_store_3d_hint(&tmC, col0 + i0 + i, t.row0 + quad * 32, WGRAD ? t.g : 0,
                                  smem_u32(buf + i / SC * kWOutBytes), policy_evict_first());
            bulk_commit();
          }
        }
      } else if (ok && row < t.row_end) {
        O* out = (O*)p.c + ((WGRAD ? (size_t)t.g * p.M : (size_t)0) + row) * p.N + col0;
        const int cols = min(WC, p.N - col0);
#pragma unroll
        for (int i = 0; i < WC; i += 16) {
          float f[16];
#pragma unroll
          for (int j = 0; j < 16; j += 2) unpair(acc[(i + j) / 2], f[j], f[j + 1]);
          if (i < cols) store16(out + i, f, cols - i, p.vec);
        }
      }
      __syncwarp();
    }
    if (CG == 2 && lane == 0) bulk_wait<0>();
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();   // neither CTA leaves while the pair's MMAs or arrivals may touch it
  tc_fence_after();
  if (warp == 1) tmem_free<CG, 512>(sm.tmem);
}

// ----------------------------------------------------------------- narrow
constexpr int kNThreads = 256, kNBufs = 4;
template <int NT> constexpr int n_stages() { return NT == 16 ? 5 : 4; }
template <int NT> constexpr int n_stage_bytes() { return (128 + NT) * BK; }
template <int NT>
struct alignas(16) NarrowSmem {
  SegSmem seg;
  uint64_t full[8], empty[8], pfull[kNBufs], pempty[kNBufs];
  uint32_t tmem;
  int abort;
};
template <int NT> constexpr int n_smem(int nkb) {
  return n_stages<NT>() * n_stage_bytes<NT>() + 1024 + (int)sizeof(NarrowSmem<NT>) + nkb * NT * 4;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Cluster of S CTAs per unit (token tile, 128 weight rows); rank r takes K blocks r nkb / S .. (r + 1) nkb / S. Two CTAs
// a SM, with rings of 5 stages (90 KB) for 16 tokens: eight in one CTA a SM were slower (below: 18.9 and 173 us).
// Measured: 128 rows over 32 experts of 7168 x 4096 in 146-150 us (93-95% of the HBM copy rate); one row x 4096 x 7168
// in 7.9 us, of which 4.3 are its bytes at that rate and the rest the start, the first copy and the joining of 8 parts
// (split in 4: 9.8, in 2: 14.8).
template <int NT, bool GATHER, typename O>
__global__ void __launch_bounds__(kNThreads, 2)
    fp8_narrow_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, GemmParams p,
                      int S) {
  constexpr int ST = n_stages<NT>(), SB = n_stage_bytes<NT>(), COLS = kNBufs * NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  NarrowSmem<NT>& sm = *reinterpret_cast<NarrowSmem<NT>*>(ring + ST * SB);
  float* sas = reinterpret_cast<float*>(ring + ST * SB + sizeof(NarrowSmem<NT>));   // [K block][token]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &sm.abort;
  const uint32_t full0 = smem_u32(sm.full), empty0 = smem_u32(sm.empty), pfull0 = smem_u32(sm.pfull),
                 pempty0 = smem_u32(sm.pempty);
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < kNBufs; ++i) {
      mbar_init(pfull0 + 8 * i, 1);
      mbar_init(pempty0 + 8 * i, 4);
    }
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();     // before the allocation, as in the wide kernel
  griddep_launch();
  if (warp == 1) tmem_alloc<1, COLS>(smem_u32(&sm.tmem));
  load_segments(sm.seg, p.off, p.G, p.rows, NT, p.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int rank = blockIdx.x % S, unit = blockIdx.x / S;
  const int nt = (p.N + 127) / 128, tt = unit / nt, n0 = (unit - tt * nt) * 128;
  const bool live = tt < sm.seg.tile[p.G];   // the same in the whole cluster
  int g = 0, row0 = 0, row_end = 0, kb0 = 0, nkb = 0;
  if (live) {
    g = segment_of(sm.seg, p.G, tt);
    row0 = sm.seg.off[g] + (tt - sm.seg.tile[g]) * NT;
    row_end = min(sm.seg.off[g + 1], row0 + NT);
    kb0 = (int)((long long)rank * p.nkb / S);
    nkb = (int)((long long)(rank + 1) * p.nkb / S) - kb0;
  }
  float acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = 0.f;
  bool ok = true;
  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    int r[4];
    if (GATHER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = row0 + 4 * lane + i;
        r[i] = gather_row(p, m, row_end);
      }
    }
    const int brow = g * p.N + n0;
    int kb = 0;
    for (; kb < nkb; ++kb) {
      const int s = kb % ST;
      ok = __all_sync(0xffffffffu, mbar_wait(empty0 + 8 * s, ((kb / ST) & 1) ^ 1, abort_flag, p.status));
      if (!ok) break;
      const uint32_t a = smem_u32(ring + s * SB), fb = full0 + 8 * s;
      const int k = (kb0 + kb) * BK;
      if (lane == 0) {
        mbar_arrive_expect_tx(fb, SB);
        tma_load_2d(a, &tmB, k, brow, fb);
        if (!GATHER) tma_load_2d(a + 128 * BK, &tmA, k, row0, fb);
      }
      if (GATHER) {
        __syncwarp();
        if (lane < NT / 4) tma_gather4(a + (128 + 4 * lane) * BK, &tmA, k, r[0], r[1], r[2], r[3], fb);
      }
    }
    if (!ok && lane == 0) {
      for (int i = max(0, kb - ST); i < kb; ++i) wait_own(full0 + 8 * (i % ST), (i / ST) & 1, p.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------------------------------------------- MMA
    if (lane == 0) {
      int last = -1;
      for (int kb = 0; kb < nkb; ++kb) {
        const int s = kb % ST, b = kb % kNBufs;
        ok = mbar_wait(pempty0 + 8 * b, ((kb / kNBufs) & 1) ^ 1, abort_flag, p.status) &&
             mbar_wait(full0 + 8 * s, (kb / ST) & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = smem_u32(ring + s * SB);
        const uint64_t da = desc_kmajor(a), db = desc_kmajor(a + 128 * BK);
#pragma unroll
        for (int k = 0; k < BK / 32; ++k)
          mma_f8<1>(tmem + b * NT, da + 2 * k, db + 2 * k, idesc_f8(128, NT), k > 0 ? 1u : 0u);
        mma_commit(empty0 + 8 * s);
        mma_commit(pfull0 + 8 * b);
        last = kb;
      }
      if (last >= 0) wait_own(pfull0 + 8 * (last % kNBufs), (last / kNBufs) & 1, p.status);
    }
    __syncwarp();
  } else if (warp < 6) {
    // -------------------------------------------------------------------- epilogue: thread = weight row
    const int quad = warp & 3;
    const uint32_t tq = tmem + ((uint32_t)(quad * 32) << 16);
    // the token tile's scales for this CTA's K blocks (zero past the segment), while the operands are on their way
    for (int i = tid - 64; i < NT * nkb; i += 128) {
      const int j = i / nkb, kb = i - j * nkb;
      float s = 0.f;
      if (row0 + j < row_end) {
        const int ar = GATHER ? p.row_index[row0 + j] : row0 + j;
        if ((unsigned)ar < (unsigned)p.a_rows) {
          s = p.sa[(size_t)ar * p.nkb + kb0 + kb];
        } else {
          set_error(p.status, MOE_ERR_DEVICE_INDEX);
        }
      }
      sas[kb * NT + j] = s;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const float* sb = p.sb + ((size_t)g * nt + n0 / 128) * p.nkb + kb0;
    float nsb = nkb > 0 ? __ldg(sb) : 0.f;
    for (int kb = 0; kb < nkb; ++kb) {
      const int b = kb % kNBufs;
      const float s = nsb;
      if (kb + 1 < nkb) nsb = __ldg(sb + kb + 1);
      ok = warp_wait(pfull0 + 8 * b, (kb / kNBufs) & 1, abort_flag, p.status);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < NT; c += 16) {
        uint32_t u[16];
        tmem_ld16(tq + b * NT + c, u);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 v = *reinterpret_cast<const float4*>(sas + kb * NT + c + i);
          acc[c + i] = fmaf(__uint_as_float(u[i]), s * v.x, acc[c + i]);
          acc[c + i + 1] = fmaf(__uint_as_float(u[i + 1]), s * v.y, acc[c + i + 1]);
          acc[c + i + 2] = fmaf(__uint_as_float(u[i + 2]), s * v.z, acc[c + i + 2]);
          acc[c + i + 3] = fmaf(__uint_as_float(u[i + 3]), s * v.w, acc[c + i + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pempty0 + 8 * b);
    }
    const int wr = quad * 32 + lane, col = n0 + wr;
    if (S == 1) {
      if (ok && col < p.N) {
        O* out = (O*)p.c + (size_t)row0 * p.N + col;
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (row0 + j < row_end) out[(size_t)j * p.N] = from_f<O>(acc[j]);
      }
    } else {   // every MMA and copy of this CTA has ended: the ring is free
      float* red = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int j = 0; j < NT; ++j) red[j * 128 + wr] = acc[j];
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free<1, COLS>(tmem);
  if (S > 1) {
    // add the parts in rank order; the CTAs share out the tokens
    cluster_sync();
    if (*abort_flag == 0) {
      const uint32_t red = smem_u32(ring);
      const int wr = tid & 127, col = n0 + wr;
      for (int j = rank * 2 + (tid >> 7); row0 + j < row_end; j += 2 * S) {
        float v = 0.f;
        for (int q = 0; q < S; ++q) v += ld_cluster(mapa_shared(red + (j * 128 + wr) * 4, q));
        if (col < p.N) ((O*)p.c)[(size_t)(row0 + j) * p.N + col] = from_f<O>(v);
      }
    }
    cluster_sync();   // no CTA leaves while another reads its part
  }
}

// -------------------------------------------------------------------- host
constexpr int kMaxSmem = 227 * 1024, kNarrowMaxKb = 128;
static_assert(w_smem<1>() <= kMaxSmem && w_smem<2>() <= kMaxSmem && n_smem<64>(kNarrowMaxKb) <= kMaxSmem && n_smem<16>(kNarrowMaxKb) <= kMaxSmem &&
                  n_smem<32>(kNarrowMaxKb) <= kMaxSmem,
              "shared memory per CTA");

// fp32 [rows][cols] (cols a multiple of 4), boxes of one row.
bool make_scale_tmap(CUtensorMap* tm, const float* base, uint64_t cols, uint64_t rows, uint32_t box) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows}, strides[1] = {4 * cols};
  cuuint32_t boxes[2] = {box, 1}, estr[2] = {1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(base), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// c [G][rows][cols] for stores of 32 rows x 128 bytes.
bool make_out_tmap(CUtensorMap* tm, void* c, uint64_t cols, uint64_t rows, uint64_t G, int fp32) {
  auto fn = encode_fn();
  if (!fn) return false;
  const uint64_t e = fp32 ? 4 : 2;
  cuuint64_t dims[3] = {cols, rows, G}, strides[2] = {cols * e, cols * rows * e};
  cuuint32_t box[3] = {(cuuint32_t)(128 / e), 32, 1}, estr[3] = {1, 1, 1};
  return fn(tm, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, c, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K>
cudaError_t set_smem(K kern) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
}
template <int CG, bool WGRAD, typename O>
cudaError_t init_wide() {
  auto kern = fp8_wide_kernel<CG, WGRAD, O>;
  cudaFuncAttributes at;
  MOE_TRY(cudaFuncGetAttributes(&at, kern));
  if (at.numRegs != kWRegs) return cudaErrorInvalidKernelImage;   // what the epilogue's registers are taken out of
  return set_smem(kern);
}
template <int NT>
cudaError_t init_narrow() {
  MOE_TRY(set_smem(fp8_narrow_kernel<NT, false, bf16>));
  MOE_TRY(set_smem(fp8_narrow_kernel<NT, false, float>));
  MOE_TRY(set_smem(fp8_narrow_kernel<NT, true, bf16>));
  return set_smem(fp8_narrow_kernel<NT, true, float>);
}

template <int CG, bool WGRAD, typename O>
cudaError_t launch_wide(const moe_ops_s* o, const CUtensorMap* tm, const GemmParams& p, long long units,
                        cudaStream_t s) {
  auto kern = fp8_wide_kernel<CG, WGRAD, O>;
  if (CG == 1) return launch_pdl(kern, dim3((unsigned)(units < o->sms ? units : o->sms)), dim3(kWThreads), w_smem<CG>(), s, tm[0], tm[1], tm[2], tm[3], tm[4], p);
  // as many pairs as run at once
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)(units < o->pairs ? units : o->pairs));
  cfg.blockDim = dim3(kWThreads);
  cfg.dynamicSmemBytes = w_smem<CG>();
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], tm[2], tm[3], tm[4], p);
}
template <bool WGRAD>
cudaError_t pick_wide(const moe_ops_s* o, int cg, const CUtensorMap* tm, GemmParams p, long long units, bool fp32,
                      cudaStream_t s) {
  const int nt = ceil_div(p.N, WN), mt = WGRAD ? ceil_div(p.M, cg * WM) : 1;
  p.nt = FastDiv(nt);
  p.mnt = FastDiv(mt * nt);
  p.rnt = FastDiv(kRasterM * nt);
  p.last = FastDiv(mt % kRasterM ? mt % kRasterM : kRasterM);
  if (cg == 1)
    return fp32 ? launch_wide<1, WGRAD, float>(o, tm, p, units, s) : launch_wide<1, WGRAD, bf16>(o, tm, p, units, s);
  return fp32 ? launch_wide<2, WGRAD, float>(o, tm, p, units, s) : launch_wide<2, WGRAD, bf16>(o, tm, p, units, s);
}

// Rows of a (and their scales) in the order of c's rows, one warp a row; an index out of range gives zeros. Rows of no
// segment are left alone, whatever row_index holds there. Most reads hit L2: 12,288 rows of 2,048 bytes in 8 us,
// 50 MB moved.
__global__ void __launch_bounds__(256) gather_rows_kernel(const uint8_t* __restrict__ a, const float* __restrict__ sa,
                                                          const int* __restrict__ row_index,
                                                          const int* __restrict__ off, int G, int M, int a_rows, int K,
                                                          int nkb, uint8_t* __restrict__ out, float* __restrict__ so,
                                                          int* status) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, m = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (m >= M) return;
  const int r = row_index[m], lo = off ? off[0] : 0, hi = off ? off[G] : M;   // (loaded together)
  if (m < lo || m >= hi) return;
  const bool in = (unsigned)r < (unsigned)a_rows;
  if (!in) set_error(status, MOE_ERR_DEVICE_INDEX);
  const uint4* src = reinterpret_cast<const uint4*>(a + (size_t)(in ? r : 0) * K);
  uint4* dst = reinterpret_cast<uint4*>(out + (size_t)m * K);
#pragma unroll 4
  for (int i = lane; i < K / 16; i += 32) dst[i] = in ? src[i] : make_uint4(0u, 0u, 0u, 0u);
  for (int i = lane; i < nkb; i += 32) so[(size_t)m * nkb + i] = in ? sa[(size_t)r * nkb + i] : 0.f;
}

template <int NT, bool GATHER, typename O>
cudaError_t launch_narrow(const CUtensorMap& a, const CUtensorMap& b, const GemmParams& p, long long units, int S,
                          cudaStream_t s) {
  auto kern = fp8_narrow_kernel<NT, GATHER, O>;
  const int smem = n_smem<NT>(ceil_div(p.nkb, S));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * S));
  cfg.blockDim = dim3(kNThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, b, p, S);
}

template <int NT>
cudaError_t pick_narrow(const CUtensorMap& a, const CUtensorMap& b, const GemmParams& p, long long units, int S,
                        bool fp32, cudaStream_t s) {
  if (p.row_index)
    return fp32 ? launch_narrow<NT, true, float>(a, b, p, units, S, s) : launch_narrow<NT, true, bf16>(a, b, p, units, S, s);
  return fp32 ? launch_narrow<NT, false, float>(a, b, p, units, S, s) : launch_narrow<NT, false, bf16>(a, b, p, units, S, s);
}

int out_vec(const void* c, long long n, int fp32) {
  const long long bytes = n * (fp32 ? 4 : 2);
  const uintptr_t at = (uintptr_t)c;
  return bytes % 32 == 0 && at % 32 == 0 ? 32 : bytes % 16 == 0 && at % 16 == 0 ? 16 : 0;
}
// Rows a segment up to which the narrow kernel is the faster one. Where the wide kernel's tiles fill the GPU, it too
// streams the weights, reads them once for up to 128 rows and loses nothing on uneven segments: 64 uneven segments of
// 2,816 x 2,048 take 80.5 us (narrow) and 81.6 (wide) with 4 rows each on average, 82.6 both with 8, 94.9 and 83.6 with
// 24; 32 of 7,168 x 4,096 156 and 159, 166 and 164, 191 and 166. Where they do not fill it, the narrow kernel has more
// tiles and splits the reduction: one segment of 4,096 x 7,168 (16 wide tiles) 17 and 33 with 32 rows, 21 and 35 with
// 64; 16,384 x 7,168 (64 tiles) 38 and 44, 50 and 44. (Cold, with an event's 2 us.)
constexpr int kNarrowAlways = 8, kNarrowHalf = 32, kNarrowMost = 64;
bool use_narrow(int M, int G, int N, int K, int sms) {
  const long long tiles = (long long)(G < M ? G : M) * ceil_div(N, WN);
  const int rows = tiles >= sms ? kNarrowAlways : 4 * tiles >= sms ? kNarrowHalf : kNarrowMost;
  return ceil_div(M, G) <= rows && ceil_div(K, BK) <= kNarrowMaxKb;
}

}  // namespace

cudaError_t fp8_init(int* pairs) {
  MOE_TRY((init_wide<1, false, bf16>()));
  MOE_TRY((init_wide<1, false, float>()));
  MOE_TRY((init_wide<1, true, bf16>()));
  MOE_TRY((init_wide<1, true, float>()));
  MOE_TRY((init_wide<2, false, bf16>()));
  MOE_TRY((init_wide<2, false, float>()));
  MOE_TRY((init_wide<2, true, bf16>()));
  MOE_TRY((init_wide<2, true, float>()));
  MOE_TRY(init_narrow<16>());
  MOE_TRY(init_narrow<32>());
  MOE_TRY(init_narrow<64>());
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1024);
  cfg.blockDim = dim3(kWThreads);
  cfg.dynamicSmemBytes = w_smem<2>();
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(pairs, (fp8_wide_kernel<2, false, bf16>), &cfg);
}

size_t fp8_matmul_workspace(int M, int G, int K, bool gathered) {
  // (whatever N is)
  if (!gathered || (ceil_div(M, G) <= kNarrowAlways && ceil_div(K, BK) <= kNarrowMaxKb)) return 0;
  return (size_t)M * K + 16 + sizeof(float) * (size_t)M * ceil_div(K, BK);
}

cudaError_t fp8_matmul(const moe_ops_s* o, const void* a, const float* sa, int a_rows, const int* row_index, int M,
                       const void* b, const float* sb, const int* off, int G, int N, int K, void* c, int out_fp32,
                       void* ws, cudaStream_t s, long long* n) {
  GemmParams p = {};
  p.sa = sa;
  p.sb = sb;
  p.row_index = row_index;
  p.off = off;
  p.G = G;
  p.rows = M;
  p.a_rows = a_rows;
  p.N = N;
  p.nkb = ceil_div(K, BK);
  p.vec = out_vec(c, N, out_fp32);
  p.c = c;
  p.status = o->status;
  CUtensorMap ta, tb;
  if (use_narrow(M, G, N, K, o->sms)) {
    // Tokens a tile, with room for uneven segments: one segment of 4,096 x 7,168 with 32 rows takes 21, 19 and 17 us
    // with tiles of 16, 32 and 64, 64 segments of 2,816 x 2,048 with 8 rows each 83, 85 and 91.
    const int avg = ceil_div(M, G), NT = avg <= 12 ? 16 : avg <= 24 ? 32 : 64;
    if (!make_tmap(&ta, a, K, a_rows, BK, row_index ? 1 : NT, 1) ||
        !make_tmap(&tb, b, K, (uint64_t)G * N, BK, 128, 1))
      return cudaErrorInvalidValue;
    const int nt = ceil_div(N, 128);
    // token tiles: at most one that is not full for each segment that holds a row
    const long long most = (G < M ? G : M), units = (M / NT + most < M ? M / NT + most : M) * (long long)nt;
    // Split while all parts run at once, two CTAs a SM: one row x 16,384 x 2,048 (128 tiles) takes 15 us whole and 17
    // split in 2, 16,384 x 7,168 36 and 33, 4,096 x 7,168 (32 tiles) 27, 21, 17 and 17 split in 1, 2, 4 and 8.
    int S = 1;
    while (S < 8 && 2 * S <= p.nkb && units * S * 2 <= 2 * o->sms) S *= 2;
    *n += 1;
    return NT == 16 ? pick_narrow<16>(ta, tb, p, units, S, out_fp32, s)
           : NT == 32 ? pick_narrow<32>(ta, tb, p, units, S, out_fp32, s)
                      : pick_narrow<64>(ta, tb, p, units, S, out_fp32, s);
  }
  if (row_index) {
    // Gathered rows are put in order once. (TMA gathers inside the product fetch them again for every column tile,
    // and one of four 128-byte rows takes about 80 cycles: 2,600 cycles a stage of 128 rows, whose MMAs take 512.)
    float* so = (float*)((char*)ws + ((size_t)M * K + 15) / 16 * 16);
    *n += 1;
    MOE_TRY(launch_pdl(gather_rows_kernel, dim3(ceil_div(M, 8)), dim3(256), 0, s, (const uint8_t*)a, sa, row_index, off, G,
                       M, a_rows, K, p.nkb, (uint8_t*)ws, so, o->status));
    a = ws;
    p.sa = so;
    p.a_rows = a_rows = M;
  }
  // Pairs take a K block of 128 rows x 256 columns a SM in 500 ns where single CTAs take 560, but cut segments into
  // tiles of 256 rows: 12,288 rows of 64 uneven segments (192 on average) x 2,816 x 2,048 take 134 us with pairs and 120
  // without, 8,192 rows of one segment x 4,096 x 7,168 196 and 214. With half a tile lost a segment the two meet near
  // 500 rows.
  const int cg = ceil_div(M, G) >= 512 ? 2 : 1;
  CUtensorMap tm[5];
  if (!make_tmap(&tm[0], a, K, a_rows, BK, WM, 1) || !make_tmap(&tm[1], b, K, (uint64_t)G * N, BK, WN / cg, 1))
    return cudaErrorInvalidValue;
  tm[2] = tm[3] = tm[4] = tm[0];      // (not read where they are not made)
  if (cg == 2 && p.vec && !make_out_tmap(&tm[4], c, N, M, 1, out_fp32)) return cudaErrorInvalidValue;
  const long long units = ((long long)ceil_div(M, cg * WM) + (G > 1 ? G : 0)) * ceil_div(N, WN);
  *n += 1;
  return pick_wide<false>(o, cg, tm, p, units, out_fp32, s);
}

cudaError_t fp8_wgrad(const moe_ops_s* o, const void* dct, const float* sdct, const void* xt, const float* sxt, int T,
                      const int* off, int G, int N, int K, void* c, int out_fp32, cudaStream_t s, long long* n) {
  GemmParams p = {};
  p.sa = sdct;
  p.sb = sxt;
  p.off = off;
  p.G = G;
  p.rows = T;
  p.M = N;
  p.N = K;
  p.vec = out_vec(c, K, out_fp32);
  p.c = c;
  p.status = o->status;
  const int Tp = quant_cols_rows(T, G), cg = N > WM ? 2 : 1;
  CUtensorMap tm[5];
  if (!make_tmap(&tm[0], dct, Tp, N, BK, WM, 1) || !make_tmap(&tm[1], xt, Tp, K, BK, WN / cg, 1) ||
      !make_scale_tmap(&tm[2], sdct, N, Tp / BK, WM) || !make_scale_tmap(&tm[3], sxt, K, Tp / BK, WN))
    return cudaErrorInvalidValue;
  tm[4] = tm[0];
  if (cg == 2 && p.vec && !make_out_tmap(&tm[4], c, K, N, G, out_fp32)) return cudaErrorInvalidValue;
  const long long units = (long long)G * ceil_div(N, cg * WM) * ceil_div(K, WN);
  *n += 1;
  return pick_wide<true>(o, cg, tm, p, units, out_fp32, s);
}

}  // namespace moe
