// fgemm_kern_w4mm.cu -- products with 4-bit weights for more rows of A than
// the few-rows kernel (fgemm_kern_w4.cu) takes: tcgen05 with the codes as the
// operand in tensor memory.
//
//   C[i][j] = epi(alpha * sum_k A[i][k] (q[j][k] - z[j][k/G]) s[j][k/G] + bias[j])
//
// As there, codes are never turned into weights: with acc = sum_k (q - z) x
// over a group, the group's part is s acc, added to a running fp32 sum.  A tile
// is 128 rows of W (the tensor core's rows) by MT rows of A.  Its codes go TMA
// -> shared memory -> registers, where a logical operation and a multiply-add
// make two fp16 operands (q - z) 2^-9 -> tensor memory; the product of a group is 2 to 8 MMAs into an accumulator of
// its own, which the fold warps read once, scale and add in registers.  So a
// weight costs about one and a half ALU operations and nothing is rounded but
// the output; the fold costs 2 fp32 operations for every group, row and column
// (the unit of the row's group, the column's scale), against 2 G of the product.
//
// A pre-pass (w4_pack_kernel) writes A as scaled fp16 in the order of the
// codes' pairs, with the unit of each group.  The main kernel is launched so that it
// may begin before the pre-pass ends (programmatic dependent launch): its
// codes are on their way by then.
//
// What bounds it: the fold's chain (products done -> tensor memory -> scale, add
// -> room for the next), not the tensor pipe nor memory.  Measured: 48 x 8192 x
// 8192 fp16, groups of 64, 32.1 us; 2048 x 4096 x 14336 bf16, groups of 128, 317
// us, 758 TFLOP/s.  (With the zero point taken off the group's sum in the fold, as
// z sum_k x: 32.4 and 341 us; but 128 x 8192 x 16384 in groups of 32 takes 242 us
// against 223.  With subnormal operands: 30.3 and 310.)
//
// Roles: warp 0 loads the codes, warp 2 A, warps 1 and 3 issue the MMAs, warps 4..
// expand the codes, the last 4 or 8 warps fold.  Every wait is bounded; a wait
// that runs out latches the error word and all roles leave.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_internal.h"
#include "fgemm_ptx.cuh"
#include "fgemm_w4.cuh"

namespace fgemm {

namespace {

constexpr int kRows = 128;   // rows of W of a tile
constexpr int kBlock = 128;  // k of one pipeline step: 64 bytes of codes a row
constexpr int kThreads = 512;
constexpr int kCodeBytes = kRows * 64;

// Most rows of A a tile takes: the accumulators of two steps' groups fit in
// tensor memory beside the expanded codes.
constexpr int kMostRows[3] = {32, 64, 128};  // groups of 32, 64, 128

template <int MT, int GROUPS>  // groups of a step
struct Cfg {
  static constexpr int kFoldWarps = MT >= 64 ? 8 : 4;
  static constexpr int kCols = MT == 128 ? 64 : MT < 32 ? MT : 32;  // of A's rows, a fold warp's
  static constexpr int kExpandWarps = 12 - kFoldWarps;
  // Tensor memory: four stages of 64 columns of expanded codes, then two or
  // four of GROUPS accumulators each.  Where it is two, the codes' stages go
  // back on their own as soon as they have been multiplied (kAhead), so that
  // codes are expanded while both accumulators are multiplied or folded; where
  // it is four, both go back together: 8192 x 16384, 16 rows, groups of 32 / 64 / 128
  // 47.6 / 36.1 / 33.9 us on their own against 45.7 / 35.9 / 33.2 together.
  static constexpr int kAStages = 4;
  static constexpr int kDCols = GROUPS * MT;
  static constexpr int kDAt = kAStages * 64;
  static constexpr int kDStages = (512 - kDAt) / kDCols < 4 ? 2 : 4;
  static constexpr int kXBytes = MT * 256;            // A's rows of one step
  static constexpr int kUnitBytes = GROUPS * MT * 4;  // units of its groups
  static constexpr int kXStages = MT == 128 ? 4 : 6;
  static constexpr int kCodeStages = MT == 128 ? 8 : 10;
  static constexpr int kBars = 2 * kCodeStages + 2 * kXStages + 2 * kAStages + 2 * kDStages + 1;
  static constexpr int kSmem = 1024 + kCodeStages * kCodeBytes + kXStages * (kXBytes + kUnitBytes) + 8 * kBars + 16;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(MT * kRows * 4 + kRows * 4 <= kCodeStages * kCodeBytes + kXStages * kXBytes, "the sums reuse the rings");
  static constexpr bool kAhead = kDStages < kAStages;
  // Warps that issue the products, a step each in turn.  One against two:
  // 2048 x 4096 x 14336 (groups of 128) 346 / 317 us, 8192 x 16384 with 128 rows (64)
  // 110.8 / 104.5, 32 rows (32) 61.5 / 60.0; with four accumulators 16 rows (128)
  // 45.1 / 33.2, 32 rows (64) 49.7 / 40.6.
  static constexpr int kIssuers = 2;
  static_assert(kDAt + kDStages * kDCols <= 512 && kDStages % kIssuers == 0, "tensor memory");
};

__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 TMEM lanes x N consecutive 32-bit columns, N = 16 or 32.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 16)
    ptx::tmem_ld_32x32b_x16(taddr, r);
  else
    ptx::tmem_ld_32x32b_x32(taddr, r);
}
template <int N>
__device__ __forceinline__ void tmem_ready(uint32_t (&r)[N]) {
  ptx::tmem_wait_ld();
  if constexpr (N == 16)
    ptx::tmem_regs_ready16(r);
  else
    ptx::tmem_regs_ready(r);
}

// Contiguous copy global -> shared of a multiple of 16 bytes, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// 16 bytes of a ring's stage.  Volatile: the read stays between the wait for
// the stage and the arrival that hands it back.  Before that arrival the reader
// needs fence.proxy.async: the barrier orders a copy's writes before reads, but
// not reads of the generic proxy before the next copy's writes.
__device__ __forceinline__ uint4 ring_read(uint32_t at) {
  uint4 v;
  asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// Two fp32 multiply-adds in one instruction.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}

// Waits for a phase; gives up when another role has (the error word) or when
// the time limit runs out, and then latches `code`.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, const W4Params& p, uint32_t code, bool honor) {
  const uint64_t t0 = ptx::globaltimer();
#pragma unroll 1
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (honor && *reinterpret_cast<volatile unsigned int*>(p.err) != 0u) return false;
    if (ptx::globaltimer() - t0 > p.spin_ns) {
      atomicCAS(p.err, 0u, code);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const W4Params& p, int role) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, p, kErrTimeout | (static_cast<uint32_t>(role) << 24) | (blockIdx.x & 0xFFFFFFu), true);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const W4Params& p, int role) {
  return __all_sync(0xFFFFFFFFu, wait(bar, parity, p, role));
}

// A ring position: stage and phase parity.
template <int N>
struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      ph ^= 1u;
    }
  }
};

// The outputs of a tile in columns with an infinite scale, term by term
// (w4_exact).  Only where an output is infinite: there every weight's sign, and
// every code at the zero point, counts.  `flags`: a word for each of the tile's rows.
template <bool BF16>
static __device__ __noinline__ void store_wild(const W4Params& p, int tile, int m0, int mt, int rank, int* flags) {
  const bool glu = p.epi == kEpiSwiglu;
  const int groups = (p.k + p.group - 1) / p.group;
  for (int r = threadIdx.x; r < kRows; r += kThreads) flags[r] = 0;
  __syncthreads();
  {
    constexpr int kEach = kThreads / kRows;  // threads a row
    const int r = threadIdx.x / kEach;
    const uint16_t* const s = p.scales + min(w4_column(p, tile, r, kRows), p.n - 1) * p.lds;
    for (int g = threadIdx.x % kEach; g < groups; g += kEach)
      if ((s[g] & 0x7FFF) == (BF16 ? 0x7F80 : 0x7C00)) flags[r] = 1;
  }
  __syncthreads();
  // (the elements that this thread has stored before)
  const int oct_log2 = glu ? 3 : 4;
  for (int e = threadIdx.x + rank * kThreads; e < (mt << oct_log2); e += kThreads * p.slices) {
    const int i = e >> oct_log2, o = (e & ((1 << oct_log2) - 1)) * 8;
    for (int q = 0; q < 8; ++q) {
      const long long j = static_cast<long long>(tile) * (8 << oct_log2) + o + q;
      const int row = (glu ? o * 2 : o) + q;
      if (j >= p.n_out || !(flags[row] || (glu && flags[row + 8]))) continue;
      float v[2];
      for (int h = 0; h < (glu ? 2 : 1); ++h) {
        const long long col = j + static_cast<long long>(h) * p.n_out;
        v[h] = p.alpha * w4_exact<BF16>(p, m0 + i, col) + (p.bias ? w4_f32<BF16>(p.bias[col]) : 0.0f);
      }
      const float y = glu ? w4_silu(v[0]) * v[1] : p.epi == kEpiSilu ? w4_silu(v[0]) : v[0];
      p.c[(m0 + i) * p.ldc + j] = BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : __half_as_ushort(__float2half_rn(y));
    }
  }
}

template <bool BF16, int MT, int GC>  // GC: group / 32
__global__ void __launch_bounds__(kThreads, 1) w4mm_kernel(const __grid_constant__ W4Params p) {
  constexpr int GROUPS = 4 / GC;  // groups of a step
  using C = Cfg<MT, GROUPS>;
  constexpr int FW = C::kFoldWarps, EW = C::kExpandWarps;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  // X stages first (1024-byte atoms), then codes, units, barriers
  auto x_at = [&](int s) { return base + s * C::kXBytes; };
  constexpr int kCodes = C::kXStages * C::kXBytes;
  constexpr int kUnits = kCodes + C::kCodeStages * kCodeBytes;
  constexpr int kBar = kUnits + C::kXStages * C::kUnitBytes;
  auto code_at = [&](int s) { return base + kCodes + s * kCodeBytes; };
  auto unit_at = [&](int s) { return base + kUnits + s * C::kUnitBytes; };
  const uint32_t bar0 = base + kBar;
  auto code_full = [&](int s) { return bar0 + 8u * s; };
  auto code_empty = [&](int s) { return bar0 + 8u * (C::kCodeStages + s); };
  auto x_full = [&](int s) { return bar0 + 8u * (2 * C::kCodeStages + s); };
  auto x_empty = [&](int s) { return bar0 + 8u * (2 * C::kCodeStages + C::kXStages + s); };
  constexpr int kABar = 2 * C::kCodeStages + 2 * C::kXStages;
  constexpr int kDBar = kABar + 2 * C::kAStages;
  auto a_full = [&](int s) { return bar0 + 8u * (kABar + s); };                 // codes expanded
  auto a_empty = [&](int s) { return bar0 + 8u * (kABar + C::kAStages + s); };  // multiplied
  auto d_full = [&](int s) { return bar0 + 8u * (kDBar + s); };                 // products done
  auto d_empty = [&](int s) { return bar0 + 8u * (kDBar + C::kDStages + s); };  // products read
  const uint32_t drain = bar0 + 8u * (C::kBars - 1);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + kBar + 8 * C::kBars);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = p.slices;
  const int rank = slices > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int tile = blockIdx.x / slices, m0 = blockIdx.y * MT;
  const int blocks = (p.k + kBlock - 1) / kBlock;
  const int b0 = min(blocks, rank * p.slice), b1 = min(blocks, b0 + p.slice);  // slice: steps of a CTA
  const bool glu = p.epi == kEpiSwiglu;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kCodeStages; ++s) {
      ptx::mbar_init(code_full(s), 1);
      ptx::mbar_init(code_empty(s), 4);
    }
    for (int s = 0; s < C::kXStages; ++s) {
      ptx::mbar_init(x_full(s), 1);
      ptx::mbar_init(x_empty(s), FW);
    }
    for (int s = 0; s < C::kAStages; ++s) {
      ptx::mbar_init(a_full(s), 4);
      ptx::mbar_init(a_empty(s), 1);
    }
    for (int s = 0; s < C::kDStages; ++s) {
      ptx::mbar_init(d_full(s), 1);
      ptx::mbar_init(d_empty(s), FW);
    }
    ptx::mbar_init(drain, C::kIssuers);
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  uint64_t sum[C::kCols / 2];  // fold warps: rows of A in pairs
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(sum) / 8); ++i) sum[i] = 0;

  if (warp == 0) {
    // ---------------------------------------------------------- codes
    if (lane == 0) {
      ptx::prefetch_tmap(&p.tmap_w);
      const int row0 = glu ? tile * 64 : tile * 128, row1 = glu ? p.n_out + tile * 64 : tile * 128 + 64;
      Ring<C::kCodeStages> rc;
      int b = b0;
      for (; b < b1; ++b, rc.next()) {
        if (!wait(code_empty(rc.s), rc.ph ^ 1u, p, 0)) break;
        ptx::mbar_arrive_expect_tx(code_full(rc.s), kCodeBytes);
        ptx::tma_load_2d(code_at(rc.s), &p.tmap_w, b * 64, row0, code_full(rc.s));
        ptx::tma_load_2d(code_at(rc.s) + kCodeBytes / 2, &p.tmap_w, b * 64, row1, code_full(rc.s));
      }
      // Whatever another role did, the copies in flight land before the CTA
      // goes on: the stages loaded last.
      for (int i = 0; i < C::kCodeStages && b - i > b0; ++i) {
        if (--rc.s < 0) rc.s = C::kCodeStages - 1, rc.ph ^= 1u;
        if (!ptx::mbar_try_wait(code_full(rc.s), rc.ph)) wait_slow(code_full(rc.s), rc.ph, p, kErrTimeout, false);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------------------------- packed A
    if (lane == 0) {
      ptx::prefetch_tmap(&p.tmap_x);
      // it is there once the pre-pass has ended
      asm volatile("griddepcontrol.wait;" ::: "memory");
      ptx::fence_proxy_async_global();
      Ring<C::kXStages> rx;
      int b = b0;
      for (; b < b1; ++b, rx.next()) {
        if (!wait(x_empty(rx.s), rx.ph ^ 1u, p, 0)) break;
        ptx::mbar_arrive_expect_tx(x_full(rx.s), C::kXBytes + GROUPS * MT * 4);
        ptx::tma_load_2d(x_at(rx.s), &p.tmap_x, b * kBlock, m0, x_full(rx.s));
        ptx::tma_load_2d(x_at(rx.s) + C::kXBytes / 2, &p.tmap_x, b * kBlock + 64, m0, x_full(rx.s));
        for (int i = 0; i < GROUPS; ++i)
          bulk_load(unit_at(rx.s) + i * MT * 4, p.units + (static_cast<long long>(b) * GROUPS + i) * p.m_pad + m0, MT * 4,
                    x_full(rx.s));
      }
      for (int i = 0; i < C::kXStages && b - i > b0; ++i) {
        if (--rx.s < 0) rx.s = C::kXStages - 1, rx.ph ^= 1u;
        if (!ptx::mbar_try_wait(x_full(rx.s), rx.ph)) wait_slow(x_full(rx.s), rx.ph, p, kErrTimeout, false);
      }
    }
    __syncwarp();
  } else if (warp == 1 || (C::kIssuers == 2 && warp == 3)) {
    // ---------------------------------------------------------- MMA
    // (The condition as `warp == 1 || warp == 3` becomes one comparison; the loop
    // behind it was 3 to 18 % slower then.)
    if (lane == 0) {
      // fp32 accumulator, fp16 operands, both K-major, N = MT, M = 128
      constexpr uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(MT >> 3) << 17) | ((128u >> 4) << 24);
      const uint64_t desc0 = ptx::sdesc(x_at(0), 16, 1024);
      Ring<C::kXStages> rx;
      Ring<C::kAStages> ra;
      Ring<C::kDStages> rd;
      // A step's products are issued by one thread, whose time counts: one
      // commit a step, on which the fold warps hand back what it used, and two
      // warps (kIssuers).
      const int turn = warp >> 1;
      if (turn) rx.next(), ra.next(), rd.next();
      for (int b = b0 + turn; b < b1; b += C::kIssuers) {
        if (!wait(x_full(rx.s), rx.ph, p, 1) || !wait(a_full(ra.s), ra.ph, p, 1) ||
            (C::kAhead && !wait(d_empty(rd.s), rd.ph ^ 1u, p, 1)))
          break;
        ptx::tc_fence_after();
        const uint64_t desc = desc0 + static_cast<uint32_t>(rx.s * (C::kXBytes >> 4));
        const uint32_t a = tmem + ra.s * 64, d = tmem + C::kDAt + rd.s * C::kDCols;
#pragma unroll
        for (int k16 = 0; k16 < 8; ++k16)
          mma_f16_ts(d + (k16 / (2 * GC)) * MT, a + k16 * 8,
                     desc + ((k16 >> 2) * (C::kXBytes >> 5) + (k16 & 3) * 2), idesc, k16 % (2 * GC) != 0 ? 1u : 0u);
        ptx::mma_commit(d_full(rd.s));
#pragma unroll
        for (int i = 0; i < C::kIssuers; ++i) rx.next(), ra.next(), rd.next();
      }
      ptx::mma_commit(drain);
      if (!ptx::mbar_try_wait(drain, 0)) wait_slow(drain, 0, p, kErrTimeout | (1u << 24), false);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + EW) {
    // ---------------------------------------------------------- expand
    // Tile row `r` of this lane, at row `sr` of the code stage.  Eight lanes
    // that read together hit different banks (64-byte swizzle).
    const int r = (warp & 3) * 32 + lane;
    const int sr = glu ? ((r >> 3) & 1) * 64 + (r >> 4) * 8 + (r & 7) : r;
    const int sw = (sr >> 1) & 3;
    constexpr int SETS = EW / 4;  // sets of four warps, which take steps in turn
    const int set = (warp - 4) >> 2;
    // zero points of this lane's row, fetched a step of its own ahead
    const uint8_t* const z_row = p.zeros + min(w4_column(p, tile, r, kRows), p.n - 1) * p.ldz;
    const int groups = (p.k + GC * 32 - 1) / (GC * 32);
    uint8_t z_next[GROUPS];
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) z_next[i] = 8;
    auto fetch = [&](int b) {
#pragma unroll
      for (int i = 0; i < GROUPS; ++i)
        if (p.zeros) z_next[i] = z_row[min(b * GROUPS + i, groups - 1)];  // past the last group A is zero
    };
    fetch(b0 + set);
    Ring<C::kCodeStages> rc;
    Ring<C::kAStages> ra;
    for (int b = b0; b < b1; ++b, rc.next(), ra.next()) {
      if (SETS > 1 && (b - b0) % SETS != set) continue;
      uint32_t zero[GROUPS];
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) zero[i] = w4_zero(z_next[i]);
      fetch(b + SETS);
      if (!wait_warp(code_full(rc.s), rc.ph, p, 3)) break;
      uint4 w[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        w[c] = ring_read(code_at(rc.s) + sr * 64 + ((c ^ sw) << 4));
      if (!wait_warp(C::kAhead ? a_empty(ra.s) : d_empty(ra.s), ra.ph ^ 1u, p, 3)) break;
      ptx::tc_fence_after();
      const uint32_t to = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + ra.s * 64;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t e[32];
        const uint32_t q[8] = {w[2 * h].x,     w[2 * h].y,     w[2 * h].z,     w[2 * h].w,
                               w[2 * h + 1].x, w[2 * h + 1].y, w[2 * h + 1].z, w[2 * h + 1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t o[4];
          w4_expand(q[i], zero[(2 * h + i / 4) / GC], o);
#pragma unroll
          for (int j = 0; j < 4; ++j) e[4 * i + j] = o[j];
        }
        tmem_st_32x32b_x32(to + h * 32, e);
      }
      tmem_wait_st();
      ptx::tc_fence_before();
      ptx::fence_proxy_async_smem();
      __syncwarp();
      // The codes' stage goes back when what was made of it has been stored.
      // Handed back right behind the reads, without the fence and before the
      // wait for the operand's stage, it was overwritten while rows of it were
      // still to be read.
      if (lane == 0) {
        ptx::mbar_arrive(a_full(ra.s));
        ptx::mbar_arrive(code_empty(rc.s));
      }
    }
  } else if (warp >= 4 + EW) {
    // ---------------------------------------------------------- fold
    constexpr int COLS = C::kCols, PART = COLS < 32 ? COLS : 32;  // PART: columns in registers at a time
    const int r = (warp & 3) * 32 + lane, col0 = ((warp - 4 - EW) >> 2) * COLS;
    const long long j = min(w4_column(p, tile, r, kRows), p.n - 1);
    const uint16_t* const s_row = p.scales + j * p.lds;
    const int groups = (p.k + GC * 32 - 1) / (GC * 32);
    // scales of the groups of AHEAD steps
    constexpr int AHEAD = GROUPS == 1 ? 4 : GROUPS == 2 ? 2 : 1, KEEP = AHEAD * GROUPS;
    uint16_t s_next[KEEP];
    auto fetch = [&](int b) {
#pragma unroll
      for (int i = 0; i < KEEP; ++i) {
        s_next[i] = s_row[min(b * GROUPS + i, groups - 1)];  // past the last group A is zero
      }
    };
    fetch(b0);
    float s[KEEP];
    Ring<C::kXStages> rx;
    Ring<C::kAStages> ra;
    Ring<C::kDStages> rd;
#pragma unroll 1
    for (int b = b0; b < b1; ++b, rx.next(), ra.next(), rd.next()) {
      if ((b - b0) % AHEAD == 0) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) s[i] = w4_f32<BF16>(s_next[i]);
        fetch(b + AHEAD);
      } else {
#pragma unroll
        for (int i = 0; i + GROUPS < KEEP; ++i) s[i] = s[i + GROUPS];
      }
      {
        const bool x = ptx::mbar_try_wait(x_full(rx.s), rx.ph), d = ptx::mbar_try_wait(d_full(rd.s), rd.ph);
        if (!__all_sync(0xFFFFFFFFu, x && d) &&
            !(wait_warp(x_full(rx.s), rx.ph, p, 2) && wait_warp(d_full(rd.s), rd.ph, p, 2)))
          break;
      }
      ptx::tc_fence_after();
      if (C::kAhead && warp == 4 + EW) {  // the step's operand has been multiplied; one warp says so
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(a_empty(ra.s));
      }
      const uint32_t from =
          tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::kDAt + rd.s * C::kDCols + col0;
#pragma unroll
      for (int i = 0; i < GROUPS * COLS / PART; ++i) {
        const int grp = i / (COLS / PART), c0 = i % (COLS / PART) * PART;
        uint32_t acc[PART];
        tmem_ld<PART>(from + grp * MT + c0, acc);
        tmem_ready<PART>(acc);
        if (i + 1 == GROUPS * COLS / PART) {  // all of the step has been read
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(d_empty(rd.s));
        }
        const uint64_t s2 = pair(s[grp], s[grp]);
        const uint32_t units = unit_at(rx.s) + (grp * MT + col0 + c0) * 4;
#pragma unroll
        for (int q = 0; q < PART / 4; ++q) {
          const uint4 x = ring_read(units + q * 16);
          uint64_t* const to = sum + c0 / 2 + 2 * q;
          const uint64_t u0 = pair(__uint_as_float(x.x), __uint_as_float(x.y));
          const uint64_t u1 = pair(__uint_as_float(x.z), __uint_as_float(x.w));
          to[0] = fma2(s2, mul2(u0, pair(__uint_as_float(acc[4 * q]), __uint_as_float(acc[4 * q + 1]))), to[0]);
          to[1] = fma2(s2, mul2(u1, pair(__uint_as_float(acc[4 * q + 2]), __uint_as_float(acc[4 * q + 3]))), to[1]);
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(x_empty(rx.s));
    }
  }

  // The sums of the tile, [row of A][row of the tile], over the rings: every
  // load has landed and every product is done.
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
  float* const part = reinterpret_cast<float*>(base_ptr);
  if (warp >= 4 + EW) {
    const int r = (warp & 3) * 32 + lane, col0 = ((warp - 4 - EW) >> 2) * C::kCols;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(sum) / 8); ++i) {
      float lo, hi;
      asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(sum[i]));
      part[(col0 + 2 * i) * kRows + r] = lo;
      part[(col0 + 2 * i + 1) * kRows + r] = hi;
    }
  }
  // no CTA ends before the pre-pass: what follows in the stream may write A and
  // the workspace
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  __syncwarp();
  if (slices > 1) ptx::cluster_sync();
  const int mt = min(MT, p.m - m0);
  const int oct_log2 = glu ? 3 : 4;  // eights of columns of C of a tile
  bool infinite = false;
  for (int e = threadIdx.x + rank * kThreads; e < (mt << oct_log2); e += kThreads * slices) {
    const int i = e >> oct_log2, o = (e & ((1 << oct_log2) - 1)) * 8;
    const long long j = static_cast<long long>(tile) * (8 << oct_log2) + o;
    const int row = glu ? o * 2 : o;
    if (j >= p.n_out) continue;
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !glu) break;
      const uint32_t here = ptx::smem_u32(part + i * kRows + row + 8 * h);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[h][q] = 0.0f;
      for (int from = 0; from < slices; ++from) {
        const uint32_t at = slices > 1 ? ptx::mapa(here, from) : here;
#pragma unroll
        for (int q = 0; q < 8; q += 4) {
          const float4 x = slices > 1 ? ld_cluster_f32x4(at + 4 * q)
                                      : *reinterpret_cast<const float4*>(part + i * kRows + row + 8 * h + q);
          v[h][q] += x.x, v[h][q + 1] += x.y, v[h][q + 2] += x.z, v[h][q + 3] += x.w;
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const long long col = j + q + static_cast<long long>(h) * p.n_out;
        const float s = v[h][q] * static_cast<float>(1 << kW4Up);
        if (j + q < p.n_out) {
          infinite |= isinf(s);
          v[h][q] = p.alpha * s + (p.bias ? w4_f32<BF16>(p.bias[col]) : 0.0f);
        }
      }
    }
    uint32_t out[4];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float y = glu ? w4_silu(v[0][q]) * v[1][q] : p.epi == kEpiSilu ? w4_silu(v[0][q]) : v[0][q];
      const uint32_t bits = BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : __half_as_ushort(__float2half_rn(y));
      if (q & 1)
        out[q >> 1] |= bits << 16;
      else
        out[q >> 1] = bits;
    }
    uint16_t* const dst = p.c + (m0 + i) * p.ldc + j;
    if (j + 8 <= p.n_out && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (j + q < p.n_out) dst[q] = static_cast<uint16_t>(out[q >> 1] >> (16 * (q & 1)));
    }
  }
  if (__syncthreads_or(infinite))
    store_wild<BF16>(p, tile, m0, mt, rank, reinterpret_cast<int*>(base_ptr + MT * kRows * 4));
  if (slices > 1) ptx::cluster_sync();  // no CTA leaves while its sums may be read
}

// A's row blockIdx.x as scaled fp16 in the order of the codes' pairs, with the
// units of its groups.
template <bool BF16, int GC>
__global__ void __launch_bounds__(256) w4_pack_kernel(const __grid_constant__ W4Params p) {
  constexpr int LANES = GC * 4;  // of a group: 8 values each
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long m = blockIdx.x;
  const int runs = p.k_pad / 8;  // a multiple of 16
  auto fetch = [&](int run) {
    const int k0 = run * 8;
    const uint16_t* const src = p.a + m * p.lda + k0;
    if (k0 + 8 <= p.k) return *reinterpret_cast<const uint4*>(src);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k0 + j < p.k) w[j >> 1] |= static_cast<uint32_t>(src[j]) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  for (int run0 = threadIdx.x & ~31; run0 < runs; run0 += 256) {
    const int run = run0 + (threadIdx.x & 31);
    const uint4 x = run < runs ? fetch(run) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    const uint32_t two = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                  __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
    uint32_t most = max(two & 0xFFFFu, two >> 16);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    if (run >= runs) continue;
    const int e = w4_shift<BF16>(most);
    const float f = w4_pow2(e);
    if (run % LANES == 0) p.units[static_cast<long long>(run / LANES) * p.m_pad + m] = w4_unit(e);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = w4_f32<BF16>(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = __floats2half2_rn(v[j] * f, v[j + 4] * f);
      out[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p.x + m * p.k_pad + run * 8) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

int m_tile(long long m, int group) {
  const int most = kMostRows[group / 64];
  int t = 16;
  while (t < m && t < most) t *= 2;
  return t;
}

template <bool BF16, int MT, int GC>
cudaError_t launch_main(const W4Params& p, const cudaLaunchConfig_t& cfg) {
  auto kernel = w4mm_kernel<BF16, MT, GC>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<MT, 4 / GC>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = cfg;
  c.dynamicSmemBytes = Cfg<MT, 4 / GC>::kSmem;
  return cudaLaunchKernelEx(&c, kernel, p);
}

template <bool BF16, int GC>
cudaError_t launch_of(W4Params p, int num_sms, cudaStream_t stream) {
  const int mt = m_tile(p.m, p.group);
  const int per_tile = p.epi == kEpiSwiglu ? kRows / 2 : kRows;
  const long long tiles = (p.n_out + per_tile - 1) / per_tile, tiles_m = (p.m + mt - 1) / mt;
  const int blocks = (p.k + kBlock - 1) / kBlock;
  // Slices of K, a CTA of a cluster each: the number that takes the fewest
  // steps over all waves, a CTA's fixed costs (fill, meeting, epilogue) counted
  // as six steps.
  double best = 0.0;
  for (int s = 1; s <= 8; ++s) {
    if (s > 1 && blocks / s < 4) break;
    const long long waves = (tiles * tiles_m + num_sms / s - 1) / (num_sms / s);
    const double cost = static_cast<double>(waves) * ((blocks + s - 1) / s + 6.0);
    if (s == 1 || cost < best) best = cost, p.slices = s;
  }
  p.slice = (blocks + p.slices - 1) / p.slices;
  w4_pack_kernel<BF16, GC><<<static_cast<unsigned>(p.m), 256, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.slices), static_cast<unsigned>(tiles_m));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(p.slices);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.slices > 1 ? 2 : 1;
  if (mt == 16) return launch_main<BF16, 16, GC>(p, cfg);
  if (mt == 32) return launch_main<BF16, 32, GC>(p, cfg);
  if constexpr (GC >= 2) {
    if (mt == 64) return launch_main<BF16, 64, GC>(p, cfg);
  }
  if constexpr (GC >= 4) {
    if (mt == 128) return launch_main<BF16, 128, GC>(p, cfg);
  }
  return cudaErrorInvalidValue;
}

// The workspace: packed A, then the groups' units.
struct Layout {
  size_t x, units, end;
  long long k_pad, m_pad;
};
Layout layout(long long m, long long k, int group) {
  Layout l;
  l.k_pad = (k + kBlock - 1) / kBlock * kBlock;
  const int mt = m_tile(m, group);
  l.m_pad = (m + mt - 1) / mt * mt;
  l.x = 0;
  l.units = static_cast<size_t>(m) * l.k_pad * 2;  // rows of a multiple of 256 bytes
  l.end = l.units + static_cast<size_t>(l.k_pad / group) * l.m_pad * 4;
  return l;
}

}  // namespace

size_t w4_workspace(long long m, long long k, int group) {
  return m <= kW4FewRows || k == 0 ? 0 : layout(m, k, group).end;
}

cudaError_t launch_w4mm(const W4Params& all, void* workspace, int num_sms, cudaStream_t stream) {
  W4Params p = all;
  const Layout l = layout(p.m, p.k, p.group);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  p.x = reinterpret_cast<uint16_t*>(ws + l.x);
  p.units = reinterpret_cast<float*>(ws + l.units);
  p.k_pad = static_cast<int>(l.k_pad);
  p.m_pad = l.m_pad;
  if (!encode_map_2d(&p.tmap_w, p.w, 1, static_cast<uint64_t>(p.k + 1) / 2, static_cast<uint64_t>(p.n),
                     static_cast<uint64_t>(p.n > 1 ? p.ldw : ((p.k + 1) / 2 + 15) / 16 * 16), 64, 64) ||
      !encode_map_2d(&p.tmap_x, p.x, 2, static_cast<uint64_t>(l.k_pad), static_cast<uint64_t>(p.m),
                     static_cast<uint64_t>(l.k_pad) * 2, 64, static_cast<uint32_t>(m_tile(p.m, p.group))))
    return cudaErrorInvalidValue;
  switch ((p.is_bf16 ? 4 : 0) + p.group / 64) {
    case 0: return launch_of<false, 1>(p, num_sms, stream);
    case 1: return launch_of<false, 2>(p, num_sms, stream);
    case 2: return launch_of<false, 4>(p, num_sms, stream);
    case 4: return launch_of<true, 1>(p, num_sms, stream);
    case 5: return launch_of<true, 2>(p, num_sms, stream);
    default: return launch_of<true, 4>(p, num_sms, stream);
  }
}

}  // namespace fgemm
