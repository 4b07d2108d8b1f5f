// fgemm_kern_w4.cu -- products with 4-bit weights and group scales, read
// straight from their codes.
//
//   C[i][j] = epi(alpha * sum_k A[i][k] (q[j][k] - z[j][k/G]) s[j][k/G] + bias[j])
//
// Codes q (0..15) lie along K, two to a byte, the even k in the low half.
// A few rows of A (a decode step's tokens) against all of W: bound by
// reading the codes, 0.5 byte a weight.
//
// The codes are never turned into weights: the scale of a group is applied to
// the fp32 sums of its codes,
//   sum_k (q - z) s x = s acc,   acc = sum_k (q - z) x,
// so no weight is rounded, and scales cost a few operations a group instead of
// one a weight.
//
// A code is an fp16 number as it stands: four bits at the bottom of one are the
// subnormal q 2^-24, four bits above them q 2^-20, so one logical operation and one
// multiply-add make two operands (q - z) 2^-9, exactly, and one shift serves four
// (w4_expand).  (The zero point taken off the group's sum, as z sum_k x, left 2^-24
// of z times an activation whose weight is 0: with one of them 2^20 times the rest,
// hundreds of times the error of the sum itself.)  A too is held as fp16, scaled
// by a power of two for each row and group (the largest value below 2^15), bf16
// as well: its 8 significant bits fit, and what falls below fp16's range is under
// 2^-39 of the group's largest value.
// Where a CTA has met an infinite scale, outputs that are not finite are computed
// again term by term (w4_exact).
//
// What bounds it: latency, from the codes' arrival to the tile's last sum.
// 5 x 28672 x 4096, SwiGLU, bf16, groups of 128: 20.6 us, 3.0 TB/s; one row 4096 x
// 4096: 6.7 us.  Measured on the first of these on the way: codes turned into
// 1 + q/16 with a ring a warp 34.3 us, two teams to a CTA 27.4, codes as
// subnormals 21.9, A loaded once and scales folded a group at a time 19.2, the
// zero point off each code 20.6.
//
// mma.sync with the codes as the 16-row operand and 8 rows of A as the other:
// the operand goes from the ring in shared memory through registers, where
// it is expanded, into the tensor core, with no second trip through shared
// memory as tcgen05 operands would take; at 8 rows of A its rate is not the
// bound.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_internal.h"
#include "fgemm_ptx.cuh"
#include "fgemm_w4.cuh"

namespace fgemm {

namespace {

constexpr int kW4Warps = 8;     // of a team, which works on one tile
constexpr int kW4Teams = 2;     // of a CTA; they share A
constexpr int kW4Threads = kW4Teams * kW4Warps * 32;
constexpr int kW4Rows = 32;    // rows of W (columns of C) of a tile
constexpr int kW4Block = 128;  // k of one ring slot: 64 bytes of codes a row
constexpr int kW4Stages = 3;
// Of A in shared memory; finer groups have more scales beside it.
template <int GC>
constexpr int kW4ABytes = (GC > 1 ? 64 : 48) * 1024;

// Shared memory of a CTA: the rings of codes and of scales, A's `chunk` values
// of m rows with the units of their groups (32 bytes a group whatever m is,
// half as much as A itself for one row in groups of 32), the warps' and teams'
// sums, a word.
constexpr size_t kW4MostSmem = 227 * 1024;
template <int GC>
constexpr size_t w4_few_fixed(int m) {
  return static_cast<size_t>(kW4Teams * kW4Warps) * kW4Stages * kW4Rows * (64 + 4 / GC * 8) +
         static_cast<size_t>(kW4Teams * (kW4Warps + 2)) * kW4Rows * m * 4 + 16;
}
template <int GC>
constexpr size_t w4_few_smem(int m, int chunk) {
  return w4_few_fixed<GC>(m) + static_cast<size_t>(chunk) * 2 * m + static_cast<size_t>(chunk / (GC * 32)) * 32;
}
// Most k of A a CTA keeps: A's own bound, and what is left beside the rest.
template <int GC>
constexpr int w4_most_chunk(int m) {
  const size_t left = (kW4MostSmem - w4_few_fixed<GC>(m)) * (GC * 32) / (2 * m * GC * 32 + 32);
  const size_t own = kW4ABytes<GC> / (2 * m);
  return static_cast<int>((left < own ? left : own) / 256 * 256);
}
template <int GC>
constexpr bool w4_few_fits() {
  for (int m = 1; m <= kW4FewRows; ++m)
    if (w4_most_chunk<GC>(m) < 8 * kW4Block || w4_few_smem<GC>(m, w4_most_chunk<GC>(m)) > kW4MostSmem) return false;
  return true;
}
static_assert(w4_few_fits<1>() && w4_few_fits<2>() && w4_few_fits<4>(), "shared memory, for every number of rows");

// 16 bytes global -> shared; bytes past `valid` (0..16) are zero and not read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The few-rows kernel: tiles of 32 rows of W against all (at most 8) rows
// of A.
//
// A sits in shared memory for as long as the CTA lives (when it fits; else a
// chunk of K at a time), its values already in the order in which expand()
// pairs codes, with the unit of each group beside it.  The codes stream
// through a ring of the warp's own: warp w of a team takes the blocks w,
// w + 8, ... of 128 k of a tile, so warps wait for each other once a tile,
// when their sums meet, while the blocks of the next tile are already on
// their way.  With few tiles, the CTAs of a cluster take a slice of K each and
// add their sums through distributed shared memory, in rank order.
template <bool BF16, int GC>  // GC: group / 32
__global__ void __launch_bounds__(kW4Threads, 1) w4_kernel(const __grid_constant__ W4Params p) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int R = kW4Rows / 16;
  constexpr int GROUPS = 4 / GC;  // groups of a block
  constexpr int G = GC * 32;
  const int team = threadIdx.x / (kW4Warps * 32), tid = threadIdx.x % (kW4Warps * 32);
  const int warp = tid >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int slices = p.slices;
  const int rank = slices > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int mt = p.m;
  // k of this CTA
  const int k_lo = rank * p.slice, k_hi = min(p.k, k_lo + p.slice);
  const int blocks = k_hi > k_lo ? (k_hi - k_lo + kW4Block - 1) / kW4Block : 0;
  const int chunk_blocks = p.chunk / kW4Block;

  // shared memory: the warps' rings of codes and of scales, A, its units, the warps'
  // sums, the teams' sums
  constexpr int kSlot = kW4Rows * 64, kScales = kW4Rows * GROUPS;
  unsigned char* const ring = smem + (threadIdx.x >> 5) * (kW4Stages * kSlot);
  float2* const scale_ring = reinterpret_cast<float2*>(smem + kW4Teams * kW4Warps * kW4Stages * kSlot) +
                             (threadIdx.x >> 5) * (kW4Stages * kScales);  // [group][row]: scale, w4_zero
  unsigned char* const a_at = smem + kW4Teams * kW4Warps * kW4Stages * (kSlot + kScales * 8);
  const int a_pitch = p.chunk * 2;
  float* const unit_at = reinterpret_cast<float*>(a_at + static_cast<size_t>(a_pitch) * mt);  // [group of the chunk][8]
  float* const sums_at = unit_at + p.chunk / G * 8;
  float* const red = sums_at + team * ((kW4Warps + 2) * kW4Rows * mt);  // [warp][row of A][row]
  float* const part = red + kW4Warps * kW4Rows * mt;  // [2][row of A][row], read by the cluster
  int* const wild = reinterpret_cast<int*>(sums_at + kW4Teams * ((kW4Warps + 2) * kW4Rows * mt));  // an infinite scale was met
  if (threadIdx.x == 0) *wild = 0;
  __syncthreads();
  const int w_bytes = (p.k + 1) / 2 - k_lo / 2;  // of a row, from this CTA's first
  const int groups = (p.k + G - 1) / G;
  const int tile_step = gridDim.x / slices * kW4Teams;
  const int first_tile = blockIdx.x / slices + team * (gridDim.x / slices);

  // this warp's blocks in the order it works on them: tile by tile, chunk by
  // chunk, block warp, warp + 8, ... of the chunk.  A lane copies 16 bytes of
  // four rows of a block and fetches the scales and zero points of row `lane`;
  // rows past the last repeat it, and their sums go nowhere.
  int load_tile = first_tile, load_chunk = 0, load_b = warp, load_slot = 0;
  const uint8_t* w_row[4];
  const uint16_t* s_row;
  const uint8_t* z_row;
  const int tile_rows = p.epi == kEpiSwiglu ? kW4Rows / 2 : kW4Rows;  // rows of W from one tile to the next
  auto aim = [&]() {  // the rows of load_tile
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w_row[i] = p.w + min(w4_column(p, load_tile, i * 8 + (lane >> 2), kW4Rows), p.n - 1) * p.ldw + (lane & 3) * 16 +
                 k_lo / 2;
    const long long row = min(w4_column(p, load_tile, lane, kW4Rows), p.n - 1);
    s_row = p.scales + row * p.lds;
    z_row = p.zeros + row * p.ldz;
  };
  const long long w_step = static_cast<long long>(tile_step) * tile_rows * p.ldw;
  const long long s_step = static_cast<long long>(tile_step) * tile_rows * p.lds;
  const long long z_step = static_cast<long long>(tile_step) * tile_rows * p.ldz;
  auto next_tile = [&]() {
    load_tile += tile_step;
    if (load_tile + 1 >= p.tiles) {  // perhaps a ragged one
      if (load_tile < p.tiles) aim();
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w_row[i] += w_step;
    s_row += s_step;
    z_row += z_step;
    // the first of these is read a block later
    asm volatile("prefetch.global.L2 [%0];" ::"l"(s_row + k_lo / G));
    if (p.zeros) asm volatile("prefetch.global.L2 [%0];" ::"l"(z_row + k_lo / G));
  };
  auto settle = [&]() {  // past what this warp has no block of
    while (load_chunk + load_b >= min(blocks, load_chunk + chunk_blocks)) {
      load_b = warp;
      load_chunk += chunk_blocks;
      if (load_chunk >= blocks) {
        load_chunk = 0;
        if (min(blocks, chunk_blocks) <= warp) load_tile = p.tiles;  // none in any tile
        next_tile();
        if (load_tile >= p.tiles) return;
      }
    }
  };
  // Scales are fetched with their block's codes, but through registers: they
  // are stored to the ring when the next block's are fetched, one block later,
  // so that no instruction waits for them.
  uint16_t s_next[GROUPS];
  uint32_t z_next[GROUPS];
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) s_next[i] = 0, z_next[i] = 8;
  auto issue = [&]() {
    const int before = load_slot == 0 ? kW4Stages - 1 : load_slot - 1;  // the slot of the block issued last
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      const float s = w4_f32<BF16>(s_next[i]);
      if (isinf(s)) *wild = 1;
      scale_ring[before * kScales + i * kW4Rows + lane] = make_float2(s, __uint_as_float(w4_zero(z_next[i])));
    }
    if (load_tile < p.tiles) {
      const int block = load_chunk + load_b, byte = block * (kW4Block / 2);
      // 16-byte chunk c of row r at chunk c ^ (r >> 1 & 3)
      const uint32_t dst = ptx::smem_u32(ring) + load_slot * kSlot + (lane >> 2) * 64 +
                           (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
      if (byte + kW4Block / 2 <= w_bytes) {
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16(dst + i * 512, w_row[i] + byte, 16);
      } else {
        const int valid = max(0, min(16, w_bytes - byte - (lane & 3) * 16));
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16(dst + i * 512, valid > 0 ? w_row[i] + byte : p.w, valid);
      }
      const int gi = k_lo / G + block * GROUPS;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) {
        const int at = min(gi + i, groups - 1);  // past the last group A is zero
        s_next[i] = s_row[at];
        if (p.zeros) z_next[i] = z_row[at];
      }
      load_b += kW4Warps;
      settle();
    }
    load_slot = load_slot + 1 == kW4Stages ? 0 : load_slot + 1;
    cp_async_commit();  // possibly empty: the count of groups stays in step
  };
  // Run `run` (8 values) of row m of A from k0 on; values from k_hi on are zero.
  auto fetch_run = [&](int m, int k0) {
    uint4 x = make_uint4(0, 0, 0, 0);
    const uint16_t* src = p.a + m * p.lda + k0;
    if (k0 + 8 <= k_hi) {
      x = *reinterpret_cast<const uint4*>(src);
    } else if (k0 < k_hi) {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k0 + j < k_hi) w[j >> 1] |= static_cast<uint32_t>(src[j]) << (16 * (j & 1));
      x = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return x;
  };
  // A's rows of one chunk into shared memory as scaled fp16, each run of 8
  // values in the order 0 4 1 5 2 6 3 7, and for each group its unit.
  // The G / 8 lanes that hold a group agree on its largest value.
  // begin(), once, runs between the first loads and their use.
  const int runs = p.chunk / 8;  // of a row of the chunk, a multiple of 32: a warp is in one row
  auto load_a = [&](int chunk0, auto begin) {
    constexpr int kBatch = 4;
    for (int run0 = 0; run0 < runs; run0 += kW4Threads) {
      const int run = run0 + threadIdx.x;
      for (int m0 = 0; m0 < mt; m0 += kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (run < runs && m0 + i < mt) x[i] = fetch_run(m0 + i, k_lo + chunk0 * kW4Block + run * 8);
        if (run0 == 0 && m0 == 0) begin();
        if (run >= runs) break;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int m = m0 + i;
          if (m >= mt) break;
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          const uint32_t pair = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                         __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
          uint32_t most = max(pair & 0xFFFFu, pair >> 16);
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = w4_f32<BF16>(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
#pragma unroll
          for (int o = 1; o < G / 8; o <<= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
          const int e = w4_shift<BF16>(most);
          if (run % (G / 8) == 0) unit_at[run / (G / 8) * 8 + m] = w4_unit(e);
          const float f = w4_pow2(e);
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __half2 h = __floats2half2_rn(v[j] * f, v[j + 4] * f);
            o[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          *reinterpret_cast<uint4*>(a_at + m * a_pitch + ((run ^ ((m & 1) << 2)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    __syncthreads();
  };

  if (blocks > 0 && load_tile < p.tiles) {
    aim();
    settle();
  } else {
    load_tile = p.tiles;
  }
  auto start = [&]() {
#pragma unroll
    for (int i = 0; i < kW4Stages - 1; ++i) issue();
  };
  const bool resident = chunk_blocks >= blocks;
  if (resident)
    load_a(0, start);
  else
    start();
  int slot_i = 0, side = 0;
  // A's rows as the tensor core's columns; those past mt repeat the last one
  // and their sums go nowhere.  Run 4 c + t of a block is at 4 (c ^ row % 2) + t.
  const unsigned char* a_row[2];  // by c % 2
  {
    const int m = min(g, mt - 1);
#pragma unroll
    for (int c = 0; c < 2; ++c) a_row[c] = a_at + m * a_pitch + ((4 * (c ^ (m & 1)) + t) << 4);
  }

  // A team without a last tile goes along where the CTA or the cluster meets.
  const bool meets = !resident || slices > 1;
  for (int tile = first_tile; meets ? tile - team * (gridDim.x / slices) < p.tiles : tile < p.tiles;
       tile += tile_step, side ^= 1) {
    const bool live = tile < p.tiles;
    float sum[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[r][i] = 0.0f;

    for (int chunk0 = 0; chunk0 < blocks; chunk0 += chunk_blocks) {
      if (!resident) {
        __syncthreads();  // every warp is done with the chunk before
        load_a(chunk0, [] {});
      }
      const int end = min(blocks - chunk0, chunk_blocks);
      for (int b = warp; live && b < end; b += kW4Warps) {
        cp_async_wait<kW4Stages - 2>();
        __syncwarp();  // every lane's copies are in, and every lane is done with the slot that is filled next
        issue();
        const unsigned char* slot = ring + slot_i * kSlot + g * 64 + t * 4;
        const float2* scales = scale_ring + slot_i * kScales + g;
        slot_i = slot_i + 1 == kW4Stages ? 0 : slot_i + 1;
#pragma unroll
        for (int grp = 0; grp < GROUPS; ++grp) {
          float acc[R][4];
          uint32_t zero[R][2];
#pragma unroll
          for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][i] = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) zero[r][h] = __float_as_uint(scales[grp * kW4Rows + r * 16 + h * 8].y);
          }
#pragma unroll
          for (int cc = 0; cc < GC; ++cc) {
            const int c = grp * GC + cc;
            const uint4 x = *reinterpret_cast<const uint4*>(a_row[c & 1] + b * 256 + (c >> 1) * 128);
            const unsigned char* at = slot + ((c ^ ((g >> 1) & 3)) << 4);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              uint32_t lo[4], hi[4];
              w4_expand(*reinterpret_cast<const uint32_t*>(at + r * 1024), zero[r][0], lo);
              w4_expand(*reinterpret_cast<const uint32_t*>(at + r * 1024 + 512), zero[r][1], hi);
              // the lower kind of codes in one product, the upper in the other
              const uint32_t a0[4] = {lo[0], hi[0], lo[2], hi[2]}, a1[4] = {lo[1], hi[1], lo[3], hi[3]};
              mma16816(acc[r], a0, x.x, x.z);
              mma16816(acc[r], a1, x.y, x.w);
            }
          }
          // unit of acc, of two rows of A
          const float2 unit = *reinterpret_cast<const float2*>(unit_at + (b * GROUPS + grp) * 8 + 2 * t);
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float scale = scales[grp * kW4Rows + r * 16 + h * 8].x;
              float* to = sum[r] + 2 * h;
              to[0] = fmaf(scale, acc[r][2 * h] * unit.x, to[0]);
              to[1] = fmaf(scale, acc[r][2 * h + 1] * unit.y, to[1]);
            }
        }
      }
    }

    // the warps' sums are added in warp order, then the CTAs' in rank order
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (2 * t + i < mt) {
        float* const to = red + (warp * mt + 2 * t + i) * kW4Rows + g;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          to[r * 16] = sum[r][i];
          to[r * 16 + 8] = sum[r][i + 2];
        }
      }
    ptx::named_bar_sync(1 + team, kW4Warps * 32);
    const bool glu = p.epi == kEpiSwiglu;
    const int outs_log2 = glu ? 4 : 5;  // columns of C of a tile
    if (slices > 1) {
      float* const mine = part + side * (kW4Rows * mt);
      for (int e = tid; e < kW4Rows * mt; e += kW4Warps * 32) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kW4Warps; ++w) s += red[w * mt * kW4Rows + e];
        mine[e] = s;
      }
      __syncwarp();
      // two buffers: a rank that reads this tile's sums keeps its cluster
      // from the next meeting, so nobody writes them before the one after
      ptx::cluster_sync();
    }
    for (int e = tid + rank * (kW4Warps * 32); live && e < (mt << outs_log2); e += kW4Warps * 32 * slices) {
      const int i = e >> outs_log2, o = e & ((1 << outs_log2) - 1);
      const int row = glu ? (o >> 3) * 16 + (o & 7) : o;
      const int j = (tile << outs_log2) + o;
      if (j >= p.n_out) continue;
      float v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !glu) break;
        const int at = i * kW4Rows + row + 8 * h;
        float s = 0.0f;
        if (slices > 1) {
          const uint32_t here = ptx::smem_u32(part + side * (kW4Rows * mt) + at);
          for (int q = 0; q < slices; ++q) s += ld_cluster_f32(ptx::mapa(here, q));
        } else {
#pragma unroll
          for (int w = 0; w < kW4Warps; ++w) s += red[w * mt * kW4Rows + at];
        }
        const long long col = j + static_cast<long long>(h) * p.n_out;
        s *= static_cast<float>(1 << kW4Up);
        if (!isfinite(s)) {
          int met = *wild;
          for (int q = 0; q < slices && slices > 1; ++q)
            met |= __float_as_int(ld_cluster_f32(ptx::mapa(ptx::smem_u32(wild), q)));
          if (met) s = w4_exact<BF16>(p, i, col);
        }
        v[h] = p.alpha * s + (p.bias ? w4_f32<BF16>(p.bias[col]) : 0.0f);
      }
      const float out = glu ? w4_silu(v[0]) * v[1] : p.epi == kEpiSilu ? w4_silu(v[0]) : v[0];
      p.c[i * p.ldc + j] = BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(out))
                                : __half_as_ushort(__float2half_rn(out));
    }
    if (slices == 1) ptx::named_bar_sync(1 + team, kW4Warps * 32);  // red is read
  }
  cp_async_wait<0>();
  __syncwarp();
  if (slices > 1) ptx::cluster_sync();  // no CTA leaves while its sums may be read
}

template <bool BF16, int GC>
cudaError_t launch_w4_few(W4Params p, int num_sms, cudaStream_t stream) {
  const int per_tile = p.epi == kEpiSwiglu ? kW4Rows / 2 : kW4Rows;
  p.tiles = (p.n_out + per_tile - 1) / per_tile;
  const int blocks = (p.k + kW4Block - 1) / kW4Block;
  // K is cut into slices, a CTA of a cluster each: while there are SMs without
  // a tile and every warp keeps a block, and until A's slice fits
  int slices = 1;
  const int most_chunk = w4_most_chunk<GC>(p.m);
  while (slices < 8 && blocks >= 2 * slices * kW4Warps && static_cast<long long>(p.tiles) * slices * 2 <= num_sms * kW4Teams)
    slices *= 2;
  while (slices < 8 && (blocks + slices - 1) / slices * kW4Block > most_chunk) slices *= 2;
  p.slices = slices;
  p.slice = ((blocks + slices - 1) / slices * kW4Block + 255) / 256 * 256;
  p.chunk = p.slice < most_chunk ? (p.slice > 0 ? p.slice : 256) : most_chunk;
  const size_t smem = w4_few_smem<GC>(p.m, p.chunk);
  auto kernel = w4_kernel<BF16, GC>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int clusters = num_sms / slices;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.tiles < clusters ? p.tiles : clusters) * slices));
  cfg.blockDim = dim3(kW4Threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(slices);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = slices > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool BF16>
cudaError_t launch_w4_type(const W4Params& p, int num_sms, cudaStream_t stream) {
  return p.group == 32   ? launch_w4_few<BF16, 1>(p, num_sms, stream)
         : p.group == 64 ? launch_w4_few<BF16, 2>(p, num_sms, stream)
                         : launch_w4_few<BF16, 4>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_w4(const W4Params& p, void* workspace, int num_sms, cudaStream_t stream) {
  if (p.k == 0) {
    KernelParams q{};
    q.C = p.c;
    q.ldc = p.ldc;
    q.bias = p.bias;
    q.M = p.m;
    q.N = p.n;
    q.n_out = p.n_out;
    q.epi = p.epi;
    q.is_bf16 = p.is_bf16;
    q.alpha = p.alpha;
    return launch_k0_fill(q, stream);
  }
  if (p.m > kW4FewRows) return launch_w4mm(p, workspace, num_sms, stream);
  return p.is_bf16 ? launch_w4_type<true>(p, num_sms, stream) : launch_w4_type<false>(p, num_sms, stream);
}

}  // namespace fgemm
