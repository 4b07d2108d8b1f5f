// fgemm_kern_w4.cu -- products with 4-bit weights and group scales, read
// straight from their codes.
//
//   C[i][j] = epi(alpha * sum_k A[i][k] (q[j][k] - z[j][k/G]) s[j][k/G] + bias[j])
//
// Codes q (0..15) lie along K, two to a byte, the even k in the low half.
// A few rows of A (a decode step's tokens) against all of W: bound by
// reading the codes, 0.5 byte a weight.
//
// The codes are never turned into weights.  q goes into the top mantissa
// bits of a 16-bit 1.0, which makes 1 + q/16 (exact in fp16 and bf16) in one
// shift and one logical operation for two codes, and the tensor cores sum
//   acc = sum_k (1 + q/16) x,   sx = sum_k x      (fp32, over one group)
// from which the group's part of the product is
//   sum_k (q - z) s x = 16 s (acc - (1 + z/16) sx),
// added to the running fp32 sum.  No weight is rounded, and scales and zero
// points cost a few operations a group instead of one a weight.  sx comes
// from one more tensor-core product with a matrix of ones, in the register
// layout of acc.  An infinite or NaN x makes acc - sx meaningless: an output
// that is not finite is computed again term by term (w4_exact).
//
// mma.sync with the codes as the 16-row operand and 8 rows of A as the other:
// the operand goes from the ring in shared memory through registers, where
// it is expanded, into the tensor core, with no second trip through shared
// memory as tcgen05 operands would take; at 8 rows of A its rate is not the
// bound.
//
// Each warp takes every eighth block of 256 k of the CTA's 16 R columns of C
// with a ring of its own (cp.async, three blocks), so warps never wait for
// each other until their sums meet in shared memory, once a tile.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_internal.h"
#include "fgemm_ptx.cuh"

namespace fgemm {

namespace {

constexpr int kW4Warps = 8;
constexpr int kW4Block = 256;  // k of one ring slot: 128 bytes of codes a row

// 16 bytes global -> shared; bytes past `valid` (0..16) are zero and not read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a)
               : "memory");
  return v;
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF16>
__device__ __forceinline__ float w4_f32(uint16_t v) {
  if (BF16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
  return __half2float(__ushort_as_half(v));
}

// The eight codes of a word as 1 + q/16, in pairs: p[i] holds code i in its
// low half and code i + 4 in its high half.
template <bool BF16>
__device__ __forceinline__ void expand(uint32_t w, uint32_t (&p)[4]) {
  constexpr uint32_t one = BF16 ? 0x3F803F80u : 0x3C003C00u;
  constexpr uint32_t mask = BF16 ? 0x00780078u : 0x03C003C0u;
  constexpr int top = BF16 ? 3 : 6;  // where a code's low bit goes
  p[0] = ((w << top) & mask) | one;
  p[1] = (top >= 4 ? (w << (top >= 4 ? top - 4 : 0)) & mask : (w >> (top >= 4 ? 0 : 4 - top)) & mask) | one;
  p[2] = ((w >> (8 - top)) & mask) | one;
  p[3] = ((w >> (12 - top)) & mask) | one;
}

__device__ __forceinline__ float w4_silu(float v) { return v / (1.0f + __expf(-v)); }

// Column j of W against row i of A, term by term.
template <bool BF16>
__device__ __noinline__ float w4_exact(const W4Params& p, long long i, long long j) {
  float sum = 0.0f;
  for (int k = 0; k < p.k; ++k) {
    const int q = (p.w[j * p.ldw + (k >> 1)] >> (4 * (k & 1))) & 15;
    const int g = k / p.group;
    const float z = p.zeros ? static_cast<float>(p.zeros[j * p.ldz + g]) : 8.0f;
    sum += w4_f32<BF16>(p.a[i * p.lda + k]) * ((static_cast<float>(q) - z) * w4_f32<BF16>(p.scales[j * p.lds + g]));
  }
  return sum;
}

// The column of W that virtual row r (0 .. 16 R - 1) of a tile stands for.
// SwiGLU: rows 0-7 of each 16 are gate columns and rows 8-15 the up columns
// they pair with, so that a tile yields 8 R outputs.
__device__ __forceinline__ int w4_column(const W4Params& p, int tile, int r, int rows) {
  if (p.epi != kEpiSwiglu) return tile * rows + r;
  const int j = tile * (rows / 2) + (r >> 4) * 8 + (r & 7);
  return j >= p.n_out ? p.n : (r & 8) ? p.n_out + j : j;
}

template <bool BF16, int R, int NT, int STAGES, int GC>  // GC: group / 32
__global__ void __launch_bounds__(kW4Warps * 32) w4_kernel(const __grid_constant__ W4Params p) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int ROWS = 16 * R;
  constexpr int GROUPS = 8 / GC;                       // groups of a block
  constexpr int PER = GROUPS > 4 ? GROUPS / 4 : 1;     // of them, a lane's
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int m0 = blockIdx.y * (8 * NT);
  const int mt = min(p.m - m0, 8 * NT);
  const uint32_t a_bytes = static_cast<uint32_t>(p.m_tile) * 512;
  const uint32_t slot_bytes = ROWS * 128 + a_bytes;
  float* red = reinterpret_cast<float*>(smem);  // [warp][row][8 NT + 1]
  constexpr int kPitch = 8 * NT + 1;
  const uint32_t ring = ptx::smem_u32(smem) + ((kW4Warps * ROWS * kPitch * 4 + 127) / 128 * 128) +
                        static_cast<uint32_t>(warp) * STAGES * slot_bytes;
  const int w_bytes = (p.k + 1) / 2;
  const int groups = (p.k + p.group - 1) / p.group;

  // this warp's blocks: (tile, kb), kb = warp, warp + 8, ... of each tile
  int load_tile = blockIdx.x, load_kb = warp, load_slot = 0;
  if (load_kb >= p.k_blocks) load_tile = p.tiles;
  auto issue = [&]() {
    if (load_tile < p.tiles) {
      const uint32_t slot = ring + static_cast<uint32_t>(load_slot) * slot_bytes;
      // codes: 16-byte chunk c of row r at chunk c ^ (r & 7)
#pragma unroll
      for (int i = 0; i < ROWS / 4; ++i) {
        const int r = i * 4 + (lane >> 3), c = lane & 7;
        const int col = w4_column(p, load_tile, r, ROWS);
        const int byte = load_kb * 128 + c * 16;
        const int valid = col < p.n ? max(0, min(16, w_bytes - byte)) : 0;
        const uint8_t* src = valid > 0 ? p.w + col * p.ldw + byte : p.w;
        cp_async16(slot + r * 128 + ((c ^ (r & 7)) << 4), src, valid);
      }
      // rows of A: chunk c of row r at chunk c ^ 4 (r & 1)
      for (int r = 0; r < mt; ++r) {
        const int k0 = load_kb * kW4Block + lane * 8;
        const int valid = max(0, min(16, (p.k - k0) * 2));
        const uint16_t* src = valid > 0 ? p.a + (m0 + r) * p.lda + k0 : p.a;
        cp_async16(slot + ROWS * 128 + r * 512 + ((lane ^ ((r & 1) << 2)) << 4), src, valid);
      }
      load_slot = load_slot + 1 == STAGES ? 0 : load_slot + 1;
      load_kb += kW4Warps;
      if (load_kb >= p.k_blocks) {
        load_kb = warp;
        load_tile += gridDim.x;
      }
    }
    cp_async_commit();  // possibly empty: the count of groups stays in step
  };
  // scales and zero points of a block: lane t of a quad holds groups t PER ..
  // of its row's GROUPS (lanes past GROUPS / PER repeat)
  struct Scales {
    float s[2 * R][PER], z[2 * R][PER];
  };
  auto fetch = [&](Scales& v, int tile, int kb) {
#pragma unroll
    for (int r = 0; r < 2 * R; ++r) {
      const long long col = w4_column(p, tile, (r >> 1) * 16 + (r & 1) * 8 + g, ROWS);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int gi = kb * GROUPS + (t * PER + i) % GROUPS;
        const bool ok = col < p.n && gi < groups;
        v.s[r][i] = ok ? 16.0f * w4_f32<BF16>(p.scales[col * p.lds + gi]) : 0.0f;
        v.z[r][i] = ok && p.zeros ? 1.0f + 0.0625f * static_cast<float>(p.zeros[col * p.ldz + gi]) : 1.5f;
      }
    }
  };

#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) issue();
  int slot_i = 0;
  const uint32_t ones[4] = {BF16 ? 0x3F803F80u : 0x3C003C00u, BF16 ? 0x3F803F80u : 0x3C003C00u,
                            BF16 ? 0x3F803F80u : 0x3C003C00u, BF16 ? 0x3F803F80u : 0x3C003C00u};

  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    float sum[R][NT][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[r][n][i] = 0.0f;

    Scales next;
    if (warp < p.k_blocks) fetch(next, tile, warp);
    for (int kb = warp; kb < p.k_blocks; kb += kW4Warps) {
      const Scales sc = next;
      if (kb + kW4Warps < p.k_blocks) fetch(next, tile, kb + kW4Warps);
      cp_async_wait<STAGES - 2>();
      __syncwarp();  // every lane's copies are in, and every lane is done with the slot that is filled next
      issue();
      const uint32_t slot = ring + static_cast<uint32_t>(slot_i) * slot_bytes;
      slot_i = slot_i + 1 == STAGES ? 0 : slot_i + 1;
#pragma unroll
      for (int grp = 0; grp < GROUPS; ++grp) {
        float acc[R][NT][4], sx[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sx[n][i] = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) acc[r][n][i] = 0.0f;
          }
#pragma unroll
        for (int cc = 0; cc < GC; ++cc) {
          const int c = grp * GC + cc;
          uint32_t b[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (8 * n + g < mt)
              x = lds128(slot + ROWS * 128 + (8 * n + g) * 512 + (((4 * c + t) ^ ((g & 1) << 2)) << 4));
            b[n][0] = __byte_perm(x.x, x.z, 0x5410);
            b[n][1] = __byte_perm(x.x, x.z, 0x7632);
            b[n][2] = __byte_perm(x.y, x.w, 0x5410);
            b[n][3] = __byte_perm(x.y, x.w, 0x7632);
            mma16816<BF16>(sx[n], ones, b[n][0], b[n][1]);
            mma16816<BF16>(sx[n], ones, b[n][2], b[n][3]);
          }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint32_t at = slot + (r * 16 + g) * 128 + ((c ^ g) << 4) + t * 4;
            uint32_t lo[4], hi[4];
            expand<BF16>(lds32(at), lo);
            expand<BF16>(lds32(at + 1024), hi);
            const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816<BF16>(acc[r][n], a0, b[n][0], b[n][1]);
              mma16816<BF16>(acc[r][n], a1, b[n][2], b[n][3]);
            }
          }
        }
        const int from = (lane & ~3) | (grp / PER);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float s0 = __shfl_sync(0xFFFFFFFFu, sc.s[2 * r][grp % PER], from);
          const float s1 = __shfl_sync(0xFFFFFFFFu, sc.s[2 * r + 1][grp % PER], from);
          const float z0 = __shfl_sync(0xFFFFFFFFu, sc.z[2 * r][grp % PER], from);
          const float z1 = __shfl_sync(0xFFFFFFFFu, sc.z[2 * r + 1][grp % PER], from);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            sum[r][n][0] = fmaf(s0, fmaf(-z0, sx[n][0], acc[r][n][0]), sum[r][n][0]);
            sum[r][n][1] = fmaf(s0, fmaf(-z0, sx[n][1], acc[r][n][1]), sum[r][n][1]);
            sum[r][n][2] = fmaf(s1, fmaf(-z1, sx[n][2], acc[r][n][2]), sum[r][n][2]);
            sum[r][n][3] = fmaf(s1, fmaf(-z1, sx[n][3], acc[r][n][3]), sum[r][n][3]);
          }
        }
      }
    }

    // the warps' sums meet in shared memory and are added in warp order
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[(warp * ROWS + r * 16 + g + (i >> 1) * 8) * kPitch + 8 * n + 2 * t + (i & 1)] = sum[r][n][i];
    __syncthreads();
    const bool glu = p.epi == kEpiSwiglu;
    const int outs = glu ? ROWS / 2 : ROWS;
    for (int e = threadIdx.x; e < outs * mt; e += kW4Warps * 32) {
      const int i = e / outs, o = e % outs;
      const int row = glu ? (o >> 3) * 16 + (o & 7) : o;
      const int j = tile * outs + o;
      if (j >= p.n_out) continue;
      float v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !glu) break;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kW4Warps; ++w) s += red[(w * ROWS + row + 8 * h) * kPitch + i];
        const long long col = j + static_cast<long long>(h) * p.n_out;
        if (!isfinite(s)) s = w4_exact<BF16>(p, m0 + i, col);
        v[h] = p.alpha * s + (p.bias ? w4_f32<BF16>(p.bias[col]) : 0.0f);
      }
      const float out = glu ? w4_silu(v[0]) * v[1] : p.epi == kEpiSilu ? w4_silu(v[0]) : v[0];
      p.c[(m0 + i) * p.ldc + j] = BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(out))
                                       : __half_as_ushort(__float2half_rn(out));
    }
    __syncthreads();
  }
  cp_async_wait<0>();
}

template <bool BF16, int R, int NT, int STAGES, int GC>
cudaError_t launch_w4_of(W4Params p, int num_sms, cudaStream_t stream) {
  constexpr int rows = 16 * R;
  const int per_tile = p.epi == kEpiSwiglu ? rows / 2 : rows;
  p.tiles = (p.n_out + per_tile - 1) / per_tile;
  p.k_blocks = (p.k + kW4Block - 1) / kW4Block;
  p.m_tile = p.m < 8 * NT ? p.m : 8 * NT;
  const size_t smem = (kW4Warps * rows * (8 * NT + 1) * 4 + 127) / 128 * 128 +
                      static_cast<size_t>(kW4Warps) * STAGES * (rows * 128 + static_cast<size_t>(p.m_tile) * 512);
  auto kernel = w4_kernel<BF16, R, NT, STAGES, GC>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int resident = static_cast<int>(227 * 1024 / (smem + 1024));
  const long long slots = static_cast<long long>(num_sms) * (resident < 1 ? 1 : resident > 4 ? 4 : resident);
  const dim3 grid(static_cast<unsigned>(p.tiles < slots ? p.tiles : slots),
                  static_cast<unsigned>((p.m + 8 * NT - 1) / (8 * NT)));
  kernel<<<grid, kW4Warps * 32, smem, stream>>>(p);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_w4_type(const W4Params& p, int num_sms, cudaStream_t stream) {
#define FGEMM_W4_GROUP(R, NT, ST)                                        \
  (p.group == 32    ? launch_w4_of<BF16, R, NT, ST, 1>(p, num_sms, stream) \
   : p.group == 64  ? launch_w4_of<BF16, R, NT, ST, 2>(p, num_sms, stream) \
                    : launch_w4_of<BF16, R, NT, ST, 4>(p, num_sms, stream))
  if (p.m > 8) return FGEMM_W4_GROUP(2, 2, 2);
  return FGEMM_W4_GROUP(2, 1, 3);
#undef FGEMM_W4_GROUP
}

}  // namespace

cudaError_t launch_w4(const W4Params& all, int num_sms, cudaStream_t stream) {
  constexpr int kSlab = 65535 * 8;  // rows of one launch: tiles of at least 8 along a grid dimension of at most 65535
  for (long long m0 = 0; m0 < all.m; m0 += kSlab) {
    W4Params p = all;
    p.a += m0 * p.lda;
    p.c += m0 * p.ldc;
    p.m = all.m - m0 < kSlab ? static_cast<int>(all.m - m0) : kSlab;
    const cudaError_t e = p.is_bf16 ? launch_w4_type<true>(p, num_sms, stream) : launch_w4_type<false>(p, num_sms, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace fgemm
