// fgemm_kern_norm.cu -- root-mean-square norm with the residual's addition:
// forward into 16 bits, forward into block-scaled 8 bits (MX), backward.
//
// Forward, for each row (n values, gain g):
//   t_j = round16(x_j + res_j)                (t = x without a residual)
//   r   = 1 / sqrt(mean_j t_j^2 + eps)
//   y_j = t_j r g_j                           (rounded once, on the store)
// The norm is taken of t as stored (16 bits): the next layer's residual, the
// backward pass and a recomputation all read that t, and all see the same
// norm.  Squares, sums, r and y are fp32.
// bf16 reaches further than fp32's squares do.  Where the sum of a row's squares
// overflows, or is so small with eps that squares were lost, the row is scaled
// by a power of two and summed again, and y formed from the scaled values
// (far_row).
// MX output (blocks of 32 along the row): the scale is 2^e with
// e = floor(log2 max|y|) - emax (8 for E4M3, 15 for E5M2) held to E8M0's
// range, the elements y / 2^e rounded to nearest even, those past the
// largest finite value set to it.  y goes from fp32 to 8 bits in one rounding.
//
// Backward, with u_j = t_j r and a_j = dy_j g_j:
//   dt_j = r (a_j - u_j mean_k(a_k u_k)) + dtotal_j
//   dg_j = sum over rows of dy_j u_j
// x and the residual enter through their sum, so dt is the gradient of both.
//
// Memory-bound: a row is read once into registers (16-byte loads, one row a
// CTA or, for short rows, one row a warp), reduced, and written from them.
// Measured: 8192 x 4096 bf16 with a residual into 16 bits 42.4 us, 6.3 TB/s, into
// 8-bit blocks 43.2 us, 5.5 TB/s; backward of the same with the residual's
// gradient 57.5 us, 4.7 TB/s (one row on its way a CTA: too little in flight);
// one row of 4096 3.1 us, a launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_internal.h"

namespace fgemm {

namespace {

template <bool BF16>
__device__ __forceinline__ float to_f32(uint32_t bits16) {
  if (BF16) return __uint_as_float(bits16 << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(bits16)));
}

template <bool BF16>
__device__ __forceinline__ uint32_t to_16(float v) {
  if (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// VEC consecutive 16-bit elements, two to a word (VEC 1: the low half).
template <int VEC>
struct Chunk {
  uint32_t w[(VEC + 1) / 2];
};

template <bool BF16, int VEC>
__device__ __forceinline__ float elem(const Chunk<VEC>& c, int i) {
  return to_f32<BF16>((i & 1) ? c.w[i >> 1] >> 16 : c.w[i >> 1] & 0xFFFFu);
}

// The chunk at columns [c0, c0 + VEC) of a row; columns outside [0, n) read as
// zero.  row + c0 is on 16 bytes.
template <int VEC>
__device__ __forceinline__ void load_chunk(Chunk<VEC>& c, const uint16_t* row, int c0, int n) {
  if (VEC == 1) {
    c.w[0] = c0 < n ? row[c0] : 0u;
    return;
  }
  if (c0 >= 0 && c0 + VEC <= n) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + c0);
    c.w[0] = v.x;
    c.w[1 % ((VEC + 1) / 2)] = v.y;
    c.w[2 % ((VEC + 1) / 2)] = v.z;
    c.w[3 % ((VEC + 1) / 2)] = v.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i) {
    const uint32_t lo = c0 + 2 * i >= 0 && c0 + 2 * i < n ? row[c0 + 2 * i] : 0u;
    const uint32_t hi = c0 + 2 * i + 1 >= 0 && c0 + 2 * i + 1 < n ? row[c0 + 2 * i + 1] : 0u;
    c.w[i] = lo | (hi << 16);
  }
}

// The same of a vector that is on 16 bytes itself, at any c0.
template <int VEC>
__device__ __forceinline__ void load_chunk_any(Chunk<VEC>& c, const uint16_t* v, int c0, int n) {
  if (VEC == 1 || (c0 & 7) == 0) {
    load_chunk<VEC>(c, v, c0, n);
    return;
  }
  if (c0 < 0 || c0 + 10 > n) {
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i) {
      const uint32_t lo = c0 + 2 * i >= 0 && c0 + 2 * i < n ? v[c0 + 2 * i] : 0u;
      const uint32_t hi = c0 + 2 * i + 1 >= 0 && c0 + 2 * i + 1 < n ? v[c0 + 2 * i + 1] : 0u;
      c.w[i] = lo | (hi << 16);
    }
    return;
  }
  const uint32_t* const w = reinterpret_cast<const uint32_t*>(v) + (c0 >> 1);
  uint32_t x[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) x[i] = w[i];
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i) c.w[i] = __funnelshift_r(x[i], x[i + 1], (c0 & 1) * 16);
}

template <int VEC>
__device__ __forceinline__ void store_chunk(const Chunk<VEC>& c, uint16_t* row, int c0, int n, bool vec = true) {
  if (VEC == 1) {
    if (c0 < n) row[c0] = static_cast<uint16_t>(c.w[0]);
    return;
  }
  if (vec && c0 >= 0 && c0 + VEC <= n) {
    *reinterpret_cast<uint4*>(row + c0) =
        make_uint4(c.w[0], c.w[1 % ((VEC + 1) / 2)], c.w[2 % ((VEC + 1) / 2)], c.w[3 % ((VEC + 1) / 2)]);
    return;
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    if (c0 + i >= 0 && c0 + i < n) row[c0 + i] = static_cast<uint16_t>(c.w[i >> 1] >> (16 * (i & 1)));
}

// Sum over the tpr threads of a row; every one of them gets it.  tpr is 32
// (a warp) or the whole CTA.  `red` holds 32 floats for each call site.
__device__ __forceinline__ float row_sum(float v, int tpr, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (tpr == 32) return v;
  const int warps = tpr >> 5;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The 8-bit form of one chunk of y and its block's scale.  A block of 32
// columns is held by 32 / VEC neighbouring lanes.  A block with an infinity
// or a NaN gets the NaN scale (255), so that nothing non-finite is hidden.
template <int VEC>
__device__ __forceinline__ void store_mx(const float (&y)[VEC], const NormParams& p, long long row, int c0) {
  uint32_t most = 0;  // |y| ordered by its bits: NaN above infinity above numbers
#pragma unroll
  for (int i = 0; i < VEC; ++i) most = max(most, __float_as_uint(y[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < 32 / VEC; o <<= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  if (c0 >= p.n) return;
  const int emax = p.mx_format == 0 ? 8 : 15;
  const int field = static_cast<int>(most >> 23);
  // subnormal and zero blocks: the smallest scale
  const int e = field == 255 ? 255 : max(field - emax, 0);
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - min(e, 253)) << 23);  // 2^(127 - e), exact
  if ((c0 & 31) == 0) p.scales[row * p.lds + (c0 >> 5)] = static_cast<uint8_t>(e);
  const __nv_fp8_interpretation_t f8 = p.mx_format == 0 ? __NV_E4M3 : __NV_E5M2;
  uint8_t* dst = p.q + row * p.ldq + c0;
  if (VEC == 8 && p.out_vec && c0 + VEC <= p.n) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a = __nv_cvt_float2_to_fp8x2(
          make_float2(y[(4 * h) % VEC] * inv, y[(4 * h + 1) % VEC] * inv), __NV_SATFINITE, f8);
      const uint32_t b = __nv_cvt_float2_to_fp8x2(
          make_float2(y[(4 * h + 2) % VEC] * inv, y[(4 * h + 3) % VEC] * inv), __NV_SATFINITE, f8);
      w[h] = a | (b << 16);
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    return;
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    if (c0 + i < p.n) dst[i] = __nv_cvt_float_to_fp8(y[i] * inv, __NV_SATFINITE, f8);
}

template <bool BF16, int VEC, bool MX>
__device__ __forceinline__ void finish_chunk(const NormParams& p, const Chunk<VEC>& t, float r, long long row,
                                             int c0) {
  Chunk<VEC> g;
  load_chunk_any<VEC>(g, p.gain, c0, p.n);
  float y[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) y[i] = elem<BF16, VEC>(t, i) * r * elem<BF16, VEC>(g, i);
  if (MX) {
    store_mx<VEC>(y, p, row, c0);
  } else {
    Chunk<VEC> o;
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i)
      o.w[i] = VEC == 1 ? to_16<BF16>(y[0]) : pack2<BF16>(y[(2 * i) % VEC], y[(2 * i + 1) % VEC]);
    store_chunk<VEC>(o, p.y + row * p.ldy, c0, p.n, p.out_vec);
  }
}

// t of one chunk: x, or the rounded sum with the residual, which is stored.
template <bool BF16, int VEC>
__device__ __forceinline__ void total_chunk(const NormParams& p, Chunk<VEC>& t, long long row, int c0) {
  load_chunk<VEC>(t, p.x + row * p.ldx, c0, p.n);
  if (p.res) {
    Chunk<VEC> b;
    load_chunk<VEC>(b, p.res + row * p.ldr, c0, p.n);
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i) {
      if (VEC == 1)
        t.w[0] = to_16<BF16>(elem<BF16, VEC>(t, 0) + elem<BF16, VEC>(b, 0));
      else
        t.w[i] = pack2<BF16>(elem<BF16, VEC>(t, 2 * i) + elem<BF16, VEC>(b, 2 * i),
                             elem<BF16, VEC>(t, 2 * i + 1) + elem<BF16, VEC>(b, 2 * i + 1));
    }
  }
}

// Whether a bf16 row's sum of squares is none: overflown (or infinite; a NaN is
// what it is), or so small that squares below fp32's range count (each is off
// by 2^-150 at most).
__device__ __forceinline__ bool is_far(float sum, const NormParams& p) {
  return sum == INFINITY || sum / static_cast<float>(p.n) + p.eps < 0x1p-120f;
}

// Such a row, read again element by element from the total (or x and the
// residual) behind the barrier of its sum: rare, so it is kept out of the
// kernels' registers (8192 x 4096 of 1e20: 163 us instead of 43).  A thread reads
// and writes the same columns in all passes (y may be x).
template <bool MX>
__device__ __noinline__ void far_row(const NormParams& p, long long row, int lane, int tpr) {
  __shared__ float red[32];
  __shared__ uint32_t red_most[32];
  auto value = [&](int c) {
    Chunk<1> t;
    if (p.total)
      load_chunk<1>(t, p.total + row * p.ldt, c, p.n);
    else
      total_chunk<true, 1>(p, t, row, c);
    return t.w[0];
  };
  if (tpr == 32) __syncwarp();  // the row's total, stored by other threads
  uint32_t most = 0;
  for (long long c = lane; c < p.n; c += tpr) most = max(most, value(static_cast<int>(c)) & 0x7FFFu);
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (tpr > 32) {
    if ((threadIdx.x & 31) == 0) red_most[threadIdx.x >> 5] = most;
    __syncthreads();
    most = __reduce_max_sync(0xFFFFFFFFu, (threadIdx.x & 31) < (tpr >> 5) ? red_most[threadIdx.x & 31] : 0u);
  }
  // the largest magnitude to about 2^40; nothing helps zeros, infinities and NaN
  const int k = most == 0 || most >= 0x7F80u ? 0 : min(120, 40 + 127 - static_cast<int>(most >> 7));
  const float a = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
  float sum = 0.0f;
  for (long long c = lane; c < p.n; c += tpr) {
    const float e = to_f32<true>(value(static_cast<int>(c))) * a;
    sum = fmaf(e, e, sum);
  }
  sum = row_sum(sum, tpr, red);
  const float r = 1.0f / sqrtf(sum / static_cast<float>(p.n) + p.eps * a * a);
  if (lane == 0 && p.inv_rms) p.inv_rms[row] = r * a;
  for (long long c0 = lane & ~31; c0 < p.n; c0 += tpr) {
    const int c = c0 + (lane & 31) < p.n ? static_cast<int>(c0) + (lane & 31) : p.n;
    Chunk<1> t;
    // (what a takes below bf16's range has a y below it)
    t.w[0] = to_16<true>(to_f32<true>(value(c)) * a);
    finish_chunk<true, 1, MX>(p, t, r, row, c);
  }
}

// One row on tpr = blockDim.x / rows_per_cta threads, VPT chunks a thread in
// registers.
template <bool BF16, int VEC, int VPT, bool MX, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[32];
  const int tpr = p.tpr;
  const long long row = static_cast<long long>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  if (row >= p.m) return;  // whole warps (tpr 32) or the whole CTA
  const int lane = threadIdx.x % tpr;
  // rows that do not start on 16 bytes: chunks from the boundary before them
  const int shift = VEC == 1 ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(p.x + row * p.ldx) % 16 / 2);
  Chunk<VEC> t[VPT];
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < VPT; ++v) total_chunk<BF16, VEC>(p, t[v], row, (v * tpr + lane) * VEC - shift);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c0 = (v * tpr + lane) * VEC - shift;
    if (p.total) store_chunk<VEC>(t[v], p.total + row * p.ldt, c0, p.n);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float e = elem<BF16, VEC>(t[v], i);
      sum = fmaf(e, e, sum);
    }
  }
  sum = row_sum(sum, tpr, red);
  if (BF16 && is_far(sum, p)) {
    far_row<MX>(p, row, lane, tpr);
    return;
  }
  const float r = 1.0f / sqrtf(sum / static_cast<float>(p.n) + p.eps);
  if (lane == 0 && p.inv_rms) p.inv_rms[row] = r;
  if (MX && p.shifted) {  // chunks would straddle blocks of 32: element by element
    __syncwarp();  // the row's total, stored above by other threads (a CTA's row: the sum's barrier)
    for (int c0 = lane & ~31; c0 < p.n; c0 += tpr) {
      const int c = c0 + (lane & 31) < p.n ? c0 + (lane & 31) : p.n;
      Chunk<1> one;
      if (p.total)
        load_chunk<1>(one, p.total + row * p.ldt, c, p.n);
      else
        total_chunk<BF16, 1>(p, one, row, c);
      finish_chunk<BF16, 1, MX>(p, one, r, row, c);
    }
    return;
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c0 = (v * tpr + lane) * VEC - shift;
    if ((v * tpr + (lane & ~31)) * VEC - shift < p.n)  // whole warps: a block's lanes stay together
      finish_chunk<BF16, VEC, MX>(p, t[v], r, row, c0);
  }
}

// Rows that do not fit in registers: one row a CTA, read twice (the second
// time mostly from L2).
template <bool BF16, int VEC, bool MX>
__global__ void __launch_bounds__(1024, 2) norm_long_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[32];
  const long long row = blockIdx.x;
  float sum = 0.0f;
  for (long long c = threadIdx.x; c * VEC < p.n; c += blockDim.x) {
    const int c0 = static_cast<int>(c * VEC);
    Chunk<VEC> t;
    total_chunk<BF16, VEC>(p, t, row, c0);
    if (p.total) store_chunk<VEC>(t, p.total + row * p.ldt, c0, p.n);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float e = elem<BF16, VEC>(t, i);
      sum = fmaf(e, e, sum);
    }
  }
  sum = row_sum(sum, blockDim.x, red);
  if (BF16 && is_far(sum, p)) {
    far_row<MX>(p, row, threadIdx.x, blockDim.x);
    return;
  }
  const float r = 1.0f / sqrtf(sum / static_cast<float>(p.n) + p.eps);
  if (threadIdx.x == 0 && p.inv_rms) p.inv_rms[row] = r;
  for (long long c = threadIdx.x & ~31; c * VEC < p.n; c += blockDim.x) {
    const long long mine = c + (threadIdx.x & 31);
    const int c0 = mine * VEC < p.n ? static_cast<int>(mine * VEC) : p.n;
    Chunk<VEC> t;
    if (p.total)  // this thread's own stores; x or the residual may share their memory
      load_chunk<VEC>(t, p.total + row * p.ldt, c0, p.n);
    else
      total_chunk<BF16, VEC>(p, t, row, c0);
    finish_chunk<BF16, VEC, MX>(p, t, r, row, c0);
  }
}

// Backward.  CTA b takes rows b, b + gridDim.x, ..., the next row's loads on
// their way while a row is reduced and written; a thread keeps the gain's
// gradient of its columns over them in registers and stores it to row b of the
// partials, which norm_dgain_kernel adds up in row order, so that results do
// not depend on which CTA ends first.  (Clusters that add theirs up first were
// slower: 304 CTAs in clusters of 8 do not fit the GPCs at once, 90 us for
// 8192 x 4096.)
template <bool BF16, int VEC, int VPT, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_back_kernel(const __grid_constant__ NormBackParams p) {
  __shared__ float red[2][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tpr = blockDim.x;
  float dg[VPT][VEC];
  Chunk<VEC> g[VPT], t[VPT], dy[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    load_chunk<VEC>(g[v], p.gain, (v * tpr + threadIdx.x) * VEC, p.n);
#pragma unroll
    for (int i = 0; i < VEC; ++i) dg[v][i] = 0.0f;
  }
  float r = 0.0f;
  auto fetch = [&](long long row) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c0 = (v * tpr + threadIdx.x) * VEC;
      load_chunk<VEC>(t[v], p.total + row * p.ldt, c0, p.n);
      load_chunk<VEC>(dy[v], p.dy + row * p.lddy, c0, p.n);
    }
    r = p.inv_rms[row];
  };
  const float inv_n = 1.0f / static_cast<float>(p.n);
  int side = 0;
  if (blockIdx.x < p.m) fetch(blockIdx.x);
  for (long long row = blockIdx.x; row < p.m; row += gridDim.x, side ^= 1) {
    Chunk<VEC> dt[VPT], tc[VPT], dc[VPT];  // this row's
    float dot = 0.0f;
    const float rr = r;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (p.dtotal) load_chunk<VEC>(dt[v], p.dtotal + row * p.lddt, (v * tpr + threadIdx.x) * VEC, p.n);
      tc[v] = t[v];
      dc[v] = dy[v];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float u = elem<BF16, VEC>(tc[v], i) * rr, d = elem<BF16, VEC>(dc[v], i);
        dot = fmaf(d * elem<BF16, VEC>(g[v], i), u, dot);
        dg[v][i] = fmaf(d, u, dg[v][i]);
      }
    }
    if (row + gridDim.x < p.m) fetch(row + gridDim.x);
    dot = row_sum(dot, tpr, red[side]) * inv_n;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        // r (a - u mean(a u)) with u = t r, in this order: r^2 leaves fp32's range
        // where r does not
        const float u = elem<BF16, VEC>(tc[v], i) * rr;
        const float w = fmaf(-u, dot, elem<BF16, VEC>(dc[v], i) * elem<BF16, VEC>(g[v], i));
        o[i] = p.dtotal ? fmaf(rr, w, elem<BF16, VEC>(dt[v], i)) : rr * w;
      }
      Chunk<VEC> c;
#pragma unroll
      for (int i = 0; i < (VEC + 1) / 2; ++i)
        c.w[i] = VEC == 1 ? to_16<BF16>(o[0]) : pack2<BF16>(o[(2 * i) % VEC], o[(2 * i + 1) % VEC]);
      store_chunk<VEC>(c, p.dx + row * p.lddx, (v * tpr + threadIdx.x) * VEC, p.n);
    }
  }
  if (p.partials) {
    float* dst = p.partials + static_cast<long long>(blockIdx.x) * p.n;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int c = (v * tpr + threadIdx.x) * VEC + i;
        if (c < p.n) dst[c] = dg[v][i];
      }
  }
}

// dg[c] = sum of the partials' column c, warps over slices of the rows, then
// the slices in order.
__global__ void __launch_bounds__(1024) norm_dgain_kernel(const float* partials, int rows, int n, float* dgain) {
  __shared__ float part[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the partials
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < n)
#pragma unroll 8
    for (int r = warp; r < rows; r += 32) s += partials[static_cast<long long>(r) * n + c];
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < n) {
    s = 0.0f;
    for (int w = 0; w < 32; ++w) s += part[w][lane];
    dgain[c] = s;
  }
}

// Backward of rows that do not fit in registers, first step: each row's
// mean(a u), one row a CTA.
template <bool BF16>
__global__ void __launch_bounds__(1024) norm_back_dot_kernel(const __grid_constant__ NormBackParams p) {
  __shared__ float red[32];
  const long long row = blockIdx.x;
  const float r = p.inv_rms[row];
  float dot = 0.0f;
  for (int c = threadIdx.x; c < p.n; c += blockDim.x) {
    const float u = to_f32<BF16>(p.total[row * p.ldt + c]) * r;
    dot = fmaf(to_f32<BF16>(p.dy[row * p.lddy + c]) * to_f32<BF16>(p.gain[c]), u, dot);
  }
  dot = row_sum(dot, blockDim.x, red);
  if (threadIdx.x == 0) p.dots[row] = dot / static_cast<float>(p.n);
}

// Second step: a thread takes one column of the rows blockIdx.y,
// blockIdx.y + gridDim.y, ...
template <bool BF16>
__global__ void __launch_bounds__(256) norm_back_cols_kernel(const __grid_constant__ NormBackParams p) {
  const long long c = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= p.n) return;
  const float g = to_f32<BF16>(p.gain[c]);
  float dg = 0.0f;
  for (long long row = blockIdx.y; row < p.m; row += gridDim.y) {
    const float r = p.inv_rms[row], u = to_f32<BF16>(p.total[row * p.ldt + c]) * r;
    const float d = to_f32<BF16>(p.dy[row * p.lddy + c]);
    dg = fmaf(d, u, dg);
    float o = r * fmaf(-u, p.dots[row], d * g);
    if (p.dtotal) o += to_f32<BF16>(p.dtotal[row * p.lddt + c]);
    p.dx[row * p.lddx + c] = static_cast<uint16_t>(to_16<BF16>(o));
  }
  if (p.partials) p.partials[static_cast<long long>(blockIdx.y) * p.n + c] = dg;
}

bool aligned16(const void* p, long long ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0;
}

template <bool BF16, int VEC, bool MX>
cudaError_t launch_fwd(NormParams p, cudaStream_t stream) {
  const int chunks = (p.n + VEC - 1) / VEC + (p.shifted ? 1 : 0);
  if (chunks <= 128) {  // a warp a row, four rows a CTA
    p.tpr = 32;
    const unsigned grid = static_cast<unsigned>((p.m + 3) / 4);
    if (chunks <= 32)
      norm_kernel<BF16, VEC, 1, MX, 128><<<grid, 128, 0, stream>>>(p);
    else
      norm_kernel<BF16, VEC, 4, MX, 128><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
  }
  const unsigned grid = static_cast<unsigned>(p.m);
  // 8192 x 4096 to 8 bits: two chunks a thread 43.3 us, four 44.4, eight 56.5
  if (chunks <= 2048) {
    p.tpr = (chunks + 63) / 64 * 32;
    norm_kernel<BF16, VEC, 2, MX, 1024><<<grid, p.tpr, 0, stream>>>(p);
  } else if (chunks <= 8192) {
    p.tpr = (chunks + 255) / 256 * 32;
    norm_kernel<BF16, VEC, 8, MX, 1024><<<grid, p.tpr, 0, stream>>>(p);
  } else {
    norm_long_kernel<BF16, VEC, MX><<<grid, 1024, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_fwd_of(NormParams p, cudaStream_t stream) {
  // The output's form and alignment only decide how it is stored: every form
  // comes from the same sums.
  const bool vec = aligned16(p.x, p.ldx) && aligned16(p.gain, 0) && (!p.res || aligned16(p.res, p.ldr)) &&
                   (!p.total || aligned16(p.total, p.ldt));
  // Rows that all start equally far behind a 16-byte boundary: chunks from
  // there (f16, 1537 x 5127: 19.4 us element by element).
  auto like_x = [&](const void* a, long long ld) {
    return reinterpret_cast<uintptr_t>(a) % 16 == reinterpret_cast<uintptr_t>(p.x) % 16 && (ld - p.ldx) % 8 == 0;
  };
  p.shifted = !vec && p.n <= 65528 && aligned16(p.gain, 0) && (!p.res || like_x(p.res, p.ldr)) &&
              (!p.total || like_x(p.total, p.ldt));
  p.out_vec = p.q ? reinterpret_cast<uintptr_t>(p.q) % 8 == 0 && p.ldq % 8 == 0
                  : p.shifted ? like_x(p.y, p.ldy) : aligned16(p.y, p.ldy);
  if (p.q)
    return vec || p.shifted ? launch_fwd<BF16, 8, true>(p, stream) : launch_fwd<BF16, 1, true>(p, stream);
  return vec || p.shifted ? launch_fwd<BF16, 8, false>(p, stream) : launch_fwd<BF16, 1, false>(p, stream);
}

// Columns a row of the register kernel may have.
constexpr int kBackRegs16 = 16384, kBackRegs2 = 8192;

bool back_vec(const NormBackParams& p) {
  return aligned16(p.total, p.ldt) && aligned16(p.dy, p.lddy) && aligned16(p.gain, 0) && aligned16(p.dx, p.lddx) &&
         (!p.dtotal || aligned16(p.dtotal, p.lddt));
}

template <bool BF16, int VEC, int VPT, int MAXT, int MINB>
cudaError_t launch_back_regs(const NormBackParams& p, cudaStream_t stream) {
  const int chunks = (p.n + VEC - 1) / VEC;
  norm_back_kernel<BF16, VEC, VPT, MAXT, MINB>
      <<<static_cast<unsigned>(p.ctas), static_cast<unsigned>((chunks + 32 * VPT - 1) / (32 * VPT) * 32), 0, stream>>>(p);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_back(const NormBackParams& p, cudaStream_t stream) {
  const bool vec = back_vec(p);
  cudaError_t e;
  if (vec && p.n <= kBackRegs16) {
    e = p.n <= 2048   ? launch_back_regs<BF16, 8, 1, 256, 4>(p, stream)
        : p.n <= 4096 ? launch_back_regs<BF16, 8, 1, 512, 2>(p, stream)
        : p.n <= 8192 ? launch_back_regs<BF16, 8, 2, 512, 1>(p, stream)
                      : launch_back_regs<BF16, 8, 4, 512, 1>(p, stream);
  } else if (!vec && p.n <= kBackRegs2) {
    e = p.n <= 1024 ? launch_back_regs<BF16, 1, 1, 1024, 1>(p, stream)
                    : launch_back_regs<BF16, 1, 8, 1024, 1>(p, stream);
  } else {
    norm_back_dot_kernel<BF16><<<static_cast<unsigned>(p.m), 1024, 0, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    norm_back_cols_kernel<BF16><<<dim3(static_cast<unsigned>((p.n + 255) / 256), static_cast<unsigned>(p.ctas)), 256, 0,
                                  stream>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !p.partials) return e;
  // launched while the rows are still worked on; it waits for their end
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.n + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_dgain_kernel, static_cast<const float*>(p.partials), p.ctas, p.n, p.dgain);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
  return p.is_bf16 ? launch_fwd_of<true>(p, stream) : launch_fwd_of<false>(p, stream);
}

int norm_back_ctas(long long m, int n, int num_sms) {
  // two an SM of rows up to 4096, else one; of few rows one an SM, or the partials
  // outweigh the rows
  const long long most = m >= 8ll * num_sms ? (n <= 4096 ? 2ll : 1ll) * num_sms : num_sms;
  return static_cast<int>(m < most ? m : most);
}

size_t norm_back_workspace(long long m, int n, int num_sms) {
  // the partials of the gain's gradient, then each row's mean
  return (static_cast<size_t>(norm_back_ctas(m, n, num_sms)) * static_cast<size_t>(n) + static_cast<size_t>(m)) *
         sizeof(float);
}

cudaError_t launch_norm_back(const NormBackParams& p, cudaStream_t stream) {
  return p.is_bf16 ? launch_back<true>(p, stream) : launch_back<false>(p, stream);
}

}  // namespace fgemm
