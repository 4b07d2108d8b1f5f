// fgemm_kern_rotary.cu -- rotary positions of queries and keys, and the write
// of keys and values into a paged cache, in one launch.
//
//   angle = position * inv_freq[i],  (a, b) -> (a cos - b sin, b cos + a sin)
//
// A token's angles are the same for all of its heads: a CTA takes a few
// tokens, forms their cosines and sines once in shared memory and then passes
// over the heads, 8 values of 16 bits (or 8 pairs) a thread. The angle is
// formed and reduced to one turn in 64 bits: at position 10^6 a 32-bit product
// is off by 0.06 radians. The reduced angle goes on in 32 bits (off by 2^-23
// at most), where the rotation's own roundings are.
//
// Memory-bound: each value is read and written once.
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_attn.cuh"
#include "fgemm_internal.h"

namespace fgemm {

namespace {

using namespace attn;

constexpr int kThreads = 256;

// cos and sin of position * inv_freq.
__device__ __forceinline__ float2 turn(int position, float inv_freq) {
  constexpr double kTurns = 0.15915494309189533577;    // 1 / 2 pi
  constexpr double kTwoPi = 6.28318530717958647693;    // 2 pi, and what 64 bits leave of it
  constexpr double kTwoPiLow = 2.4492935982947064e-16;
  constexpr double kHalfTurns = 0.31830988618379067154;  // 1 / pi
  const double angle = static_cast<double>(position) * static_cast<double>(inv_freq);
  const double n = rint(angle * kTurns);
  const double rest = fma(-n, kTwoPiLow, fma(-n, kTwoPi, angle));
  float s, c;
  sincospif(static_cast<float>(rest * kHalfTurns), &s, &c);
  return make_float2(c, s);
}

template <bool BF16>
__device__ __forceinline__ void rotate(uint32_t a, uint32_t b, const float2 t0, const float2 t1, uint32_t& to_a,
                                       uint32_t& to_b) {
  const float a0 = lo_f32<BF16>(a), a1 = hi_f32<BF16>(a), b0 = lo_f32<BF16>(b), b1 = hi_f32<BF16>(b);
  to_a = pack2<BF16>(a0 * t0.x - b0 * t0.y, a1 * t1.x - b1 * t1.y);
  to_b = pack2<BF16>(b0 * t0.x + a0 * t0.y, b1 * t1.x + a1 * t1.y);
}

// One head of a token: part `part` of its parts (parts_of).
// MODE 0: pairs (i, i + rot / 2) with rot a multiple of 16, 16-byte accesses;
// MODE 1: pairs (2 i, 2 i + 1), 16-byte accesses; MODE 2: pairs (i, i + rot / 2)
// one at a time.
template <bool BF16, int MODE>
__device__ __forceinline__ void head_part(const uint16_t* from, uint16_t* to, int part, int rot, const float2* turns) {
  if (MODE == 2) {
    const int half = rot / 2;
    if (part < half) {
      const float a = to_f32<BF16>(from[part]), b = to_f32<BF16>(from[part + half]);
      const float2 t = turns[part];
      to[part] = to_16<BF16>(a * t.x - b * t.y);
      to[part + half] = to_16<BF16>(b * t.x + a * t.y);
    } else {
      to[part + half] = from[part + half];
    }
    return;
  }
  const uint4* const in = reinterpret_cast<const uint4*>(from);
  uint4* const out = reinterpret_cast<uint4*>(to);
  if (MODE == 0) {
    const int pairs = rot / 16;
    if (part >= pairs) {
      out[part + pairs] = in[part + pairs];
      return;
    }
    const uint4 a = in[part], b = in[part + pairs];
    const float2* const t = turns + part * 8;
    uint4 x, y;
    rotate<BF16>(a.x, b.x, t[0], t[1], x.x, y.x);
    rotate<BF16>(a.y, b.y, t[2], t[3], x.y, y.y);
    rotate<BF16>(a.z, b.z, t[4], t[5], x.z, y.z);
    rotate<BF16>(a.w, b.w, t[6], t[7], x.w, y.w);
    out[part] = x;
    out[part + pairs] = y;
  } else {
    uint4 v = in[part];
    uint32_t* const w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = part * 4 + i;
      if (2 * pair < rot) {
        const float a = lo_f32<BF16>(w[i]), b = hi_f32<BF16>(w[i]);
        const float2 t = turns[pair];
        w[i] = pack2<BF16>(a * t.x - b * t.y, b * t.x + a * t.y);
      }
    }
    out[part] = v;
  }
}

template <int MODE>
__host__ __device__ inline int parts_of(int dim, int rot) {
  return MODE == 2 ? dim - rot / 2 : MODE == 1 ? dim / 8 : dim / 8 - rot / 16;
}

// blockIdx.x: `each` tokens.
template <bool BF16, int MODE>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p, int each) {
  extern __shared__ float2 turns[];  // [token][rot / 2]
  const int half = p.rot / 2;
  const long long t0 = static_cast<long long>(blockIdx.x) * each;
  const int count = static_cast<int>(min(static_cast<long long>(each), p.tokens - t0));
  for (int i = threadIdx.x; i < count * half; i += kThreads)
    turns[i] = turn(p.positions[t0 + i / half], p.inv_freq[i % half]);
  __syncthreads();
  const int parts = parts_of<MODE>(p.dim, p.rot), chunks = p.dim / 8;
  const int queries = p.heads * parts, keys = p.kv_heads * parts, tasks = queries + keys + p.kv_heads * chunks;
  for (int i = 0; i < count; ++i) {
    const long long t = t0 + i;
    const int slot = p.slots[t];
    const bool kept = slot >= 0 && slot < p.cache_slots;
    const long long page = kept ? slot / p.page_size : 0, in_page = kept ? slot % p.page_size : 0;
    for (int task = threadIdx.x; task < tasks; task += kThreads) {
      if (task < queries) {
        const int head = task / parts, part = task - head * parts;
        head_part<BF16, MODE>(p.q.p + t * p.q.ld + head * p.q.hs, p.out.p + t * p.out.ld + head * p.out.hs, part, p.rot,
                              turns + i * half);
      } else if (kept && task < queries + keys) {
        const int head = (task - queries) / parts, part = task - queries - head * parts;
        head_part<BF16, MODE>(p.k.p + t * p.k.ld + head * p.k.hs,
                              p.k_cache + page * p.k_page + in_page * p.k_token + head * p.k_head, part, p.rot,
                              turns + i * half);
      } else if (kept) {
        const int head = (task - queries - keys) / chunks, c = task - queries - keys - head * chunks;
        reinterpret_cast<uint4*>(p.v_cache + page * p.v_page + in_page * p.v_token + head * p.v_head)[c] =
            reinterpret_cast<const uint4*>(p.v.p + t * p.v.ld + head * p.v.hs)[c];
      }
    }
  }
}

template <bool BF16>
cudaError_t launch_of(const RotaryParams& p, cudaStream_t stream) {
  const int each = p.tokens >= 4096 ? 4 : 1;
  const unsigned grid = static_cast<unsigned>((p.tokens + each - 1) / each);
  const size_t smem = static_cast<size_t>(each) * (p.rot / 2) * sizeof(float2);
  if (p.interleaved)
    rotary_kernel<BF16, 1><<<grid, kThreads, smem, stream>>>(p, each);
  else if (p.rot % 16 == 0)
    rotary_kernel<BF16, 0><<<grid, kThreads, smem, stream>>>(p, each);
  else
    rotary_kernel<BF16, 2><<<grid, kThreads, smem, stream>>>(p, each);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  return p.is_bf16 ? launch_of<true>(p, stream) : launch_of<false>(p, stream);
}

}  // namespace fgemm
