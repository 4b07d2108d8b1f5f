// fgemm_kern_rotary.cu -- rotary positions of queries and keys, and the write
// of keys and values into a paged cache, in one launch.
//
//   angle = position * inv_freq[i],  (a, b) -> (a cos - b sin, b cos + a sin)
//
// A token's angles are the same for all of its heads: a CTA takes one or a few
// tokens, forms their cosines and sines once in shared memory and then passes over the
// heads, 8 values of 16 bits (or 8 pairs) a thread. Angles are counted in turns, in
// fixed point modulo one turn, so far positions lose nothing: at position 10^6 a 32-bit
// product is off by 0.06 radians. What is left of a turn, at most half of one to either
// side, goes on as a 32-bit floating-point number (off by 2^-24 of itself), where the
// rotation's own roundings are.
//
// Memory-bound: each value is read and written once. Measured, 8191 tokens, 32 heads of
// 128 over 8 key heads: pairs (i, i + rot / 2) bf16 32 us (6.2 TB/s), with 64 heads 53 us
// (6.3 TB/s); pairs (2 i, 2 i + 1) 36 us (5.6 TB/s); one token 2.6 us, a launch. Before,
// with angles in 64-bit floating point and the turns of a part side by side, where a warp
// met the same banks, the first took 65 us, 1024 tokens 10.5 us (now 7.3).
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_attn.cuh"
#include "fgemm_internal.h"

namespace fgemm {

namespace {

using namespace attn;

constexpr int kMostThreads = 256;

// inv_freq / 2 pi less its whole turns, in units of 2^-64 of a turn: positions are
// integers, so that is all that matters of it. In integers (the 64-bit floating-point
// units of this device are few), the reduction of M. Payne and R. Hanek ("Radian
// reduction for trigonometric functions", 1983): with |inv_freq| = m 2^e, m times the
// first 128 bits of 1 / 2 pi shifted by e. Off by less than two units, 2^-32 turns at the
// last position.
__device__ __forceinline__ unsigned long long pace_of(float inv_freq) {
  // the first 256 bits behind the point of 1 / 2 pi
  constexpr unsigned long long kBits[4] = {0x28BE60DB9391054Aull, 0x7F09D5F47D4D3770ull, 0x36D8A5664F10E410ull,
                                           0x7F9458EAF7AEF158ull};
  const uint32_t bits = __float_as_uint(inv_freq);
  const int exponent = static_cast<int>(bits >> 23 & 255u), e = max(exponent, 1) - 150;
  const unsigned long long m = (bits & 0x7FFFFFu) | (exponent > 0 ? 0x800000u : 0u);
  unsigned long long r;
  if (e < 0) {
    const unsigned long long low = m * kBits[0], sum = low + __umul64hi(m, kBits[1]);
    const unsigned long long high = __umul64hi(m, kBits[0]) + (sum < low ? 1u : 0u);
    r = e > -64 ? high << (64 + e) | sum >> -e : high >> min(-e - 64, 63);
  } else {
    const int s = e & 63;
    const bool far = e >= 64;
    const unsigned long long a = far ? kBits[1] : kBits[0], b = far ? kBits[2] : kBits[1], c = far ? kBits[3] : kBits[2];
    r = m * (a << s | b >> 1 >> (63 - s)) + __umul64hi(m, b << s | c >> 1 >> (63 - s));
  }
  return bits >> 31 ? 0ull - r : r;
}

// cos and sin of position * inv_freq: the product's whole turns run over the 64 bits.
__device__ __forceinline__ float2 turn(int position, float inv_freq, unsigned long long pace) {
  const unsigned long long at = pace * static_cast<unsigned long long>(static_cast<long long>(position));
  float half_turns = static_cast<float>(static_cast<long long>(at)) * 0x1p-63f;
  if (!isfinite(inv_freq)) half_turns = NAN;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c, s);
}

template <bool BF16>
__device__ __forceinline__ void rotate(uint32_t a, uint32_t b, const float2 t0, const float2 t1, uint32_t& to_a,
                                       uint32_t& to_b) {
  const float a0 = lo_f32<BF16>(a), a1 = hi_f32<BF16>(a), b0 = lo_f32<BF16>(b), b1 = hi_f32<BF16>(b);
  to_a = pack2<BF16>(a0 * t0.x - b0 * t0.y, a1 * t1.x - b1 * t1.y);
  to_b = pack2<BF16>(b0 * t0.x + a0 * t0.y, b1 * t1.x + a1 * t1.y);
}

// A head is passed over in parts (parts_of). MODE 0: pairs (i, i + rot / 2) with rot a
// multiple of 16, 16-byte accesses; MODE 1: pairs (2 i, 2 i + 1), 16-byte accesses;
// MODE 2: pairs (i, i + rot / 2) one at a time.
template <int MODE>
__host__ __device__ inline int parts_of(int dim, int rot) {
  return MODE == 2 ? dim - rot / 2 : MODE == 1 ? dim / 8 : dim / 8 - rot / 16;
}

// Pairs of a part; the turns of a token lie in shared memory by pair of the part, then
// by part (neighbours in a warp have neighbouring parts), `line` of them.
template <int MODE>
constexpr int kPairs = MODE == 0 ? 8 : MODE == 1 ? 4 : 1;
template <int MODE>
__host__ __device__ inline int line_of(int rot) {
  return (rot / 2 + kPairs<MODE> - 1) / kPairs<MODE> * kPairs<MODE>;
}

// What a part reads: up to two vectors of 16 bytes, or two values.
struct Loaded {
  uint4 a, b;
};

template <int MODE>
__device__ __forceinline__ Loaded load_part(const uint16_t* from, int part, int rot) {
  Loaded v;
  if (MODE == 2) {
    const int half = rot / 2;
    v.a.x = part < half ? from[part] : 0u;
    v.b.x = from[part + half];
  } else {
    const uint4* const in = reinterpret_cast<const uint4*>(from);
    const int pairs = rot / 16;
    v.a = in[MODE == 1 || part < pairs ? part : part + pairs];
    if (MODE == 0 && part < pairs) v.b = in[part + pairs];
  }
  return v;
}

template <bool BF16, int MODE>
__device__ __forceinline__ void store_part(uint16_t* to, const Loaded& v, int part, int rot, const float2* turns) {
  if (MODE == 2) {
    const int half = rot / 2;
    if (part < half) {
      const float a = to_f32<BF16>(v.a.x), b = to_f32<BF16>(v.b.x);
      const float2 t = turns[part];
      to[part] = to_16<BF16>(a * t.x - b * t.y);
      to[part + half] = to_16<BF16>(b * t.x + a * t.y);
    } else {
      to[part + half] = static_cast<uint16_t>(v.b.x);
    }
    return;
  }
  uint4* const out = reinterpret_cast<uint4*>(to);
  if (MODE == 0) {
    const int pairs = rot / 16;
    if (part >= pairs) {
      out[part + pairs] = v.a;
      return;
    }
    const float2* const t = turns + part;
    uint4 x, y;
    rotate<BF16>(v.a.x, v.b.x, t[0], t[pairs], x.x, y.x);
    rotate<BF16>(v.a.y, v.b.y, t[2 * pairs], t[3 * pairs], x.y, y.y);
    rotate<BF16>(v.a.z, v.b.z, t[4 * pairs], t[5 * pairs], x.z, y.z);
    rotate<BF16>(v.a.w, v.b.w, t[6 * pairs], t[7 * pairs], x.w, y.w);
    out[part] = x;
    out[part + pairs] = y;
  } else {
    uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * (part * 4 + i) < rot) {
        const float a = lo_f32<BF16>(w[i]), b = hi_f32<BF16>(w[i]);
        const float2 t = turns[i * ((rot + 7) / 8) + part];
        w[i] = pack2<BF16>(a * t.x - b * t.y, b * t.x + a * t.y);
      }
    }
    out[part] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// blockIdx.x: EACH tokens. A thread takes the same part of each, all loads first.
template <bool BF16, int MODE, int EACH>
__global__ void __launch_bounds__(kMostThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  extern __shared__ float2 turns[];  // [token][pair of a part][part]
  __shared__ long long k_at[EACH], v_at[EACH];  // of the tokens' places in the cache, -1: none
  const int half = p.rot / 2, line = line_of<MODE>(p.rot);
  const long long t0 = static_cast<long long>(blockIdx.x) * EACH;
  const int count = static_cast<int>(min(static_cast<long long>(EACH), p.tokens - t0));
  if (threadIdx.x < count) {
    const int slot = p.slots[t0 + threadIdx.x];
    const bool kept = slot >= 0 && slot < p.cache_slots;
    const long long page = kept ? slot / p.page_size : 0, in_page = kept ? slot % p.page_size : 0;
    k_at[threadIdx.x] = kept ? page * p.k_page + in_page * p.k_token : -1;
    v_at[threadIdx.x] = kept ? page * p.v_page + in_page * p.v_token : -1;
  }
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const float inv_freq = p.inv_freq[i];
    const unsigned long long pace = pace_of(inv_freq);
    float2* const to = turns + i % kPairs<MODE> * (line / kPairs<MODE>) + i / kPairs<MODE>;
#pragma unroll
    for (int j = 0; j < EACH; ++j)
      if (j < count) to[j * line] = turn(p.positions[t0 + j], inv_freq, pace);
  }
  const int parts = parts_of<MODE>(p.dim, p.rot), chunks = p.dim / 8;
  const int queries = p.heads * parts, keys = p.kv_heads * parts, tasks = queries + keys + p.kv_heads * chunks;
  bool formed = false;
  for (int task = threadIdx.x; task < tasks || !formed; task += blockDim.x) {
    // queries, keys, then values (copied as they are)
    const int kind = task < queries ? 0 : task < queries + keys ? 1 : 2;
    const int at = kind == 0 ? task : kind == 1 ? task - queries : task - queries - keys;
    const int head = at / (kind == 2 ? chunks : parts), part = at - head * (kind == 2 ? chunks : parts);
    Loaded v[EACH];
    if (task < tasks) {
      const Heads& from = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
#pragma unroll
      for (int i = 0; i < EACH; ++i)
        if (i < count) {
          const uint16_t* const x = from.p + (t0 + i) * from.ld + head * from.hs;
          if (kind == 2)
            v[i].a = reinterpret_cast<const uint4*>(x)[part];
          else
            v[i] = load_part<MODE>(x, part, p.rot);
        }
    }
    if (!formed) __syncthreads();  // the turns (the first loads are on their way)
    formed = true;
    if (task >= tasks) continue;
#pragma unroll
    for (int i = 0; i < EACH; ++i)
      if (i < count) {
        if (kind == 0) {
          store_part<BF16, MODE>(p.out.p + (t0 + i) * p.out.ld + head * p.out.hs, v[i], part, p.rot, turns + i * line);
        } else if (kind == 1) {
          if (k_at[i] >= 0)
            store_part<BF16, MODE>(p.k_cache + k_at[i] + head * p.k_head, v[i], part, p.rot, turns + i * line);
        } else if (v_at[i] >= 0) {
          reinterpret_cast<uint4*>(p.v_cache + v_at[i] + head * p.v_head)[part] = v[i].a;
        }
      }
  }
}

template <bool BF16, int MODE>
cudaError_t launch_mode(const RotaryParams& p, int num_sms, cudaStream_t stream) {
  // Several tokens a CTA once there are enough for every SM, where a part is small: pairs
  // of vectors are fastest one token at a time (34 us; two 42, four 47), single vectors
  // four (37 us; two 40, one 43).
  constexpr int kEach = MODE == 0 ? 1 : 4;
  const int each = p.tokens >= static_cast<long long>(num_sms) * kEach * 4 ? kEach : 1;
  const unsigned grid = static_cast<unsigned>((p.tokens + each - 1) / each);
  // As many threads as leave few without a part in the last pass (28 heads of 64 over 4,
  // 16384 tokens 37 us; with 256 threads 49).
  const int tasks = (p.heads + p.kv_heads) * parts_of<MODE>(p.dim, p.rot) + p.kv_heads * (p.dim / 8);
  const int passes = (tasks + kMostThreads - 1) / kMostThreads;
  const int threads = ((tasks + passes - 1) / passes + 31) / 32 * 32;
  const size_t smem = static_cast<size_t>(each) * line_of<MODE>(p.rot) * sizeof(float2);
  if (kEach == 1 || each == 1)
    rotary_kernel<BF16, MODE, 1><<<grid, threads, smem, stream>>>(p);
  else
    rotary_kernel<BF16, MODE, kEach><<<grid, threads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_of(const RotaryParams& p, int num_sms, cudaStream_t stream) {
  if (p.interleaved) return launch_mode<BF16, 1>(p, num_sms, stream);
  if (p.rot % 16 == 0) return launch_mode<BF16, 0>(p, num_sms, stream);
  return launch_mode<BF16, 2>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, int num_sms, cudaStream_t stream) {
  return p.is_bf16 ? launch_of<true>(p, num_sms, stream) : launch_of<false>(p, num_sms, stream);
}

}  // namespace fgemm
