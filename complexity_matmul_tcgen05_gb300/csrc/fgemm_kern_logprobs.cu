// fgemm_kern_logprobs.cu -- log probability of a given token, entropy and the
// most probable tokens of rows of logits.
//
// For a row x with largest value m (NaN counts as -inf), d_i = x_i - m:
//   z = 1 + r,  r = sum of e^d_i over all but one entry at m
//   log p_i = d_i - log z,   entropy = log z - (sum e^d_i d_i) / z
// One entry at m stays out of the sum: with log(1 + r) what is left to the other
// tokens keeps its bits beside a probability near 1.
//
// One pass over the row: a thread takes 64 bytes at a time, follows the largest
// value with its sums relative to it (they are scaled when a batch brings a larger
// one), and the threads' sums meet at the row's end. d is held to -200 and above:
// that leaves e^d 0 and the product with d too, for masked logits and NaN alike.
//
// The most probable tokens: the n-th largest of the threads' maxima is a value that
// at least n logits reach, so the first n are among the logits from there on. A
// search on the maxima finds such a value that at most 2 n threads reach, these
// threads read their logits again and leave the ones from there on in a list, and
// the list is ranked by counting. A list that does not fit (ties) is not used: the
// tokens are then found one by one, a pass each.
//
// A row is shared by a cluster of up to 8 CTAs where there are few rows.
// Memory-bound with many rows, bound by the meetings with few.
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_attn.cuh"
#include "fgemm_internal.h"
#include "fgemm_ptx.cuh"

namespace fgemm {

namespace {

using namespace attn;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kDeep = 4;         // vectors of 16 bytes a thread has on their way
constexpr int kList = 1024;      // logits that may be ranked
constexpr int kMostTop = 32;
constexpr int kMostSplit = 8;
constexpr int kCtasPerSm = 4;
constexpr float kLog2e = 1.4426950408889634f;

using Key = unsigned long long;

__device__ __forceinline__ uint32_t ordered(float x) {  // as an integer; -0 as 0
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// Larger value first, then lower index, as one integer; 0 for -inf (and NaN).
__device__ __forceinline__ Key key_of(float x, int i) {
  if (!(x > -INFINITY)) return 0;
  return (static_cast<Key>(ordered(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float value_of(Key key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ int index_of(Key key) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key)); }

// Sums of some logits relative to their largest, m (-inf: there are none): r and t
// are those of e^d and e^d d without one entry at m.
struct Part {
  float m, r, t;
};
__device__ __forceinline__ Part join(Part a, Part b) {
  if (b.m > a.m) {
    const Part c = a;
    a = b;
    b = c;
  }
  if (b.m == -INFINITY) return a;
  const float d = b.m == a.m ? 0.0f : b.m - a.m;  // (infinite ones may be equal)
  const float f = expf(d);
  if (f > 0.0f) {
    a.r += f * (b.r + 1.0f);
    a.t += f * (b.t + d * (b.r + 1.0f));
  }
  return a;
}

template <int TYPE>
struct Row {
  static constexpr int kVec = TYPE == 2 ? 4 : 8;
  const uint8_t* base;  // on 16 bytes, at or before the row's first logit
  int skip, vocab;      // logits from there to it; of the row
  int vectors;

  __device__ __forceinline__ Row(const LogprobParams& p, long long row) {
    constexpr int kSize = TYPE == 2 ? 4 : 2;
    const uint8_t* const first = static_cast<const uint8_t*>(p.logits) + row * p.ld * kSize;
    skip = static_cast<int>(reinterpret_cast<uintptr_t>(first) % 16) / kSize;
    base = first - skip * kSize;
    vocab = p.vocab;
    vectors = (skip + vocab + kVec - 1) / kVec;
  }
  __device__ __forceinline__ float one(int i) const {
    if (TYPE == 2) return reinterpret_cast<const float*>(base)[skip + i];
    return to_f32<TYPE == 1>(reinterpret_cast<const uint16_t*>(base)[skip + i]);
  }
  // Vector v; logits that are not the row's read as -inf.
  __device__ __forceinline__ uint4 load(int v) const {
    const int i0 = v * kVec - skip;
    if (i0 >= 0 && i0 + kVec <= vocab) return reinterpret_cast<const uint4*>(base)[v];
    uint32_t w[4];
    if (TYPE == 2) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = i0 + k >= 0 && i0 + k < vocab ? reinterpret_cast<const uint32_t*>(base)[v * 4 + k] : 0xFF800000u;
    } else {
      constexpr uint32_t kLow = TYPE == 1 ? 0xFF80u : 0xFC00u;  // -inf
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint16_t* const at = reinterpret_cast<const uint16_t*>(base) + v * 8 + 2 * k;
        const int i = i0 + 2 * k;
        const uint32_t lo = i >= 0 && i < vocab ? at[0] : kLow;
        const uint32_t hi = i + 1 >= 0 && i + 1 < vocab ? at[1] : kLow;
        w[k] = lo | hi << 16;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ static uint4 none() {
    constexpr uint32_t kLow = TYPE == 2 ? 0xFF800000u : TYPE == 1 ? 0xFF80FF80u : 0xFC00FC00u;
    return make_uint4(kLow, kLow, kLow, kLow);
  }
  __device__ __forceinline__ static float elem(const uint4& v, int k) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (TYPE == 2) return __uint_as_float(w[k]);
    return k & 1 ? hi_f32<TYPE == 1>(w[k >> 1]) : lo_f32<TYPE == 1>(w[k >> 1]);
  }
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A batch of vectors into the thread's sums.
template <int TYPE>
__device__ __forceinline__ void add_batch(Part& s, const uint4 (&v)[kDeep]) {
  using R = Row<TYPE>;
  float most = -INFINITY;
#pragma unroll
  for (int n = 0; n < kDeep; ++n)
#pragma unroll
    for (int k = 0; k < R::kVec; ++k) most = fmaxf(most, R::elem(v[n], k));
  if (most > s.m) {
    // Sums go to the new largest value, which is among these logits: its entries
    // are counted, one of them not.
    const Part before = s;
    s = Part{most, 0.0f, 0.0f};
    s = join(s, before);
    float count = 0.0f;
#pragma unroll
    for (int n = 0; n < kDeep; ++n)
#pragma unroll
      for (int k = 0; k < R::kVec; ++k) {
        const float x = R::elem(v[n], k);
        const float d = fmaxf(x - most, -200.0f);
        const float w = x == most ? 0.0f : exp2_fast(d * kLog2e);
        count += x == most ? 1.0f : 0.0f;
        s.r += w;
        s.t = fmaf(w, d, s.t);
      }
    s.r += count - 1.0f;
  } else if (s.m == INFINITY) {
#pragma unroll
    for (int n = 0; n < kDeep; ++n)
#pragma unroll
      for (int k = 0; k < R::kVec; ++k) s.r += R::elem(v[n], k) == INFINITY ? 1.0f : 0.0f;
  } else if (s.m > -INFINITY) {
    const uint64_t less = pair(-s.m, -s.m);
    uint64_t r2 = pair(0.0f, 0.0f), t2 = pair(0.0f, 0.0f);
#pragma unroll
    for (int n = 0; n < kDeep; ++n)
#pragma unroll
      for (int k = 0; k < R::kVec; k += 2) {
        float d0, d1;
        unpair(add2(pair(R::elem(v[n], k), R::elem(v[n], k + 1)), less), d0, d1);
        d0 = fmaxf(d0, -200.0f);
        d1 = fmaxf(d1, -200.0f);
        const uint64_t w = pair(exp2_fast(d0 * kLog2e), exp2_fast(d1 * kLog2e));
        r2 = add2(r2, w);
        t2 = fma2(w, pair(d0, d1), t2);
      }
    float a, b;
    unpair(r2, a, b);
    s.r += a + b;
    unpair(t2, a, b);
    s.t += a + b;
  }
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ Key ld_cluster_key(uint32_t at) {
  Key v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
  return v;
}

// A CTA of a cluster of `split` takes a part of row blockIdx.x / split.
template <int TYPE>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) logprobs_kernel(const __grid_constant__ LogprobParams p,
                                                                        int split) {
  using R = Row<TYPE>;
  __shared__ Key list[kList];
  __shared__ Key sorted[kMostTop];
  __shared__ Key best[kWarps];
  __shared__ Part parts[kWarps];
  __shared__ float sums[3];
  __shared__ int listed;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const long long row = blockIdx.x / split;
  const R x(p, row);
  const int each = (x.vectors + split - 1) / split;
  const int v0 = min(x.vectors, rank * each), v1 = min(x.vectors, v0 + each);
  const int token = rank == 0 && threadIdx.x == 0 ? p.tokens[row] : 0;
  const float given = rank == 0 && threadIdx.x == 0 && token >= 0 && token < p.vocab ? x.one(token) : -INFINITY;

  Part s{-INFINITY, 0.0f, 0.0f};
  for (int v = v0 + threadIdx.x; v < v1; v += kThreads * kDeep) {
    uint4 batch[kDeep];
#pragma unroll
    for (int n = 0; n < kDeep; ++n) batch[n] = v + n * kThreads < v1 ? x.load(v + n * kThreads) : R::none();
    add_batch<TYPE>(s, batch);
  }
  const float mine = s.m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    s = join(s, Part{__shfl_xor_sync(0xFFFFFFFFu, s.m, d), __shfl_xor_sync(0xFFFFFFFFu, s.r, d),
                     __shfl_xor_sync(0xFFFFFFFFu, s.t, d)});
  if (lane == 0) parts[warp] = s;
  if (threadIdx.x == 0) listed = 0;
  if (threadIdx.x < kMostTop) sorted[threadIdx.x] = 0;
  __syncthreads();

  const int top = p.top;
  if (top > 0) {
    // A value that at least `top` threads reach, if so many have one above -inf,
    // and not many more: keys in [lo, hi), those from lo on are enough.
    const uint32_t my = mine > -INFINITY ? ordered(mine) : 0u;
    uint32_t lo = 1u, hi = 0xFFFFFFFFu;
    if (__syncthreads_count(my >= lo) > top) {
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int count = __syncthreads_count(my >= mid);
        if (count < top) {
          hi = mid;
        } else {
          lo = mid;
          if (count <= 2 * top) break;
        }
      }
    }
    if (my >= lo) {
      for (int v = v0 + threadIdx.x; v < v1; v += kThreads * kDeep) {
        uint4 batch[kDeep];
#pragma unroll
        for (int n = 0; n < kDeep; ++n) batch[n] = v + n * kThreads < v1 ? x.load(v + n * kThreads) : R::none();
#pragma unroll
        for (int n = 0; n < kDeep; ++n)
#pragma unroll
          for (int k = 0; k < R::kVec; ++k) {
            const Key key = key_of(R::elem(batch[n], k), (v + n * kThreads) * R::kVec - x.skip + k);
            if (static_cast<uint32_t>(key >> 32) >= lo) {
              const int at = atomicAdd(&listed, 1);
              if (at < kList) list[at] = key;
            }
          }
      }
    }
    __syncthreads();
    const int count = listed;
    if (count <= kList) {
      for (int i = threadIdx.x; i < count; i += kThreads) {
        const Key key = list[i];
        int before = 0;
        for (int j = 0; j < count; ++j) before += list[j] > key;
        if (before < top) sorted[before] = key;
      }
    } else {
      Key last = ~0ull;
      for (int n = 0; n < top; ++n) {
        Key most = 0;
        for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
          const uint4 w = x.load(v);
#pragma unroll
          for (int k = 0; k < R::kVec; ++k) {
            const Key key = key_of(R::elem(w, k), v * R::kVec - x.skip + k);
            if (key < last && key > most) most = key;
          }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          const Key other = __shfl_xor_sync(0xFFFFFFFFu, most, d);
          most = other > most ? other : most;
        }
        if (lane == 0) best[warp] = most;
        __syncthreads();
        most = 0;
        for (int w = 0; w < kWarps; ++w) most = best[w] > most ? best[w] : most;
        last = most;
        if (threadIdx.x == 0) sorted[n] = most;
        __syncthreads();
      }
    }
  }

  // The CTA's sums, then the cluster's in its first CTA.
  if (threadIdx.x == 0) {
    s = parts[0];
    for (int w = 1; w < kWarps; ++w) s = join(s, parts[w]);
    sums[0] = s.m, sums[1] = s.r, sums[2] = s.t;
  }
  __syncthreads();
  if (split > 1) {
    ptx::cluster_sync();
    if (rank == 0) {
      if (threadIdx.x == 0) {
        for (int c = 1; c < split; ++c) {
          const uint32_t at = ptx::mapa(ptx::smem_u32(sums), c);
          s = join(s, Part{ld_cluster_f32(at), ld_cluster_f32(at + 4), ld_cluster_f32(at + 8)});
        }
        sums[0] = s.m, sums[1] = s.r, sums[2] = s.t;
      }
      Key key = 0;  // at most 8 x 32 of them
      if (top > 0 && threadIdx.x < split * kMostTop) {
        const uint32_t at = ptx::mapa(ptx::smem_u32(sorted + threadIdx.x % kMostTop), threadIdx.x / kMostTop);
        key = ld_cluster_key(at);
      }
      list[threadIdx.x] = key;
      __syncthreads();
      if (threadIdx.x < kMostTop) sorted[threadIdx.x] = 0;
      __syncthreads();
      if (key != 0) {
        int before = 0;
        for (int j = 0; j < split * kMostTop; ++j) before += list[j] > key;
        if (before < top) sorted[before] = key;
      }
      __syncthreads();
    }
    ptx::cluster_sync();  // no CTA leaves while it may be read
    if (rank != 0) return;
  }
  const float m = sums[0], r = sums[1], t = sums[2], log_z = log1pf(r);
  const auto log_p = [&](float v) { return !(v > -INFINITY) ? -INFINITY : v == m ? -log_z : v - m - log_z; };
  if (threadIdx.x == 0) {
    p.logprob[row] = m == -INFINITY ? -INFINITY : log_p(given);
    if (p.entropy) p.entropy[row] = m == -INFINITY ? 0.0f : log_z - t / (1.0f + r);
  }
  if (threadIdx.x < top) {
    const Key key = sorted[threadIdx.x];
    p.top_tokens[row * top + threadIdx.x] = key ? index_of(key) : -1;
    p.top_logprobs[row * top + threadIdx.x] = key ? log_p(value_of(key)) : -INFINITY;
  }
}

template <int TYPE>
cudaError_t launch_of(const LogprobParams& p, int num_sms, cudaStream_t stream) {
  // CTAs of a row: as many as the device holds beside the other rows', each with
  // a vector a thread at least.
  const long long vectors = (p.vocab + Row<TYPE>::kVec - 1) / Row<TYPE>::kVec;
  int split = kMostSplit;
  while (split > 1 && (static_cast<long long>(p.rows) * split > static_cast<long long>(num_sms) * kCtasPerSm ||
                       vectors < static_cast<long long>(split) * kThreads))
    split /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * static_cast<unsigned>(split));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(split);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<TYPE>, p, split);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, int num_sms, cudaStream_t stream) {
  if (p.type == 0) return launch_of<0>(p, num_sms, stream);
  if (p.type == 1) return launch_of<1>(p, num_sms, stream);
  return launch_of<2>(p, num_sms, stream);
}

}  // namespace fgemm
