// fgemm_kern_logprobs.cu -- log probability of a given token, entropy and the
// most probable tokens of rows of logits.
//
// For a row x with largest value m (NaN counts as -inf), d_i = x_i - m:
//   z = 1 + r,  r = sum of e^d_i over all but one entry at m
//   log p_i = d_i - log z,   entropy = log z - (sum e^d_i d_i) / z
// One entry at m stays out of the sum: with log(1 + r) what is left to the other
// tokens keeps its bits beside a probability near 1.
//
// One pass over the row: a warp takes 2 KB at a time, follows the largest value with
// its lanes' sums relative to it (they are scaled when a batch brings a larger one),
// and the warps' sums meet at the row's end. d is held to -200 and above:
// that leaves e^d 0 and the product with d too, for masked logits and NaN alike.
//
// The most probable tokens: the n-th largest of the threads' maxima is a value that
// at least n logits reach, so the first n are among the logits from there on. A
// search on the maxima finds such a value that at most 2 n threads reach (ties
// apart), these threads' logits are read again, the ones from there on go to a list,
// and the list is ranked by counting. A list that does not fit (ties) is not used: the
// tokens are then found one by one, a pass each.
//
// A row is shared by a cluster of up to 8 CTAs where there are few rows; the others
// write to its first one.
// Measured: 4096 x 50257 fp16 70 us (5.9 TB/s; with sums by thread, whose lanes took
// different branches, 140); 64 x 131072 fp32 9.3 us without alternatives, 14.4 with 20
// (the search, the second read and two rankings come one after the other); one row of
// 32000 bf16 4.5 us, with 5 alternatives 6.9.
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_attn.cuh"
#include "fgemm_internal.h"
#include "fgemm_ptx.cuh"

namespace fgemm {

namespace {

using namespace attn;

constexpr int kDeep = 4;         // vectors of 16 bytes a thread has on their way
constexpr int kList = 1024;      // logits that may be ranked
constexpr int kMostTop = 32;
constexpr int kMostSplit = 8;
constexpr int kThreadsPerSm = 1024;  // that the registers allow
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

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <int TYPE>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {  // a number before a NaN
  if (TYPE == 2) return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  if (TYPE == 1) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// A warp's sums of what it has seen: the largest value m is the warp's, r and t are
// a lane's share, without one entry at m (a lane has left it out).
struct Running {
  float m, r, t;
  float mine;  // the lane's largest
};

// A batch of vectors of each lane of a warp. The lanes go the same ways: a branch
// by a lane's own maximum was taken by some lane in nearly every batch.
template <int TYPE>
__device__ __forceinline__ void add_batch(Running& s, uint4 (&v)[kDeep]) {
  using R = Row<TYPE>;
  uint32_t w = v[0].x;
#pragma unroll
  for (int n = 0; n < kDeep; ++n) {
    w = max_word<TYPE>(w, max_word<TYPE>(v[n].x, v[n].y));
    w = max_word<TYPE>(w, max_word<TYPE>(v[n].z, v[n].w));
  }
  const float most = TYPE == 2 ? fmaxf(-INFINITY, __uint_as_float(w))
                               : fmaxf(fmaxf(-INFINITY, lo_f32<TYPE == 1>(w)), hi_f32<TYPE == 1>(w));
  s.mine = fmaxf(s.mine, most);
  const bool above = most > s.m;
  if (__any_sync(0xFFFFFFFFu, above)) {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, most > -INFINITY ? ordered(most) : 0u);
    const float m = __uint_as_float(top & 0x80000000u ? top & 0x7FFFFFFFu : ~top);
    if (s.m > -INFINITY) {
      const float d = s.m - m, f = exp2_fast(fmaxf(d, -200.0f) * kLog2e);
      if ((threadIdx.x & 31) == 0) s.r += 1.0f;  // the entry at the old m counts now
      s.t = f > 0.0f ? f * (s.t + d * s.r) : 0.0f;
      s.r *= f;
    }
    s.m = m;
    // one lane leaves out one entry at m
    const uint32_t has = __ballot_sync(0xFFFFFFFFu, most == m);
    if ((threadIdx.x & 31) == __ffs(has) - 1) {
      bool out = false;
#pragma unroll
      for (int n = 0; n < kDeep; ++n) {
        uint32_t x[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (TYPE == 2) {
            const bool hit = !out && __uint_as_float(x[k]) == m;
            x[k] = hit ? 0xFF800000u : x[k];
            out |= hit;
          } else {
            constexpr uint32_t kLow = TYPE == 1 ? 0xFF80u : 0xFC00u;
            const bool lo = !out && lo_f32<TYPE == 1>(x[k]) == m;
            x[k] = lo ? (x[k] & 0xFFFF0000u) | kLow : x[k];
            out |= lo;
            const bool hi = !out && hi_f32<TYPE == 1>(x[k]) == m;
            x[k] = hi ? (x[k] & 0xFFFFu) | kLow << 16 : x[k];
            out |= hi;
          }
        }
        v[n] = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
    __syncwarp();
  }
  if (s.m == -INFINITY) return;
  if (s.m == INFINITY) {
#pragma unroll
    for (int n = 0; n < kDeep; ++n)
#pragma unroll
      for (int k = 0; k < R::kVec; ++k) s.r += R::elem(v[n], k) == INFINITY ? 1.0f : 0.0f;
    return;
  }
  const uint64_t less = pair(-s.m, -s.m), log2e = pair(kLog2e, kLog2e);
  uint64_t r2 = pair(s.r, 0.0f), t2 = pair(s.t, 0.0f);
#pragma unroll
  for (int n = 0; n < kDeep; ++n)
#pragma unroll
    for (int k = 0; k < R::kVec; k += 2) {
      float d0, d1, e0, e1;
      unpair(add2(pair(R::elem(v[n], k), R::elem(v[n], k + 1)), less), d0, d1);
      const uint64_t d = pair(fmaxf(d0, -200.0f), fmaxf(d1, -200.0f));
      unpair(mul2(d, log2e), e0, e1);
      const uint64_t w2 = pair(exp2_fast(e0), exp2_fast(e1));
      r2 = add2(r2, w2);
      t2 = fma2(w2, d, t2);
    }
  float a, b;
  unpair(r2, a, b);
  s.r = a + b;
  unpair(t2, a, b);
  s.t = a + b;
}

__device__ __forceinline__ void st_cluster_f32(uint32_t at, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_key(uint32_t at, Key v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The first `top` of `count` different keys, in order, by all threads of a CTA; four
// threads a key.
template <int kThreads>
__device__ __forceinline__ void rank_list(const Key* list, int count, Key* sorted, int top) {
  for (int i = threadIdx.x / 4; i < (count + 7) / 8 * 8; i += kThreads / 4) {  // (whole warps)
    const Key key = i < count ? list[i] : 0;
    int before = 0;
#pragma unroll 4
    for (int j = threadIdx.x % 4; j < count; j += 4) before += list[j] > key;
    before += __shfl_xor_sync(0xFFFFFFFFu, before, 1);
    before += __shfl_xor_sync(0xFFFFFFFFu, before, 2);
    if (i < count && before < top && threadIdx.x % 4 == 0) sorted[before] = key;
  }
}

constexpr uint32_t kLowest = 0x00800000u;  // ordered(-FLT_MAX)

// Of 32 EACH ordered values one that at least `top` of them reach and not many more,
// by a warp; kLowest if fewer than `top` are above -inf.
template <int EACH>
__device__ __forceinline__ uint32_t search(const uint32_t* values, int top) {
  uint32_t v[EACH];
#pragma unroll
  for (int i = 0; i < EACH; i += 4) {
    const uint4 w = reinterpret_cast<const uint4*>(values)[(threadIdx.x & 31) * (EACH / 4) + i / 4];
    v[i] = w.x, v[i + 1] = w.y, v[i + 2] = w.z, v[i + 3] = w.w;
  }
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) lo = min(lo, v[i]), hi = max(hi, v[i]);
  lo = max(__reduce_min_sync(0xFFFFFFFFu, lo), kLowest);
  hi = max(__reduce_max_sync(0xFFFFFFFFu, hi), lo) + 1;
  // at least `top` reach lo (or lo is kLowest), fewer reach hi; three borders at a time
  uint32_t reach = 32 * EACH;
  while (reach > 2u * top && hi - lo > 1) {
    const uint32_t step = max((hi - lo) / 4, 1u), a = lo + step, b = min(a + step, hi), c = min(b + step, hi);
    uint32_t count = 0;  // ten bits each
#pragma unroll
    for (int i = 0; i < EACH; ++i) count += (v[i] >= a ? 1u : 0u) + (v[i] >= b ? 1u << 10 : 0u) + (v[i] >= c ? 1u << 20 : 0u);
    count = __reduce_add_sync(0xFFFFFFFFu, count);
    const uint32_t na = count & 1023u, nb = count >> 10 & 1023u, nc = count >> 20;
    const uint32_t need = static_cast<uint32_t>(top);
    if (nc >= need)
      lo = c, reach = nc;
    else if (nb >= need)
      lo = b, hi = c, reach = nb;
    else if (na >= need)
      lo = a, hi = b, reach = na;
    else
      hi = a;
  }
  return lo;
}

// A CTA of a cluster of `split` takes a part of row blockIdx.x / split.
template <int TYPE, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreadsPerSm / kThreads)
    logprobs_kernel(const __grid_constant__ LogprobParams p, int split) {
  using R = Row<TYPE>;
  constexpr int kWarps = kThreads / 32;
  __shared__ __align__(16) Key list[kList];
  __shared__ __align__(16) Key theirs[kMostSplit * kMostTop];  // first CTA: every CTA's first tokens
  __shared__ Key sorted[kMostTop];
  __shared__ Key best[kWarps];
  __shared__ Part parts[kWarps];
  __shared__ __align__(16) uint32_t maxima[kThreads];
  __shared__ uint32_t threshold;
  __shared__ uint8_t lanes[kWarps][32];
  __shared__ float sums[kMostSplit][3];  // first CTA: every CTA's
  __shared__ int listed;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const long long row = blockIdx.x / split;
  const R x(p, row);
  const int each = (x.vectors + split - 1) / split;
  const int v0 = min(x.vectors, rank * each), v1 = min(x.vectors, v0 + each);
  if (split > 1) cluster_arrive();  // this CTA is there
  const int token = rank == 0 && threadIdx.x == 0 ? p.tokens[row] : 0;
  const float given = rank == 0 && threadIdx.x == 0 && token >= 0 && token < p.vocab ? x.one(token) : -INFINITY;

  // A warp takes kDeep x 32 vectors in a row; the next ones are on their way.
  constexpr int kChunk = kDeep * 32;
  auto fetch = [&](uint4 (&batch)[kDeep], int v) {
    const int end = v + kChunk;  // (the same for the lanes: the warp's first vector)
    if (end <= v1 && v * R::kVec >= x.skip && end * R::kVec <= x.skip + x.vocab) {
#pragma unroll
      for (int n = 0; n < kDeep; ++n) batch[n] = reinterpret_cast<const uint4*>(x.base)[v + n * 32 + lane];
    } else {
#pragma unroll
      for (int n = 0; n < kDeep; ++n) batch[n] = v + n * 32 + lane < v1 ? x.load(v + n * 32 + lane) : R::none();
    }
  };
  Running seen{-INFINITY, 0.0f, 0.0f, -INFINITY};
  {
    uint4 batch[kDeep], next[kDeep];
    int v = v0 + warp * kChunk;
    if (v < v1) fetch(batch, v);
    while (v < v1) {
      v += kThreads * kDeep;
      if (v < v1) fetch(next, v);
      add_batch<TYPE>(seen, batch);
#pragma unroll
      for (int n = 0; n < kDeep; ++n) batch[n] = next[n];
    }
  }
  const float mine = seen.mine;
  Part s{seen.m, seen.r, seen.t};
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    s.r += __shfl_xor_sync(0xFFFFFFFFu, s.r, d);
    s.t += __shfl_xor_sync(0xFFFFFFFFu, s.t, d);
  }
  const int top = p.top;
  const uint32_t my = mine > -INFINITY ? ordered(mine) : 0u;
  if (lane == 0) parts[warp] = s;
  if (top > 0) {
    maxima[threadIdx.x] = my;
    if (threadIdx.x == 0) listed = 0;
    if (threadIdx.x < kMostTop) sorted[threadIdx.x] = 0;
  }
  __syncthreads();

  if (top > 0) {
    if (warp == 0) {
      const uint32_t from = search<kThreads / 32>(maxima, top);
      if (lane == 0) threshold = from;
    }
    __syncthreads();
    // The lanes with a maximum from there on: the warp reads their logits again,
    // a vector a lane.
    const uint32_t from = threshold;
    const uint32_t has = __ballot_sync(0xFFFFFFFFu, my >= from);
    if (has) {
      const float least = value_of(static_cast<Key>(from) << 32);
      uint8_t* const who = lanes[warp];
      if (my >= from) who[__popc(has & ((1u << lane) - 1))] = static_cast<uint8_t>(lane);
      __syncwarp();
      const int first = v0 + warp * kChunk;  // vector `first + b kThreads kDeep + n 32 + lane`, b from 0, n below kDeep
      const int per = first < v1 ? ((v1 - first + kThreads * kDeep - 1) / (kThreads * kDeep)) * kDeep : 0;
      const int all = per * __popc(has);
#pragma unroll 4
      for (int e = lane; e < all; e += 32) {
        const int i = e % per;
        const int v = first + i / kDeep * (kThreads * kDeep) + i % kDeep * 32 + who[e / per];
        if (v >= v1) continue;
        const uint4 w = x.load(v);
#pragma unroll
        for (int k = 0; k < R::kVec; ++k) {
          const float value = R::elem(w, k);
          if (value >= least) {
            const int at = atomicAdd(&listed, 1);
            if (at < kList) list[at] = key_of(value, v * R::kVec - x.skip + k);
          }
        }
      }
    }
    __syncthreads();
    const int count = listed;
    if (count <= kList) {
      rank_list<kThreads>(list, count, sorted, top);
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

  // The CTA's sums; the cluster's meet in its first CTA, to which the others write.
  if (threadIdx.x == 0) {
    s = parts[0];
    for (int w = 1; w < kWarps; ++w) s = join(s, parts[w]);
    if (split == 1) sums[0][0] = s.m, sums[0][1] = s.r, sums[0][2] = s.t;
  }
  __syncthreads();
  if (split > 1) {
    cluster_wait();
    if (threadIdx.x == 0) {
      const uint32_t at = ptx::mapa(ptx::smem_u32(sums[rank]), 0);
      st_cluster_f32(at, s.m);
      st_cluster_f32(at + 4, s.r);
      st_cluster_f32(at + 8, s.t);
    }
    if (threadIdx.x < top) st_cluster_key(ptx::mapa(ptx::smem_u32(theirs + rank * top + threadIdx.x), 0), sorted[threadIdx.x]);
    __syncwarp();
    cluster_arrive();
    if (rank != 0) return;  // (what is over counts as arrived; nobody writes to this CTA)
    cluster_wait();
    if (threadIdx.x == 0) {
      for (int c = 1; c < split; ++c) s = join(s, Part{sums[c][0], sums[c][1], sums[c][2]});
      sums[0][0] = s.m, sums[0][1] = s.r, sums[0][2] = s.t;
    }
    if (top > 0) {
      // At least `top` keys reach the least of the CTAs' k-th ones, k = ceil(top / split):
      // those are ranked.
      const int k = (top + split - 1) / split - 1;
      Key least = ~0ull;
      for (int c = 0; c < split; ++c) least = min(least, theirs[c * top + k]);
      if (threadIdx.x == 0) listed = 0;
      if (threadIdx.x < kMostTop) sorted[threadIdx.x] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < split * top; i += kThreads) {
        const Key key = theirs[i];
        if (key != 0 && key >= least) list[atomicAdd(&listed, 1)] = key;
      }
      __syncthreads();
      rank_list<kThreads>(list, listed, sorted, top);
    }
    __syncthreads();
  }
  const float m = sums[0][0], r = sums[0][1], t = sums[0][2], log_z = log1pf(r);
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

template <int TYPE, int kThreads>
cudaError_t launch_split(const LogprobParams& p, int split, cudaStream_t stream) {
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
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<TYPE, kThreads>, p, split);
}

template <int TYPE>
cudaError_t launch_of(const LogprobParams& p, int num_sms, cudaStream_t stream) {
  // CTAs of a row: as many as the device holds beside the other rows', each with
  // a vector a thread at least.
  constexpr int kMany = 256, kFew = 128;
  const long long vectors = (p.vocab + Row<TYPE>::kVec - 1) / Row<TYPE>::kVec;
  int split = kMostSplit;
  while (split > 1 && (static_cast<long long>(p.rows) * split > static_cast<long long>(num_sms) * (kThreadsPerSm / kMany) ||
                       vectors < static_cast<long long>(split) * kMany))
    split /= 2;
  // Twice the rows on their way on an SM hide each other's ends better, but the n-th
  // largest of fewer threads' maxima leaves more logits to read again. 128 threads against
  // 256, 4096 x 50257 fp16 with 0, 1, 2, 3, 5, 8, 20 alternatives: 70 / 77 us, 78 / 87, 83 / 88,
  // 92 / 90, 102 / 95, 115 / 100, 145 / 134; 700 x 131072 fp32: 58 / 66, 69 / 74, 77 / 75, 83 / 75,
  // 93 / 81, 107 / 87, 134 / 105.
  return split == 1 && p.top <= 1 ? launch_split<TYPE, kFew>(p, split, stream) : launch_split<TYPE, kMany>(p, split, stream);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, int num_sms, cudaStream_t stream) {
  if (p.type == 0) return launch_of<0>(p, num_sms, stream);
  if (p.type == 1) return launch_of<1>(p, num_sms, stream);
  return launch_of<2>(p, num_sms, stream);
}

}  // namespace fgemm
