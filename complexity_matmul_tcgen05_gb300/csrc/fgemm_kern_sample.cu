// fgemm_kern_sample.cu -- sampling from rows of logits with temperature,
// top-k, top-p and min-p, each row from one given uniform number.
//
// For a row x (NaN counts as -inf) with largest value m:
//   w_i = exp((x_i - m) / T); order: larger x first, then lower index
//   top-k: the first k of the order
//   top-p: of those the shortest prefix whose w add up to at least p of theirs
//   min-p: of those the ones with w_i >= min_p (w of the largest is 1)
//   token: the first index i, in index order, at which the running sum of the
//   kept w exceeds u times the whole sum.
//
// Where a threshold falls is decided by sums over up to a million terms, and
// a token changes when a sum moves across a border, so the sums here are
// exact: w is computed to about 36 bits (mass()) and held as an integer in
// units of 2^-44.  Integer sums do not depend on their order, which also
// makes the shared-memory atomics below deterministic.
//
// The vocabulary is not sorted: top-k and top-p are each a threshold on x,
// found by histograms.  The first one bins x linearly between m and m - 32 T
// (masses below are under 2^-46).  When top-k's threshold falls in a bin and
// that bin and those above hold at most 2048 logits, these are gathered in one
// CTA, sorted there, and the rest of the work is on a short list.  Otherwise
// the bin is searched again with bins over its key range (keys: x's bits,
// ordered as integers) until one key is left, and ties at that key are cut by
// index.
//
// A cluster of CTAs works on a row, each on a slice kept in shared memory,
// so the logits are read from memory once; the CTAs read each other's
// histograms and sums through distributed shared memory.  What bounds it:
// with many rows the arithmetic of the masses, with few the cluster's meetings.
// Measured: 64 x 131072 fp32, top-p 0.9, 123 us (memory alone would take 5; 264
// instructions a logit); 200 x 50257 fp16, half masked, min-p, 38 us; one row of
// 32000, top-k 50 and top-p 0.95, 12.6 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "fgemm_internal.h"

namespace cg = cooperative_groups;

namespace fgemm {

namespace {

using u64 = unsigned long long;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kUnit = 44;  // masses are multiples of 2^-44
constexpr u64 kOne = 1ull << kUnit;
constexpr int kMaxCluster = 8;

// 2^(j/32) in units of 2^-44.
__constant__ u64 kPow[32] = {
    17592186044416ull, 17977404757381ull, 18371058661769ull, 18773332464219ull,
    19184414915921ull, 19604498901178ull, 20033781527906ull, 20472464220127ull,
    20920752812471ull, 21378857646762ull, 21846993670708ull, 22325380538761ull,
    22814242715178ull, 23313809579344ull, 23824315533396ull, 24346000112214ull,
    24879108095804ull, 25423889624159ull, 25980600314626ull, 26549501381838ull,
    27130859760289ull, 27724948229574ull, 28332045542385ull, 28952436555301ull,
    29586412362452ull, 30234270432094ull, 30896314746195ull, 31572855943056ull,
    32264211463077ull, 32970705697691ull, 33692670141585ull, 34430443548229ull,
};

// Bins that masses above 2^-14 fall into: (m - x) / T < 14 ln 2 = 9.71, 32 bins to 1.
constexpr int kFewBins = 311;
constexpr int kList = 2048;
constexpr int kLimb = 15;  // bits: a CTA's slice of 2^17 logits cannot overflow a 32-bit sum of limbs

struct SampleShared {
  unsigned int hist[3][kBins];  // sums of the masses' limbs (counts: the first)
  u64 list[kList];              // the short list (rank 0): key, then the index from above
  u64 mass[kList];              // its masses; before, this CTA's part of the list
  u64 pow[32];
  float powf[32];
  u64 warp64[kWarps];
  u64 warp64b[kWarps];
  u64 total;         // this CTA's sum, read by the others
  u64 sel_before;    // what lies above the selected bin
  u64 sel_upto;      // and with it
  unsigned int gathered, place;
  int sel_bin;
  unsigned int warp32[kWarps];
  unsigned int best; // this CTA's largest key
  unsigned int count;
  int found;         // index located by locate(), in the CTA that finds it
  u64 found_mass;
  unsigned int range[2];
  float ch, cl;      // log2(e) / temperature in two floats
};

// Keys: order of floats as unsigned integers (x is never NaN, -0 never).
__device__ __forceinline__ unsigned int key_of(float x) {
  const unsigned int b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned int k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// exp((x - m) / T) in units of 2^-44, to about 2^-36 (of its value, or of 1 for
// masses below 2^-14).  y = (x - m) log2(e) / T is held as a sum of two floats (x - m and its
// rounding error by a two-sum, the product's error by an fma); then
// 2^y = 2^n 2^(j/32) 2^r with a table for 2^(j/32) and the exponential series
// for 2^r, |r| <= 1/64, whose first-order term is again kept in two floats.
// Numbers become integers by adding 1.5 2^23, whose unit in the last place is
// 1: the conversion instruction runs at a fraction of the rate.
struct Masses {
  float m, ch, cl;  // ch + cl = log2(e) / T
  const u64* pow;
  const float* powf;  // 2^(j/32)
  // How small a mass is: y rounded, from which low() or high() goes on.
  __device__ __forceinline__ float size(float x) const { return x == m ? 0.0f : fmaf(x - m, ch, (x - m) * cl); }
  // A mass below 2^-14: fp32 is enough for its 30 bits (the error is below
  // 2^-36 of m's mass, and not of one sign).
  static constexpr float kSmall = -14.0f;
  __device__ __forceinline__ unsigned int low(float y) const {
    constexpr float magic = 12582912.0f;
    constexpr int magic_bits = 0x4B400000;
    // without branches, so that a thread's logits go through side by side
    const float c = fminf(fmaxf(y, -46.0f), kSmall);
    const float t = fmaf(c, 32.0f, magic);  // 32 y, rounded
    const int j = __float_as_int(t) - magic_bits;
    const float z = fmaf(t - magic, -0.03125f, c) * 0.693147182464599609375f;
    const float p = z * fmaf(z, fmaf(z, 1.0f / 6, 0.5f), 1.0f);
    const float f = powf[j & 31];
    const unsigned int w = __float2uint_rn(fmaf(f, p, f) * __int_as_float((44 + (j >> 5) + 127) << 23));
    return y > -46.0f ? w : 0;
  }
  __device__ __forceinline__ u64 operator()(float x) const {
    const float y = size(x);
    return y > kSmall ? high(x) : low(y);
  }
  __device__ __forceinline__ u64 high(float x) const {
    constexpr float magic = 12582912.0f;
    constexpr int magic_bits = 0x4B400000;
    if (x == m) return kOne;
    const float s = x - m;
    const float yh = __fmul_rn(s, ch);  // rounded here: not to be fused into a sum below
    const float bb = s - x;
    const float e = (x - (s - bb)) + (-m - bb);
    const float yl = fmaf(s, ch, -yh) + fmaf(s, cl, e * ch);
    const float t = fmaf(yh, 32.0f, magic);  // 32 y, rounded
    const int j = __float_as_int(t) - magic_bits;
    const float r = fmaf(t - magic, -0.03125f, yh);
    constexpr float l1 = 0.693147182464599609375f, l2 = -1.90465429995776804525e-09f;  // ln 2
    const float zh = __fmul_rn(r, l1);
    const float zl = fmaf(r, l1, -zh) + fmaf(r, l2, yl * l1);
    const float q = zh * zh * fmaf(zh, fmaf(zh, fmaf(zh, 1.0f / 120, 1.0f / 24), 1.0f / 6), 0.5f);
    // zh + q + zl in units of 2^-37: the upper part in units of 2^-22, the rest
    const float t2 = fmaf(zh + q, 4194304.0f, magic);
    const float rest = (fmaf(t2 - magic, -2.384185791015625e-07f, zh) + q) + zl;
    const float t3 = fmaf(rest, 137438953472.0f, magic);
    const int series = ((__float_as_int(t2) - magic_bits) << 15) + (__float_as_int(t3) - magic_bits);
    const u64 p = pow[j & 31];
    const u64 v = p + static_cast<u64>((static_cast<long long>(static_cast<int>(p >> 15)) * series) >> 22);
    const int shift = -(j >> 5);
    return (v + ((1ull << shift) >> 1)) >> shift;
  }
};

// a f for 0 < f < 1 exactly, rounded down or up.
__device__ __forceinline__ u64 times(u64 a, float f, bool up) {
  if (!(f < 1.0f)) return a;
  const int b = __float_as_int(f), field = b >> 23;
  const u64 m = field ? (b & 0x7FFFFF) | 0x800000 : b;
  const int e = 150 - (field ? field : 1);  // f = m 2^-e, e >= 24
  const u64 lo = a * m, hi = __umul64hi(a, m);
  u64 v, rest;
  if (e < 64) {
    v = (hi << (64 - e)) | (lo >> e);
    rest = lo & ((1ull << e) - 1);
  } else {
    const int h = e - 64;
    v = h < 64 ? hi >> h : 0;
    rest = lo | (h < 64 ? hi & ((1ull << h) - 1) : hi);
  }
  return v + (up && rest ? 1 : 0);
}

template <typename T>
__device__ __forceinline__ float raw_value(T v);
template <>
__device__ __forceinline__ float raw_value<float>(float v) { return v; }
template <>
__device__ __forceinline__ float raw_value<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float raw_value<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : x + 0.0f; }

// A CTA's slice [first, first + len) of its row.  Vector v of thread lane:
// E consecutive elements, E = 16 bytes' worth; a warp's vectors are
// consecutive, so (round, warp, lane, element) is index order.
template <typename T, bool CACHED>
struct Slice {
  static constexpr int E = 16 / sizeof(T);
  const T* global;  // the slice's first logit
  T* cache;
  int len, rounds;
  __device__ __forceinline__ void get(int vec, float (&x)[E]) const {
    if (CACHED) {
      const uint4 raw = reinterpret_cast<const uint4*>(cache)[vec];
      const T* v = reinterpret_cast<const T*>(&raw);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = clean(raw_value<T>(v[e]));
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = vec * E + e < len ? clean(raw_value<T>(global[vec * E + e])) : -INFINITY;
    }
  }
  // f(x, index in the slice) for every element of this thread
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int r = 0; r < rounds; ++r) {
      const int vec = r * kThreads + threadIdx.x;
      float x[E];
      get(vec, x);
#pragma unroll
      for (int e = 0; e < E; ++e) f(x[e], vec * E + e);
    }
  }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 a = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += a;
  }
  return v;
}

struct Threshold {
  unsigned int key;  // larger keys are in
  int bin;           // of the first histogram, when the search stopped there (key 0)
  u64 above;         // the count or mass of larger keys
  u64 upto;          // the sum of the first histogram's bins down to the one found
  u64 target;
  int last;          // of the logits at `key`: the index of the last one in, -1 when not known
};

// Descending bitonic sort of n (a power of two, at most kList) numbers.
__device__ void sort_down(u64* a, int n) {
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < n / 2; i += kThreads) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const u64 x = a[lo], y = a[hi];
        if ((x < y) == ((lo & k) == 0)) {
          a[lo] = y;
          a[hi] = x;
        }
      }
      __syncthreads();
    }
}

// Inclusive sums of v[0 .. n) in place; n <= kList.  Returns the whole.
__device__ u64 scan_list(SampleShared& sh, u64* v, int n) {
  constexpr int kEach = kList / kThreads;
  u64 x[kEach], s = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = threadIdx.x * kEach + i;
    x[i] = at < n ? v[at] : 0;
    s += x[i];
  }
  const u64 upto = warp_scan(s);
  if ((threadIdx.x & 31) == 31) sh.warp64b[threadIdx.x >> 5] = upto;
  __syncthreads();
  u64 before = upto - s, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < (threadIdx.x >> 5)) before += sh.warp64b[w];
    all += sh.warp64b[w];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    before += x[i];
    const int at = threadIdx.x * kEach + i;
    if (at < n) v[at] = before;
  }
  __syncthreads();
  return all;
}

// How many of the ascending v[0 .. n) are below t (by every thread).
__device__ __forceinline__ int below(const u64* v, int n, u64 t) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] < t) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// The logits with in(x), of all CTAs, gathered in rank 0's list.  Returns how
// many there are (to every CTA); above kList the list is not complete.
template <typename S, typename P>
__device__ int gather(const S& slice, SampleShared& sh, cg::cluster_group& cluster, int first, P in) {
  slice.each([&](float x, int i) {
    if (!in(x)) return;
    const unsigned int at = atomicAdd(&sh.gathered, 1u);
    if (at < kList)
      sh.mass[at] = static_cast<u64>(key_of(x)) << 32 | (0xFFFFFFFFu - static_cast<unsigned int>(first + i));
  });
  __syncthreads();
  const unsigned int mine = sh.gathered;
  if (threadIdx.x == 0) sh.found = static_cast<int>(atomicAdd(cluster.map_shared_rank(&sh.place, 0), mine));
  __syncthreads();
  const unsigned int base = static_cast<unsigned int>(sh.found);
  if (base + mine <= kList) {
    u64* const to = cluster.map_shared_rank(&sh.list[0], 0) + base;
    for (unsigned int i = threadIdx.x; i < mine; i += kThreads) to[i] = sh.mass[i];
  }
  cluster.sync();
  return static_cast<int>(*cluster.map_shared_rank(&sh.place, 0));
}

// The threshold's bin, when few logits are in it: sorted and summed in rank 0.
template <typename S, typename P>
__device__ bool short_border(const S& slice, SampleShared& sh, cg::cluster_group& cluster, int first,
                             const Masses& mass, Threshold& res, P in) {
  const int n = gather(slice, sh, cluster, first, in);
  if (n > kList) {
    cluster.sync();  // sh.place has been read
    return false;
  }
  if (cluster.block_rank() == 0) {
    if (n <= kThreads) {  // each entry finds what is before it by itself
      const u64 mine = threadIdx.x < n ? sh.list[threadIdx.x] : 0;
      const u64 w = threadIdx.x < n ? mass(value_of(static_cast<unsigned int>(mine >> 32))) : 0;
      if (threadIdx.x < n) sh.mass[threadIdx.x] = w;
      if (threadIdx.x == 0) sh.range[0] = 0;
      __syncthreads();
      u64 before = res.above;
      if (threadIdx.x < n)
        for (int i = 0; i < n; ++i) before += sh.list[i] > mine ? sh.mass[i] : 0;
      if (threadIdx.x < n && before < res.target && res.target <= before + w) {
        sh.range[0] = static_cast<unsigned int>(mine >> 32);
        sh.found = static_cast<int>(0xFFFFFFFFu - static_cast<unsigned int>(mine));
      }
    } else {
      int size = 2;
      while (size < n) size <<= 1;
      for (int i = n + threadIdx.x; i < size; i += kThreads) sh.list[i] = 0;
      __syncthreads();
      sort_down(sh.list, size);
      for (int i = threadIdx.x; i < n; i += kThreads)
        sh.mass[i] = mass(value_of(static_cast<unsigned int>(sh.list[i] >> 32)));
      __syncthreads();
      scan_list(sh, sh.mass, n);
    }
    if (n > kThreads && threadIdx.x == 0) {
      const int at = min(below(sh.mass, n, res.target - res.above), n - 1);
      sh.range[0] = static_cast<unsigned int>(sh.list[at] >> 32);
      sh.found = static_cast<int>(0xFFFFFFFFu - static_cast<unsigned int>(sh.list[at]));
    }
  }
  cluster.sync();
  res.key = cluster.map_shared_rank(&sh.range[0], 0)[0];
  res.last = *cluster.map_shared_rank(&sh.found, 0);
  cluster.sync();  // both have been read
  return true;
}

// The key at which the sum of 1 (COUNT) or of the masses over the logits with
// is_in(x), from the largest down, reaches target_of(the whole sum; for counts:
// of the bins).  Counts: the search stops after the first histogram (key 0) when the bins down to the one found
// hold at most kList.  Masses: it stops there (key 0) when the target lies
// above their sum.  Every thread of the cluster gets the result.
//
// Masses are summed in three 32-bit limbs of 15 bits: shared-memory atomics
// of 32 bits are native, those of 64 a loop.
template <bool COUNT, typename S, typename I, typename G>
__device__ Threshold find_threshold(const S& slice, SampleShared& sh, cg::cluster_group& cluster, const Masses& mass,
                                    float scale, int first_index, I is_in, G target_of) {
  const float m = mass.m;
  const int ranks = cluster.num_blocks();
  Threshold res;
  res.key = 0;
  res.bin = 0;
  res.above = 0;
  res.upto = 0;
  res.target = 0;
  res.last = -1;
  unsigned int lo = 0, hi = 0xFFFFFFFFu;  // keys still in question, once `linear` is done
  bool linear = true;
  bool few = !COUNT;  // the first histogram has bins for large masses only
  int shift = 0;
  auto bin_of = [&](float x) -> int {
    if (linear) return x == m ? 0 : static_cast<int>(fminf((m - x) * scale, kBins - 1.0f));
    const unsigned int k = key_of(x);
    return k < lo || k > hi ? -1 : static_cast<int>((hi - k) >> shift);
  };
  while (true) {
    for (int b = threadIdx.x; b < kBins; b += kThreads) {
      sh.hist[0][b] = 0;
      if (!COUNT) {
        sh.hist[1][b] = 0;
        sh.hist[2][b] = 0;
      }
    }
    if (threadIdx.x == 0) sh.sel_bin = kBins - 1;
    __syncthreads();
    u64 rest = 0;  // in units of 2^-44, of this thread's small masses (first histogram)
    if (COUNT) {
      // the last linear bin holds all that lies far below: it is what is left
      slice.each([&](float x, int) {
        const int b = bin_of(x);
        if (b < 0 || (linear && b == kBins - 1)) return;
        if (is_in(x)) atomicAdd(&sh.hist[0][b], 1u);
      });
    } else {
      constexpr unsigned int mask = (1u << kLimb) - 1;
      constexpr int E = S::E;
      const int lane = threadIdx.x & 31;
      float* const room = reinterpret_cast<float*>(sh.mass) + (threadIdx.x >> 5) * (32 * E);
      for (int r = 0; r < slice.rounds; ++r) {
        float x[E];
        slice.get(r * kThreads + threadIdx.x, x);
        bool dense[E];  // its mass takes long: on full warps
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float y = mass.size(x[e]);
          const bool in = is_in(x[e]);
          if (few) {  // large masses into bins; small ones only into their sum
            dense[e] = in && y > Masses::kSmall;
            const unsigned int w = mass.low(y);
            rest += in && !dense[e] ? w : 0;
          } else {
            dense[e] = in && y > -46.0f && bin_of(x[e]) >= 0;
          }
        }
        int n = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const unsigned int who = __ballot_sync(0xFFFFFFFFu, dense[e]);
          if (dense[e]) room[n + __popc(who & ((1u << lane) - 1))] = x[e];
          n += __popc(who);
        }
        __syncwarp();
        for (int i = lane; i < n; i += 32) {
          const float v = room[i];
          const int b = bin_of(v);
          const u64 w = mass(v);
          atomicAdd(&sh.hist[0][b], static_cast<unsigned int>(w) & mask);
          if (w >> kLimb) atomicAdd(&sh.hist[1][b], static_cast<unsigned int>(w >> kLimb) & mask);
          if (w >> (2 * kLimb)) atomicAdd(&sh.hist[2][b], static_cast<unsigned int>(w >> (2 * kLimb)));
        }
        __syncwarp();
      }
      if (few) {
        rest = warp_sum(rest);
        if (lane == 0) sh.warp64b[threadIdx.x >> 5] = rest;
        __syncthreads();
        if (threadIdx.x < 32) {
          rest = warp_sum(lane < kWarps ? sh.warp64b[lane] : 0);
          if (lane == 0) sh.total = rest;
        }
      }
    }
    cluster.sync();
    // thread t: bins 2t and 2t + 1 over all CTAs
    u64 v[2] = {0, 0};
    u64 rests = 0;
    if (COUNT) {
      unsigned int h[kMaxCluster][2];  // all on their way together
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        const unsigned int* const at = cluster.map_shared_rank(&sh.hist[0][0], r < ranks ? r : 0) + 2 * threadIdx.x;
        h[r][0] = at[0];
        h[r][1] = at[1];
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < ranks) v[0] += h[r][0], v[1] += h[r][1];
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (few && 2 * threadIdx.x + i >= kFewBins) break;
        unsigned int h[kMaxCluster][3];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          const unsigned int* const at =
              cluster.map_shared_rank(&sh.hist[0][0], r < ranks ? r : 0) + 2 * threadIdx.x + i;
          h[r][0] = at[0];
          h[r][1] = at[kBins];
          h[r][2] = at[2 * kBins];
        }
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < ranks)
            v[i] += h[r][0] + (static_cast<u64>(h[r][1]) << kLimb) + (static_cast<u64>(h[r][2]) << (2 * kLimb));
      }
      if (few)
        for (int r = 0; r < ranks; ++r) rests += *cluster.map_shared_rank(&sh.total, r);
    }
    const u64 mine = warp_scan(v[0] + v[1]);
    if ((threadIdx.x & 31) == 31) sh.warp64[threadIdx.x >> 5] = mine;
    __syncthreads();
    u64 before = res.above + mine - v[0] - v[1];
    u64 all = res.above;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < (threadIdx.x >> 5)) before += sh.warp64[w];
      all += sh.warp64[w];
    }
    if (linear) res.target = target_of(all + rests);
    const u64 target = res.target;
    if (threadIdx.x == 0) {  // the last linear bin, unless another bin reaches the target
      sh.sel_before = all;
      sh.sel_upto = ~0ull;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (before < target && target <= before + v[i]) {
        sh.sel_bin = 2 * threadIdx.x + i;
        sh.sel_before = before;
        sh.sel_upto = before + v[i];
      }
      before += v[i];
    }
    cluster.sync();  // the others are done with this CTA's histogram
    const int bin = sh.sel_bin;
    res.above = sh.sel_before;
    if (linear) {
      res.bin = bin;
      res.upto = sh.sel_upto;
      if (COUNT && res.upto <= kList) return res;
      if (!COUNT && few) {
        if (res.target > res.above && res.upto == ~0ull && res.target > res.above + rests) return res;
        // (above is what the bins hold when none of them reaches the target;
        // the last of them also has small masses that are not in it)
        if (res.upto == ~0ull || bin >= kFewBins - 1) {  // among the small masses: all over again with bins for them
          few = false;
          res.above = 0;
          __syncthreads();
          continue;
        }
      }
      if (!COUNT && res.upto == ~0ull) return res;
      if (!COUNT && short_border(slice, sh, cluster, first_index, mass, res,
                                 [&](float x) { return bin_of(x) == bin && is_in(x); }))
        return res;
      // The bin's key range: keys at which bin_of, which falls as keys grow, is
      // `bin`.  Thread 0: the smallest key with bin_of <= bin; thread 1: the
      // largest with bin_of >= bin.  Each begins where the bin's edge lies
      // before rounding and widens its step until the key is enclosed.
      if (threadIdx.x < 2) {
        const bool low = threadIdx.x == 0;
        const unsigned int first = key_of(-INFINITY), last = key_of(m);
        const float edge = m - (static_cast<float>(bin) + (low ? 1.0f : 0.0f)) / scale;
        unsigned int at = edge == edge ? key_of(edge + 0.0f) : last;
        at = at < first ? first : at > last ? last : at;
        auto ok = [&](unsigned int k) { return low ? bin_of(value_of(k)) <= bin : bin_of(value_of(k)) >= bin; };
        unsigned int good, bad, step = 4;  // the key sought lies from good towards bad, bad excluded
        const unsigned int end_good = low ? last : first, end_bad = low ? first : last;
        if (ok(at)) {
          good = at;
          while (true) {  // towards bad
            const unsigned int room = low ? good - end_bad : end_bad - good;
            if (room == 0) break;
            const unsigned int d = step < room ? step : room;
            const unsigned int k = low ? good - d : good + d;
            if (!ok(k)) {
              bad = k;
              break;
            }
            good = k;
            step = step < 0x40000000u ? step * 4 : step;
          }
          if (good == end_bad) bad = good;
        } else {
          bad = at;
          good = end_good;
          while (true) {  // towards good
            const unsigned int room = low ? end_good - bad : bad - end_good;
            const unsigned int d = step < room ? step : room;
            const unsigned int k = low ? bad + d : bad - d;
            if (d == 0 || ok(k)) {
              good = k;
              break;
            }
            bad = k;
            step = step < 0x40000000u ? step * 4 : step;
          }
        }
        while (low ? good > bad + 1 && good != bad : bad > good + 1) {
          const unsigned int mid = low ? bad + (good - bad) / 2 : good + (bad - good) / 2;
          if (ok(mid)) good = mid; else bad = mid;
        }
        sh.range[threadIdx.x] = good;
      }
      __syncthreads();
      lo = sh.range[0];
      hi = sh.range[1];
      linear = false;
      few = false;
    } else {
      const unsigned int top = hi - (static_cast<unsigned int>(bin) << shift);
      const unsigned int width = (1u << shift) - 1;
      lo = top - lo > width ? top - width : lo;
      hi = top;
    }
    // sel_bin, sel_before and range have been read: the next round, or the next
    // search, writes sel_bin before its first barrier
    __syncthreads();
    if (lo >= hi) break;
    const int bits = 32 - __clz(hi - lo);
    shift = bits > 10 ? bits - 10 : 0;
  }
  res.key = lo;
  return res;
}

// The first index of the row at which the running sum of weight(x, index)
// exceeds target(whole sum); -1 if the whole sum is 0.  Every thread of the
// cluster gets it; *mass is full_of that element and *whole the sum.
//
// A warp sums the weights of its vectors of a round; with DENSE, in_sum(x,
// index) says which of them have one (none below floor_x), and those are first
// moved together, so that weight_of (costly) is evaluated on full warps.
template <bool DENSE, typename S, typename I, typename V, typename F, typename G>
__device__ int locate(const S& slice, SampleShared& sh, u64* segs, cg::cluster_group& cluster, int first, float floor_x, I in_sum,
                      V weight_of, F full_of, G target_of, u64* mass, u64* whole) {
  auto weight = [&](float x, int i) -> u64 { return in_sum(x, i) ? weight_of(x) : 0; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  constexpr int E = S::E;
  u64 sum = 0;
  for (int r = 0; r < slice.rounds; ++r) {
    const int vec = r * kThreads + threadIdx.x;
    float x[E];
    slice.get(vec, x);
    u64 s = 0;
    if (DENSE) {
      float* const room = reinterpret_cast<float*>(sh.mass) + warp * (32 * E);
      int n = 0;
      float most = x[0];
#pragma unroll
      for (int e = 1; e < E; ++e) most = fmaxf(most, x[e]);
      if (__any_sync(0xFFFFFFFFu, most >= floor_x))
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool in = in_sum(x[e], vec * E + e);
        const unsigned int who = __ballot_sync(0xFFFFFFFFu, in);
        if (in) room[n + __popc(who & ((1u << lane) - 1))] = x[e];
        n += __popc(who);
      }
      __syncwarp();
      for (int i = lane; i < n; i += 32) s += weight_of(room[i]);
      __syncwarp();
      if (n) s = warp_sum(s);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) s += weight(x[e], vec * E + e);
      s = warp_sum(s);
    }
    if (lane == 0) segs[r * kWarps + warp] = s;
    sum += s;
  }
  if (lane == 0) sh.warp64[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    const u64 t = warp_sum(lane < kWarps ? sh.warp64[lane] : 0);
    if (lane == 0) {
      sh.total = t;
      sh.found = -1;
    }
  }
  cluster.sync();
  u64 all = 0, before = 0, own = 0, totals[kMaxCluster];
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) totals[r] = *cluster.map_shared_rank(&sh.total, r < ranks ? r : 0);
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) {
    const u64 t = r < ranks ? totals[r] : 0;
    if (r < rank) before += t;
    if (r == rank) own = t;
    all += t;
  }
  const u64 target = all ? target_of(all) : 0;
  *whole = all;
  if (all && before <= target && target < before + own) {
    // the segment, as many at a time as there are threads, then the element in it
    const int n = slice.rounds * kWarps;
    u64 base = before;
    if (threadIdx.x == 0) sh.sel_bin = -1;
    for (int s0 = 0; s0 < n; s0 += kThreads) {
      const int seg = s0 + threadIdx.x;
      const u64 v = seg < n ? segs[seg] : 0;
      const u64 upto = warp_scan(v);
      if (lane == 31) sh.warp64b[warp] = upto;
      __syncthreads();
      u64 from = base + upto - v;
      for (int w = 0; w < kWarps; ++w) {
        const u64 t = sh.warp64b[w];
        if (w < warp) from += t;
        base += t;
      }
      if (from <= target && target < from + v) {
        sh.sel_bin = seg;
        sh.sel_before = from;
      }
      __syncthreads();
      if (sh.sel_bin >= 0) break;
    }
    if (warp == 0) {
      const int seg = sh.sel_bin;
      const int vec = (seg / kWarps) * kThreads + (seg % kWarps) * 32 + lane;
      float x[E];
      slice.get(vec, x);
      u64 w[E], s = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        w[e] = weight(x[e], vec * E + e);
        s += w[e];
      }
      u64 run = sh.sel_before + warp_scan(s) - s;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (run <= target && target < run + w[e]) {
          sh.found = first + vec * E + e;
          sh.found_mass = full_of(x[e]);
        }
        run += w[e];
      }
    }
  }
  cluster.sync();
  int found = -1, at[kMaxCluster];
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) at[r] = *cluster.map_shared_rank(&sh.found, r < ranks ? r : 0);
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < ranks && at[r] >= 0) {
      found = at[r];
      *mass = *cluster.map_shared_rank(&sh.found_mass, r);
    }
  cluster.sync();  // sh.total and sh.found may be written again
  return found;
}

// One CTA finishes on the short list: all logits of the row that can be kept
// are among its n entries.
__device__ void finish_list(SampleShared& sh, const Masses& mass, int n, int top_k, float top_p, u64 least, float u,
                            int* token, float* prob) {
  if (n <= kThreads) {
    // Without a sort: each entry adds up what comes before it, by rank, then
    // by index.
    const bool here = threadIdx.x < n;
    const u64 mine = here ? sh.list[threadIdx.x] : 0;
    int rank = 0;
    if (here)
      for (int i = 0; i < n; ++i) rank += sh.list[i] > mine;
    u64 w = here && rank < top_k ? mass(value_of(static_cast<unsigned int>(mine >> 32))) : 0;
    if (here) sh.mass[threadIdx.x] = w;
    __syncthreads();
    if (top_p < 1.0f) {
      u64 before = 0, whole = 0;
      if (here)
        for (int i = 0; i < n; ++i) {
          const u64 v = sh.mass[i];
          whole += v;
          before += sh.list[i] > mine ? v : 0;
        }
      const u64 target = times(whole, top_p, true);
      if (before >= (target < 1 ? 1 : target)) w = 0;
    }
    if (rank > 0 && w < least) w = 0;
    __syncthreads();
    if (here) sh.mass[threadIdx.x] = w;
    __syncthreads();
    u64 before = 0, kept = 0;
    if (here && w)
      for (int i = 0; i < n; ++i) {
        const u64 v = sh.mass[i];
        kept += v;  // a lower index is a larger lower half
        before += static_cast<unsigned int>(sh.list[i]) > static_cast<unsigned int>(mine) ? v : 0;
      }
    const u64 at = times(kept, u, false);
    if (here && w && before <= at && at < before + w) {
      *token = static_cast<int>(0xFFFFFFFFu - static_cast<unsigned int>(mine));
      w = mass.high(value_of(static_cast<unsigned int>(mine >> 32)));  // (its probability is told to fp32 precision)
      if (prob) *prob = static_cast<float>(static_cast<double>(w) / static_cast<double>(kept));
    }
    return;
  }
  int size = 2;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kThreads) sh.list[i] = 0;
  __syncthreads();
  sort_down(sh.list, size);
  n = min(n, top_k);
  for (int i = threadIdx.x; i < n; i += kThreads) sh.mass[i] = mass(value_of(static_cast<unsigned int>(sh.list[i] >> 32)));
  __syncthreads();
  const u64 whole = scan_list(sh, sh.mass, n);
  int keep = n;
  if (top_p < 1.0f) {
    const u64 target = times(whole, top_p, true);
    keep = min(n, below(sh.mass, n, target < 1 ? 1 : target) + 1);
  }
  if (least > 0) {  // masses fall along the list
    int lo = 1, hi = keep;
    while (lo < hi) {  // the first entry from 1 on that is too small
      const int mid = (lo + hi) >> 1;
      if (mass(value_of(static_cast<unsigned int>(sh.list[mid] >> 32))) >= least) lo = mid + 1; else hi = mid;
    }
    keep = lo;
  }
  __syncthreads();
  // by index: the entries' lower half is the index from above, so its order
  // is that of falling entries
  size = 2;
  while (size < keep) size <<= 1;
  for (int i = threadIdx.x; i < size; i += kThreads)
    sh.list[i] = i < keep ? (sh.list[i] << 32) | (sh.list[i] >> 32) : 0;
  __syncthreads();
  sort_down(sh.list, size);
  for (int i = threadIdx.x; i < keep; i += kThreads) sh.mass[i] = mass(value_of(static_cast<unsigned int>(sh.list[i])));
  __syncthreads();
  const u64 kept = scan_list(sh, sh.mass, keep);
  if (threadIdx.x == 0) {
    const int at = below(sh.mass, keep, times(kept, u, false) + 1);  // the first sum above u times the whole
    const u64 w = mass.high(value_of(static_cast<unsigned int>(sh.list[at])));
    *token = static_cast<int>(0xFFFFFFFFu - static_cast<unsigned int>(sh.list[at] >> 32));
    if (prob) *prob = static_cast<float>(static_cast<double>(w) / static_cast<double>(kept));
  }
}

template <typename T, bool CACHED>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ SampleShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int row = blockIdx.x / ranks;
  constexpr int E = 16 / sizeof(T);

  Slice<T, CACHED> slice;
  const int per = p.slice;
  // The slice takes per - pad logits: as many as fit behind a start that is
  // not on 16 bytes.  `first` is the index of the vectors' first element.
  const int begin = min(rank * (per - p.pad), p.vocab), len = min(p.vocab - begin, per - p.pad);
  const T* const from = static_cast<const T*>(p.logits) + row * p.ld + begin;
  const int shift = CACHED ? static_cast<int>(reinterpret_cast<uintptr_t>(from) % 16 / sizeof(T)) : 0;
  const int first = begin - shift;
  slice.len = len;
  slice.rounds = per / (kThreads * E);
  slice.global = from - shift;
  u64* segs = reinterpret_cast<u64*>(dyn);
  slice.cache = reinterpret_cast<T*>(dyn + static_cast<size_t>(slice.rounds) * kWarps * 8);
  if (threadIdx.x < 32) {
    sh.pow[threadIdx.x] = kPow[threadIdx.x];
    sh.powf[threadIdx.x] = static_cast<float>(kPow[threadIdx.x]) * 0x1p-44f;
  }

  // the slice into shared memory, its largest key and its candidates
  float top = -INFINITY;
  unsigned int count = 0;
  if (CACHED) {
    // Vectors from the 16-byte boundary at or before the slice; what lies
    // outside it counts as -inf.
#pragma unroll 4
    for (int v = threadIdx.x; v < per / E; v += kThreads) {
      uint4 raw;
      const int i0 = v * E - shift;  // of the slice
      if (i0 >= 0 && i0 + E <= len) {
        raw = *reinterpret_cast<const uint4*>(slice.global + v * E);
      } else {
        T part[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
          part[e] = i0 + e >= 0 && i0 + e < len ? slice.global[v * E + e] : static_cast<T>(-INFINITY);
        memcpy(&raw, part, 16);
      }
      reinterpret_cast<uint4*>(slice.cache)[v] = raw;
      T part[E];
      memcpy(part, &raw, 16);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = clean(raw_value<T>(part[e]));
        top = fmaxf(top, x);
        count += x > -INFINITY;
      }
    }
  } else {
    slice.each([&](float x, int) {
      top = fmaxf(top, x);
      count += x > -INFINITY;
    });
  }
  const float temperature = p.temperature ? p.temperature[row] : p.temperature0;
  const float top_p = p.top_p ? p.top_p[row] : p.top_p0;
  const float min_p = p.min_p ? p.min_p[row] : p.min_p0;
  const int top_k = p.top_k ? p.top_k[row] : p.top_k0;
  // the largest float below 1 stands for anything above it, 0 for anything below and for NaN
  const float u = fminf(fmaxf(p.u[row], 0.0f), 0.999999940395355224609375f);
  const bool greedy = !(temperature > 0.0f) || top_k == 1 || top_p <= 0.0f || min_p > 1.0f;
  if (threadIdx.x == 0) {
    sh.gathered = 0;
    sh.place = 0;
    const double c = 1.4426950408889634074 / static_cast<double>(greedy ? 1.0f : temperature);
    sh.ch = static_cast<float>(c);
    sh.cl = isinf(sh.ch) ? 0.0f : static_cast<float>(c - static_cast<double>(sh.ch));
  }
  unsigned int best = key_of(top);
  best = __reduce_max_sync(0xFFFFFFFFu, best);
  count = __reduce_add_sync(0xFFFFFFFFu, count);
  if ((threadIdx.x & 31) == 0) {
    sh.warp32[threadIdx.x >> 5] = best;
    sh.warp64[threadIdx.x >> 5] = count;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    count = 0;
    for (int w = 0; w < kWarps; ++w) {
      best = max(best, sh.warp32[w]);
      count += static_cast<unsigned int>(sh.warp64[w]);
    }
    sh.best = best;
    sh.count = count;
  }
  cluster.sync();
  best = 0;
  count = 0;
  for (int r = 0; r < ranks; ++r) {
    best = max(best, *cluster.map_shared_rank(&sh.best, r));
    count += *cluster.map_shared_rank(&sh.count, r);
  }
  const float m = value_of(best);
  int token = -1;
  float prob = 0.0f;
  if (count) {
    Masses mass;
    mass.m = m;
    mass.pow = sh.pow;
    mass.powf = sh.powf;
    mass.ch = sh.ch;
    mass.cl = sh.cl;
    // logits below this have no mass, or less than min_p
    float floor_x = m - 32.5f * temperature;
    if (min_p > 0.0f) floor_x = fmaxf(floor_x, m + temperature * (__logf(min_p) - 0.01f) - fabsf(m) * 1e-6f);
    if (!(floor_x == floor_x)) floor_x = -INFINITY;
    const float scale = kBins / (32.0f * (greedy ? 1.0f : temperature));

    // kept: keys above `cut`, and those at `cut` up to index `last`
    unsigned int cut = 0;
    int last = p.vocab;
    u64 ties = 0;  // how many at `cut`; 0: all
    u64 above = 0;
    if (greedy) {
      cut = best;
      ties = 1;
    } else {
      if (top_k > 0 && static_cast<unsigned int>(top_k) < count) {
        const Threshold t = find_threshold<true>(
            slice, sh, cluster, mass, scale, first, [](float x) { return x > -INFINITY; },
            [&](u64) { return static_cast<u64>(top_k); });
        if (t.key == 0) {  // a short list: everything in the bins down to t.bin
          gather(slice, sh, cluster, first, [&](float x) {
            return x > -INFINITY && (x == m || fminf((m - x) * scale, kBins - 1.0f) < t.bin + 1.0f);
          });
          cluster.sync();  // sh.place has been read
          if (rank == 0)
            finish_list(sh, mass, static_cast<int>(t.upto), top_k, top_p, min_p > 0.0f ? times(kOne, min_p, true) : 0, u,
                        p.token + row, p.prob ? p.prob + row : nullptr);
          return;  // nobody reads another CTA's memory any more
        }
        cut = t.key;
        ties = static_cast<u64>(top_k) - t.above;
      }
      if (top_p < 1.0f) {
        // of what top-k keeps: the mass above its threshold, and the ties'
        const u64 at_cut = ties ? mass(value_of(cut)) : 0;
        const Threshold t = find_threshold<false>(
            slice, sh, cluster, mass, scale, first,
            [&](float x) { return x > -INFINITY && key_of(x) > cut; },
            [&](u64 all) {
              above = all;
              const u64 target = times(all + ties * at_cut, top_p, true);
              return target < 1 ? static_cast<u64>(1) : target;
            });
        if (t.target > above) {  // the prefix ends among the ties at top-k's threshold
          const u64 need = (t.target - above + at_cut - 1) / at_cut;
          ties = need < ties ? need : ties;
        } else {
          cut = t.key;
          if (t.last >= 0) {
            last = t.last;
            ties = 0;
          } else {
            const u64 each = mass(value_of(cut));
            ties = (t.target - t.above + each - 1) / each;
          }
        }
      }
    }
    u64 chosen = 0, whole = 0;
    if (ties)  // the index of the last tie that is kept
      last = locate<false>(
          slice, sh, segs, cluster, first, -INFINITY, [&](float x, int) { return key_of(x) == cut; },
          [](float) -> u64 { return 1; }, [](float) -> u64 { return 1; },
          [&](u64 all) -> u64 { return (ties < all ? ties : all) - 1; }, &chosen, &whole);
    if (greedy) {
      token = last;
      prob = 1.0f;
    } else {
      const u64 least = min_p > 0.0f ? times(kOne, min_p, true) : 0;
      const float limit = cut ? value_of(cut) : -INFINITY, lowest = fmaxf(floor_x, limit);
      token = locate<true>(
          slice, sh, segs, cluster, first, lowest,
          [&](float x, int i) { return x > lowest || (x == lowest && x > -INFINITY && (x > limit || first + i <= last)); },
          [&](float x) -> u64 {
            const u64 w = mass(x);
            return w >= least ? w : 0;
          },
          [&](float x) -> u64 { return mass.high(x); },  // (its probability is told to fp32 precision)
          [&](u64 all) -> u64 { return times(all, u, false); },
          &chosen, &whole);
      if (threadIdx.x == 0) prob = static_cast<float>(static_cast<double>(chosen) / static_cast<double>(whole));
    }
  }
  if (rank == 0 && threadIdx.x == 0) {
    p.token[row] = token;
    if (p.prob) p.prob[row] = prob;
  }
  cluster.sync();  // no CTA leaves while another may still read its shared memory
}

template <typename T>
cudaError_t launch_sample_of(SampleParams p, int num_sms, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(T);
  constexpr int step = kThreads * E;
  int ranks = 1;
  while (ranks < kMaxCluster && static_cast<long long>(p.rows) * ranks * 2 <= 4ll * num_sms &&
         p.vocab > ranks * step)
    ranks *= 2;
  // rows on 16 bytes need no room in front
  p.pad = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.ld * sizeof(T) % 16 == 0 ? 0 : E;
  auto slice_of = [&](int r) { return ((p.vocab + r - 1) / r + p.pad + step - 1) / step * step; };
  // enough CTAs that the slice fits in shared memory
  constexpr size_t most = 176 * 1024;
  while (ranks < kMaxCluster && static_cast<size_t>(slice_of(ranks)) * sizeof(T) > most) ranks *= 2;
  p.slice = slice_of(ranks);
  const size_t segs = static_cast<size_t>(p.slice / step) * kWarps * 8;
  const bool cached = p.slice * sizeof(T) <= most;
  const size_t smem = segs + (cached ? p.slice * sizeof(T) : 0);
  void (*kernel)(SampleParams) = cached ? sample_kernel<T, true> : sample_kernel<T, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, int num_sms, cudaStream_t stream) {
  if (p.type == 2) return launch_sample_of<float>(p, num_sms, stream);
  if (p.type == 1) return launch_sample_of<__nv_bfloat16>(p, num_sms, stream);
  return launch_sample_of<__half>(p, num_sms, stream);
}

}  // namespace fgemm
