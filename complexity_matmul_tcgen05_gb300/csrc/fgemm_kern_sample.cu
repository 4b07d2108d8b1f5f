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
// No sort: top-k and top-p are each a threshold on x, found by histograms.
// The first one bins x linearly between m and m - 32 T (the masses below are
// under 2^-46); the bin the threshold falls in is searched again with bins
// over its key range (keys: x's bits, ordered as integers) until one key is
// left.  Ties at that key are cut by index.
//
// A cluster of CTAs works on a row, each on a slice kept in shared memory,
// so the logits are read from memory once; the CTAs read each other's
// histograms and sums through distributed shared memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

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

// 2^(j/32) for j = -16 .. 16 in units of 2^-44.
__constant__ u64 kPow[33] = {
    12439554047902ull, 12711944812080ull, 12990300157313ull, 13274750690919ull, 13565429880144ull,
    13862474114787ull, 14166022771192ull, 14476218277651ull, 14793206181226ull, 15117135216047ull,
    15448157373097ull, 15786427971528ull, 16132105731538ull, 16485352848846ull, 16846335070792ull,
    17215221774115ull, 17592186044416ull, 17977404757381ull, 18371058661769ull, 18773332464219ull,
    19184414915921ull, 19604498901178ull, 20033781527906ull, 20472464220127ull, 20920752812471ull,
    21378857646762ull, 21846993670708ull, 22325380538761ull, 22814242715178ull, 23313809579344ull,
    23824315533396ull, 24346000112214ull, 24879108095804ull,
};

struct SampleShared {
  u64 hist[kBins];
  u64 pow[33];
  u64 warp64[kWarps];
  u64 total;         // this CTA's sum, read by the others
  u64 sel_before;    // what lies above the selected bin
  int sel_bin;
  unsigned int warp32[kWarps];
  unsigned int best; // this CTA's largest key
  unsigned int count;
  int found;         // index located by locate(), in the CTA that finds it
  u64 found_mass;
  unsigned int range[2];
};

// Keys: order of floats as unsigned integers (x is never NaN, -0 never).
__device__ __forceinline__ unsigned int key_of(float x) {
  const unsigned int b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned int k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// exp((x - m) / T) in units of 2^-44, to about 2^-36 of its value.
// y = (x - m) log2(e) / T is held as a sum of two floats (x - m and its
// rounding error by a two-sum, the product's error by an fma); then
// 2^y = 2^n 2^(j/32) 2^r with a table for 2^(j/32) and the exponential series
// for 2^r, |r| <= 1/64, whose first-order term is again kept in two floats.
struct Masses {
  float m, ch, cl;  // ch + cl = log2(e) / T
  const u64* pow;
  __device__ __forceinline__ u64 operator()(float x) const {
    if (x == m) return kOne;
    const float s = x - m;
    const float yh = __fmul_rn(s, ch);  // rounded here: not to be fused into the subtraction below
    if (!(yh > -46.0f)) return 0;
    const float bb = s - x;
    const float e = (x - (s - bb)) + (-m - bb);
    const float yl = fmaf(s, ch, -yh) + fmaf(s, cl, e * ch);
    const float n = rintf(yh);
    const float f = yh - n;
    const float j = rintf(f * 32.0f);
    const float r = fmaf(j, -0.03125f, f);
    constexpr float l1 = 0.693147182464599609375f, l2 = -1.90465429995776804525e-09f;  // ln 2
    const float zh = __fmul_rn(r, l1);
    const float zl = fmaf(r, l1, -zh) + fmaf(r, l2, yl * l1);
    const float q = zh * zh * fmaf(zh, fmaf(zh, fmaf(zh, 1.0f / 120, 1.0f / 24), 1.0f / 6), 0.5f);
    const int series = __float2int_rn(zh * 137438953472.0f) + __float2int_rn((zl + q) * 137438953472.0f);  // 2^37
    const u64 t = pow[static_cast<int>(j) + 16];
    const long long v =
        static_cast<long long>(t) + ((static_cast<long long>(t >> 13) * static_cast<long long>(series)) >> 24);
    const int shift = -static_cast<int>(n);
    return (static_cast<u64>(v) + ((1ull << shift) >> 1)) >> shift;
  }
};

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
  u64 above;         // their count or mass
};

// The key at which the sum of weight(x) over the candidates, from the
// largest down, reaches target (1 <= target <= the whole sum).  weight 0:
// not a candidate.  Every thread of the cluster gets the result.
template <typename S, typename W>
__device__ Threshold find_threshold(const S& slice, SampleShared& sh, cg::cluster_group& cluster, float m, float scale,
                                    u64 target, W weight) {
  const int ranks = cluster.num_blocks();
  Threshold res{0, 0};
  unsigned int lo = 0, hi = 0xFFFFFFFFu;  // keys still in question, once `linear` is done
  bool linear = true;
  int shift = 0;
  auto bin_of = [&](float x) -> int {
    if (linear) return x == m ? 0 : static_cast<int>(fminf((m - x) * scale, kBins - 1.0f));
    const unsigned int k = key_of(x);
    return k < lo || k > hi ? -1 : static_cast<int>((hi - k) >> shift);
  };
  while (true) {
    for (int b = threadIdx.x; b < kBins; b += kThreads) sh.hist[b] = 0;
    if (threadIdx.x == 0) sh.sel_bin = kBins - 1;
    __syncthreads();
    slice.each([&](float x, int) {
      const int b = bin_of(x);
      // the last linear bin holds all that lies far below: it is what is left
      if (b < 0 || (linear && b == kBins - 1)) return;
      const u64 w = weight(x);
      if (w) atomicAdd(&sh.hist[b], w);
    });
    cluster.sync();
    // thread t: bins 2t and 2t + 1 over all CTAs
    u64 v[2] = {0, 0};
    for (int r = 0; r < ranks; ++r) {
      const u64* h = cluster.map_shared_rank(sh.hist, r);
      v[0] += h[2 * threadIdx.x];
      v[1] += h[2 * threadIdx.x + 1];
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
    if (threadIdx.x == 0) sh.sel_before = all;  // the last linear bin, unless another bin reaches the target
    __syncthreads();
    if (before < target && target <= before + v[0]) {
      sh.sel_bin = 2 * threadIdx.x;
      sh.sel_before = before;
    } else if (before + v[0] < target && target <= before + v[0] + v[1]) {
      sh.sel_bin = 2 * threadIdx.x + 1;
      sh.sel_before = before + v[0];
    }
    cluster.sync();  // the others are done with this CTA's histogram
    const int bin = sh.sel_bin;
    res.above = sh.sel_before;
    if (linear) {
      // the bin's key range: keys at which bin_of, which falls as keys grow, is `bin`
      if (threadIdx.x < 2) {
        // thread 0: the smallest key with bin_of <= bin; thread 1: the largest with bin_of >= bin
        unsigned int a = key_of(-INFINITY), b = key_of(m);
        while (a < b) {
          const unsigned int mid = threadIdx.x == 0 ? a + (b - a) / 2 : a + (b - a) / 2 + 1;
          const int at = bin_of(value_of(mid));
          if (threadIdx.x == 0) {
            if (at <= bin) b = mid; else a = mid + 1;
          } else {
            if (at >= bin) a = mid; else b = mid - 1;
          }
        }
        sh.range[threadIdx.x] = a;
      }
      __syncthreads();
      lo = sh.range[0];
      hi = sh.range[1];
      linear = false;
    } else {
      const unsigned int top = hi - (static_cast<unsigned int>(bin) << shift);
      const unsigned int width = (1u << shift) - 1;
      lo = top - lo > width ? top - width : lo;
      hi = top;
    }
    if (lo == hi) break;
    const int bits = 32 - __clz(hi - lo);
    shift = bits > 10 ? bits - 10 : 0;
    __syncthreads();
  }
  res.key = lo;
  return res;
}

// The first index of the row at which the running sum of weight(x, index)
// exceeds target(whole sum); -1 if the whole sum is 0.  Every thread of the
// cluster gets it; *mass is that element's weight and *whole the sum.
template <typename S, typename W, typename G>
__device__ int locate(const S& slice, SampleShared& sh, u64* segs, cg::cluster_group& cluster, int first, W weight,
                      G target_of, u64* mass, u64* whole) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  constexpr int E = S::E;
  u64 sum = 0;
  for (int r = 0; r < slice.rounds; ++r) {
    const int vec = r * kThreads + threadIdx.x;
    float x[E];
    slice.get(vec, x);
    u64 s = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) s += weight(x[e], vec * E + e);
    s = warp_sum(s);
    if (lane == 0) segs[r * kWarps + warp] = s;
    sum += s;
  }
  if (lane == 0) sh.warp64[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    u64 t = 0;
    for (int w = 0; w < kWarps; ++w) t += sh.warp64[w];
    sh.total = t;
    sh.found = -1;
  }
  cluster.sync();
  u64 all = 0, before = 0, own = 0;
  for (int r = 0; r < ranks; ++r) {
    const u64 t = *cluster.map_shared_rank(&sh.total, r);
    if (r < rank) before += t;
    if (r == rank) own = t;
    all += t;
  }
  const u64 target = all ? target_of(all) : 0;
  *whole = all;
  if (all && before <= target && target < before + own && warp == 0) {
    // the segment, 32 at a time, then the element in it
    const int n = slice.rounds * kWarps;
    u64 base = before;
    for (int s0 = 0; s0 < n; s0 += 32) {
      const u64 v = s0 + lane < n ? segs[s0 + lane] : 0;
      const u64 upto = base + warp_scan(v);
      const unsigned int hit = __ballot_sync(0xFFFFFFFFu, upto > target);
      if (hit) {
        const int at = __ffs(hit) - 1;
        const u64 seg_before = __shfl_sync(0xFFFFFFFFu, upto - v, at);
        const int seg = s0 + at;
        const int vec = (seg / kWarps) * kThreads + (seg % kWarps) * 32 + lane;
        float x[E];
        slice.get(vec, x);
        u64 w[E], s = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          w[e] = weight(x[e], vec * E + e);
          s += w[e];
        }
        u64 run = seg_before + warp_scan(s) - s;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (run <= target && target < run + w[e]) {
            sh.found = first + vec * E + e;
            sh.found_mass = w[e];
          }
          run += w[e];
        }
        break;
      }
      base = __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
  }
  cluster.sync();
  int found = -1;
  for (int r = 0; r < ranks; ++r) {
    const int f = *cluster.map_shared_rank(&sh.found, r);
    if (f >= 0) {
      found = f;
      *mass = *cluster.map_shared_rank(&sh.found_mass, r);
    }
  }
  cluster.sync();  // sh.total and sh.found may be written again
  return found;
}

template <typename T, bool CACHED>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ SampleShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int row = blockIdx.x / ranks;
  constexpr int E = 16 / sizeof(T);

  Slice<T, CACHED> slice;
  const int per = p.slice;
  const int first = min(rank * per, p.vocab);
  slice.len = min(p.vocab - first, per);
  slice.rounds = per / (kThreads * E);
  slice.global = static_cast<const T*>(p.logits) + row * p.ld + first;
  u64* segs = reinterpret_cast<u64*>(dyn);
  slice.cache = reinterpret_cast<T*>(dyn + static_cast<size_t>(slice.rounds) * kWarps * 8);
  if (threadIdx.x < 33) sh.pow[threadIdx.x] = kPow[threadIdx.x];

  // the slice into shared memory, its largest key and its candidates
  float top = -INFINITY;
  unsigned int count = 0;
  if (CACHED) {
    for (int i = threadIdx.x; i < per; i += kThreads) {
      const T v = i < slice.len ? slice.global[i] : static_cast<T>(-INFINITY);
      slice.cache[i] = v;
      const float x = clean(raw_value<T>(v));
      top = fmaxf(top, x);
      count += x > -INFINITY;
    }
  } else {
    slice.each([&](float x, int) {
      top = fmaxf(top, x);
      count += x > -INFINITY;
    });
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
  const float temperature = p.temperature ? p.temperature[row] : p.temperature0;
  const float top_p = p.top_p ? p.top_p[row] : p.top_p0;
  const float min_p = p.min_p ? p.min_p[row] : p.min_p0;
  const int top_k = p.top_k ? p.top_k[row] : p.top_k0;
  const bool greedy = !(temperature > 0.0f) || top_k == 1 || top_p <= 0.0f || min_p > 1.0f;

  int token = -1;
  float prob = 0.0f;
  if (count) {
    Masses mass;
    mass.m = m;
    mass.pow = sh.pow;
    const double c = 1.4426950408889634074 / static_cast<double>(greedy ? 1.0f : temperature);
    mass.ch = static_cast<float>(c);
    mass.cl = isinf(mass.ch) ? 0.0f : static_cast<float>(c - static_cast<double>(mass.ch));
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
        const Threshold t = find_threshold(slice, sh, cluster, m, scale, static_cast<u64>(top_k),
                                           [](float x) -> u64 { return x > -INFINITY ? 1 : 0; });
        cut = t.key;
        ties = static_cast<u64>(top_k) - t.above;
      }
      if (top_p < 1.0f) {
        // the mass of what top-k keeps
        u64 whole = 0, unused = 0;
        const u64 at_cut = ties ? mass(value_of(cut)) : 0;
        locate(slice, sh, segs, cluster, first,
               [&](float x, int) -> u64 { return x > -INFINITY && key_of(x) > cut ? mass(x) : 0; },
               [](u64) -> u64 { return 0; }, &unused, &above);
        whole = above + ties * at_cut;
        u64 target = static_cast<u64>(ceil(static_cast<double>(top_p) * static_cast<double>(whole)));
        target = target < 1 ? 1 : target > whole ? whole : target;
        if (target > above) {  // the prefix ends among the ties at top-k's threshold
          const u64 need = (target - above + at_cut - 1) / at_cut;
          ties = need < ties ? need : ties;
        } else {
          const Threshold t = find_threshold(
              slice, sh, cluster, m, scale, target,
              [&](float x) -> u64 { return x > -INFINITY && key_of(x) > cut ? mass(x) : 0; });
          cut = t.key;
          const u64 each = mass(value_of(cut));
          ties = (target - t.above + each - 1) / each;
        }
      }
    }
    u64 chosen = 0, whole = 0;
    if (ties)  // the index of the last tie that is kept
      last = locate(slice, sh, segs, cluster, first, [&](float x, int) -> u64 { return key_of(x) == cut ? 1 : 0; },
                    [&](u64 all) -> u64 { return (ties < all ? ties : all) - 1; }, &chosen, &whole);
    if (greedy) {
      token = last;
      prob = 1.0f;
    } else {
      const u64 least = min_p > 0.0f ? static_cast<u64>(ceil(static_cast<double>(min_p) * kOne)) : 0;
      // the largest float below 1 stands for anything above it, 0 for anything below and for NaN
      const double u = static_cast<double>(fminf(fmaxf(p.u[row], 0.0f), 0.999999940395355224609375f));
      token = locate(
          slice, sh, segs, cluster, first,
          [&](float x, int i) -> u64 {
            const unsigned int k = key_of(x);
            if (!(x > -INFINITY) || k < cut || (k == cut && first + i > last)) return 0;
            const u64 w = mass(x);
            return w >= least ? w : 0;
          },
          [&](u64 all) -> u64 {
            const u64 at = static_cast<u64>(u * static_cast<double>(all));
            return at < all ? at : all - 1;
          },
          &chosen, &whole);
      prob = static_cast<float>(static_cast<double>(chosen) / static_cast<double>(whole));
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
  while (ranks < kMaxCluster && static_cast<long long>(p.rows) * ranks * 2 <= 2ll * num_sms &&
         p.vocab > ranks * step)
    ranks *= 2;
  auto slice_of = [&](int r) { return ((p.vocab + r - 1) / r + step - 1) / step * step; };
  // enough CTAs that the slice fits in shared memory
  constexpr size_t most = 200 * 1024;
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
