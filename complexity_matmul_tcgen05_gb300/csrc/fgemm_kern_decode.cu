// fgemm_kern_decode.cu -- attention of one new token a sequence over a paged
// cache.
//
//   x_j = scale q.k_j,   out = sum_j e^(x_j - lse) v_j,   lse = log sum_j e^(x_j)
//
// One pass over the keys and values with a running reference r of the maximum
// and sums relative to it: w_j = 2^(x_j log2 e - r). The reference follows the
// maximum only when that is more than 8 above it (the weights stay below 2^8, or
// below 2^14 in fp16, where small ones would lose bits, and sums below 2^46, far
// inside fp32), so that the outputs in registers are seldom scaled. Weights are
// rounded to 16 bits for the product with the values, their sum is of the 32-bit ones.
//
// Memory-bound: a key and a value are read once for the up to 16 query heads
// that share them. The query heads of a key head are the 16 rows of a matrix
// instruction (mma.sync: with 4 flop a byte for each query head, its rate is not
// what counts), 16 tokens its columns, so scores stay in the registers that the
// product with the values takes them from. Every warp streams blocks of 16
// tokens of its own through its own ring of asynchronous copies and keeps its own
// sums; the warps of a CTA meet once at the end of a sequence's part.
//
// Measured, bf16, 32 heads of 128 over 8 key heads: 64 sequences of up to 16384 tokens
// 210 us (6.26 TB/s); one of 4097 tokens 10.9 us, of which the memory's part is 2.5: two
// launches, the lengths, the page table, the keys and the parts come one after the
// other. fp16, 28 heads of 64 over 4, 3 sequences of 131071 tokens 68 us (5.9 TB/s).
//
// The work of all sequences, in blocks of 64 tokens laid end to end, is cut into
// equal shares on the device: lengths are not known to the host. A share is taken by
// a CTA for each key head, neighbours in the grid, so that the keys and values that
// lie side by side are read at about the same time (ragged batch of 64 sequences, 8
// key heads of 128: 213 us; with the heads of a sequence one after the other in the
// shares 239). A sequence whose blocks lie in more than one share is joined from its
// parts, in their order, by a second kernel, launched so that it is there when the
// first ends. Sums do not depend on timing.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fgemm_attn.cuh"
#include "fgemm_internal.h"
#include "fgemm_ptx.cuh"

namespace fgemm {

namespace {

using namespace attn;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTokens = 16;                 // of a warp's block
constexpr int kBlock = kWarps * kTokens;    // tokens of a share's block
constexpr int kRows = 16;                   // query heads of a CTA
constexpr int kMostScanned = 512;           // sequences whose blocks the join adds up itself
constexpr long long kMostTokens = (1LL << 31) - 4096;  // of a sequence: its blocks stay inside 32 bits
constexpr float kSlack = 8.0f;              // log2 of how far the maximum may be above the reference
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int DP>  // values of a head, padded
struct Cfg {
  static constexpr int kCtasPerSm = DP == 128 ? 2 : 3;
  static constexpr int kStages = DP == 128 ? 3 : 4;
  static constexpr int kTile = kTokens * DP * 2;                  // keys (or values) of a block
  static constexpr int kRing = kStages * 2 * kTile;               // of a warp
  static constexpr int kPart = kRows * DP + 2 * kRows;            // floats of a part: outputs, references, sums
  static constexpr int kSmem = kWarps * kRing;
  static_assert(kWarps * kPart * 4 <= kSmem, "the parts of the warps reuse the rings");
  static_assert((kSmem + 4096) * kCtasPerSm <= 227 * 1024, "shared memory");
};

struct Plan {
  long long* before;  // seqs + 1: blocks of the sequences before
  float* parts;       // two a CTA
  int tiles;   // groups of kRows query heads of a key head
  int units;   // of a sequence: key heads by tiles
  int shares;  // of the blocks of all sequences, each taken by `units` CTAs
};

struct Span {
  int first, count;  // tokens seen
};
__device__ __forceinline__ Span span_of(const DecodeParams& p, int s) {
  const long long most = min(static_cast<long long>(p.table_pages) * p.page_size, kMostTokens);
  const int length = static_cast<int>(min(static_cast<long long>(max(p.lengths[s], 0)), most));
  Span r;
  r.first = p.window > 0 ? max(0, length - p.window) : 0;
  r.count = length - r.first;
  return r;
}
__device__ __forceinline__ int blocks_of(const DecodeParams& p, int s) {
  return (span_of(p, s).count + kBlock - 1) / kBlock;
}

// Blocks of a share; share i begins at block i times that.
__device__ __forceinline__ long long share_of(long long total, int shares) { return max((total + shares - 1) / shares, 1LL); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Factor of sums relative to `ref` when they go to `top`. Sums without a
// reference are zeros, or NaN where every score was.
__device__ __forceinline__ float scale_of(float ref, float top) { return ref == -INFINITY ? 1.0f : exp2_fast(ref - top); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreads, Cfg<DP>::kCtasPerSm) decode_kernel(const __grid_constant__ DecodeParams p,
                                                                      const __grid_constant__ Plan plan) {
  using C = Cfg<DP>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long sums[kThreads + 1];  // blocks before the sequences of a thread
  __shared__ uint32_t there[kWarps][C::kStages];  // tokens of a block that are seen, a bit each
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- shares: a prefix sum over the sequences, `each` of them a thread
  const int share = blockIdx.x / plan.units, unit = blockIdx.x % plan.units;
  const int each = (p.seqs + kThreads - 1) / kThreads;
  {
    const int s0 = min(p.seqs, static_cast<int>(threadIdx.x) * each), s1 = min(p.seqs, s0 + each);
    long long n = 0;
    for (int s = s0; s < s1; ++s) n += blocks_of(p, s);
    long long scan = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(0xFFFFFFFFu, scan, d);
      if (lane >= d) scan += x;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    long long start = 0;
    for (int w = 0; w < warp; ++w) start += sums[w];
    __syncthreads();
    sums[threadIdx.x] = start + scan - n;
    if (threadIdx.x == kThreads - 1) sums[kThreads] = start + scan;
    __syncthreads();
    if (blockIdx.x == 0) {  // for the join
      long long at = sums[threadIdx.x];
      for (int s = s0; s < s1; ++s) {
        plan.before[s] = at;
        at += blocks_of(p, s);
      }
      if (threadIdx.x == 0) plan.before[p.seqs] = sums[kThreads];
    }
  }
  const long long total = sums[kThreads];
  const long long size = share_of(total, plan.shares), b0 = share * size, b1 = min(b0 + size, total);
  if (b0 >= b1) return;
  // the sequence of block b0
  int seq;
  long long at;  // blocks before it
  {
    int t = 0;
    for (int step = kThreads / 2; step > 0; step >>= 1)
      if (sums[t + step] <= b0) t += step;
    seq = t * each;
    at = sums[t];
    while (true) {
      const int n = blocks_of(p, seq);
      if (at + n > b0) break;
      at += n;
      ++seq;
    }
  }

  const uint32_t ring = ptx::smem_u32(smem) + warp * C::kRing;
  const int group = p.heads / p.kv_heads;
  const float to_log2 = p.scale * kLog2e;
  constexpr float kLift = BF16 ? 0.0f : 6.0f;  // log2 of the weights' factor
  const bool alike = p.k_page == p.v_page && p.k_token == p.v_token && p.k_head == p.v_head;

  for (long long b = b0; b < b1;) {
    // ---- a part: blocks [b, end) of one sequence
    const int blocks = blocks_of(p, seq);
    if (blocks == 0) {
      ++seq;
      continue;
    }
    const long long unit0 = at, unit1 = at + blocks;
    const long long end = min(b1, unit1);
    const Span span = span_of(p, seq);
    const int t0 = static_cast<int>(b - unit0) * kBlock;
    const int t1 = min(span.count, static_cast<int>(end - unit0) * kBlock);
    const int kv = unit / plan.tiles, head0 = kv * group + (unit % plan.tiles) * kRows;
    const int rows = min(kRows, (kv + 1) * group - head0);
    const int* const table = p.page_table + seq * p.ld_table;
    const uint16_t* const k_base = p.k_cache + kv * p.k_head;
    const uint16_t* const v_base = p.v_cache + kv * p.v_head;

    // queries: rows lane / 4 and + 8
    uint32_t q[DP / 16][4];
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = lane / 4 + (i & 1) * 8, c = k * 16 + (lane & 3) * 2 + (i >> 1) * 8;
        q[k][i] = r < rows && c < p.dim
                      ? *reinterpret_cast<const uint32_t*>(p.q.p + seq * p.q.ld + (head0 + r) * p.q.hs + c)
                      : 0u;
      }
    float o[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
    float ref[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};

    const int mine = t1 - t0 > warp * kTokens ? (t1 - t0 - warp * kTokens + kBlock - 1) / kBlock : 0;  // blocks of this warp
    auto token = [&](int i) { return t0 + warp * kTokens + i * kBlock + (lane & 15); };  // of the span
    auto page_of = [&](int i) {  // lanes 0..15 (and again 16..31): the page of a token of block i, -1: not seen
      const int t = token(i);
      if (i >= mine || t >= t1) return -1;
      const int page = table[(span.first + t) / p.page_size];
      return page >= 0 && page < p.pages ? page : -1;
    };
    int page = page_of(0);
    auto load = [&](int i) {
      const int stage = i % C::kStages;
      if (i < mine) {
        const bool seen = page >= 0;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, seen) & 0xFFFFu;
        if (lane == 0) there[warp][stage] = mask;
        const long long in_page = seen ? (span.first + token(i)) % p.page_size : 0;
        const long long k_off = seen ? page * p.k_page + in_page * p.k_token : 0;
        const long long v_off = alike || !seen ? k_off : page * p.v_page + in_page * p.v_token;
        page = page_of(i + 1);
        constexpr int kChunks = DP / 8, kRowsAtOnce = 32 / kChunks;
        const int chunk = lane % kChunks;
        const uint32_t to = ring + stage * 2 * C::kTile;
#pragma unroll
        for (int j = 0; j < kTokens / kRowsAtOnce; ++j) {
          const int r = j * kRowsAtOnce + lane / kChunks;
          const long long ko = __shfl_sync(0xFFFFFFFFu, k_off, r);
          const long long vo = alike ? ko : __shfl_sync(0xFFFFFFFFu, v_off, r);
          const uint32_t bytes = ((mask >> r) & 1u) && chunk * 8 < p.dim ? 16u : 0u;
          const uint32_t dst = to + r * DP * 2 + ((chunk ^ (r & 7)) << 4);
          const int c = bytes ? chunk * 8 : 0;
          copy16(dst, k_base + ko + c, bytes);
          copy16(dst + C::kTile, v_base + vo + c, bytes);
        }
      }
      copies_commit();
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) load(i);

    for (int i = 0; i < mine; ++i) {
      copies_wait<C::kStages - 2>();
      __syncwarp();
      const int stage = i % C::kStages;
      const uint32_t keys = ring + stage * 2 * C::kTile, values = keys + C::kTile;
      // scores of 16 heads by 16 tokens
      float s[2][4] = {};
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
        uint32_t kb[4];
        const int r = (lane & 7) + (lane >> 4) * 8, c = 2 * k + ((lane >> 3) & 1);
        ldmatrix4(keys + r * DP * 2 + ((c ^ (r & 7)) << 4), kb);
        mma<BF16>(s[0], q[k], kb[0], kb[1]);
        mma<BF16>(s[1], q[k], kb[2], kb[3]);
      }
      const uint32_t mask = there[warp][stage];
      float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool seen = (mask >> (n * 8 + (lane & 3) * 2 + (e & 1))) & 1u;
          s[n][e] = seen ? s[n][e] * to_log2 : -INFINITY;
          most[e >> 1] = fmaxf(most[e >> 1], s[n][e]);
        }
      bool far = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        most[h] = fmaxf(most[h], __shfl_xor_sync(0xFFFFFFFFu, most[h], 1));
        most[h] = fmaxf(most[h], __shfl_xor_sync(0xFFFFFFFFu, most[h], 2));
        far |= most[h] > ref[h] + kSlack;
      }
      if (__any_sync(0xFFFFFFFFu, far)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float to = fmaxf(ref[h], most[h]);
          const float f = to == -INFINITY ? 1.0f : exp2_fast(ref[h] - to);
          ref[h] = to;
          sum[h] *= f;
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            o[n][2 * h] *= f;
            o[n][2 * h + 1] *= f;
          }
        }
      }
      float base[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) base[h] = ref[h] == -INFINITY ? 0.0f : ref[h] - kLift;
      uint32_t w[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = exp2_fast(s[n][2 * h] - base[h]), y = exp2_fast(s[n][2 * h + 1] - base[h]);
          sum[h] += x + y;
          w[n * 2 + h] = pack2<BF16>(x, y);
        }
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        uint32_t vb[4];
        const int r = lane & 15, c = 2 * n + (lane >> 4);
        ldmatrix4_t(values + r * DP * 2 + ((c ^ (r & 7)) << 4), vb);
        mma<BF16>(o[2 * n], w, vb[0], vb[1]);
        mma<BF16>(o[2 * n + 1], w, vb[2], vb[3]);
      }
      __syncwarp();  // the stage that is loaded next has been read
      load(i + C::kStages - 1);
    }
    copies_wait<0>();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sum[h] += __shfl_xor_sync(0xFFFFFFFFu, sum[h], 1);
      sum[h] += __shfl_xor_sync(0xFFFFFFFFu, sum[h], 2);
    }
    // ---- the warps meet over their rings
    __syncthreads();
    float* const parts = reinterpret_cast<float*>(smem);
    {
      float* const part = parts + warp * C::kPart;
#pragma unroll
      for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(part + (lane / 4 + h * 8) * DP + n * 8 + (lane & 3) * 2) =
              make_float2(o[n][2 * h], o[n][2 * h + 1]);
      if ((lane & 3) == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          part[kRows * DP + lane / 4 + h * 8] = ref[h] - kLift;
          part[kRows * DP + kRows + lane / 4 + h * 8] = sum[h];
        }
      }
    }
    __syncthreads();
    const bool whole = unit0 >= b0 && unit1 <= b1;
    float* const to = plan.parts + (2LL * blockIdx.x + (unit0 >= b0 ? 1 : 0)) * C::kPart;
    for (int e = threadIdx.x; e < rows * (DP / 4); e += kThreads) {
      const int r = e / (DP / 4), c = e % (DP / 4) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, parts[w * C::kPart + kRows * DP + r]);
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float z = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* const part = parts + w * C::kPart;
        const float mr = part[kRows * DP + r];
        const float f = scale_of(mr, top);
        const float4 x = *reinterpret_cast<const float4*>(part + r * DP + c);
        z += f * part[kRows * DP + kRows + r];
        acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
      }
      if (!whole) {
        *reinterpret_cast<float4*>(to + r * DP + c) = acc;
        if (c == 0) {
          to[kRows * DP + r] = top;
          to[kRows * DP + kRows + r] = z;
        }
      } else if (c < p.dim) {
        const float inv = z == 0.0f ? 0.0f : 1.0f / z;
        *reinterpret_cast<uint2*>(p.out.p + seq * p.out.ld + (head0 + r) * p.out.hs + c) =
            make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
        if (p.lse && c == 0)
          p.lse[static_cast<long long>(seq) * p.heads + head0 + r] = z == 0.0f ? -INFINITY : (top + log2f(z)) * kLn2;
      }
    }
    __syncthreads();  // the rings are free again
    b = end;
    if (b == unit1) {
      at = b;
      ++seq;
    }
  }
}

// One CTA a query head: the parts of its unit, warp w taking part w and every
// kJoinWarps-th behind it, or zeros where there is nothing. What does not come from
// the first kernel is done while that one runs.
constexpr int kJoinWarps = 8, kJoinThreads = kJoinWarps * 32;
template <bool BF16, int DP>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ DecodeParams p,
                                                                   const __grid_constant__ Plan plan) {
  using C = Cfg<DP>;
  __shared__ float4 outs[kJoinWarps][32];
  __shared__ float refs[kJoinWarps], sums[kJoinWarps];
  __shared__ long long blocks_sum[2][kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seq = blockIdx.x / p.heads, head = blockIdx.x % p.heads, group = p.heads / p.kv_heads;
  long long before, total;
  const long long blocks = blocks_of(p, seq);
  if (p.seqs <= kMostScanned) {
    long long all = 0, ahead = 0;
    for (int s = threadIdx.x; s < p.seqs; s += kJoinThreads) {
      const int n = blocks_of(p, s);
      all += n;
      ahead += s < seq ? n : 0;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
      ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, d);
    }
    if (lane == 0) blocks_sum[0][warp] = all, blocks_sum[1][warp] = ahead;
    __syncthreads();
    total = before = 0;
    for (int w = 0; w < kJoinWarps; ++w) total += blocks_sum[0][w], before += blocks_sum[1][w];
    asm volatile("griddepcontrol.wait;" ::: "memory");
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    before = plan.before[seq];
    total = plan.before[p.seqs];
  }
  uint16_t* const out = p.out.p + seq * p.out.ld + head * p.out.hs;
  if (blocks == 0) {
    if (threadIdx.x < p.dim / 8) reinterpret_cast<uint4*>(out)[threadIdx.x] = make_uint4(0, 0, 0, 0);
    if (p.lse && threadIdx.x == 0) p.lse[blockIdx.x] = -INFINITY;
    return;
  }
  const int unit = head / group * plan.tiles + head % group / kRows, r = head % group % kRows;
  const long long size = share_of(total, plan.shares);
  const int c0 = static_cast<int>(before / size), c1 = static_cast<int>((before + blocks - 1) / size);
  if (c0 == c1) return;
  float top = -INFINITY, z = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto part = [&](int c) {
    return plan.parts + (2LL * (c * plan.units + unit) + (c == c0 ? 1 : 0)) * C::kPart;
  };
#pragma unroll 1
  for (int c = c0 + warp; c <= c1; c += 4 * kJoinWarps) {
    // four parts at once
    float ref[4], sum[4];
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = c + i * kJoinWarps;
      ref[i] = -INFINITY, sum[i] = 0.0f, v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (at <= c1) {
        const float* const x = part(at);
        ref[i] = x[kRows * DP + r];
        sum[i] = x[kRows * DP + kRows + r];
        if (lane * 4 < DP) v[i] = *reinterpret_cast<const float4*>(x + r * DP + lane * 4);
      }
    }
    const float to = fmaxf(top, fmaxf(fmaxf(ref[0], ref[1]), fmaxf(ref[2], ref[3])));
    const float f0 = scale_of(top, to);
    z *= f0;
    acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
    top = to;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = scale_of(ref[i], to);
      z += f * sum[i];
      acc.x += f * v[i].x, acc.y += f * v[i].y, acc.z += f * v[i].z, acc.w += f * v[i].w;
    }
  }
  outs[warp][lane] = acc;
  if (lane == 0) refs[warp] = top, sums[warp] = z;
  __syncthreads();
  if (warp != 0) return;
  top = refs[0];
  for (int w = 1; w < kJoinWarps; ++w) top = fmaxf(top, refs[w]);
  acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  z = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float f = scale_of(refs[w], top);
    const float4 v = outs[w][lane];
    z += f * sums[w];
    acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
  }
  const float inv = z == 0.0f ? 0.0f : 1.0f / z;
  if (lane * 4 < p.dim)
    *reinterpret_cast<uint2*>(out + lane * 4) =
        make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
  if (p.lse && lane == 0) p.lse[blockIdx.x] = z == 0.0f ? -INFINITY : (top + log2f(z)) * kLn2;
}

size_t before_bytes(int seqs) { return (static_cast<size_t>(seqs) + 1 + 1) / 2 * 16; }

template <bool BF16, int DP>
cudaError_t launch_of(const DecodeParams& p, const Plan& plan, cudaStream_t stream) {
  static unsigned long long devices = 0;
  auto kernel = decode_kernel<BF16, DP>;
  cudaError_t e = with_smem(kernel, Cfg<DP>::kSmem, devices);
  if (e != cudaSuccess) return e;
  kernel<<<plan.shares * plan.units, kThreads, Cfg<DP>::kSmem, stream>>>(p, plan);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.seqs) * static_cast<unsigned>(p.heads));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_join_kernel<BF16, DP>, p, plan);
}

}  // namespace

namespace {
int tiles_of(int heads, int kv_heads) { return (heads / kv_heads + kRows - 1) / kRows; }
int shares_held(int units, int dim, int num_sms) {
  return std::max(num_sms * (dim > 64 ? Cfg<128>::kCtasPerSm : Cfg<64>::kCtasPerSm) / units, 1);
}
}  // namespace

size_t decode_workspace(int seqs, int heads, int kv_heads, int dim, int num_sms) {
  const size_t part = static_cast<size_t>(dim > 64 ? Cfg<128>::kPart : Cfg<64>::kPart) * 4;
  const int units = kv_heads * tiles_of(heads, kv_heads);
  return before_bytes(seqs) + static_cast<size_t>(shares_held(units, dim, num_sms)) * units * 2 * part;
}

cudaError_t launch_decode(const DecodeParams& p, void* workspace, int num_sms, cudaStream_t stream) {
  Plan plan;
  plan.before = static_cast<long long*>(workspace);
  plan.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + before_bytes(p.seqs));
  plan.tiles = tiles_of(p.heads, p.kv_heads);
  plan.units = p.kv_heads * plan.tiles;
  plan.shares = shares_held(plan.units, p.dim, num_sms);
  if (p.dim > 64)
    return p.is_bf16 ? launch_of<true, 128>(p, plan, stream) : launch_of<false, 128>(p, plan, stream);
  return p.is_bf16 ? launch_of<true, 64>(p, plan, stream) : launch_of<false, 64>(p, plan, stream);
}

}  // namespace fgemm
