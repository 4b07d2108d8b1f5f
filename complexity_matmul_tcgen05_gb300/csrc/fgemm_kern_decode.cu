// fgemm_kern_decode.cu -- attention of one new token a sequence over a paged
// cache.
//
//   x_j = scale q.k_j,   out = sum_j e^(x_j - lse) v_j,   lse = log sum_j e^(x_j)
//
// One pass over the keys and values with a running reference r of the maximum
// and sums relative to it: w_j = 2^(x_j log2 e - r). The reference follows the
// maximum only when that is more than 8 above it, so that the outputs in registers are
// seldom scaled. In bf16 the weights are lowered by 2^8 and stay at most 1: no sum is
// larger than it were relative to the maximum, and values may be near the end of fp32. In
// fp16, where small ones would lose bits, they are lifted by 2^6 and stay below 2^14, sums
// below 2^61. Weights are rounded to 16 bits for the product with the values, their sum is
// of the 32-bit ones.
//
// Memory-bound: a key and a value are read once for the up to 16 query heads
// that share them. 16 tokens are the rows of a matrix instruction (mma.sync) and 8
// query heads its columns, one or two of them; a sequence's few heads are the short
// side, where padding costs least (as the 16 rows, 4 heads of 128 took twice the
// instructions: one sequence of 512 tokens 8.3 us against 6.9, a ragged batch 211
// against 205 then). Scores stay in the registers, transposed eight by eight, for the
// product with the values. Every warp streams blocks of 16 tokens of its own through
// its own ring of asynchronous copies and keeps its own sums; the warps of a CTA meet
// once at the end of a sequence's part.
//
// Measured, bf16, 32 heads of 128 over 8 key heads: 64 sequences of up to 16384 tokens
// 197 to 203 us (6.5 to 6.7 TB/s), 256 of 300 tokens 65 us (4.8 TB/s); one of 4097 tokens
// 9.2 us, of which the memory's part is 2.5: two launches, the lengths, the page table, the keys and
// the parts come one after the other. fp16, 28 heads of 64 over 4, 3 sequences of 131071
// tokens 64 to 67 us (6.0 to 6.2 TB/s).
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
constexpr long long kMostTokens = (1LL << 31) - 4096;  // of a sequence: its blocks stay inside 32 bits
constexpr float kSlack = 8.0f;              // log2 of how far the maximum may be above the reference
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int DP, int NT>  // values of a head, padded; eights of query heads
struct Cfg {
  static constexpr int kRows = 8 * NT;  // query heads of a CTA
  static constexpr int kCtasPerSm = DP == 128 ? 2 : 3;
  static constexpr int kStages = DP == 128 ? 3 : 4;
  static constexpr int kTile = kTokens * DP * 2;                  // keys (or values) of a block
  static constexpr int kRing = kStages * 2 * kTile;               // of a warp
  static constexpr int kLine = DP + 4;                            // floats of a head's outputs in a part
  static constexpr int kPart = kRows * kLine + 2 * kRows;         // of a part: outputs, references, sums
  static constexpr int kSmem = kWarps * kRing;
  static_assert(kWarps * kPart * 4 <= kSmem, "the parts of the warps reuse the rings");
  static_assert((kSmem + 4096) * kCtasPerSm <= 227 * 1024, "shared memory");
};

// The sequence that begins in a share and ends in a later one, `last`; seq -1: none.
struct Straddle {
  int seq, last;
};

struct Plan {
  Straddle* straddles;  // by share
  float* parts;         // two a CTA
  int tiles;   // groups of 8 NT query heads of a key head
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
__device__ __forceinline__ long long share_of(long long total, int shares) {
  return max((total + shares - 1) / shares, 1LL);
}

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
// Eight rows of eight 16-bit values, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
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

template <bool BF16, int DP, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<DP, NT>::kCtasPerSm) decode_kernel(const __grid_constant__ DecodeParams p,
                                                                      const __grid_constant__ Plan plan) {
  using C = Cfg<DP, NT>;
  constexpr int kRows = C::kRows;
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
  }
  // Sequences of which nothing is seen: rows of zeros.
  for (int s = share + static_cast<int>(threadIdx.x) * plan.shares; s < p.seqs; s += kThreads * plan.shares)
    if (blocks_of(p, s) == 0) {
      const int group = p.heads / p.kv_heads, kv = unit / plan.tiles, row0 = unit % plan.tiles * kRows;
      for (int head = kv * group + row0; head < kv * group + min(group, row0 + kRows); ++head) {
        uint4* const out = reinterpret_cast<uint4*>(p.out.p + s * p.out.ld + head * p.out.hs);
        for (int c = 0; c < p.dim / 8; ++c) out[c] = make_uint4(0, 0, 0, 0);
        if (p.lse) p.lse[static_cast<long long>(s) * p.heads + head] = -INFINITY;
      }
    }
  const long long total = sums[kThreads];
  const long long size = share_of(total, plan.shares), b0 = share * size, b1 = min(b0 + size, total);
  Straddle straddle{-1, 0};
  if (b0 >= b1) {
    if (unit == 0 && threadIdx.x == 0) plan.straddles[share] = straddle;
    return;
  }
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
  constexpr float kLift = BF16 ? -kSlack : 6.0f;  // log2 of the weights' factor
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

    // queries: heads 8 h + lane / 4
    uint32_t q[DP / 16][NT][2];
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = h * 8 + lane / 4, c = k * 16 + (lane & 3) * 2 + i * 8;
          q[k][h][i] = r < rows && c < p.dim
                           ? *reinterpret_cast<const uint32_t*>(p.q.p + seq * p.q.ld + (head0 + r) * p.q.hs + c)
                           : 0u;
        }
    // outputs: values lane / 4 (and + 8) of sixteen, heads 8 h + (lane & 3) * 2 (and + 1)
    float o[DP / 16][NT][4];
#pragma unroll
    for (int n = 0; n < DP / 16; ++n)
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][h][i] = 0.0f;
    float ref[NT][2], sum[NT][2];  // of these heads
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) ref[h][e] = -INFINITY, sum[h][e] = 0.0f;

    // blocks of this warp
    const int mine = t1 - t0 > warp * kTokens ? (t1 - t0 - warp * kTokens + kBlock - 1) / kBlock : 0;
    auto token = [&](int i) { return t0 + warp * kTokens + i * kBlock + (lane & 15); };  // of the span
    // Lanes 0..15 (and again 16..31): the page of a token of block i, as the table has
    // it (looked up two blocks ahead); -1: not seen.
    auto page_of = [&](int i) {
      const int t = token(i);
      if (i >= mine || t >= t1) return -1;
      return table[(span.first + t) / p.page_size];
    };
    int page = page_of(0), page_next = page_of(1);
    auto load = [&](int i) {
      const int stage = i % C::kStages;
      if (i < mine) {
        const bool seen = page >= 0 && page < p.pages;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, seen) & 0xFFFFu;
        if (lane == 0) there[warp][stage] = mask;
        const long long in_page = seen ? (span.first + token(i)) % p.page_size : 0;
        const long long k_off = seen ? page * p.k_page + in_page * p.k_token : 0;
        const long long v_off = alike || !seen ? k_off : page * p.v_page + in_page * p.v_token;
        page = page_next;
        page_next = page_of(i + 2);
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
      // scores of 16 tokens by 8 NT heads, in two sums
      float s[NT][4] = {}, s2[NT][4] = {};
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
        uint32_t ka[4];
        const int r = lane & 15, c = 2 * k + (lane >> 4);
        ldmatrix4(keys + r * DP * 2 + ((c ^ (r & 7)) << 4), ka);
#pragma unroll
        for (int h = 0; h < NT; ++h) mma<BF16>(NT == 1 && (k & 1) ? s2[h] : s[h], ka, q[k][h][0], q[k][h][1]);
      }
      const uint32_t mask = there[warp][stage] >> (lane / 4);  // bits 0 and 8: this lane's tokens
      float most[NT][2];
      bool far = false;
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int i = e; i < 4; i += 2) {
            const float x = NT == 1 ? s[h][i] + s2[h][i] : s[h][i];
            s[h][i] = (mask >> (i >> 1) * 8) & 1u ? x * to_log2 : -INFINITY;
          }
          most[h][e] = fmaxf(s[h][e], s[h][e + 2]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) most[h][e] = fmaxf(most[h][e], __shfl_xor_sync(0xFFFFFFFFu, most[h][e], d));
          far |= most[h][e] > ref[h][e] + kSlack;
        }
      if (__any_sync(0xFFFFFFFFu, far)) {
#pragma unroll
        for (int h = 0; h < NT; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float to = fmaxf(ref[h][e], most[h][e]);
            const float f = to == -INFINITY ? 1.0f : exp2_fast(ref[h][e] - to);
            ref[h][e] = to;
            sum[h][e] *= f;
#pragma unroll
            for (int n = 0; n < DP / 16; ++n) {
              o[n][h][e] *= f;
              o[n][h][e + 2] *= f;
            }
          }
      }
      uint32_t w[NT][2];
#pragma unroll
      for (int h = 0; h < NT; ++h) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float base = ref[h][e] == -INFINITY ? 0.0f : ref[h][e] - kLift;
#pragma unroll
          for (int i = e; i < 4; i += 2) {
            s[h][i] = exp2_fast(s[h][i] - base);
            sum[h][e] += s[h][i];
          }
        }
        w[h][0] = transposed(pack2<BF16>(s[h][0], s[h][1]));
        w[h][1] = transposed(pack2<BF16>(s[h][2], s[h][3]));
      }
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        uint32_t va[4];
        const int r = (lane & 7) + (lane >> 4) * 8, c = 2 * n + ((lane >> 3) & 1);
        ldmatrix4_t(values + r * DP * 2 + ((c ^ (r & 7)) << 4), va);
#pragma unroll
        for (int h = 0; h < NT; ++h) mma<BF16>(o[n][h], va, w[h][0], w[h][1]);
      }
      __syncwarp();  // the stage that is loaded next has been read
      load(i + C::kStages - 1);
    }
    copies_wait<0>();
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum[h][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[h][e], d);
    // ---- the warps meet over their rings
    __syncthreads();
    float* const parts = reinterpret_cast<float*>(smem);
    {
      float* const part = parts + warp * C::kPart;
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = h * 8 + (lane & 3) * 2 + e;
#pragma unroll
          for (int n = 0; n < DP / 16; ++n) {
            part[r * C::kLine + n * 16 + lane / 4] = o[n][h][e];
            part[r * C::kLine + n * 16 + lane / 4 + 8] = o[n][h][e + 2];
          }
          if (lane < 4) {
            part[kRows * C::kLine + r] = ref[h][e] - kLift;
            part[kRows * C::kLine + kRows + r] = sum[h][e];
          }
        }
    }
    __syncthreads();
    const bool whole = unit0 >= b0 && unit1 <= b1;
    if (unit0 >= b0 && unit1 > b1) straddle = {seq, static_cast<int>((unit1 - 1) / size)};
    float* const to = plan.parts + (2LL * blockIdx.x + (unit0 >= b0 ? 1 : 0)) * C::kPart;
    for (int e = threadIdx.x; e < rows * (DP / 4); e += kThreads) {
      const int r = e / (DP / 4), c = e % (DP / 4) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, parts[w * C::kPart + kRows * C::kLine + r]);
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float z = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* const part = parts + w * C::kPart;
        const float mr = part[kRows * C::kLine + r];
        const float f = scale_of(mr, top);
        const float4 x = *reinterpret_cast<const float4*>(part + r * C::kLine + c);
        z += f * part[kRows * C::kLine + kRows + r];
        acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
      }
      if (!whole) {
        *reinterpret_cast<float4*>(to + r * C::kLine + c) = acc;
        if (c == 0) {
          to[kRows * C::kLine + r] = top;
          to[kRows * C::kLine + kRows + r] = z;
        }
      } else if (c < p.dim) {
        const float inv = z == 0.0f ? 0.0f : 1.0f / z;
        *reinterpret_cast<uint2*>(p.out.p + seq * p.out.ld + (head0 + r) * p.out.hs + c) =
            make_uint2(pack_means<BF16>(acc.x, acc.y, inv), pack_means<BF16>(acc.z, acc.w, inv));
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
  if (unit == 0 && threadIdx.x == 0) plan.straddles[share] = straddle;
}

// Joins the parts of a query head's unit, warp w taking part w and every kJoinWarps-th
// behind it. A CTA a sequence and head, which finds the sequence's shares while the first
// kernel runs; or, where the sequences are more than the shares, a CTA a share and head:
// of many short sequences few lie in two shares (256 of 300 tokens, 32 heads of 128
// over 8: 68 us; with 8192 CTAs, most of them without parts, 86).
constexpr int kJoinWarps = 8, kJoinThreads = kJoinWarps * 32;
template <bool BF16, int DP, int NT>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ DecodeParams p,
                                                                   const __grid_constant__ Plan plan) {
  using C = Cfg<DP, NT>;
  constexpr int kRows = C::kRows;
  __shared__ float4 outs[kJoinWarps][32];
  __shared__ float refs[kJoinWarps], sums[kJoinWarps];
  __shared__ long long blocks_sum[2][kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int seq = blockIdx.x / p.heads;
  const int head = blockIdx.x % p.heads, group = p.heads / p.kv_heads;
  int c0, c1;  // the sequence's shares
  if (p.seqs <= plan.shares) {
    const long long blocks = blocks_of(p, seq);
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
    long long total = 0, before = 0;
    for (int w = 0; w < kJoinWarps; ++w) total += blocks_sum[0][w], before += blocks_sum[1][w];
    const long long size = share_of(total, plan.shares);
    c0 = static_cast<int>(before / size);
    c1 = blocks > 0 ? static_cast<int>((before + blocks - 1) / size) : c0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
  } else {
    c0 = seq;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Straddle x = plan.straddles[c0];
    seq = x.seq;
    c1 = seq >= 0 ? x.last : c0;
  }
  if (c0 == c1) return;
  uint16_t* const out = p.out.p + seq * p.out.ld + head * p.out.hs;
  const int unit = head / group * plan.tiles + head % group / kRows, r = head % group % kRows;
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
        ref[i] = x[kRows * C::kLine + r];
        sum[i] = x[kRows * C::kLine + kRows + r];
        if (lane * 4 < DP) v[i] = *reinterpret_cast<const float4*>(x + r * C::kLine + lane * 4);
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
        make_uint2(pack_means<BF16>(acc.x, acc.y, inv), pack_means<BF16>(acc.z, acc.w, inv));
  if (p.lse && lane == 0)
    p.lse[static_cast<long long>(seq) * p.heads + head] = z == 0.0f ? -INFINITY : (top + log2f(z)) * kLn2;
}

// Query heads of a CTA in eights: matrix instructions of 16 tokens by 8 heads.
int eights_of(int heads, int kv_heads) { return heads / kv_heads <= 8 ? 1 : 2; }

size_t straddle_bytes(int shares) { return (static_cast<size_t>(shares) + 1) / 2 * 16; }

template <bool BF16, int DP, int NT>
cudaError_t launch_of(const DecodeParams& p, const Plan& plan, cudaStream_t stream) {
  static unsigned long long devices = 0;
  auto kernel = decode_kernel<BF16, DP, NT>;
  cudaError_t e = with_smem(kernel, Cfg<DP, NT>::kSmem, devices);
  if (e != cudaSuccess) return e;
  kernel<<<plan.shares * plan.units, kThreads, Cfg<DP, NT>::kSmem, stream>>>(p, plan);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(p.seqs, plan.shares)) * static_cast<unsigned>(p.heads));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_join_kernel<BF16, DP, NT>, p, plan);
}

template <bool BF16, int DP>
cudaError_t launch_rows(const DecodeParams& p, const Plan& plan, cudaStream_t stream) {
  return eights_of(p.heads, p.kv_heads) == 1 ? launch_of<BF16, DP, 1>(p, plan, stream)
                                             : launch_of<BF16, DP, 2>(p, plan, stream);
}

int tiles_of(int heads, int kv_heads) {
  const int rows = 8 * eights_of(heads, kv_heads);
  return (heads / kv_heads + rows - 1) / rows;
}
// A share is taken by `units` CTAs, so places are left over where units do not divide
// them: 16 sequences of the same bytes take 160 us with 8, 32, 38 or 76 key heads of 128
// (304, 288, 304 and 304 of 304 places), 162 with 40 (280), 163 with 48 or 64 (288, 256).
int shares_held(int units, int dim, int num_sms) {
  return std::max(num_sms * (dim > 64 ? Cfg<128, 1>::kCtasPerSm : Cfg<64, 1>::kCtasPerSm) / units, 1);
}
template <int DP>
size_t part_bytes(int heads, int kv_heads) {
  return (eights_of(heads, kv_heads) == 1 ? Cfg<DP, 1>::kPart : Cfg<DP, 2>::kPart) * sizeof(float);
}

}  // namespace

size_t decode_workspace(int heads, int kv_heads, int dim, int num_sms) {
  const size_t part = dim > 64 ? part_bytes<128>(heads, kv_heads) : part_bytes<64>(heads, kv_heads);
  const int units = kv_heads * tiles_of(heads, kv_heads), shares = shares_held(units, dim, num_sms);
  return straddle_bytes(shares) + static_cast<size_t>(shares) * units * 2 * part;
}

cudaError_t launch_decode(const DecodeParams& p, void* workspace, int num_sms, cudaStream_t stream) {
  Plan plan;
  plan.tiles = tiles_of(p.heads, p.kv_heads);
  plan.units = p.kv_heads * plan.tiles;
  plan.shares = shares_held(plan.units, p.dim, num_sms);
  plan.straddles = static_cast<Straddle*>(workspace);
  plan.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + straddle_bytes(plan.shares));
  if (p.dim > 64)
    return p.is_bf16 ? launch_rows<true, 128>(p, plan, stream) : launch_rows<false, 128>(p, plan, stream);
  return p.is_bf16 ? launch_rows<true, 64>(p, plan, stream) : launch_rows<false, 64>(p, plan, stream);
}

}  // namespace fgemm
