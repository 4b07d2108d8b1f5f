// fgemm_kern_prompt.cu -- attention over packed prompts, on tcgen05.
//
//   S = Q K^T (fp32),  x = scale S,  w = 2^(x log2 e - r),  O = w V,
//   out = O / sum w,  lse = (r + log2 sum w) ln 2
//
// One pass over the keys of a tile of 128 queries, 128 keys a step: S goes from the
// tensor core to tensor memory, a thread takes one row of it (a query) to registers,
// so a row's maximum and sum need no other thread, and writes the weights, rounded to
// 16 bits, over S in tensor memory, from where they are an operand of the product
// with the values. The reference r follows the row's maximum only when that is more
// than 8 above it, so that O is seldom scaled; in bf16 the weights are lowered by 2^8 and
// stay at most 1, so that O is never larger than the sum of w |V| with the maximum as
// reference (values may be near the end of fp32), in fp16 they are lifted by 2^6 and stay
// below 2^14, so that small ones keep their bits.
//
// A CTA has two tiles of queries at a time: while the tensor core works on one tile's
// products the threads of the other tile form its weights. A tile's round is about
// 1300 clocks for the weights (512 of them the exponentials' rate) and 1024 for the
// two products of 128 x 128 x 128, with about 100 for each of the waits between them;
// the two tiles' rounds overlap, so products fill most of the time.
// Warps 0 and 1 issue the products of a tile each, warp 2 loads (TMA, rings of key
// and value tiles), warp 3 looks after the values of steps in which not every row
// sees every key, warps 4-7 and 8-11 are the two tiles' rows.
//
// Those are the steps on the diagonal, at a window's edge and at the end of a
// sequence. A weight there may be 0 because its key is hidden, and 0 times a value
// that is not finite would be NaN: warp 3 clears the values behind the sequence's end
// (another sequence's) and looks for others that are not finite. If there are any,
// the step's product is taken row by row over the keys that each row sees
// (product_by_rows), without the tensor core.
//
// Measured, bf16 with 32 heads of 128 over 8 key heads: 16384 tokens, causal, 1.22 to 1.36
// ms (1.8 to 1.6 PFLOP/s: a card comes to its power limit); 8192 tokens 328 to 350 us
// causal, 620 to 660 us not (1.77 to 1.67 PFLOP/s); 13 packed prompts of 177 to 1819 tokens
// 141 us, bound by the fill and the end of every job, in which the two tiles have nothing
// to run under; 37 tokens 7.1 us. Heads of 64 are bound by the weights: 1.0 PFLOP/s.
//
// Every wait is bounded; a wait that runs out latches the error word and all roles
// leave.
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "fgemm_attn.cuh"
#include "fgemm_internal.h"
#include "fgemm_ptx.cuh"

namespace fgemm {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {

using namespace attn;

constexpr int kTile = 128;            // queries of a tile, keys of a step
constexpr int kEarly = 96;            // keys of a step whose weights are handed over first
constexpr int kThreads = 384;
constexpr int kIssue = 0, kLoad = 2, kLook = 3, kWeights = 4;  // warps (two that issue)
constexpr float kSlack = 8.0f;        // log2 of how far the maximum may be above the reference
constexpr float kFar = 65536.0f;      // size of a reference from which on it is held as a score
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int DP>  // values of a head, padded: 64 or 128
struct Cfg {
  static constexpr int kBytes = kTile * DP * 2;  // of a tile of queries, keys or values
  // Rings of their own for keys and values: who passes over one of them waits for
  // each of its tiles in turn. (In a ring of both, the warps that look after the
  // values alone took a stage whose key tile was still on its way for the next one.)
  static constexpr int kValues = DP == 128 ? 2 : 4, kKeys = kValues + 1;
  static constexpr int kBars = 20 + kKeys + 3 * kValues;
  static constexpr int kBarAt = (2 + kKeys + kValues) * kBytes;
  static constexpr int kJobAt = kBarAt + (8 * kBars + 15) / 16 * 16;  // two jobs, an answer, flags
  static constexpr int kSmem = 1024 + kJobAt + 2 * 32 + 16 + 4 * kValues + 16;
  static constexpr int kOAt = 256;  // tensor memory: scores of the two tiles, then their outputs
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct Args {
  CUtensorMap q, k, v;
  PromptParams p;
  // The two tiles of a job: the same queries of two heads that share their keys
  // (by_heads), or 256 queries in a row of one head.
  int by_heads;
  int rows;   // queries of a job
  int slots;  // of so many queries, over all sequences
  int wide;   // rows of out are on 32 bytes
};

// ------------------------------------------------------------------- PTX

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc].
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_x8(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Eight columns, with the wait for them.
__device__ __forceinline__ void tmem_ld_x8(uint32_t at, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 32 bytes in one store.
__device__ __forceinline__ void store32(void* at, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Asks for a CTA of the grid that has not been launched: it will not be, and its
// work is the asker's. The answer (16 bytes) is counted on `bar`.
__device__ __forceinline__ void ask_for_cta(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   answer),
               "r"(bar)
               : "memory");
}
// Whether there was one, and its index.
__device__ __forceinline__ bool answered_cta(uint32_t answer, unsigned& index) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "=r"(index)
      : "r"(answer)
      : "memory");
  return ok != 0;
}

// Two fp32 operations in one instruction.
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

// One lane of a warp whose lanes are all here; the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// A value that is the same in all lanes, known as such to the compiler.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

template <int V>
struct Constant {
  static constexpr int value = V;
};

// A ring position: stage and phase parity.
template <int N>
struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      ph ^= 1u;
    }
  }
};

// ----------------------------------------------------------------- waits

// One try that may sleep for up to about 20 us.
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}

// Waits for a phase; gives up when another role has (the error word) or when
// the time limit runs out, and then latches `code`.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, unsigned int* err, unsigned long long spin_ns,
                                       uint32_t code, bool honor) {
  const uint64_t t0 = ptx::globaltimer();
#pragma unroll 1
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (honor && *reinterpret_cast<volatile unsigned int*>(err) != 0u) return false;
    if (ptx::globaltimer() - t0 > spin_ns) {
      atomicCAS(err, 0u, code);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const PromptParams& p, int role) {
  // (reading the clock first costs a wait about 400 clocks)
  if (try_wait_long(bar, parity) || try_wait_long(bar, parity)) return true;
  return wait_slow(bar, parity, p.err, p.spin_ns,
                   kErrTimeout | (static_cast<uint32_t>(role) << 24) | (blockIdx.x & 0xFFFFFFu), true);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const PromptParams& p, int role) {
  return __all_sync(0xFFFFFFFFu, wait(bar, parity, p, role));
}
__device__ __forceinline__ void wait_out(uint32_t bar, uint32_t parity, const PromptParams& p, int role) {
  if (!ptx::mbar_try_wait(bar, parity))
    wait_slow(bar, parity, p.err, p.spin_ns, kErrTimeout | (static_cast<uint32_t>(role) << 24), false);
}

// ------------------------------------------------------------------ tiles

__device__ __forceinline__ int held(int v, int lo, long long hi) {
  return static_cast<int>(min(max(static_cast<long long>(v), static_cast<long long>(lo)), hi));
}

// The sequence of slot `slot`. With R queries a job sequence i begins at slot
// floor(start_i / R) + i, which leaves it at least ceil(length / R) slots before the
// next one begins. All lanes of a warp search together. -1: the slot lies before the
// first.
__device__ __forceinline__ int sequence_of(const PromptParams& p, int rows, int slot) {
  const int lane = threadIdx.x & 31;
  auto first = [&](int i) { return held(p.starts[i], 0, p.tokens) / rows + i; };
  int lo = 0, hi = p.seqs;  // the last i in [lo, hi) with first(i) <= slot, if first(lo) is
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const bool ok = lane == 0 || (i < hi && first(i) <= slot);
    const int n = __ffs(~__ballot_sync(0xFFFFFFFFu, ok)) - 1;  // lanes from 0 on that hold it
    const int at = lo + ((n < 0 ? 32 : n) - 1) * step;
    hi = min(hi, at + step);
    lo = at;
  }
  return first(lo) <= slot ? lo : -1;
}

// A tile of queries: its rows, the steps that the keys of any row lie in, and of
// these the ones whose keys every row sees.
struct Tile {
  int rows;  // 0: none
  int from, to;
  int all_from, all_to;
  // a step that it has and of which some row does not see some key
  __device__ __forceinline__ bool masked(int j) const {
    return j >= from && j < to && (j < all_from || j >= all_to);
  }
};
// Keys [lo, hi) that a query at position `at` sees.
__device__ __forceinline__ int key_end(const PromptParams& p, int at, int keys) {
  return p.causal ? max(0, min(at + 1, keys)) : keys;
}
// (a query in front of the first key has a position below 0, and a window may be the
// largest number there is: the difference is formed only where it stays inside 32 bits)
__device__ __forceinline__ int key_begin(const PromptParams& p, int at) {
  return p.window > 0 && at >= p.window ? at + 1 - p.window : 0;
}
__device__ __forceinline__ Tile tile_of(const PromptParams& p, int row0, int queries, int keys) {
  Tile t;
  t.rows = min(kTile, queries - row0);
  t.from = t.to = t.all_from = t.all_to = 0;
  if (t.rows <= 0) {
    t.rows = 0;
    return t;
  }
  const int at0 = keys - queries + row0, at1 = at0 + t.rows - 1;
  const int lo = key_begin(p, at0), hi = key_end(p, at1, keys);
  if (lo < hi) {
    t.from = lo / kTile;
    t.to = (hi + kTile - 1) / kTile;
    t.all_from = (key_begin(p, at1) + kTile - 1) / kTile;
    t.all_to = key_end(p, at0, keys) / kTile;
  }
  return t;
}

// Columns of the weights of keys 16 k to 16 k + 15 of a step from its scores on: each
// 32 keys' weights lie over the first half of their scores.
__device__ __forceinline__ constexpr int weights_at(int k) { return (k >> 1) * 32 + (k & 1) * 8; }

// O (+)= w V of one step for the rows of a warp, over the keys [lo, hi) of the
// step that each row sees; all lanes together. w is read from tensor memory.
template <bool BF16, int DP>
__device__ __forceinline__ void product_by_rows(uint32_t w_at, uint32_t o_at, uint32_t values, int lo, int hi, bool first) {
#pragma unroll 1
  for (int d = 0; d < DP / 8; ++d) {
    float acc[8] = {};
#pragma unroll 1
    for (int c = 0; c < kTile; c += 16) {
      uint32_t w[8];
      tmem_ld_x8(w_at + weights_at(c / 16), w);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int key = c + k;
        if (key < lo || key >= hi) continue;
        const float f = k & 1 ? hi_f32<BF16>(w[k >> 1]) : lo_f32<BF16>(w[k >> 1]);
        uint32_t v[4];
        asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(values + (d >> 3) * (kTile * 128) + key * 128 + (((d & 7) ^ (key & 7)) << 4))
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[2 * i] += f * lo_f32<BF16>(v[i]);
          acc[2 * i + 1] += f * hi_f32<BF16>(v[i]);
        }
      }
      __syncwarp();
    }
    uint32_t o[8];
    if (!first) tmem_ld_x8(o_at + d * 8, o);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(first ? acc[i] : __uint_as_float(o[i]) + acc[i]);
    tmem_st_x8(o_at + d * 8, o);
    tmem_wait_st();
  }
}

// A job: two tiles of one sequence, as the loading warp finds it.
struct Job {
  int head, q0, queries, k0, keys, row0;
  int more;  // 0: there are no more
  int pad;
};

// The job of CTA `index` of the grid; false if there is none (the slots are more than
// the jobs). All lanes of a warp together.
__device__ __forceinline__ bool job_of(const Args& a, unsigned index, Job& job) {
  const PromptParams& p = a.p;
  const unsigned heads = static_cast<unsigned>(p.heads) >> a.by_heads;
  job.head = static_cast<int>(index % heads) << a.by_heads;
  // the last slots first: with a causal mask they have the most keys
  const int slot = a.slots - 1 - static_cast<int>(index / heads);
  const int seq = sequence_of(p, a.rows, slot);
  if (seq < 0) return false;
  job.q0 = held(p.starts[seq], 0, p.tokens);
  job.queries = held(p.starts[seq + 1], job.q0, p.tokens) - job.q0;
  job.k0 = held(p.k_starts[seq], 0, p.k_tokens);
  job.keys = held(p.k_starts[seq + 1], job.k0, p.k_tokens) - job.k0;
  job.row0 = (slot - (job.q0 / a.rows + seq)) * a.rows;
  return job.row0 < job.queries;
}

// The two tiles of a job and the steps of both (the second tile's begin no later
// than the first's end).
struct Tiles {
  Tile t0, t1;
  int from, to;
  __device__ __forceinline__ Tiles(const Args& a, const Job& job) {
    t0 = tile_of(a.p, job.row0, job.queries, job.keys);
    t1 = a.by_heads ? t0 : tile_of(a.p, job.row0 + kTile, job.queries, job.keys);
    from = t0.from < t0.to ? t0.from : t1.from;
    to = t1.from < t1.to ? max(t0.to, t1.to) : t0.to;
  }
  __device__ __forceinline__ const Tile& operator[](int t) const { return t == 0 ? t0 : t1; }
};

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Args a) {
  using C = Cfg<DP>;
  const PromptParams& p = a.p;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  auto q_at = [&](int t) { return base + t * C::kBytes; };
  auto k_at = [&](int s) { return base + (2 + s) * C::kBytes; };
  auto v_at = [&](int s) { return base + (2 + C::kKeys + s) * C::kBytes; };
  const uint32_t bar0 = base + C::kBarAt;
  auto bar = [&](int i) { return bar0 + 8u * i; };
  // by tile
  auto q_full = [&](int t) { return bar(t); };
  auto q_empty = [&](int t) { return bar(2 + t); };
  auto s_full = [&](int t) { return bar(4 + t); };    // scores are there
  auto w_early = [&](int t) { return bar(6 + t); };   // weights of the first keys are there
  auto w_full = [&](int t) { return bar(8 + t); };    // all are
  auto o_full = [&](int t) { return bar(10 + t); };   // outputs are there
  auto go = [&](int t) { return bar(12 + t); };       // it is the tile's turn to issue
  // of the two places for jobs
  auto job_full = [&](int s) { return bar(14 + s); };
  auto job_empty = [&](int s) { return bar(16 + s); };
  const uint32_t taken = bar(18);  // the answer to a request for a job
  const uint32_t drain = bar(19);
  // of the rings
  auto k_full = [&](int s) { return bar(20 + s); };
  constexpr int kVBar = 20 + C::kKeys;
  auto v_full = [&](int s) { return bar(kVBar + s); };
  auto v_ok = [&](int s) { return bar(kVBar + C::kValues + s); };       // looked after
  auto empty = [&](int s) { return bar(kVBar + 2 * C::kValues + s); };  // a step is done
  const uint32_t answer = base + C::kJobAt + 2 * sizeof(Job);
  // of the value tiles in their ring: 1 where not all of it is finite
  volatile int* const wild = reinterpret_cast<volatile int*>(base_ptr + C::kJobAt + 2 * sizeof(Job) + 16);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + C::kJobAt + 2 * sizeof(Job) + 16 + 4 * C::kValues);

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(q_full(t), 1);
      ptx::mbar_init(q_empty(t), 1);
      ptx::mbar_init(s_full(t), 1);
      ptx::mbar_init(w_early(t), 4);
      ptx::mbar_init(w_full(t), 4);
      ptx::mbar_init(o_full(t), 1);
      ptx::mbar_init(go(t), 1);
      ptx::mbar_init(job_full(t), 1);
      ptx::mbar_init(job_empty(t), kThreads / 32 - 1);
    }
    ptx::mbar_init(taken, 1);
    ptx::mbar_init(drain, 2);
    for (int s = 0; s < C::kKeys; ++s) ptx::mbar_init(k_full(s), 1);
    for (int s = 0; s < C::kValues; ++s) {
      ptx::mbar_init(v_full(s), 1);
      ptx::mbar_init(v_ok(s), 1);
      ptx::mbar_init(empty(s), 2);
    }
    ptx::fence_mbar_init();
  }
  volatile Job* const jobs = reinterpret_cast<volatile Job*>(base_ptr + C::kJobAt);
  Job job = {};
  bool any_more = true;
  auto store_job = [&](int place, bool more) {
    if (lane == 0) {
      volatile Job& to = jobs[place];
      to.head = job.head, to.q0 = job.q0, to.queries = job.queries, to.k0 = job.k0, to.keys = job.keys;
      to.row0 = job.row0, to.more = more ? 1 : 0;
    }
  };
  if (warp == kLoad) {  // the first job; an empty one if the CTA's slot is
    if (!job_of(a, blockIdx.x, job)) job.head = job.q0 = job.queries = job.k0 = job.keys = job.row0 = 0;
    store_job(0, true);
  }
  if (warp == kIssue) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  // (all columns: the address is 0, known when this is compiled)
  constexpr uint32_t tmem = 0;
  const int next_row = a.by_heads ? 0 : kTile, next_head = a.by_heads;  // of a job's second tile

  // Jobs are numbered; number n lies in place n & 1, the first since before the
  // barrier above. False: a wait ran out.
  int number = 0;
  auto job_there = [&](int role) {
    return number == 0 || wait_warp(job_full(number & 1), ((number - 1) >> 1) & 1u, p, role);
  };
  auto job_read = [&]() {
    const volatile Job& from = jobs[number & 1];
    job.head = from.head, job.q0 = from.q0, job.queries = from.queries, job.k0 = from.k0, job.keys = from.keys;
    job.row0 = from.row0;
    return from.more != 0;
  };
  auto job_done = [&]() {  // by every warp but the loading one
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(job_empty(number & 1));
    ++number;
  };

  // Registers of warps 0-3 go to the others, of 168 for each of 384 threads at launch:
  // without, a few dozen words of the rows' loop live in local memory and 16384 tokens
  // took 8 % longer. (No function of this kernel is called: with calls the
  // compiler cannot give the rows' warps more than at launch.)
  if (warp < kWeights) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");

  if (warp == kLoad) {
    // ------------------------------------------------------ jobs and loads
    // The grid has a CTA a job; one that is done with its own takes over those of
    // CTAs that have not been launched (a job ahead of its work), so the next job's
    // loads and first scores run under this one's last steps.
    if (lane == 0) {
      ptx::prefetch_tmap(&a.q);
      ptx::prefetch_tmap(&a.k);
      ptx::prefetch_tmap(&a.v);
    }
    uint32_t asked = 0;
    bool ok = true;
    // Asks for jobs until there is one or no more and leaves it for the others.
    auto publish = [&]() {
      bool found = false;
      while (ok && any_more && !found) {
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(taken, 16);
          ask_for_cta(answer, taken);
        }
        __syncwarp();
        // (waited for to its end: the answer is on its way to this CTA's memory)
        if (!wait_warp(taken, asked & 1u, p, 0)) {
          wait_out(taken, asked & 1u, p, 0);
          ok = false;
        }
        ++asked;
        unsigned index = 0;
        any_more = ok && answered_cta(answer, index);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (any_more) found = job_of(a, static_cast<unsigned>(uniform(static_cast<int>(index))), job);
      }
      ++number;
      if (ok && number >= 2) ok = wait_warp(job_empty(number & 1), ((number - 2) >> 1) & 1u, p, 0);
      if (ok) {
        store_job(number & 1, found);
        if (lane == 0) ptx::mbar_arrive(job_full(number & 1));
      }
      return ok && found;
    };
    Ring<C::kKeys> rk;
    Ring<C::kValues> rv;
    uint32_t q_turn[2] = {0, 0};
    int nk = 0, nv = 0;  // tiles loaded so far
    for (bool more = true; ok && more;) {
      const Tiles tiles(a, job);
      const int q0 = job.q0 + job.row0, q_head = job.head, k0 = job.k0 + tiles.from * kTile;
      const int kv = job.head / (p.heads / p.kv_heads), count = tiles.to - tiles.from;
      auto load = [&](int n, uint32_t at, const CUtensorMap* map, uint32_t full) {
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(full, C::kBytes);
          for (int x = 0; x < DP; x += 64)
            tma_load_3d(at + x * (kTile * 2), map, x, kv, k0 + n * kTile, full);
        }
      };
      for (int t = 0; ok && t < 2; ++t)
        if (tiles[t].from < tiles[t].to) {
          ok = wait_warp(q_empty(t), (q_turn[t] & 1u) ^ 1u, p, 0);
          if (ok && lane == 0) {
            ptx::mbar_arrive_expect_tx(q_full(t), C::kBytes);
            for (int x = 0; x < DP; x += 64)
              tma_load_3d(q_at(t) + x * (kTile * 2), &a.q, x, q_head + t * next_head, q0 + t * next_row, q_full(t));
          }
          q_turn[t] += ok ? 1 : 0;
        }
      // Keys go a step ahead of the values. A step's end hands back its values and
      // the keys of the next, whose scores it ended with; there is one stage more of
      // keys for the first of a job, which come back with its first step.
      if (count <= 0) more = publish();
      for (int n = 0; ok && n < count; ++n) {
        if (n == 0) load(0, k_at(rk.s), &a.k, k_full(rk.s)), rk.next(), ++nk;
        if (!(ok = wait_warp(empty(rv.s), rv.ph ^ 1u, p, 0))) break;
        if (n + 1 < count) load(n + 1, k_at(rk.s), &a.k, k_full(rk.s)), rk.next(), ++nk;
        load(n, v_at(rv.s), &a.v, v_full(rv.s)), rv.next(), ++nv;
        if (n == min(count, C::kValues) - 1) {  // the ring is full, or this job is loaded
          more = publish();
        }
      }
    }
    // Whatever another role did, the copies in flight land before the CTA ends.
    if (lane == 0) {
      for (int i = max(0, nk - C::kKeys); i < nk; ++i) wait_out(k_full(i % C::kKeys), (i / C::kKeys) & 1u, p, 0);
      for (int i = max(0, nv - C::kValues); i < nv; ++i) wait_out(v_full(i % C::kValues), (i / C::kValues) & 1u, p, 0);
      for (int t = 0; t < 2; ++t)
        if (q_turn[t] > 0) wait_out(q_full(t), (q_turn[t] - 1) & 1u, p, 0);
    }
    __syncwarp();
  } else if (warp < kIssue + 2) {
    // --------------------------------------------------------- products
    // A thread a tile, in turns: a thread's waits and commits (about 100 clocks each)
    // run under the other's products, of which the tensor core holds about eight.
    // By one thread alone 16384 tokens took 1.75 ms where this took 1.50; by two
    // without turns, whose tiles fell in step, 2.2. All lanes go through the loop, so
    // that what a product takes (descriptors, addresses) is known to be the warp's
    // (1.68 ms without); one lane issues.
    constexpr uint32_t fmt = BF16 ? 1u : 0u;
    // fp32 accumulator, M = 128; scores: both operands K-major, N = 128;
    // outputs: the values MN-major (bit 16), N = dim
    constexpr uint32_t i_s = (1u << 4) | (fmt << 7) | (fmt << 10) | ((kTile >> 3) << 17) | ((kTile >> 4) << 24);
    // (of the padded width only what dim, in sixteens, has)
    const int sixteens = (p.dim + 15) / 16;
    const uint32_t i_o = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 16) |
                         (static_cast<uint32_t>(2 * sixteens) << 17) | ((kTile >> 4) << 24);
    const int t = warp - kIssue;
    const uint32_t s_to = tmem + t * kTile, o_to = tmem + C::kOAt + t * 128;
    const uint64_t q_desc = ptx::sdesc(q_at(t), 16, 1024);
    const bool leader = elect_one();
    uint32_t turn = 0, q_turn = 0;
    Ring<C::kKeys> rk;
    Ring<C::kValues> rv;
    // (the first tile's first turn needs no word of the second)
    uint32_t mine = t == 0 ? 1u : 0u;
    bool ok = true;
    for (; ok && (ok = job_there(1)) && job_read(); job_done()) {
      const Tiles tiles(a, job);
      const int first = uniform(tiles.from), last = uniform(tiles.to);
      const int tile_from = uniform(tiles[t].from), tile_to = uniform(tiles[t].to);
      const int all_from = uniform(tiles[t].all_from), all_to = uniform(tiles[t].all_to);
      if (tile_from < tile_to) {
        if (!(ok = wait_warp(q_full(t), q_turn, p, 1))) break;
        q_turn ^= 1u;
      }
      for (int j = first - 1; first < last && j < last; ++j) {
        // the product of step j with the values, then the scores of step j + 1
        const bool begun = j >= first, product = begun && j >= tile_from && j < tile_to;
        const bool scores = j + 1 >= tile_from && j + 1 < tile_to, keys_too = j + 1 < last;
        const uint64_t k_desc = ptx::sdesc(k_at(rk.s), 16, 1024), v_desc = ptx::sdesc(v_at(rv.s), kTile * 128, 1024);
        auto form_scores = [&]() {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const uint32_t step = (k >> 2) * (kTile * 128 >> 4) + (k & 3) * 2;
            if (k < sixteens) ptx::mma_f16(s_to, q_desc + step, k_desc + step, i_s, k != 0 ? 1u : 0u);
          }
          ptx::mma_commit(s_full(t));
          if (j + 2 == tile_to) ptx::mma_commit(q_empty(t));
        };
        // products with the values of which the weights are there
        auto take = [&](int from, int to) {
          const uint32_t more = j != tile_from ? 1u : 0u;
#pragma unroll
          for (int n = 0; n < kTile / 16; ++n) {
            const int k = (n + 4) % 8;  // (the second half of the keys comes first)
            if (n >= from && n < to) mma_ts(o_to, s_to + weights_at(k), v_desc + k * 128, i_o, n != 0 ? 1u : more);
          }
        };
        {
          const bool x = !begun || ptx::mbar_try_wait(v_full(rv.s), rv.ph);
          const bool y = !begun || ptx::mbar_try_wait(v_ok(rv.s), rv.ph);
          const bool z = !keys_too || ptx::mbar_try_wait(k_full(rk.s), rk.ph);
          ok = __all_sync(0xFFFFFFFFu, x && y && z) ||
               ((!begun || (wait_warp(v_full(rv.s), rv.ph, p, 1) && wait_warp(v_ok(rv.s), rv.ph, p, 1))) &&
                (!keys_too || wait_warp(k_full(rk.s), rk.ph, p, 1)));
        }
        ok = ok && wait_warp(go(t), mine, p, 1) && (!product || wait_warp(w_early(t), turn, p, 1));
        if (!ok) break;
        mine ^= 1u;
        ptx::tc_fence_after();
        if (product) {
          const bool issue = leader && ((j >= all_from && j < all_to) || wild[rv.s] == 0);
          if (issue) take(0, kEarly / 16);
          if (!(ok = wait_warp(w_full(t), turn, p, 1))) break;
          turn ^= 1u;
          ptx::tc_fence_after();
          if (issue) take(kEarly / 16, kTile / 16);
        }
        if (leader) {
          if (scores)
            form_scores();
          else if (product)
            ptx::mma_commit(o_full(t));
          ptx::mbar_arrive(go(1 - t));
          if (begun) ptx::mma_commit(empty(rv.s));
        }
        if (keys_too) rk.next();
        if (begun) rv.next();
      }
    }
    // Every product of this warp is complete before tensor memory goes back.
    if (leader) {
      ptx::mma_commit(drain);
      wait_out(drain, 0, p, 1);
    }
    __syncwarp();
  } else if (warp == kLook) {
    // ----------------------------------------------- values that are hidden
    Ring<C::kValues> rv;
    bool ok = true;
    for (; ok && (ok = job_there(3)) && job_read(); job_done()) {
      const Tiles tiles(a, job);
      for (int j = tiles.from; j < tiles.to; ++j, rv.next()) {
        if (!(ok = wait_warp(v_full(rv.s), rv.ph, p, 3))) break;
        uint32_t most = 0;  // magnitudes as integers, two halves
        if (tiles.t0.masked(j) || tiles.t1.masked(j)) {
          const int count = min(kTile, job.keys - j * kTile);
          for (int x = 0; x < DP; x += 64) {
            const uint32_t at = v_at(rv.s) + x * (kTile * 2) + lane * 16;  // 4 rows at a time
#pragma unroll 8
            for (int r = lane >> 3; r < count; r += 4) {
              uint32_t v[4];
              asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                           : "r"(at + (r >> 2) * 512));
#pragma unroll
              for (int i = 0; i < 4; ++i) most = __vmaxu2(most, v[i] & 0x7FFF7FFFu);
            }
            if (count < kTile)
              for (int r = count + (((lane >> 3) - count) & 3); r < kTile; r += 4)
                asm volatile("st.volatile.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + (r >> 2) * 512), "r"(0u)
                             : "memory");
          }
          ptx::fence_proxy_async_smem();
        }
        constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
        const bool any = __any_sync(0xFFFFFFFFu, (most & 0xFFFFu) >= kInf || (most >> 16) >= kInf);
        if (lane == 0) {
          wild[rv.s] = any ? 1 : 0;
          ptx::mbar_arrive(v_ok(rv.s));
        }
      }
    }
  } else {
    // ---------------------------------------------------------- weights
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int t = (warp - kWeights) >> 2, row = (warp & 3) * 32 + lane;  // row of the tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + t * kTile, o_at = tmem + lanes + C::kOAt + t * 128;
    const float to_log2 = p.scale * kLog2e;
    constexpr float kLift = BF16 ? -kSlack : 6.0f;  // log2 of the weights' factor
    uint32_t turn = 0, o_turn = 0;
    bool ok = true;
    // (What a step seldom needs of its job is read again there: registers are short.)
    auto keys_seen = [&](int j, int& lo, int& hi) {  // of step j by this row
      const volatile Job& of = jobs[number & 1];
      const int keys = of.keys, at = keys - of.queries + of.row0 + t * next_row + row;
      lo = key_begin(p, at) - j * kTile, hi = key_end(p, at, keys) - j * kTile;
    };
    int ahead = 0;  // value tiles before step 0 of the job
    for (; ok && (ok = job_there(2)) && job_read(); job_done()) {
      int tile_from, tile_to, all_from, all_to;
      {
        const Tiles tiles(a, job);
        ahead -= tiles.from;
        tile_from = tiles[t].from, tile_to = tiles[t].to, all_from = tiles[t].all_from, all_to = tiles[t].all_to;
      }
      // Rounded to fp32 the reference is off by up to half of its last place: nothing to
      // the weights of a row, which are all off alike, but at 2^27 it is 8, beyond what
      // a weight of 16 bits holds. From kFar on the reference is a score itself, and the
      // other scores' differences from it (exact near it) meet scale log2 e.
      float ref = -INFINITY, sum = 0.0f;
      bool far = false;    // of some row of the warp
      float shift = 0.0f;  // log2 of what sums gain when ref becomes a score
      // One step. Three copies of the code, so that the one that runs again and again
      // stays short enough for the instruction cache: for steps in which every row sees
      // every key, for the others, and, in a loop of its own, for both behind a far
      // reference. The step that finds one is left as it was and taken again there.
      // (As a branch of the first two copies this cost packed prompts 3.5 %; so 0.4 %,
      // heads of 64 3 %.)
      constexpr int kAll = 0, kSome = 1, kFarRows = 2;
      auto step = [&](auto kind, int j) {
        constexpr bool MASKED = decltype(kind)::value != kAll, FAR = decltype(kind)::value == kFarRows;
        if (!(ok = wait_warp(s_full(t), turn, p, 2))) return;
        turn ^= 1u;
        ptx::tc_fence_after();
        // The scores, in chunks of 32 keys.
        uint32_t s[4][32];
        int lo = 0, hi = kTile;
        if (MASKED) keys_seen(j, lo, hi);
        auto chunk = [&](uint32_t (&x)[32], int c) {  // arrived: keys 32 c on
          ptx::tmem_regs_ready(x);
          if (MASKED) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i < lo || 32 * c + i >= hi) x[i] = 0xFF800000u;  // -inf
          }
        };
        float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 4; ++i) ptx::tmem_ld_32x32b_x32(s_at + i * 32, s[i]);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) chunk(s[i], i);
#pragma unroll
        for (int c = 0; c < 32; c += 2)
#pragma unroll
          for (int i = 0; i < 4; ++i) m[i] = max3(m[i], __uint_as_float(s[i][c]), __uint_as_float(s[i][c + 1]));
        const float unit = FAR ? to_log2 : 1.0f;  // of the reference and the maximum
        const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * (FAR ? 1.0f : to_log2);
        const bool above = most * unit > fmaf(ref, unit, kSlack);
        if (__any_sync(0xFFFFFFFFu, above || (FAR && shift != 0.0f))) {
          if (!FAR) {
            far = __any_sync(0xFFFFFFFFu, above && fabsf(most) > kFar);
            if (far) {
              turn ^= 1u;
              return;
            }
          }
          const float next = above ? most : ref;
          const float f = next == -INFINITY ? 1.0f : exp2_fast((ref - next) * unit + (FAR ? shift : 0.0f));
          if (FAR) shift = 0.0f;
          ref = next;
          sum *= f;
          if (j != tile_from) {
            // (the scores of this step are there, so the product before them is done)
#pragma unroll 1
            for (int d = 0; d < DP; d += 8) {
              uint32_t o[8];
              tmem_ld_x8(o_at + d, o);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st_x8(o_at + d, o);
            }
          }
        }
        if (FAR) {
          const float base = ref == -INFINITY ? 0.0f : ref;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 32; ++c) s[i][c] = __float_as_uint(__uint_as_float(s[i][c]) - base);
        }
        const uint64_t to_log2_2 = pair(to_log2, to_log2);
        const float less = ref == -INFINITY ? 0.0f : FAR ? kLift : kLift - ref;
        const uint64_t less2 = pair(less, less);
        uint64_t sum2[2] = {pair(sum, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int i = (n + 2) & 3;  // chunk
          uint32_t (&x)[32] = s[i];
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float u, v;
            unpair(fma2(pair(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), to_log2_2, less2), u, v);
            u = exp2_fast(u);
            v = exp2_fast(v);
            sum2[c & 1] = add2(sum2[c & 1], pair(u, v));
            w[c] = pack2<BF16>(u, v);
          }
          tmem_st_x16(s_at + weights_at(2 * i), w);  // over its own scores
          if (n == kEarly / 32 - 1) {  // the product with these values may begin
            tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(w_early(t));
          }
        }
        tmem_wait_st();
        {
          float x, y;
          unpair(add2(sum2[0], sum2[1]), x, y);
          sum = x + y;
        }
        if (MASKED) {
          const int n = ahead + j, st = n % C::kValues;
          const uint32_t ph = (n / C::kValues) & 1u;
          if (!(ok = wait_warp(v_full(st), ph, p, 2) && wait_warp(v_ok(st), ph, p, 2))) return;
          if ((!FAR || j < all_from || j >= all_to) && wild[st] != 0) {
            product_by_rows<BF16, DP>(s_at, o_at, v_at(st), lo, hi, j == tile_from);
            ptx::fence_proxy_async_smem();
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(w_full(t));
      };
      int j = tile_from;
      for (; ok && j < tile_to; ++j) {
        if (j >= all_from && j < all_to)
          step(Constant<kAll>{}, j);
        else
          step(Constant<kSome>{}, j);
        if (far) break;
      }
      if (far) {
        const float score = __fdividef(ref, to_log2);
        if (ref > -INFINITY) shift = fmaf(-score, to_log2, ref - kLift) + kLift;  // (ref - kLift: as rounded for the weights)
        ref = score;
        for (; ok && j < tile_to; ++j) step(Constant<kFarRows>{}, j);
        ref *= to_log2;
      }
      // outputs: a row a thread
      if (!ok) break;
      const bool any = tile_from < tile_to;
      if (any) {
        if (!(ok = wait_warp(o_full(t), o_turn, p, 2))) break;
        o_turn ^= 1u;
        ptx::tc_fence_after();
      }
      job_read();
      ahead += Tiles(a, job).to;
      const int head = job.head + t * next_head, at = job.row0 + t * next_row + row;
      const bool mine = at < job.queries;
      const long long token = static_cast<long long>(job.q0) + at;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      uint16_t* const out = p.out.p + token * p.out.ld + head * p.out.hs;
#pragma unroll 1
      for (int d = 0; d < DP; d += 32) {
        uint32_t o[32], w[16];
        if (any) {
          ptx::tmem_ld_32x32b_x32(o_at + d, o);
          ptx::tmem_wait_ld();
          ptx::tmem_regs_ready(o);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = sum == 0.0f ? 0u : pack_sat<BF16>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
        if (!BF16) {
          // pack_means, by saturation where all sums are finite (seen by their products
          // with 0): element by element it cost 64 x 256 tokens 8 %
          uint64_t none = 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) none = fma2(pair(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), 0, none);
          float x, y;
          unpair(none, x, y);
          if (__any_sync(0xFFFFFFFFu, sum != 0.0f && !(x + y == 0.0f))) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[i] = sum == 0.0f ? 0u : pack_means<BF16>(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]), inv);
          }
        }
        if (mine && a.wide) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (d + 16 * i < p.dim) store32(out + d + 16 * i, &w[8 * i]);
        } else if (mine) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (d + 8 * i < p.dim)
              *reinterpret_cast<uint4*>(out + d + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        __syncwarp();
      }
      if (mine && p.lse) p.lse[token * p.heads + head] = sum == 0.0f ? -INFINITY : (ref - kLift + log2f(sum)) * kLn2;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kIssue) ptx::tmem_dealloc(*tmem_slot, 512);
}

// A map of tokens x heads x dim in boxes of 64 values x 128 tokens of a head.
bool encode(CUtensorMap* map, const Heads& t, long long tokens, int heads, int dim, bool bf16) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(t.hs) * 2, static_cast<cuuint64_t>(t.ld) * 2};
  const cuuint32_t box[3] = {64, 1, kTile}, step[3] = {1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, t.p, dims, strides, box,
             step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16, int DP>
cudaError_t launch_of(const Args& a, unsigned grid, cudaStream_t stream) {
  static unsigned long long devices = 0;
  auto kernel = prompt_kernel<BF16, DP>;
  cudaError_t e = with_smem(kernel, Cfg<DP>::kSmem, devices);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, Cfg<DP>::kSmem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

// At most, with either kind of job.
long long prompt_ctas(long long tokens, int seqs, int heads) { return (tokens / kTile + seqs) * heads; }

cudaError_t launch_prompt(const PromptParams& p, int num_sms, cudaStream_t stream) {
  Args a;
  a.p = p;
  // Two heads with the same keys begin and end together, two tiles of one head do
  // not: packed prompts of 177 to 1819 tokens 160 us against 180. Where that leaves
  // SMs without a job, short sequences have one tile a CTA instead: 37 tokens 7.5 us
  // against 9.2. (Odd groups have no such pairs: 13 packed prompts of 28 heads over 4 key
  // heads take 147 us, of 28 over 14 129.)
  const long long pairs = (p.tokens + kTile - 1) / kTile * (p.heads / 2);
  a.by_heads = p.heads / p.kv_heads % 2 == 0 && pairs >= num_sms;
  a.rows = a.by_heads ? kTile : 2 * kTile;
  a.slots = static_cast<int>(p.tokens / a.rows) + p.seqs;
  a.wide = reinterpret_cast<uintptr_t>(p.out.p) % 32 == 0 && p.out.ld % 16 == 0 && p.out.hs % 16 == 0 && p.dim % 16 == 0;
  if (!encode(&a.q, p.q, p.tokens, p.heads, p.dim, p.is_bf16)) return cudaErrorInvalidValue;
  if (p.k_tokens == 0) {  // nothing is loaded
    a.k = a.v = a.q;
  } else if (!encode(&a.k, p.k, p.k_tokens, p.kv_heads, p.dim, p.is_bf16) ||
             !encode(&a.v, p.v, p.k_tokens, p.kv_heads, p.dim, p.is_bf16)) {
    return cudaErrorInvalidValue;
  }
  const unsigned grid = static_cast<unsigned>(a.slots) * static_cast<unsigned>(p.heads >> a.by_heads);
  if (p.dim > 64) return p.is_bf16 ? launch_of<true, 128>(a, grid, stream) : launch_of<false, 128>(a, grid, stream);
  return p.is_bf16 ? launch_of<true, 64>(a, grid, stream) : launch_of<false, 64>(a, grid, stream);
}

}  // namespace fgemm
