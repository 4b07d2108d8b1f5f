// fgemm_kern_prompt.cu -- attention over packed prompts: one warp a query and
// head, keys one after the other with the running maximum and sum of the
// softmax.
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_attn.cuh"
#include "fgemm_internal.h"

namespace fgemm {

namespace {

using namespace attn;

__device__ __forceinline__ int held(int v, long long lo, long long hi) {
  return static_cast<int>(min(max(static_cast<long long>(v), lo), hi));
}

template <bool BF16>
__global__ void __launch_bounds__(128) prompt_rows_kernel(const __grid_constant__ PromptParams p) {
  const int lane = threadIdx.x & 31, head = blockIdx.y;
  const long long t = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  int lo = 0, hi = p.seqs;  // the last sequence that starts at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (p.starts[mid] <= t) lo = mid; else hi = mid;
  }
  // (empty sequences start where the next one does: the last of them holds t)
  const int q0 = held(p.starts[lo], 0, p.tokens), q1 = held(p.starts[lo + 1], q0, p.tokens);
  if (t < q0 || t >= q1) return;
  const int k0 = held(p.k_starts[lo], 0, p.k_tokens), k1 = held(p.k_starts[lo + 1], k0, p.k_tokens);
  const long long at = (k1 - k0) - (q1 - q0) + (t - q0);  // the query's position
  const long long last = p.causal ? min(at + 1, static_cast<long long>(k1 - k0)) : k1 - k0;
  const long long first = p.window > 0 ? max(0LL, at + 1 - p.window) : 0;
  const int kv = head / (p.heads / p.kv_heads);
  const bool mine = lane * 4 < p.dim;
  float q[4] = {}, o[4] = {}, m = -INFINITY, l = 0.0f;
  if (mine)
    for (int i = 0; i < 4; ++i) q[i] = to_f32<BF16>(p.q.p[t * p.q.ld + head * p.q.hs + lane * 4 + i]);
  for (long long j = k0 + first; j < k0 + last; ++j) {
    float x = 0.0f;
    if (mine)
      for (int i = 0; i < 4; ++i) x += q[i] * to_f32<BF16>(p.k.p[j * p.k.ld + kv * p.k.hs + lane * 4 + i]);
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    x *= p.scale;
    const float to = fmaxf(m, x);
    const float keep = to == -INFINITY ? 1.0f : expf(m - to), w = x == -INFINITY ? 0.0f : expf(x - to);
    m = to;
    l = l * keep + w;
    if (mine)
      for (int i = 0; i < 4; ++i) o[i] = o[i] * keep + w * to_f32<BF16>(p.v.p[j * p.v.ld + kv * p.v.hs + lane * 4 + i]);
  }
  if (mine)
    for (int i = 0; i < 4; ++i)
      p.out.p[t * p.out.ld + head * p.out.hs + lane * 4 + i] = to_16<BF16>(l == 0.0f ? 0.0f : o[i] / l);
  if (p.lse && lane == 0) p.lse[t * p.heads + head] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_prompt(const PromptParams& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const dim3 grid(static_cast<unsigned>((p.tokens + 3) / 4), static_cast<unsigned>(p.heads));
  if (p.is_bf16)
    prompt_rows_kernel<true><<<grid, 128, 0, stream>>>(p);
  else
    prompt_rows_kernel<false><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fgemm
