// fgemm_kern_logprobs.cu -- log probability of a given token, entropy and the
// most probable tokens of rows of logits: one CTA a row, passes over the row.
//
// For a row x with largest value m (NaN counts as -inf), held by c entries, and
// r = sum over the others of e^(x_i - m):
//   log p_i = x_i - m - log(c + r),   entropy = log(c + r) - sum e^(x_i - m)(x_i - m) / (c + r)
// One of the c is kept out of the sum, log(1 + (c - 1 + r)), so that what is
// left to the other tokens keeps its bits beside a probability near 1.
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_attn.cuh"
#include "fgemm_internal.h"

namespace fgemm {

namespace {

using namespace attn;

constexpr int kThreads = 256;

template <int TYPE>
__device__ __forceinline__ float logit(const LogprobParams& p, long long row, int i) {
  float x;
  if (TYPE == 2)
    x = static_cast<const float*>(p.logits)[row * p.ld + i];
  else
    x = to_f32<TYPE == 1>(static_cast<const uint16_t*>(p.logits)[row * p.ld + i]);
  return isnan(x) ? -INFINITY : x;
}

// Larger value first, then lower index, as one integer; 0 for -inf.
__device__ __forceinline__ unsigned long long key_of(float x, int i) {
  if (x == -INFINITY) return 0;
  if (x == 0.0f) x = 0.0f;  // -0 and 0 are equal
  const uint32_t b = __float_as_uint(x);
  const uint32_t ordered = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (static_cast<unsigned long long>(ordered) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float value_of(unsigned long long key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

template <class T, class F>
__device__ __forceinline__ T reduce(T v, T* shared, F f) {
  for (int d = 16; d > 0; d >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  v = shared[0];
  for (int i = 1; i < kThreads / 32; ++i) v = f(v, shared[i]);
  return v;
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads) logprobs_rows_kernel(const __grid_constant__ LogprobParams p) {
  __shared__ unsigned long long buffer[kThreads / 32];
  float* const floats = reinterpret_cast<float*>(buffer);
  const auto most = [](auto a, auto b) { return a > b ? a : b; };
  const auto add = [](float a, float b) { return a + b; };
  const long long row = blockIdx.x;
  float m = -INFINITY;
  for (int i = threadIdx.x; i < p.vocab; i += kThreads) m = fmaxf(m, logit<TYPE>(p, row, i));
  m = reduce(m, floats, most);
  float count = 0.0f, r = 0.0f, t = 0.0f;
  for (int i = threadIdx.x; i < p.vocab; i += kThreads) {
    const float x = logit<TYPE>(p, row, i);
    if (x == m) {
      count += 1.0f;
    } else if (x > -INFINITY) {
      const float w = expf(x - m);
      r += w;
      if (w > 0.0f) t += w * (x - m);
    }
  }
  count = reduce(count, floats, add);
  r = reduce(r, floats, add);
  t = reduce(t, floats, add);
  const bool empty = m == -INFINITY;
  const float log_z = log1pf(count - 1.0f + r);
  const auto log_p = [&](float x) { return empty || x == -INFINITY ? -INFINITY : x == m ? -log_z : x - m - log_z; };
  if (threadIdx.x == 0) {
    const int token = p.tokens[row];
    p.logprob[row] = token >= 0 && token < p.vocab ? log_p(logit<TYPE>(p, row, token)) : -INFINITY;
    if (p.entropy) p.entropy[row] = empty ? 0.0f : log_z - t / (count + r);
  }
  unsigned long long before = ~0ull;
  for (int n = 0; n < p.top; ++n) {
    unsigned long long best = 0;
    for (int i = threadIdx.x; i < p.vocab; i += kThreads) {
      const unsigned long long k = key_of(logit<TYPE>(p, row, i), i);
      if (k < before && k > best) best = k;
    }
    best = before = reduce(best, buffer, most);
    if (threadIdx.x == 0) {
      p.top_tokens[row * p.top + n] = best ? static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : -1;
      p.top_logprobs[row * p.top + n] = best ? log_p(value_of(best)) : -INFINITY;
    }
  }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const unsigned grid = static_cast<unsigned>(p.rows);
  if (p.type == 0)
    logprobs_rows_kernel<0><<<grid, kThreads, 0, stream>>>(p);
  else if (p.type == 1)
    logprobs_rows_kernel<1><<<grid, kThreads, 0, stream>>>(p);
  else
    logprobs_rows_kernel<2><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fgemm
