// fgemm_kern_decode.cu -- attention of one new token a sequence over a paged
// cache: one warp a query head, keys one after the other with the running
// maximum and sum of the softmax.
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_attn.cuh"
#include "fgemm_internal.h"

namespace fgemm {

namespace {

using namespace attn;

template <bool BF16>
__global__ void __launch_bounds__(128) decode_rows_kernel(const __grid_constant__ DecodeParams p) {
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= p.seqs * p.heads) return;
  const int s = row / p.heads, head = row % p.heads, kv = head / (p.heads / p.kv_heads);
  const bool mine = lane * 4 < p.dim;
  const long long most = static_cast<long long>(p.table_pages) * p.page_size;
  const int length = static_cast<int>(min(static_cast<long long>(max(p.lengths[s], 0)), most));
  const int first = p.window > 0 ? max(0, length - p.window) : 0;
  float q[4] = {}, o[4] = {}, m = -INFINITY, l = 0.0f;
  if (mine)
    for (int i = 0; i < 4; ++i) q[i] = to_f32<BF16>(p.q.p[s * p.q.ld + head * p.q.hs + lane * 4 + i]);
  for (int j = first; j < length; ++j) {
    const int page = p.page_table[s * p.ld_table + j / p.page_size], at = j % p.page_size;
    if (page < 0 || page >= p.pages) continue;
    float x = 0.0f;
    if (mine)
      for (int i = 0; i < 4; ++i)
        x += q[i] * to_f32<BF16>(p.k_cache[page * p.k_page + at * p.k_token + kv * p.k_head + lane * 4 + i]);
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    x *= p.scale;
    const float to = fmaxf(m, x);
    const float keep = to == -INFINITY ? 1.0f : expf(m - to), w = x == -INFINITY ? 0.0f : expf(x - to);
    m = to;
    l = l * keep + w;
    if (mine)
      for (int i = 0; i < 4; ++i)
        o[i] = o[i] * keep +
               w * to_f32<BF16>(p.v_cache[page * p.v_page + at * p.v_token + kv * p.v_head + lane * 4 + i]);
  }
  if (mine)
    for (int i = 0; i < 4; ++i)
      p.out.p[s * p.out.ld + head * p.out.hs + lane * 4 + i] = to_16<BF16>(l == 0.0f ? 0.0f : o[i] / l);
  if (p.lse && lane == 0) p.lse[row] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t decode_workspace(int, int, int, int, int) { return 0; }

cudaError_t launch_decode(const DecodeParams& p, void*, int, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.seqs) * p.heads + 3) / 4);
  if (p.is_bf16)
    decode_rows_kernel<true><<<grid, 128, 0, stream>>>(p);
  else
    decode_rows_kernel<false><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fgemm
