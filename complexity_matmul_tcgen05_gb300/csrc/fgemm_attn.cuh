// fgemm_attn.cuh -- what the kernels around a key-value cache share: 16-bit
// conversions and the place of a token in a paged cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace fgemm {
namespace attn {

template <bool BF16>
__device__ __forceinline__ float lo_f32(uint32_t w) {
  if (BF16) return __uint_as_float(w << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(w & 0xFFFFu)));
}
template <bool BF16>
__device__ __forceinline__ float hi_f32(uint32_t w) {
  if (BF16) return __uint_as_float(w & 0xFFFF0000u);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16)));
}

template <bool BF16>
__device__ __forceinline__ float to_f32(uint16_t bits) {
  return lo_f32<BF16>(bits);
}

template <bool BF16>
__device__ __forceinline__ uint16_t to_16(float v) {
  if (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}

// Two values in one word, lo in the low half, each rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// As pack2, but what would be infinity in fp16 is its largest number.
template <bool BF16>
__device__ __forceinline__ uint32_t pack_sat(float lo, float hi) {
  if (BF16) return pack2<true>(lo, hi);
  uint32_t w;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// Two outputs of attention in one word: sums of weighted values a and b times the
// reciprocal of the weights' sum. An output is a mean of values, but weights of 16 bits
// and their 32-bit sum differ by up to 2^-11: at 65504 that would be infinity, so in fp16 a
// finite sum stays finite. (In bf16 the types end alike: such a sum is no number of fp32.)
template <bool BF16>
__device__ __forceinline__ uint32_t pack_means(float a, float b, float inv) {
  const float x = a * inv, y = b * inv;
  if (BF16) return pack2<true>(x, y);
  return pack2<false>(fabsf(a) < INFINITY ? fminf(fmaxf(x, -65504.0f), 65504.0f) : x,
                      fabsf(b) < INFINITY ? fminf(fmaxf(y, -65504.0f), 65504.0f) : y);
}

// A kernel's shared memory, asked for once on each device; `devices` is a word of the
// kernel's own.
template <class K>
cudaError_t with_smem(K kernel, int bytes, unsigned long long& devices) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (device & 63);
  if (device < 64 && (__atomic_load_n(&devices, __ATOMIC_ACQUIRE) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && device < 64) __atomic_fetch_or(&devices, bit, __ATOMIC_RELEASE);
  return e;
}

}  // namespace attn
}  // namespace fgemm
