// fgemm_ops_api.cu -- entry points of the operators of a token step: the
// root-mean-square norm, products with 4-bit weights, sampling.  Argument
// checks and launches; the kernels are in fgemm_kern_norm.cu,
// fgemm_kern_w4.cu and fgemm_kern_sample.cu.  Nothing here allocates,
// synchronises or throws: the calls may be captured into a graph.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fgemm.h"
#include "fgemm_internal.h"

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1024;

fgemm_status_t bad(fgemm_handle_t h, fgemm_status_t s, const char* text) {
  return static_cast<fgemm_status_t>(fgemm::handle_fail(h, s, text));
}
fgemm_status_t bad_arg(fgemm_handle_t h, const char* text) { return bad(h, FGEMM_ERR_INVALID_ARG, text); }

// The handle is checked last, so that the other checks work without a device.
fgemm_status_t no_handle() { return bad(nullptr, FGEMM_ERR_INVALID_ARG, "handle is NULL"); }
fgemm_status_t nothing(fgemm_handle_t h) { return h ? FGEMM_OK : no_handle(); }

fgemm_status_t launched(fgemm_handle_t h, cudaError_t e) {
  if (e == cudaSuccess) return FGEMM_OK;
  cudaGetLastError();  // told here, not again by the next call's launch
  return bad(h, FGEMM_ERR_CUDA, cudaGetErrorString(e));
}

bool off(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

bool is_16bit(int dtype) { return dtype == FGEMM_F16 || dtype == FGEMM_BF16; }

fgemm_status_t rms_forward(fgemm_handle_t h, fgemm::NormParams& p, int64_t M, int64_t N, const void* x, int64_t ldx,
                           const void* residual, int64_t ldr, const void* gain, float eps, fgemm_dtype_t dtype,
                           void* total, int64_t ldt, float* inv_rms) {
  if (!is_16bit(dtype)) return bad_arg(h, "dtype must be FGEMM_F16 or FGEMM_BF16");
  if (M < 0 || N < 0 || M > kMaxDim || N > kMaxDim) return bad_arg(h, "sizes must be in 0 .. 2^31 - 1024");
  if (!(eps >= 0.0f) || std::isinf(eps)) return bad_arg(h, "eps must be finite and not negative");
  if (M == 0) return nothing(h);
  if (N == 0) return bad_arg(h, "a row needs at least one value");
  if (!x || !gain) return bad_arg(h, "x and gain must not be NULL");
  if (ldx < N || (residual && ldr < N) || (total && ldt < N))
    return bad_arg(h, "a leading dimension is below the row length");
  if (off(x, 2) || off(residual, 2) || off(gain, 2) || off(total, 2) || off(inv_rms, 4))
    return bad(h, FGEMM_ERR_ALIGNMENT, "16-bit data must be 2-byte aligned, inv_rms 4-byte");
  p = fgemm::NormParams{};
  p.x = static_cast<const uint16_t*>(x);
  p.res = static_cast<const uint16_t*>(residual);
  p.gain = static_cast<const uint16_t*>(gain);
  p.total = static_cast<uint16_t*>(total);
  p.inv_rms = inv_rms;
  p.m = M;
  p.n = static_cast<int>(N);
  p.ldx = ldx;
  p.ldr = ldr;
  p.ldt = ldt;
  p.eps = eps;
  p.is_bf16 = dtype == FGEMM_BF16;
  return FGEMM_OK;
}

}  // namespace

extern "C" {

fgemm_status_t fgemm_rms_norm(fgemm_handle_t h, int64_t M, int64_t N, const void* x, int64_t ldx,
                              const void* residual, int64_t ldr, const void* gain, float eps, fgemm_dtype_t dtype,
                              void* total, int64_t ldt, void* y, int64_t ldy, float* inv_rms) {
  fgemm::NormParams p;
  fgemm_status_t s = rms_forward(h, p, M, N, x, ldx, residual, ldr, gain, eps, dtype, total, ldt, inv_rms);
  if (s != FGEMM_OK || M == 0) return s;
  if (!y) return bad_arg(h, "y must not be NULL");
  if (y == total) return bad_arg(h, "y and total must not be the same memory");
  if (ldy < N) return bad_arg(h, "a leading dimension is below the row length");
  if (off(y, 2)) return bad(h, FGEMM_ERR_ALIGNMENT, "16-bit data must be 2-byte aligned, inv_rms 4-byte");
  if (!h) return no_handle();
  p.y = static_cast<uint16_t*>(y);
  p.ldy = ldy;
  return launched(h, fgemm::launch_norm(p, fgemm::handle_stream(h)));
}

fgemm_status_t fgemm_rms_norm_mx(fgemm_handle_t h, int64_t M, int64_t N, const void* x, int64_t ldx,
                                 const void* residual, int64_t ldr, const void* gain, float eps, fgemm_dtype_t dtype,
                                 void* total, int64_t ldt, int32_t format, void* q, int64_t ldq, void* scales,
                                 int64_t lds, float* inv_rms) {
  if (format != FGEMM_FP8_E4M3 && format != FGEMM_FP8_E5M2)
    return bad_arg(h, "format must be FGEMM_FP8_E4M3 or FGEMM_FP8_E5M2");
  fgemm::NormParams p;
  fgemm_status_t s = rms_forward(h, p, M, N, x, ldx, residual, ldr, gain, eps, dtype, total, ldt, inv_rms);
  if (s != FGEMM_OK || M == 0) return s;
  if (!q || !scales) return bad_arg(h, "q and scales must not be NULL");
  if (ldq < N || lds < (N + 31) / 32)
    return bad_arg(h, "ldq >= N and lds >= ceil(N / 32) are needed");
  if (!h) return no_handle();
  p.q = static_cast<uint8_t*>(q);
  p.ldq = ldq;
  p.scales = static_cast<uint8_t*>(scales);
  p.lds = lds;
  p.mx_format = format;
  return launched(h, fgemm::launch_norm(p, fgemm::handle_stream(h)));
}

size_t fgemm_rms_norm_backward_workspace(fgemm_handle_t h, int64_t M, int64_t N) {
  if (!h || M <= 0 || N <= 0 || M > kMaxDim || N > kMaxDim) return 0;
  return fgemm::norm_back_workspace(M, static_cast<int>(N), fgemm::handle_sms(h));
}

fgemm_status_t fgemm_rms_norm_backward(fgemm_handle_t h, int64_t M, int64_t N, const void* dy, int64_t lddy,
                                       const void* total, int64_t ldt, const void* gain, const float* inv_rms,
                                       const void* dtotal, int64_t lddt, fgemm_dtype_t dtype, void* dx, int64_t lddx,
                                       float* dgain, void* workspace, size_t workspace_bytes) {
  if (!is_16bit(dtype)) return bad_arg(h, "dtype must be FGEMM_F16 or FGEMM_BF16");
  if (M < 0 || N < 0 || M > kMaxDim || N > kMaxDim) return bad_arg(h, "sizes must be in 0 .. 2^31 - 1024");
  if (N == 0) return M == 0 ? nothing(h) : bad_arg(h, "a row needs at least one value");
  if (off(dgain, 4)) return bad(h, FGEMM_ERR_ALIGNMENT, "dgain must be 4-byte aligned");
  if (M == 0 && !h) return no_handle();
  if (M == 0)  // no rows: the gain's gradient is an empty sum
    return dgain ? launched(h, cudaMemsetAsync(dgain, 0, static_cast<size_t>(N) * 4, fgemm::handle_stream(h)))
                 : FGEMM_OK;
  if (!dy || !total || !gain || !inv_rms || !dx) return bad_arg(h, "dy, total, gain, inv_rms and dx must not be NULL");
  if (lddy < N || ldt < N || (dtotal && lddt < N) || lddx < N)
    return bad_arg(h, "a leading dimension is below the row length");
  if (off(dy, 2) || off(total, 2) || off(gain, 2) || off(dtotal, 2) || off(dx, 2) || off(inv_rms, 4))
    return bad(h, FGEMM_ERR_ALIGNMENT, "16-bit data must be 2-byte aligned, inv_rms 4-byte");
  if (!h) return no_handle();
  const int sms = fgemm::handle_sms(h);
  if (!workspace || workspace_bytes < fgemm::norm_back_workspace(M, static_cast<int>(N), sms))
    return bad_arg(h, "the workspace is smaller than fgemm_rms_norm_backward_workspace says");
  if (off(workspace, 4)) return bad(h, FGEMM_ERR_ALIGNMENT, "workspace must be 4-byte aligned");
  fgemm::NormBackParams p{};
  p.dy = static_cast<const uint16_t*>(dy);
  p.total = static_cast<const uint16_t*>(total);
  p.gain = static_cast<const uint16_t*>(gain);
  p.dtotal = static_cast<const uint16_t*>(dtotal);
  p.inv_rms = inv_rms;
  p.dx = static_cast<uint16_t*>(dx);
  p.dgain = dgain;
  p.m = M;
  p.n = static_cast<int>(N);
  p.lddy = lddy;
  p.ldt = ldt;
  p.lddt = lddt;
  p.lddx = lddx;
  p.is_bf16 = dtype == FGEMM_BF16;
  p.ctas = fgemm::norm_back_ctas(M, static_cast<int>(N), sms);
  p.partials = dgain ? static_cast<float*>(workspace) : nullptr;
  p.dots = static_cast<float*>(workspace) + static_cast<size_t>(p.ctas) * static_cast<size_t>(N);
  return launched(h, fgemm::launch_norm_back(p, fgemm::handle_stream(h)));
}

size_t fgemm_matmul_w4_workspace(int64_t M, int64_t K, int32_t group) {
  if (M <= 0 || K <= 0 || M > (int64_t{1} << 20) || K > (int64_t{1} << 30) || (group != 32 && group != 64 && group != 128)) return 0;
  return fgemm::w4_workspace(M, K, group);
}

fgemm_status_t fgemm_matmul_w4(fgemm_handle_t h, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                               const void* W, int64_t ldw, const void* scales, int64_t lds, const void* zeros,
                               int64_t ldz, int32_t group, void* C, int64_t ldc, fgemm_dtype_t dtype,
                               const fgemm_epilogue_t* epi, void* workspace, size_t workspace_bytes) {
  if (!is_16bit(dtype)) return bad_arg(h, "dtype must be FGEMM_F16 or FGEMM_BF16");
  if (M < 0 || N < 0 || K < 0 || M > (int64_t{1} << 20) || N > kMaxDim || K > (int64_t{1} << 30))
    return bad_arg(h, "sizes must be in 0 .. 2^31 - 1024, M in 0 .. 2^20, K in 0 .. 2^30");
  if (group != 32 && group != 64 && group != 128) return bad_arg(h, "group must be 32, 64 or 128");
  const int32_t kind = epi ? epi->kind : FGEMM_EPI_NONE;
  if (kind < FGEMM_EPI_NONE || kind > FGEMM_EPI_SWIGLU) return bad_arg(h, "unknown epilogue kind");
  if (kind == FGEMM_EPI_SWIGLU && N % 2 != 0) return bad_arg(h, "SWIGLU needs an even N (gate | up)");
  const void* bias = epi ? epi->bias : nullptr;
  if (kind == FGEMM_EPI_SCALE_BIAS && !bias) return bad_arg(h, "SCALE_BIAS needs a bias vector");
  const int64_t n_out = kind == FGEMM_EPI_SWIGLU ? N / 2 : N;
  if (M == 0 || n_out == 0) return nothing(h);
  if (!C) return bad_arg(h, "C must not be NULL");
  if (ldc < n_out) return bad_arg(h, "ldc is below the output width");
  if (off(C, 2) || off(bias, 2)) return bad(h, FGEMM_ERR_ALIGNMENT, "C and the bias must be 2-byte aligned");
  if (K > 0) {
    const int64_t groups = (K + group - 1) / group;
    if (!A || !W || !scales) return bad_arg(h, "A, W and scales must not be NULL");
    if (lda < K || ldw < (K + 1) / 2 || lds < groups || (zeros && ldz < groups))
      return bad_arg(h, "lda >= K, ldw >= ceil(K / 2), lds and ldz >= ceil(K / group) are needed");
    // a single row has no stride to keep aligned
    if (off(A, 16) || off(W, 16) || (M > 1 && lda % 8 != 0) || (N > 1 && ldw % 16 != 0))
      return bad(h, FGEMM_ERR_ALIGNMENT, "A and W must be 16-byte aligned, lda a multiple of 8 and ldw of 16");
    if (off(scales, 2)) return bad(h, FGEMM_ERR_ALIGNMENT, "scales must be 2-byte aligned");
    const size_t need = fgemm::w4_workspace(M, K, group);
    if (need > 0 && (!workspace || workspace_bytes < need))
      return bad_arg(h, "the workspace is smaller than fgemm_matmul_w4_workspace says");
    if (need > 0 && off(workspace, 256)) return bad(h, FGEMM_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  }
  if (!h) return no_handle();
  fgemm::W4Params p{};
  p.a = static_cast<const uint16_t*>(A);
  p.w = static_cast<const uint8_t*>(W);
  p.scales = static_cast<const uint16_t*>(scales);
  p.zeros = static_cast<const uint8_t*>(zeros);
  p.bias = static_cast<const uint16_t*>(bias);
  p.c = static_cast<uint16_t*>(C);
  p.lda = lda;
  p.ldw = ldw;
  p.lds = lds;
  p.ldz = ldz;
  p.ldc = ldc;
  p.m = static_cast<int>(M);
  p.n = static_cast<int>(N);
  p.k = static_cast<int>(K);
  p.n_out = static_cast<int>(n_out);
  p.group = group;
  p.epi = kind;
  p.is_bf16 = dtype == FGEMM_BF16;
  p.alpha = epi ? epi->alpha : 1.0f;
  p.err = fgemm::handle_err(h);
  p.spin_ns = fgemm::handle_spin_ns(h);
  return launched(h, fgemm::launch_w4(p, workspace, fgemm::handle_sms(h), fgemm::handle_stream(h)));
}

fgemm_status_t fgemm_sample(fgemm_handle_t h, int64_t rows, int64_t vocab, const void* logits, int64_t ld,
                            int32_t logits_type, const float* u, const fgemm_sampling_t* how, int32_t* token,
                            float* prob) {
  if (logits_type != FGEMM_F16 && logits_type != FGEMM_BF16 && logits_type != FGEMM_LOGITS_F32)
    return bad_arg(h, "logits_type must be FGEMM_F16, FGEMM_BF16 or FGEMM_LOGITS_F32");
  if (rows < 0 || vocab < 0 || rows > (int64_t{1} << 27)) return bad_arg(h, "rows must be in 0 .. 2^27, vocab not negative");
  if (vocab > FGEMM_SAMPLE_MAX_VOCAB) return bad(h, FGEMM_ERR_UNSUPPORTED, "vocab above FGEMM_SAMPLE_MAX_VOCAB");
  if (rows == 0) return nothing(h);
  if (!how || !u || !token || (vocab > 0 && !logits)) return bad_arg(h, "logits, u, how and token must not be NULL");
  if (ld < vocab) return bad_arg(h, "ld is below vocab");
  if (off(logits, logits_type == FGEMM_LOGITS_F32 ? 4 : 2) || off(u, 4) || off(token, 4) || off(prob, 4) ||
      off(how->temperatures, 4) || off(how->top_ks, 4) || off(how->top_ps, 4) || off(how->min_ps, 4))
    return bad(h, FGEMM_ERR_ALIGNMENT, "pointers must be aligned to their elements");
  if (!h) return no_handle();
  fgemm::SampleParams p{};
  p.logits = logits;
  p.ld = ld;
  p.u = u;
  p.temperature = how->temperatures;
  p.top_k = how->top_ks;
  p.top_p = how->top_ps;
  p.min_p = how->min_ps;
  p.temperature0 = how->temperature;
  p.top_k0 = how->top_k;
  p.top_p0 = how->top_p;
  p.min_p0 = how->min_p;
  p.token = token;
  p.prob = prob;
  p.rows = static_cast<int>(rows);
  p.vocab = static_cast<int>(vocab);
  p.type = logits_type;
  return launched(h, fgemm::launch_sample(p, fgemm::handle_sms(h), fgemm::handle_stream(h)));
}

}  // extern "C"
