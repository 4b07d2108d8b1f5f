// fgemm_cache_api.cu -- entry points of the operators around a key-value
// cache: rotary positions with the write into the cache, attention of one
// token over it, attention over packed prompts, log probabilities. Argument
// checks and launches; the kernels are in fgemm_kern_rotary.cu,
// fgemm_kern_decode.cu, fgemm_kern_prompt.cu and fgemm_kern_logprobs.cu.
// Nothing here allocates, synchronises or throws: the calls may be captured
// into a graph.
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm.h"
#include "fgemm_internal.h"

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1024;
constexpr int64_t kMaxStride = int64_t{1} << 36;  // elements; a tensor map takes strides below 2^40 bytes
constexpr int32_t kMaxHeads = 1024;
constexpr float kMaxScale = 18446744073709551616.0f;  // with log2 e it stays finite
constexpr int64_t kMaxSeqs = int64_t{1} << 20;

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

fgemm_status_t check_sizes(fgemm_handle_t h, int64_t tokens, int32_t heads, int32_t kv_heads, int32_t dim, int dtype,
                           bool grouped) {
  if (dtype != FGEMM_F16 && dtype != FGEMM_BF16) return bad_arg(h, "dtype must be FGEMM_F16 or FGEMM_BF16");
  if (tokens < 0 || tokens > kMaxDim) return bad_arg(h, "sizes must be in 0 .. 2^31 - 1024");
  if (heads < 1 || kv_heads < 1 || heads > kMaxHeads || kv_heads > kMaxHeads)
    return bad_arg(h, "heads and kv_heads must be in 1 .. 1024");
  if (grouped && heads % kv_heads != 0) return bad_arg(h, "heads must be a multiple of kv_heads");
  if (dim < 8 || dim > FGEMM_MAX_HEAD_DIM || dim % 8 != 0)
    return bad_arg(h, "dim must be a multiple of 8 in 8 .. FGEMM_MAX_HEAD_DIM");
  return FGEMM_OK;
}

// A tensor of tokens x heads x dim; a stride over one token or head is replaced.
fgemm_status_t check_heads(fgemm_handle_t h, fgemm::Heads& t, const void* p, int64_t ld, int64_t hs, int64_t tokens,
                           int32_t heads, int32_t dim, bool written) {
  if (!p) return bad_arg(h, "a tensor of heads must not be NULL");
  if (heads == 1) hs = dim;
  if (tokens <= 1) ld = dim;
  if (ld < dim || hs < dim || ld > kMaxStride || hs > kMaxStride)
    return bad_arg(h, "a token or head stride is below dim or above 2^36");
  // (hs - dim < (tokens - 1) * ld, without that product: it may pass 64 bits)
  if (written && tokens > 1 && heads > 1 && ld < (heads - 1) * hs + dim && (hs - dim) / ld < tokens - 1)
    return bad_arg(h, "rows of out must not overlap");
  if (off(p, 16) || ld % 8 != 0 || hs % 8 != 0)
    return bad(h, FGEMM_ERR_ALIGNMENT, "tensors of heads must be 16-byte aligned, their strides multiples of 8");
  t.p = static_cast<uint16_t*>(const_cast<void*>(p));
  t.ld = ld;
  t.hs = hs;
  return FGEMM_OK;
}

fgemm_status_t check_cache(fgemm_handle_t h, const fgemm_kv_cache_t* c, int32_t dim) {
  if (!c) return bad_arg(h, "cache must not be NULL");
  if (c->pages < 0 || c->page_size < 1 || c->pages > (int64_t{1} << 31) - 1 ||
      c->pages * c->page_size > (int64_t{1} << 31) - 1)
    return bad_arg(h, "a cache needs page_size >= 1 and pages * page_size below 2^31");
  if (c->pages == 0) return FGEMM_OK;
  if (!c->k || !c->v) return bad_arg(h, "the cache's k and v must not be NULL");
  const int64_t strides[6] = {c->k_page, c->k_token, c->k_head, c->v_page, c->v_token, c->v_head};
  for (int64_t s : strides)
    if (s < dim || s > kMaxStride) return bad_arg(h, "a stride of the cache is below dim or above 2^36");
  for (int64_t s : strides)
    if (s % 8 != 0) return bad(h, FGEMM_ERR_ALIGNMENT, "the cache must be 16-byte aligned, its strides multiples of 8");
  if (off(c->k, 16) || off(c->v, 16))
    return bad(h, FGEMM_ERR_ALIGNMENT, "the cache must be 16-byte aligned, its strides multiples of 8");
  return FGEMM_OK;
}

template <class P>
void set_cache(P& p, const fgemm_kv_cache_t& c) {
  p.k_page = c.k_page;
  p.k_token = c.k_token;
  p.k_head = c.k_head;
  p.v_page = c.v_page;
  p.v_token = c.v_token;
  p.v_head = c.v_head;
  p.page_size = c.page_size;
}

fgemm_status_t check_softmax(fgemm_handle_t h, float scale, int32_t window, const float* lse) {
  if (!(scale > 0.0f) || scale > kMaxScale) return bad_arg(h, "scale must be positive and at most 2^64");
  if (window < 0) return bad_arg(h, "window must not be negative");
  if (off(lse, 4)) return bad(h, FGEMM_ERR_ALIGNMENT, "lse must be 4-byte aligned");
  return FGEMM_OK;
}

}  // namespace

extern "C" {

fgemm_status_t fgemm_rotary_cache(fgemm_handle_t h, int64_t T, int32_t heads, int32_t kv_heads, int32_t dim,
                                  const void* q, int64_t ldq, int64_t hsq, const void* k, int64_t ldk, int64_t hsk,
                                  const void* v, int64_t ldv, int64_t hsv, const int32_t* positions,
                                  const int32_t* slots, const float* inv_freq, int32_t rot, int32_t interleaved,
                                  fgemm_dtype_t dtype, void* out, int64_t ldo, int64_t hso,
                                  const fgemm_kv_cache_t* cache) {
  fgemm_status_t s = check_sizes(h, T, heads, kv_heads, dim, dtype, false);
  if (s != FGEMM_OK) return s;
  if (rot < 0 || rot > dim || rot % 2 != 0) return bad_arg(h, "rot must be even and in 0 .. dim");
  if (T == 0) return nothing(h);
  if (!positions || !slots || (rot > 0 && !inv_freq))
    return bad_arg(h, "positions, slots and inv_freq must not be NULL");
  if (off(positions, 4) || off(slots, 4) || off(inv_freq, 4))
    return bad(h, FGEMM_ERR_ALIGNMENT, "positions, slots and inv_freq must be 4-byte aligned");
  fgemm::RotaryParams p{};
  if ((s = check_heads(h, p.q, q, ldq, hsq, T, heads, dim, false)) != FGEMM_OK ||
      (s = check_heads(h, p.k, k, ldk, hsk, T, kv_heads, dim, false)) != FGEMM_OK ||
      (s = check_heads(h, p.v, v, ldv, hsv, T, kv_heads, dim, false)) != FGEMM_OK ||
      (s = check_heads(h, p.out, out, ldo, hso, T, heads, dim, true)) != FGEMM_OK ||
      (s = check_cache(h, cache, dim)) != FGEMM_OK)
    return s;
  if (out == q && (p.q.ld != p.out.ld || p.q.hs != p.out.hs))
    return bad_arg(h, "out over q needs q's strides");
  if (!h) return no_handle();
  set_cache(p, *cache);
  p.k_cache = static_cast<uint16_t*>(cache->k);
  p.v_cache = static_cast<uint16_t*>(cache->v);
  p.cache_slots = cache->pages * cache->page_size;
  p.positions = positions;
  p.slots = slots;
  p.inv_freq = inv_freq;
  p.tokens = T;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.dim = dim;
  p.rot = rot;
  p.interleaved = interleaved != 0;
  p.is_bf16 = dtype == FGEMM_BF16;
  return launched(h, fgemm::launch_rotary(p, fgemm::handle_sms(h), fgemm::handle_stream(h)));
}

size_t fgemm_attention_paged_workspace(fgemm_handle_t h, int64_t seqs, int32_t heads, int32_t kv_heads, int32_t dim) {
  if (!h || seqs <= 0 || seqs > kMaxSeqs || heads < 1 || heads > kMaxHeads || kv_heads < 1 || heads % kv_heads != 0 ||
      dim < 8 || dim > FGEMM_MAX_HEAD_DIM || dim % 8 != 0)
    return 0;
  return fgemm::decode_workspace(heads, kv_heads, dim, fgemm::handle_sms(h));
}

fgemm_status_t fgemm_attention_paged(fgemm_handle_t h, int64_t seqs, int32_t heads, int32_t kv_heads, int32_t dim,
                                     const void* q, int64_t ldq, int64_t hsq, const fgemm_kv_cache_t* cache,
                                     const int32_t* page_table, int64_t ld_table, int64_t table_pages,
                                     const int32_t* lengths, float scale, int32_t window, fgemm_dtype_t dtype,
                                     void* out, int64_t ldo, int64_t hso, float* lse, void* workspace,
                                     size_t workspace_bytes) {
  fgemm_status_t s = check_sizes(h, seqs, heads, kv_heads, dim, dtype, true);
  if (s != FGEMM_OK) return s;
  if (seqs > kMaxSeqs) return bad_arg(h, "seqs must be in 0 .. 2^20");
  if ((s = check_softmax(h, scale, window, lse)) != FGEMM_OK) return s;
  if (table_pages < 0 || table_pages > kMaxDim) return bad_arg(h, "sizes must be in 0 .. 2^31 - 1024");
  if (seqs == 0) return nothing(h);
  if (!lengths || (table_pages > 0 && !page_table)) return bad_arg(h, "lengths and page_table must not be NULL");
  if (seqs > 1 && ld_table < table_pages) return bad_arg(h, "ld_table is below table_pages");
  if (off(lengths, 4) || off(page_table, 4))
    return bad(h, FGEMM_ERR_ALIGNMENT, "lengths and page_table must be 4-byte aligned");
  fgemm::DecodeParams p{};
  if ((s = check_heads(h, p.q, q, ldq, hsq, seqs, heads, dim, false)) != FGEMM_OK ||
      (s = check_heads(h, p.out, out, ldo, hso, seqs, heads, dim, true)) != FGEMM_OK ||
      (s = check_cache(h, cache, dim)) != FGEMM_OK)
    return s;
  if (out == q && (p.q.ld != p.out.ld || p.q.hs != p.out.hs))
    return bad_arg(h, "out over q needs q's strides");
  if (!h) return no_handle();
  const int sms = fgemm::handle_sms(h);
  const size_t need = fgemm::decode_workspace(heads, kv_heads, dim, sms);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return bad_arg(h, "the workspace is smaller than fgemm_attention_paged_workspace says");
  if (need > 0 && off(workspace, 16)) return bad(h, FGEMM_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  set_cache(p, *cache);
  p.k_cache = static_cast<const uint16_t*>(cache->k);
  p.v_cache = static_cast<const uint16_t*>(cache->v);
  p.pages = cache->pages;
  p.page_table = page_table;
  p.ld_table = ld_table;
  p.table_pages = static_cast<int>(table_pages);
  p.lengths = lengths;
  p.lse = lse;
  p.seqs = static_cast<int>(seqs);
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.dim = dim;
  p.window = window;
  p.scale = scale;
  p.is_bf16 = dtype == FGEMM_BF16;
  return launched(h, fgemm::launch_decode(p, workspace, sms, fgemm::handle_stream(h)));
}

fgemm_status_t fgemm_attention(fgemm_handle_t h, int64_t seqs, int64_t T, int64_t T_k, int32_t heads,
                               int32_t kv_heads, int32_t dim, const void* q, int64_t ldq, int64_t hsq,
                               const void* k, int64_t ldk, int64_t hsk, const void* v, int64_t ldv, int64_t hsv,
                               const int32_t* starts, const int32_t* k_starts, int32_t causal, int32_t window,
                               float scale, fgemm_dtype_t dtype, void* out, int64_t ldo, int64_t hso, float* lse) {
  fgemm_status_t s = check_sizes(h, T, heads, kv_heads, dim, dtype, true);
  if (s != FGEMM_OK) return s;
  if (T_k < 0 || T_k > kMaxDim) return bad_arg(h, "sizes must be in 0 .. 2^31 - 1024");
  if (seqs < 0 || seqs > kMaxSeqs) return bad_arg(h, "seqs must be in 0 .. 2^20");
  if ((s = check_softmax(h, scale, window, lse)) != FGEMM_OK) return s;
  if (window > 0 && !causal) return bad_arg(h, "a window needs causal");
  if (fgemm::prompt_ctas(T, static_cast<int>(seqs), heads) > kMaxDim)
    return bad(h, FGEMM_ERR_UNSUPPORTED, "(T / 128 + seqs) * heads must be below 2^31");
  if (T == 0 || seqs == 0) return nothing(h);
  if (!starts) return bad_arg(h, "starts must not be NULL");
  if (off(starts, 4) || off(k_starts, 4))
    return bad(h, FGEMM_ERR_ALIGNMENT, "starts and k_starts must be 4-byte aligned");
  fgemm::PromptParams p{};
  if ((s = check_heads(h, p.q, q, ldq, hsq, T, heads, dim, false)) != FGEMM_OK ||
      (s = check_heads(h, p.out, out, ldo, hso, T, heads, dim, true)) != FGEMM_OK)
    return s;
  if (T_k > 0 && ((s = check_heads(h, p.k, k, ldk, hsk, T_k, kv_heads, dim, false)) != FGEMM_OK ||
                  (s = check_heads(h, p.v, v, ldv, hsv, T_k, kv_heads, dim, false)) != FGEMM_OK))
    return s;
  if (out == q || out == k || out == v) return bad_arg(h, "out must not be q, k or v");
  if (!h) return no_handle();
  p.starts = starts;
  p.k_starts = k_starts ? k_starts : starts;
  p.lse = lse;
  p.tokens = T;
  p.k_tokens = T_k;
  p.seqs = static_cast<int>(seqs);
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.dim = dim;
  p.causal = causal != 0;
  p.window = window;
  p.scale = scale;
  p.is_bf16 = dtype == FGEMM_BF16;
  p.err = fgemm::handle_err(h);
  p.spin_ns = fgemm::handle_spin_ns(h);
  return launched(h, fgemm::launch_prompt(p, fgemm::handle_sms(h), fgemm::handle_stream(h)));
}

fgemm_status_t fgemm_logprobs(fgemm_handle_t h, int64_t rows, int64_t vocab, const void* logits, int64_t ld,
                              int32_t logits_type, const int32_t* tokens, int32_t top, float* logprob,
                              float* entropy, int32_t* top_tokens, float* top_logprobs) {
  if (logits_type != FGEMM_F16 && logits_type != FGEMM_BF16 && logits_type != FGEMM_LOGITS_F32)
    return bad_arg(h, "logits_type must be FGEMM_F16, FGEMM_BF16 or FGEMM_LOGITS_F32");
  if (rows < 0 || vocab < 0 || rows > (int64_t{1} << 27)) return bad_arg(h, "rows must be in 0 .. 2^27, vocab not negative");
  if (vocab > FGEMM_SAMPLE_MAX_VOCAB) return bad(h, FGEMM_ERR_UNSUPPORTED, "vocab above FGEMM_SAMPLE_MAX_VOCAB");
  if (top < 0 || top > FGEMM_LOGPROBS_MAX_TOP) return bad_arg(h, "top must be in 0 .. FGEMM_LOGPROBS_MAX_TOP");
  if (rows == 0) return nothing(h);
  if (!tokens || !logprob || (vocab > 0 && !logits) || (top > 0 && (!top_tokens || !top_logprobs)))
    return bad_arg(h, "logits, tokens, logprob, top_tokens and top_logprobs must not be NULL");
  if (rows > 1 && ld < vocab) return bad_arg(h, "ld is below vocab");
  if (off(logits, logits_type == FGEMM_LOGITS_F32 ? 4 : 2) || off(tokens, 4) || off(logprob, 4) || off(entropy, 4) ||
      off(top_tokens, 4) || off(top_logprobs, 4))
    return bad(h, FGEMM_ERR_ALIGNMENT, "pointers must be aligned to their elements");
  if (!h) return no_handle();
  fgemm::LogprobParams p{};
  p.logits = logits;
  p.ld = ld;
  p.tokens = tokens;
  p.logprob = logprob;
  p.entropy = entropy;
  p.top_tokens = top_tokens;
  p.top_logprobs = top_logprobs;
  p.rows = static_cast<int>(rows);
  p.vocab = static_cast<int>(vocab);
  p.type = logits_type;
  p.top = top;
  return launched(h, fgemm::launch_logprobs(p, fgemm::handle_sms(h), fgemm::handle_stream(h)));
}

}  // extern "C"
