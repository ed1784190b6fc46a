// C-ABI entry points of the 8-bit cache and of the norm and rotation before
// a cache: argument checks and launches.
#include <climits>
#include <cmath>

#include "tq_q8.cuh"

using namespace tq;

namespace {

bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }

bool good_stride(int64_t s) { return s >= 0 && s % 8 == 0; }

tq_status check_sizes(const tq_q8_cache* c) {
  if (!c || c->batch < 1 || c->num_kv_heads < 1 || c->head_dim < 1 || c->capacity < 1 ||
      c->capacity % kQ8Block != 0 || (c->format != TQ_Q8_INT8 && c->format != TQ_Q8_E4M3) ||
      (c->dtype != TQ_DTYPE_FP16 && c->dtype != TQ_DTYPE_BF16))
    return TQ_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return TQ_ERR_UNSUPPORTED;
  // units are a grid's y, positions 32-bit
  if (c->batch > kQ8MaxRows || (int64_t)c->batch * c->num_kv_heads > 65535 || c->capacity > INT_MAX - kQ8Block)
    return TQ_ERR_UNSUPPORTED;
  return TQ_OK;
}

tq_status check_cache(const tq_q8_cache* c) {
  const tq_status st = check_sizes(c);
  if (st != TQ_OK) return st;
  for (const void* p : {(const void*)c->k_codes, (const void*)c->v_codes, (const void*)c->k_recent, (const void*)c->v_recent})
    if (!p || !aligned(p, 16)) return TQ_ERR_INVALID_ARG;
  for (const void* p : {(const void*)c->k_scales, (const void*)c->v_scales, (const void*)c->status})
    if (!p || !aligned(p, 4)) return TQ_ERR_INVALID_ARG;
  return TQ_OK;
}

tq_status check_attention(const tq_q8_cache* c, int32_t hq, int32_t n) {
  if (hq < 1 || n < 1 || hq % c->num_kv_heads != 0) return TQ_ERR_INVALID_ARG;
  if (hq / c->num_kv_heads > kQ8MaxGroup || n > kQ8MaxQueries) return TQ_ERR_UNSUPPORTED;
  return TQ_OK;
}

cudaError_t sm_count(int* sms) {
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace

extern "C" {

tq_status tq_q8_append(const tq_q8_cache* c, const void* k, const void* v, int64_t k_row_stride,
                       int64_t k_head_stride, int64_t k_token_stride, int64_t v_row_stride,
                       int64_t v_head_stride, int64_t v_token_stride, int32_t n,
                       const int32_t* lens, const int32_t* n_rows, cudaStream_t stream) {
  const tq_status st = check_cache(c);
  if (st != TQ_OK) return st;
  if (n < 0) return TQ_ERR_INVALID_ARG;
  if (n == 0) return TQ_OK;
  if (!k || !v || !lens || !aligned(k, 16) || !aligned(v, 16) || !aligned(lens, 4) || !aligned(n_rows, 4) ||
      !good_stride(k_row_stride) || !good_stride(k_head_stride) || !good_stride(k_token_stride) ||
      !good_stride(v_row_stride) || !good_stride(v_head_stride) || !good_stride(v_token_stride))
    return TQ_ERR_INVALID_ARG;
  if (n > c->capacity && !n_rows) return TQ_ERR_CAPACITY;
  const Q8AppendArgs a{*c, {k, v}, {k_row_stride, v_row_stride}, {k_head_stride, v_head_stride},
                       {k_token_stride, v_token_stride}, n, lens, n_rows};
  return launch_q8_append(a, stream) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

tq_status tq_q8_read(const tq_q8_cache* c, const int32_t* lens, int64_t start, int32_t n,
                     void* k_out, void* v_out, cudaStream_t stream) {
  const tq_status st = check_cache(c);
  if (st != TQ_OK) return st;
  if (n < 0 || start < 0) return TQ_ERR_INVALID_ARG;
  if (n == 0) return TQ_OK;
  if (!lens || !k_out || !v_out || !aligned(lens, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return TQ_ERR_INVALID_ARG;
  if (start >= c->capacity) return TQ_OK;               // no row holds such a token
  const Q8ReadArgs a{*c, lens, start, n, {k_out, v_out}};
  return launch_q8_read(a, stream) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

tq_status tq_q8_attention_bytes(const tq_q8_cache* c, int32_t num_q_heads, int32_t n, size_t* bytes) {
  tq_status st = check_sizes(c);
  if (st != TQ_OK) return st;
  if (!bytes) return TQ_ERR_INVALID_ARG;
  st = check_attention(c, num_q_heads, n);
  if (st != TQ_OK) return st;
  int sms;
  if (sm_count(&sms) != cudaSuccess) return TQ_ERR_CUDA;
  *bytes = q8_attend_scratch(*c, num_q_heads, n, sms);
  return TQ_OK;
}

tq_status tq_q8_attention(const tq_q8_cache* c, const void* q, int64_t row_stride, int64_t token_stride,
                          int64_t head_stride, int32_t num_q_heads, int32_t n, const int32_t* lens,
                          const int32_t* n_rows, float softmax_scale, void* out, void* scratch,
                          size_t scratch_bytes, cudaStream_t stream) {
  tq_status st = check_cache(c);
  if (st != TQ_OK) return st;
  if (!q || !lens || !out || !scratch || !aligned(q, 16) || !aligned(out, 16) || !aligned(lens, 4) ||
      !aligned(n_rows, 4) || !aligned(scratch, 256) || !good_stride(row_stride) || !good_stride(token_stride) ||
      !good_stride(head_stride) || !std::isfinite(softmax_scale))
    return TQ_ERR_INVALID_ARG;
  st = check_attention(c, num_q_heads, n);
  if (st != TQ_OK) return st;
  int sms;
  if (sm_count(&sms) != cudaSuccess) return TQ_ERR_CUDA;
  if (scratch_bytes < q8_attend_scratch(*c, num_q_heads, n, sms)) return TQ_ERR_INVALID_ARG;
  const double sigma = softmax_scale == 0.f ? 1.0 / std::sqrt((double)c->head_dim) : (double)softmax_scale;
  const Q8AttendArgs a{*c, q, row_stride, token_stride, head_stride, num_q_heads, num_q_heads / c->num_kv_heads,
                       n, lens, n_rows, (float)(sigma * 1.4426950408889634), out, (uint8_t*)scratch};
  return launch_q8_attend(a, sms, stream) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

tq_status tq_q8_get_status(const tq_q8_cache* c, cudaStream_t stream) {
  if (!c || !c->status) return TQ_ERR_INVALID_ARG;
  int32_t w = 0;
  if (cudaMemcpyAsync(&w, c->status, sizeof(w), cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaMemsetAsync(c->status, 0, sizeof(w), stream) != cudaSuccess || cudaStreamSynchronize(stream) != cudaSuccess)
    return TQ_ERR_CUDA;
  return w & kQ8StatusCapacity ? TQ_ERR_CAPACITY : w ? TQ_ERR_INVALID_ARG : TQ_OK;
}

tq_status tq_qk_norm_rope(int32_t batch, int32_t n, int32_t num_q_heads, int32_t num_kv_heads,
                          int32_t head_dim, int32_t dtype, const void* q, int64_t q_row_stride,
                          int64_t q_token_stride, int64_t q_head_stride, const void* k, int64_t k_row_stride,
                          int64_t k_token_stride, int64_t k_head_stride, const int32_t* positions,
                          const float* inv_freq, const void* q_weight, const void* k_weight, float eps,
                          int32_t interleaved, void* q_out, void* k_out, cudaStream_t stream) {
  if (batch < 0 || n < 0 || num_q_heads < 0 || num_kv_heads < 0 || head_dim < 1 ||
      (dtype != TQ_DTYPE_FP16 && dtype != TQ_DTYPE_BF16) || (interleaved != 0 && interleaved != 1) ||
      !(eps >= 0.f) || std::isinf(eps))
    return TQ_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return TQ_ERR_UNSUPPORTED;
  if ((int64_t)num_q_heads + num_kv_heads > 65535 || (int64_t)batch * n > INT_MAX) return TQ_ERR_UNSUPPORTED;
  if (batch == 0 || n == 0 || num_q_heads + num_kv_heads == 0) return TQ_OK;
  if (!positions || !inv_freq || !aligned(positions, 4) || !aligned(inv_freq, 4)) return TQ_ERR_INVALID_ARG;
  if (num_q_heads > 0 && (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(q_weight, 16) ||
                          !good_stride(q_row_stride) || !good_stride(q_token_stride) || !good_stride(q_head_stride)))
    return TQ_ERR_INVALID_ARG;
  if (num_kv_heads > 0 && (!k || !k_out || !aligned(k, 16) || !aligned(k_out, 16) || !aligned(k_weight, 16) ||
                           !good_stride(k_row_stride) || !good_stride(k_token_stride) || !good_stride(k_head_stride)))
    return TQ_ERR_INVALID_ARG;
  const NormRopeArgs a{batch, n, num_q_heads, num_kv_heads, head_dim, dtype, q, k, q_row_stride, q_token_stride,
                       q_head_stride, k_row_stride, k_token_stride, k_head_stride, positions, inv_freq, q_weight,
                       k_weight, eps, interleaved, q_out, k_out};
  return launch_norm_rope(a, stream) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
