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

tq_status tq_q8_append(const tq_q8_cache* c, const tq_q8_append_args* x, cudaStream_t stream) {
  const tq_status st = check_cache(c);
  if (st != TQ_OK) return st;
  if (!x || x->n < 0) return TQ_ERR_INVALID_ARG;
  if (x->n == 0) return TQ_OK;
  if (!x->k || !x->v || !x->lens || !aligned(x->k, 16) || !aligned(x->v, 16) || !aligned(x->lens, 4) ||
      !aligned(x->n_rows, 4) || !good_stride(x->k_row_stride) || !good_stride(x->k_head_stride) ||
      !good_stride(x->k_token_stride) || !good_stride(x->v_row_stride) || !good_stride(x->v_head_stride) ||
      !good_stride(x->v_token_stride))
    return TQ_ERR_INVALID_ARG;
  if (x->n > c->capacity && !x->n_rows) return TQ_ERR_CAPACITY;
  const Q8AppendArgs a{*c, {x->k, x->v}, {x->k_row_stride, x->v_row_stride}, {x->k_head_stride, x->v_head_stride},
                       {x->k_token_stride, x->v_token_stride}, x->n, x->lens, x->n_rows};
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

tq_status tq_q8_attention(const tq_q8_cache* c, const tq_q8_attention_args* x, cudaStream_t stream) {
  tq_status st = check_cache(c);
  if (st != TQ_OK) return st;
  if (!x || !x->q || !x->lens || !x->out || !x->scratch || !aligned(x->q, 16) || !aligned(x->out, 16) ||
      !aligned(x->lens, 4) || !aligned(x->n_rows, 4) || !aligned(x->scratch, 256) || !good_stride(x->row_stride) ||
      !good_stride(x->token_stride) || !good_stride(x->head_stride) || !std::isfinite(x->softmax_scale))
    return TQ_ERR_INVALID_ARG;
  st = check_attention(c, x->num_q_heads, x->n);
  if (st != TQ_OK) return st;
  int sms;
  if (sm_count(&sms) != cudaSuccess) return TQ_ERR_CUDA;
  if (x->scratch_bytes < q8_attend_scratch(*c, x->num_q_heads, x->n, sms)) return TQ_ERR_INVALID_ARG;
  const double sigma = x->softmax_scale == 0.f ? 1.0 / std::sqrt((double)c->head_dim) : (double)x->softmax_scale;
  const Q8AttendArgs a{*c, x->q, x->row_stride, x->token_stride, x->head_stride, x->num_q_heads,
                       x->num_q_heads / c->num_kv_heads, x->n, x->lens, x->n_rows,
                       (float)(sigma * 1.4426950408889634), x->out, (uint8_t*)x->scratch};
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

tq_status tq_qk_norm_rope(const tq_qk_norm_rope_args* x, cudaStream_t stream) {
  if (!x || x->batch < 0 || x->n < 0 || x->num_q_heads < 0 || x->num_kv_heads < 0 || x->head_dim < 1 ||
      (x->dtype != TQ_DTYPE_FP16 && x->dtype != TQ_DTYPE_BF16) || (x->interleaved != 0 && x->interleaved != 1) ||
      !(x->eps >= 0.f) || std::isinf(x->eps))
    return TQ_ERR_INVALID_ARG;
  if (x->head_dim != 64 && x->head_dim != 128) return TQ_ERR_UNSUPPORTED;
  if ((int64_t)x->num_q_heads + x->num_kv_heads > 65535 || (int64_t)x->batch * x->n > INT_MAX) return TQ_ERR_UNSUPPORTED;
  if (x->batch == 0 || x->n == 0 || x->num_q_heads + x->num_kv_heads == 0) return TQ_OK;
  if (!x->positions || !x->inv_freq || !aligned(x->positions, 4) || !aligned(x->inv_freq, 4)) return TQ_ERR_INVALID_ARG;
  if (x->num_q_heads > 0 &&
      (!x->q || !x->q_out || !aligned(x->q, 16) || !aligned(x->q_out, 16) || !aligned(x->q_weight, 16) ||
       !good_stride(x->q_row_stride) || !good_stride(x->q_token_stride) || !good_stride(x->q_head_stride)))
    return TQ_ERR_INVALID_ARG;
  if (x->num_kv_heads > 0 &&
      (!x->k || !x->k_out || !aligned(x->k, 16) || !aligned(x->k_out, 16) || !aligned(x->k_weight, 16) ||
       !good_stride(x->k_row_stride) || !good_stride(x->k_token_stride) || !good_stride(x->k_head_stride)))
    return TQ_ERR_INVALID_ARG;
  const NormRopeArgs a = norm_rope_args(*x);
  int sms;
  if (sm_count(&sms) != cudaSuccess) return TQ_ERR_CUDA;
  return launch_norm_rope(a, sms, stream) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
