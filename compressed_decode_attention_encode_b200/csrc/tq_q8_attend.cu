// Attention over the 8-bit cache (include/tq.h has the contract).
//
// The simplest kernel that is right for every case: one CTA per (row, query
// token, query head), a warp per token, float32 throughout, and one online
// softmax per warp; the warps' partial results meet in shared memory.
#include <cmath>

#include "tq_q8.cuh"

namespace tq {
namespace {

constexpr int kAttThreads = 256;

template <typename T, int FMT, int D>
__global__ void __launch_bounds__(kAttThreads) q8_attend_simple(const Q8AttendArgs a) {
  constexpr int E = D / 32, W = kAttThreads / 32;
  __shared__ float so[W][D], sm[W], sl[W];
  const int h = blockIdx.x % a.Hq, i = blockIdx.x / a.Hq, b = blockIdx.y;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int len = a.lens[b], nr = a.n_rows ? a.n_rows[b] : a.n;
  T* out = static_cast<T*>(a.out) + (((size_t)b * a.n + i) * a.Hq + h) * D;
  if (len < 0 || len > a.c.capacity || nr < 0 || nr > a.n) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.c.status, kQ8StatusInvalid);
    for (int e = threadIdx.x; e < D / 2; e += kAttThreads) reinterpret_cast<uint32_t*>(out)[e] = 0x7fff7fffu;
    return;
  }
  if (i >= nr) return;
  const int end = len - nr + 1 + i, whole = len / kQ8Block * kQ8Block;
  const int unit = b * a.c.num_kv_heads + h / a.G;
  const T* q = static_cast<const T*>(a.q) + b * a.row_stride + i * a.token_stride + h * a.head_stride;
  float qv[E], o[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) qv[e] = (float)q[e * 32 + lane], o[e] = 0.f;
  auto value = [&](bool v, int p, int e) {
    const int x = e * 32 + lane;
    if (p >= whole) return (float)static_cast<const T*>(v ? a.c.v_recent : a.c.k_recent)[((size_t)unit * kQ8Ring + p % kQ8Ring) * D + x];
    const uint32_t w = static_cast<const uint8_t*>(v ? a.c.v_codes : a.c.k_codes)[((size_t)unit * a.c.capacity + p) * D + x];
    return unpack16<__half>(codes_to_half2<FMT>(w)).x *
           (v ? a.c.v_scales : a.c.k_scales)[(size_t)unit * (a.c.capacity / kQ8Block) + p / kQ8Block];
  };
  for (int p = warp; p < end; p += W) {
    float s = 0.f, kv[E], vv[E];
    bool bad = false;
    for (int e = 0; e < E; ++e) {
      kv[e] = value(false, p, e), vv[e] = value(true, p, e);
      bad |= !isfinite(kv[e]) || !isfinite(vv[e]);
      s = fmaf(qv[e], kv[e], s);
    }
    for (int x = 16; x; x /= 2) s += __shfl_xor_sync(~0u, s, x);
    s = __any_sync(~0u, bad) ? NAN : s * a.scale_log2;
    const float mn = s > m || isnan(s) ? s : m, c = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * c + w;
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + w * vv[e];
  }
  for (int e = 0; e < E; ++e) so[warp][e * 32 + lane] = o[e];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  __syncthreads();
  float mx = -INFINITY, tot = 0.f;
  for (int w = 0; w < W; ++w) mx = sm[w] > mx || isnan(sm[w]) ? sm[w] : mx;
  for (int w = 0; w < W; ++w) tot += mx == -INFINITY ? 0.f : exp2f(sm[w] - mx) * sl[w];
  for (int x = threadIdx.x; x < D; x += kAttThreads) {
    float r = 0.f;
    for (int w = 0; w < W; ++w) r += mx == -INFINITY ? 0.f : exp2f(sm[w] - mx) * so[w][x];
    out[x] = (T)(end <= 0 ? 0.f : r / tot);
  }
}

}  // namespace

size_t q8_attend_scratch(const tq_q8_cache&, int, int, int) { return 256; }

cudaError_t launch_q8_attend(const Q8AttendArgs& a, int, cudaStream_t s) {
  const dim3 grid((unsigned)(a.Hq * a.n), (unsigned)a.c.batch);
  auto go = [&](auto fn) { fn<<<grid, kAttThreads, 0, s>>>(a); };
  const bool h = a.c.dtype == TQ_DTYPE_FP16, i8 = a.c.format == TQ_Q8_INT8;
#define TQ_ATT(D)                                                                               \
  h ? (i8 ? go(q8_attend_simple<__half, TQ_Q8_INT8, D>) : go(q8_attend_simple<__half, TQ_Q8_E4M3, D>)) \
    : (i8 ? go(q8_attend_simple<__nv_bfloat16, TQ_Q8_INT8, D>) : go(q8_attend_simple<__nv_bfloat16, TQ_Q8_E4M3, D>))
  if (a.c.head_dim == 64) TQ_ATT(64);
  else TQ_ATT(128);
#undef TQ_ATT
  return cudaGetLastError();
}

}  // namespace tq
