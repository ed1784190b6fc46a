// The 8-bit cache: writing tokens, reading them back, and the norm and
// rotation before a cache (include/tq.h has the contracts).
//
// All three move data: each is bound by HBM for long inputs and by launch
// latency for a decode step's.
#include "tq_q8.cuh"

namespace tq {
namespace {

constexpr float kQ8Tiny = 7.888609052210118e-31f;   // 2^-100

template <int FMT>
__device__ __forceinline__ float q8_top() {
  return FMT == TQ_Q8_INT8 ? 127.f : 448.f;
}

// ---- append ---------------------------------------------------------------
// One CTA per (touched block, row x kv head, K or V).  A block that the call
// completes is gathered (its old tokens from the ring, the others from the
// input), reduced to its largest magnitude, and coded; a thread keeps its
// share of the 64 x D values in registers, so each is read once.
//
// The 16-bit ring takes the new tokens of the newest two blocks.  A block
// writes its own, with one exception: the first touched block reads its old
// tokens from the ring half of its parity, so a later block of that parity
// leaves its ring tokens to the first CTA, which writes them after its
// reads.  So no CTA writes what another one reads.
//
// Bound by HBM: 4096 tokens in 8 rows (8 kv heads of 128, fp16 to int8) take
// 32.9 us, 6.2 TB/s.  A thread has four chunks of 8 values for either head
// dim: with the 256 threads of d = 128 for d = 64 too, 13 padded prompts of
// up to 1777 tokens took 7.3 us instead of 5.8.
__host__ __device__ constexpr int append_threads(int d) { return 2 * d; }

template <typename T, int FMT, int D>
__global__ void __launch_bounds__(append_threads(D)) q8_append_kernel(const Q8AppendArgs a) {
  constexpr int kAppendThreads = append_threads(D);
  constexpr int CH = D / 8;                              // 16-byte chunks per token
  constexpr int ITEMS = kQ8Block * CH / kAppendThreads;  // chunks per thread
  __shared__ unsigned red[kAppendThreads / 32];
  const int unit = blockIdx.y, kv = blockIdx.z, tid = threadIdx.x;
  wait_for_stream();
  const int b = unit / a.c.num_kv_heads, h = unit % a.c.num_kv_heads;
  const int len = a.lens[b], fresh = a.n_rows ? a.n_rows[b] : a.n;
  const bool invalid = len < 0 || fresh < 0 || fresh > a.n;
  if (invalid || (int64_t)len + fresh > a.c.capacity) {
    if (blockIdx.x == 0 && tid == 0) atomicOr(a.c.status, invalid ? kQ8StatusInvalid : kQ8StatusCapacity);
    return;
  }
  if (fresh == 0) return;
  const int end = len + fresh, first = len / kQ8Block, last = (end - 1) / kQ8Block;
  const int blk = first + (int)blockIdx.x;
  if (blk > last) return;
  const uint4* in = reinterpret_cast<const uint4*>(
      static_cast<const T*>(a.in[kv]) + b * a.row_stride[kv] + h * a.head_stride[kv]);
  const int64_t tstride = a.token_stride[kv] / 8;
  uint4* ring = reinterpret_cast<uint4*>(kv ? a.c.v_recent : a.c.k_recent) + (size_t)unit * kQ8Ring * CH;

  if ((blk + 1) * kQ8Block <= end) {
    uint4 x[ITEMS];
    unsigned mx = 0;                                     // magnitudes' bits, two 16-bit lanes
    constexpr int TOKS = kAppendThreads / CH;            // tokens at a time
    const int p0 = blk * kQ8Block + tid / CH, c = tid % CH;
    const uint4* src = in + (int64_t)(p0 - len) * tstride + c;
    if (blk * kQ8Block >= len) {
#pragma unroll
      for (int j = 0; j < ITEMS; ++j) x[j] = src[j * TOKS * tstride];
    } else {
#pragma unroll
      for (int j = 0; j < ITEMS; ++j) {
        const int p = p0 + j * TOKS;
        x[j] = p < len ? ring[(p % kQ8Ring) * CH + c] : src[j * TOKS * tstride];
      }
    }
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const unsigned w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = __vmaxu2(mx, w[e] & 0x7fff7fffu);
    }
    mx = max(mx & 0xffffu, mx >> 16);                    // bits of a magnitude order as magnitudes do,
    mx = __reduce_max_sync(~0u, mx);                     // infinities and NaN above all numbers
    if (tid % 32 == 0) red[tid / 32] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) mx = max(mx, red[w]);
    const float amax = unpack16<T>(mx).x;
    const bool bad = mx >= (Pair16<T>::kInf & 0xffffu), live = amax >= kQ8Tiny && !bad;
    const float inv = live ? __fdiv_rn(q8_top<FMT>(), amax) : 0.f;
    uint2* codes = reinterpret_cast<uint2*>(kv ? a.c.v_codes : a.c.k_codes) +
                   ((size_t)unit * a.c.capacity + (size_t)blk * kQ8Block) * CH;
    if (bad) {                                           // 0 * NaN would leave a NaN code
#pragma unroll
      for (int j = 0; j < ITEMS; ++j) x[j] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const unsigned w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      unsigned o[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float2 lo = unpack16<T>(w[2 * e]), hi = unpack16<T>(w[2 * e + 1]);
        lo.x = __fmul_rn(lo.x, inv), lo.y = __fmul_rn(lo.y, inv);
        hi.x = __fmul_rn(hi.x, inv), hi.y = __fmul_rn(hi.y, inv);
        if (FMT == TQ_Q8_E4M3) {
          o[e] = __nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3) |
                 (unsigned)__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3) << 16;
        } else {
          // |y| <= 127 (1 + 2^-23): the low byte of y + 1.5 2^23, which the sum rounds to nearest even
          const float m = 12582912.f;
          const unsigned p0 = __byte_perm(__float_as_uint(lo.x + m), __float_as_uint(lo.y + m), 0x0040);
          const unsigned p1 = __byte_perm(__float_as_uint(hi.x + m), __float_as_uint(hi.y + m), 0x0040);
          o[e] = __byte_perm(p0, p1, 0x5410);
        }
      }
      codes[tid + j * kAppendThreads] = make_uint2(o[0], o[1]);
    }
    if (tid == 0)
      (kv ? a.c.v_scales : a.c.k_scales)[(size_t)unit * (a.c.capacity / kQ8Block) + blk] =
          bad ? __uint_as_float(0x7fffffffu) : live ? __fdiv_rn(amax, q8_top<FMT>()) : 1.f;
  }

  auto to_ring = [&](int r) {
    const int lo = max(r * kQ8Block, len), hi = min((r + 1) * kQ8Block, end);
    for (int i = tid; i < (hi - lo) * CH; i += kAppendThreads) {
      const int p = lo + i / CH;
      ring[(p % kQ8Ring) * CH + i % CH] = in[(int64_t)(p - len) * tstride + i % CH];
    }
  };
  if (blk >= last - 1 && (blk == first || ((blk - first) & 1))) to_ring(blk);
  if (blk == first && last >= first + 2) {
    __syncthreads();                                     // after this CTA's reads of the ring
    to_ring(((last - first) & 1) ? last - 1 : last);
  }
}

// ---- read -----------------------------------------------------------------
// A thread takes kReadItems chunks of 8 values, the loads of all of them
// before any conversion: 4096 tokens of 8 rows (8 kv heads of 128, int8) take
// 32.8 us, 6.1 TB/s; with one chunk a thread they took 139.
constexpr int kReadThreads = 256, kReadItems = 4;

template <typename T, int FMT, int D>
__global__ void __launch_bounds__(kReadThreads) q8_read_kernel(const Q8ReadArgs a) {
  constexpr int CH = D / 8;
  const int unit = blockIdx.y, kv = blockIdx.z, b = unit / a.c.num_kv_heads;
  wait_for_stream();
  const int len = a.lens[b];
  if (len < 0 || len > a.c.capacity) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.c.status, kQ8StatusInvalid);
    return;
  }
  const int whole = len / kQ8Block * kQ8Block;
  const uint2* codes = reinterpret_cast<const uint2*>(kv ? a.c.v_codes : a.c.k_codes) + (size_t)unit * a.c.capacity * CH;
  const uint4* ring = reinterpret_cast<const uint4*>(kv ? a.c.v_recent : a.c.k_recent) + (size_t)unit * kQ8Ring * CH;
  const float* scales = (kv ? a.c.v_scales : a.c.k_scales) + (size_t)unit * (a.c.capacity / kQ8Block);
  uint4* out = reinterpret_cast<uint4*>(kv ? a.out[1] : a.out[0]) + (size_t)unit * a.n * CH;
  const int64_t i0 = (int64_t)blockIdx.x * kReadThreads * kReadItems + threadIdx.x;
  uint4 x[kReadItems];                                     // codes in x, y and their scale in z, or 16-bit values
#pragma unroll
  for (int j = 0; j < kReadItems; ++j) {
    const int64_t i = i0 + j * kReadThreads, t = i / CH, p = a.start + t;
    x[j] = make_uint4(0u, 0u, 0u, 0u);
    if (t < a.n && p < whole) {
      const uint2 w = codes[p * CH + i % CH];
      x[j].x = w.x, x[j].y = w.y, x[j].z = __float_as_uint(scales[p / kQ8Block]);
    } else if (t < a.n && p < len) {
      x[j] = ring[p % kQ8Ring * CH + i % CH];
    }
  }
#pragma unroll
  for (int j = 0; j < kReadItems; ++j) {
    const int64_t i = i0 + j * kReadThreads, t = i / CH, p = a.start + t;
    if (p < whole) {
      const float s = __uint_as_float(x[j].z);
      unsigned f[4], o[4];
      codes_to_half4<FMT>(x[j].x, f[0], f[1]);
      codes_to_half4<FMT>(x[j].y, f[2], f[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = unpack16<__half>(f[e]);
        o[e] = pack16<T>(__fmul_rn(v.x, s), __fmul_rn(v.y, s));
      }
      x[j] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (t < a.n && p < len) out[i] = x[j];
  }
}

// ---- norm and rotation ------------------------------------------------------
// A warp takes a token, or a part of its heads: the angles' cosines and sines
// once (position x frequency reduced to half turns in float64, then a float32
// sine and cosine), then D / 16 lanes per head, each with one 16-byte chunk of
// either half of the head, so that both elements of every pair are in one lane
// in either layout of the pairs.  A lane keeps its pairs' turns and its weights
// for all of its heads; its next heads, kRopeAhead of them, are on their way
// to shared memory meanwhile, the first before the angles.  Bound by HBM for
// prompts: 12297 tokens of 40 heads of 128 (bf16) take 45 us, 5.6 TB/s; the
// same with a head's halves loaded one head ahead into registers took 55.
constexpr int kRopeThreads = 128, kRopeWarps = kRopeThreads / 32, kRopeAhead = 2;
constexpr int kRopeCtas = 5;                               // per SM: 86 to 96 registers a thread

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) norm_rope_kernel(const NormRopeArgs a, int parts) {
  constexpr int L = D / 16, HW = 32 / L;                   // lanes per head, heads per warp
  __shared__ float2 cs[kRopeWarps][D / 2];                 // a lane's i-th turn at [i L + lane]
  __shared__ uint4 buf[kRopeAhead * kRopeThreads * 2];     // [stage][warp][half][lane]
  const int tid = threadIdx.x, lane = tid % L, warp = tid / 32;
  const int64_t part = (int64_t)blockIdx.x * kRopeWarps + warp;
  const int tok = (int)(part / parts);
  if (tok >= a.batch * a.n) return;                        // whole warps; they share nothing
  const int step = HW * parts;
  wait_for_stream();
  const int b = tok / a.n, t = tok % a.n;
  // A lane's heads: of the queries first, then of the keys.
  struct Head {
    int h, heads;
    bool keys;
    __device__ void settle(const NormRopeArgs& a) {        // from behind the queries to the keys
      if (!keys && h >= a.Hq) keys = true, h -= a.Hq, heads = a.Hkv;
    }
  };
  Head use{(int)(part % parts) * HW + tid % 32 / L, a.Hq, false};
  use.settle(a);
  Head get = use;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(buf) + (warp * 64 + tid % 32) * 16;
  auto fetch = [&](int stage) {
    if (get.h < get.heads) {
      const T* src = (get.keys ? static_cast<const T*>(a.k) + b * a.k_row + t * a.k_token + get.h * a.k_head
                               : static_cast<const T*>(a.q) + b * a.q_row + t * a.q_token + get.h * a.q_head) + 8 * lane;
      const uint32_t dst = mine + stage * (kRopeThreads * 32);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512), "l"(src + 8 * L) : "memory");
      get.h += step;
      get.settle(a);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kRopeAhead; ++i) fetch(i);
  uint4 wt[2];
  const T* weight = nullptr;                               // whose values wt holds
  auto weigh = [&](bool keys) {
    const T* own = static_cast<const T*>(keys ? a.k_weight : a.q_weight);
    if (own != weight && own) wt[0] = reinterpret_cast<const uint4*>(own)[lane], wt[1] = reinterpret_cast<const uint4*>(own)[lane + L];
    weight = own;
  };
  if (use.h < use.heads) weigh(use.keys);                  // a lane may have no head at all
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const int p = tid % 32 + 32 * i;
    const double inv_pi = 0.31830988618379067154;
    const double ang = (double)a.positions[tok] * (double)a.inv_freq[p];
    const float r = (float)fma(ang, inv_pi, -2.0 * rint(ang * inv_pi * 0.5));   // half turns, in [-1, 1]
    float s, c;
    sincospif(r, &s, &c);
    cs[warp][INTER ? (p % 4 + p / (D / 4) * 4) * L + p % (D / 4) / 4 : p % 8 * L + p / 8] = make_float2(c, s);
  }
  __syncwarp();
  float2 turn[8];                                          // of the lane's pairs: elements i, i + 8, or 2 i, 2 i + 1
#pragma unroll
  for (int i = 0; i < 8; ++i) turn[i] = cs[warp][i * L + lane];
  int stage = 0;
  while (use.h < use.heads) {                              // whole groups of L lanes leave together
    asm volatile("cp.async.wait_group %0;" ::"n"(kRopeAhead - 1) : "memory");
    const uint4* own_buf = buf + stage * (kRopeThreads * 2) + warp * 64 + tid % 32;   // a lane reads what it copied
    const uint4 cur[2] = {own_buf[0], own_buf[32]};
    uint4* dst = reinterpret_cast<uint4*>(use.keys ? static_cast<T*>(a.k_out) + (((size_t)b * a.Hkv + use.h) * a.n + t) * D
                                                   : static_cast<T*>(a.q_out) + ((size_t)tok * a.Hq + use.h) * D) + lane;
    weigh(use.keys);
    fetch(stage);
    stage = stage + 1 == kRopeAhead ? 0 : stage + 1;
    use.h += step;
    use.settle(a);
    float x[16];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const unsigned w[4] = {cur[e].x, cur[e].y, cur[e].z, cur[e].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16<T>(w[i]);
        x[8 * e + 2 * i] = f.x, x[8 * e + 2 * i + 1] = f.y;
      }
    }
    if (weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
      const unsigned mask = ((1u << L) - 1u) << (tid % 32 / L * L);
#pragma unroll
      for (int o = L / 2; o; o /= 2) ss += __shfl_xor_sync(mask, ss, o);
      if (Pair16<T>::kWide && !(ss > 1e-30f && ss < 1e38f)) {
        // bf16 squares can leave float32 at either end: such heads take float64
        double sd = 0.0;
#pragma unroll
        for (int i = 0; i < 16; ++i) sd += (double)x[i] * x[i];
#pragma unroll
        for (int o = L / 2; o; o /= 2) sd += __shfl_xor_sync(mask, sd, o);
        // in two factors, since the whole one may be no float32
        const double rd = 1.0 / sqrt(sd / D + a.eps), half = rd > 1.0 ? 1.8446744073709552e19 : 5.421010862427522e-20;
        const float r0 = (float)half, r1 = (float)(rd / half);   // 2^64 or 2^-64, and the rest
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * r0 * r1;
      } else {
        const float r = rsqrtf(fmaf(ss, 1.0f / D, a.eps));
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= r;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const unsigned w[4] = {wt[e].x, wt[e].y, wt[e].z, wt[e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack16<T>(w[i]);
          x[8 * e + 2 * i] *= f.x, x[8 * e + 2 * i + 1] *= f.y;
        }
      }
    }
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      constexpr int S = INTER ? 2 : 1, O = INTER ? 1 : 8;
      y[S * i] = x[S * i] * turn[i].x - x[S * i + O] * turn[i].y;
      y[S * i + O] = x[S * i + O] * turn[i].x + x[S * i] * turn[i].y;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      dst[e * L] = make_uint4(pack16<T>(y[8 * e], y[8 * e + 1]), pack16<T>(y[8 * e + 2], y[8 * e + 3]),
                                     pack16<T>(y[8 * e + 4], y[8 * e + 5]), pack16<T>(y[8 * e + 6], y[8 * e + 7]));
  }
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendArgs& a, cudaStream_t s) {
  // blocks that n tokens can touch, wherever they begin
  const int64_t most = ((int64_t)a.n + kQ8Block - 2) / kQ8Block + 1, blocks = a.c.capacity / kQ8Block;
  const dim3 grid((unsigned)(most < blocks ? most : blocks), (unsigned)(a.c.batch * a.c.num_kv_heads), 2);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto fn) { e = launch_dependent(fn, grid, append_threads(a.c.head_dim), 0, s, a); };
  const bool h = a.c.dtype == TQ_DTYPE_FP16, i8 = a.c.format == TQ_Q8_INT8;
#define TQ_APPEND(D)                                                                            \
  h ? (i8 ? go(q8_append_kernel<__half, TQ_Q8_INT8, D>) : go(q8_append_kernel<__half, TQ_Q8_E4M3, D>)) \
    : (i8 ? go(q8_append_kernel<__nv_bfloat16, TQ_Q8_INT8, D>) : go(q8_append_kernel<__nv_bfloat16, TQ_Q8_E4M3, D>))
  if (a.c.head_dim == 64) TQ_APPEND(64);
  else TQ_APPEND(128);
#undef TQ_APPEND
  return e;
}

cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t s) {
  const int64_t held = a.c.capacity - a.start;               // no row holds more
  const int64_t chunks = (a.n < held ? a.n : held) * (a.c.head_dim / 8);
  const int per = kReadThreads * kReadItems;
  const dim3 grid((unsigned)((chunks + per - 1) / per), (unsigned)(a.c.batch * a.c.num_kv_heads), 2);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto fn) { e = launch_dependent(fn, grid, kReadThreads, 0, s, a); };
  const bool h = a.c.dtype == TQ_DTYPE_FP16, i8 = a.c.format == TQ_Q8_INT8;
#define TQ_READ(D)                                                                              \
  h ? (i8 ? go(q8_read_kernel<__half, TQ_Q8_INT8, D>) : go(q8_read_kernel<__half, TQ_Q8_E4M3, D>)) \
    : (i8 ? go(q8_read_kernel<__nv_bfloat16, TQ_Q8_INT8, D>) : go(q8_read_kernel<__nv_bfloat16, TQ_Q8_E4M3, D>))
  if (a.c.head_dim == 64) TQ_READ(64);
  else TQ_READ(128);
#undef TQ_READ
  return e;
}

template <typename T, int D>
static cudaError_t launch_rope(const NormRopeArgs& a, int num_sms, cudaStream_t s) {
  const int64_t tokens = (int64_t)a.batch * a.n;
  const int passes = (a.Hq + a.Hkv + 32 / (D / 16) - 1) / (32 / (D / 16));
  const int parts = norm_rope_parts(tokens, passes, num_sms * kRopeCtas * kRopeWarps);
  const unsigned grid = (unsigned)((tokens * parts + kRopeWarps - 1) / kRopeWarps);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto fn) { e = launch_dependent(fn, dim3(grid), kRopeThreads, 0, s, a, parts); };
  if (a.interleaved) go(norm_rope_kernel<T, D, true>);
  else go(norm_rope_kernel<T, D, false>);
  return e;
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, int num_sms, cudaStream_t s) {
  if (a.dtype == TQ_DTYPE_FP16)
    return a.d == 64 ? launch_rope<__half, 64>(a, num_sms, s) : launch_rope<__half, 128>(a, num_sms, s);
  return a.d == 64 ? launch_rope<__nv_bfloat16, 64>(a, num_sms, s) : launch_rope<__nv_bfloat16, 128>(a, num_sms, s);
}

}  // namespace tq
