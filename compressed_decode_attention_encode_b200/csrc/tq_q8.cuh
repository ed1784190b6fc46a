// Internal declarations of the 8-bit cache (tq_q8_*) and of the norm and
// rotation before a cache: argument blocks and launchers.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/tq.h"

namespace tq {

constexpr int kQ8Block = 64;        // tokens that share a scale
constexpr int kQ8Ring = 128;        // slots of the 16-bit ring: two blocks
constexpr int kQ8MaxRows = 1024;
constexpr int kQ8MaxQueries = 64;
constexpr int kQ8MaxGroup = 16;

// Status word bits of a tq_q8_cache.
constexpr int kQ8StatusInvalid = 1;
constexpr int kQ8StatusCapacity = 2;

struct Q8AppendArgs {
  tq_q8_cache c;
  const void* in[2];                 // K, V
  int64_t row_stride[2], head_stride[2], token_stride[2];
  int n;
  const int32_t* lens;
  const int32_t* n_rows;
};

struct Q8ReadArgs {
  tq_q8_cache c;
  const int32_t* lens;
  int64_t start;
  int n;
  void* out[2];
};

struct Q8AttendArgs {
  tq_q8_cache c;
  const void* q;
  int64_t row_stride, token_stride, head_stride;
  int Hq, G, n;
  const int32_t* lens;
  const int32_t* n_rows;
  float scale_log2;                  // sigma * log2(e)
  void* out;
  uint8_t* scratch;
};

struct NormRopeArgs {
  int batch, n, Hq, Hkv, d, dtype;
  const void* q;
  const void* k;
  int64_t q_row, q_token, q_head, k_row, k_token, k_head;
  const int32_t* positions;
  const float* inv_freq;
  const void* q_weight;
  const void* k_weight;
  float eps;
  int interleaved;
  void* q_out;
  void* k_out;
};

// Parts that a token's heads (of so many passes) are split into, each a warp's:
// while all of them fit on the card at once.  A step's 8 tokens of 40 heads of
// 128 take 2.0 to 2.2 us so, 700 tokens 4.2 us in four parts (whole tokens to a
// warp 6.0), 1184 tokens 5.1 in two (6.0); one part too many, which makes a
// second, mostly empty wave, takes 1000 tokens from 5.1 to 6.6 us and 1776 from
// 7.0 to 8.2.
inline int norm_rope_parts(int64_t tokens, int passes, int warps) {
  const int64_t fit = warps / tokens;
  return (int)(fit < 1 ? 1 : fit < passes ? fit : passes);
}

// The kernel's arguments: what belongs to a side without heads is not used, so
// nothing of it goes on.
inline NormRopeArgs norm_rope_args(const tq_qk_norm_rope_args& x) {
  NormRopeArgs a{x.batch, x.n, x.num_q_heads, x.num_kv_heads, x.head_dim, x.dtype, x.q, x.k,
                 x.q_row_stride, x.q_token_stride, x.q_head_stride, x.k_row_stride, x.k_token_stride,
                 x.k_head_stride, x.positions, x.inv_freq, x.q_weight, x.k_weight, x.eps, x.interleaved,
                 x.q_out, x.k_out};
  if (x.num_q_heads == 0) a.q = a.q_weight = a.q_out = nullptr, a.q_row = a.q_token = a.q_head = 0;
  if (x.num_kv_heads == 0) a.k = a.k_weight = a.k_out = nullptr, a.k_row = a.k_token = a.k_head = 0;
  return a;
}

cudaError_t launch_q8_append(const Q8AppendArgs& a, cudaStream_t s);
cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t s);
size_t q8_attend_scratch(const tq_q8_cache& c, int Hq, int n, int num_sms);
cudaError_t launch_q8_attend(const Q8AttendArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_norm_rope(const NormRopeArgs& a, int num_sms, cudaStream_t s);

#ifdef __CUDACC__
// Launches a kernel as a programmatic dependent of the stream's last one: its
// blocks are placed while that one ends.  The kernel begins with
// wait_for_stream(), before it reads anything.
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- 16-bit values and codes in registers --------------------------------
template <typename T>
struct Pair16;                           // of a 16-bit type: two infinities, ...
template <>
struct Pair16<__half> {
  static constexpr uint32_t kInf = 0x7c007c00u;
  static constexpr bool kWide = false;   // whether squares of values can leave float32
};
template <>
struct Pair16<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7f807f80u;
  static constexpr bool kWide = true;
};

template <typename T>
__device__ __forceinline__ float2 unpack16(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack16<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack16<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four codes as fp16, which holds every code exactly: the low two, the high two.
template <int FMT>
__device__ __forceinline__ void codes_to_half4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == TQ_Q8_E4M3) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(lo), "=r"(hi) : "r"(w));
  } else {
    // 0x6400 | u is 1024 + u for a byte u; u = code + 128
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));
    w ^= 0x80808080u;
    const uint32_t l = __byte_perm(w, 0x64646464u, 0x4140), h = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&l), bias);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&h), bias);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// Whether a 16-bit pair holds a NaN or an infinity.
template <typename T>
__device__ __forceinline__ bool pair_bad(uint32_t w) {
  constexpr uint32_t inf = Pair16<T>::kInf;
  return (w & inf & 0xffffu) == (inf & 0xffffu) || (w & inf & 0xffff0000u) == (inf & 0xffff0000u);
}
#endif

}  // namespace tq
