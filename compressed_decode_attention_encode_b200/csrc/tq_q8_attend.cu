// Attention over the 8-bit cache (include/tq.h has the contract).
//
// For a query q of a row's (row, kv head) unit, with a block's scales s_k, s_v
// and codes c:
//   x_p = sigma log2(e) s_k <q, c_k>,   o = sum_p 2^x_p s_v c_v / sum_p 2^x_p
// in one pass, with two running references: ml of x for the denominator, and
// mv of x + log2 s_v for the numerator, whose weights 2^(x + log2 s_v - mv)
// take the place of an fp16 operand without a multiplication by s_v.
//
// The work is the batch's tiles (a unit's whole blocks of 64 tokens, then its
// open block), flattened and cut into equal runs, one per CTA, so that rows of
// any length share the card; every CTA finds its run from the lengths alone
// (they are device memory).  Each unit has kUnitCost places before its first
// tile, which stand for what a pass costs besides its tiles (its queries'
// latency, the open block's, the join of the warps).  A unit inside one CTA's
// run is finished there; the others leave partial results that a second
// kernel joins in a fixed order.
#include <cmath>

#include "tq_q8.cuh"

namespace tq {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kUnitCost = 3;                 // of a unit besides its tiles, in tiles
constexpr int kMinTiles = 4;                 // places that a CTA takes at least
constexpr float kLowest = -3.0e38f;          // of a reference before its first token
constexpr float kShift = 7.f;                // numerator weights are 2^7 at their reference (mv holds it less 7),
constexpr float kLazy = 8.f;                 // and a reference moves when one exceeds it by 2^8: below fp16's 2^16

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds32f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

// ---- the plan: which tiles a CTA takes -------------------------------------
__device__ __forceinline__ bool row_valid(const Q8AttendArgs& a, int len, int nr) {
  return len >= 0 && len <= a.c.capacity && nr >= 0 && nr <= a.n;
}
// Places of a unit of row b.
__device__ __forceinline__ int row_places(const Q8AttendArgs& a, int b) {
  const int len = a.lens[b], nr = a.n_rows ? a.n_rows[b] : a.n;
  return row_valid(a, len, nr) && nr > 0 && len > 0 ? kUnitCost + len / kQ8Block + (len % kQ8Block != 0) : 0;
}
// Places before each row into pre[0 .. batch] (a unit's places x units of a row).
__device__ __forceinline__ void plan_rows(const Q8AttendArgs& a, int subs, uint32_t* pre, uint32_t* warp_sums) {
  uint32_t total = 0;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int b0 = 0; b0 < a.c.batch; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const uint32_t v = b < a.c.batch ? (uint32_t)row_places(a, b) * subs : 0;
    uint32_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t y = __shfl_up_sync(~0u, s, o);
      if (lane >= o) s += y;
    }
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    uint32_t before = total;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_sums[w];
      total += warp_sums[w];
    }
    if (b < a.c.batch) pre[b] = before + s - v;
    __syncthreads();
  }
  if (threadIdx.x == 0) pre[a.c.batch] = total;
  __syncthreads();
}
__device__ __forceinline__ uint32_t plan_ctas(uint32_t tiles, uint32_t grid) {
  const uint32_t most = (tiles + kMinTiles - 1) / kMinTiles;
  return most < grid ? most : grid;
}
__device__ __forceinline__ uint32_t cta_start(uint32_t c, uint32_t tiles, uint32_t ctas) {
  return (uint32_t)((uint64_t)c * tiles / ctas);
}
// The CTA whose run holds place t.
__device__ __forceinline__ uint32_t cta_of(uint32_t t, uint32_t tiles, uint32_t ctas) {
  return (uint32_t)((((uint64_t)t + 1) * ctas + tiles - 1) / tiles) - 1;
}

// A CTA's run, segment by segment: a segment is the run's tiles [begin, end) of one unit (kv head x query
// group of a row), never empty.
struct Walk {
  int row, sub;
  uint32_t left;                           // places of the run behind this segment
  int whole, tiles, begin, end;            // of the unit: whole blocks, tiles; of the segment: tiles
  __device__ void enter(const Q8AttendArgs& a, uint32_t pos) {
    const int len = a.lens[row];
    whole = len / kQ8Block;
    tiles = whole + (len % kQ8Block != 0);
    const uint32_t take = min(left, (uint32_t)(kUnitCost + tiles) - pos);
    begin = max((int)pos - kUnitCost, 0);
    end = (int)(pos + take) - kUnitCost;
    left -= take;
  }
  // To the next segment; false at the end of the run.
  __device__ bool next(const Q8AttendArgs& a, const uint32_t* pre, int subs) {
    do {
      if (left == 0) return false;
      if (++sub == subs) {
        sub = 0;
        do ++row;
        while (pre[row + 1] == pre[row]);
      }
      enter(a, 0);
    } while (end <= begin);
    return true;
  }
  __device__ bool first(const Q8AttendArgs& a, const uint32_t* pre, int subs, uint32_t t0, uint32_t t1) {
    int lo = 0, hi = a.c.batch;            // pre[lo] <= t0 < pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      (pre[mid] <= t0 ? lo : hi) = mid;
    }
    row = lo;
    const uint32_t off = t0 - pre[row], places = (pre[row + 1] - pre[row]) / subs;
    sub = off / places;
    left = t1 - t0;
    enter(a, off % places);
    return end > begin || next(a, pre, subs);
  }
};

template <int D, int NT>
struct Shape {
  static constexpr int ROWS = 8 * NT;                      // query rows of a unit's pass
  static constexpr int SLAB = 16 * D;                      // bytes of 16 tokens' codes
  static constexpr int STAGE = 2 * SLAB + 16;              // K, V, scales
  static constexpr int RING = kWarps * kStages * STAGE;
  static constexpr int OROW = D + 4;                       // a row of partial results: o, ml, mv, l
  static constexpr int JOIN = 2 * ROWS * OROW * 4;
  static constexpr int STATS = kWarps * ROWS * 4 * 4;
};
// CTAs per SM: what registers and shared memory allow.
constexpr int ctas_per_sm(int d, int nt) { return nt > 1 ? 2 : d == 128 ? 3 : 4; }
template <int D, int NT>
int smem_bytes(int batch) {
  return Shape<D, NT>::RING + Shape<D, NT>::JOIN + Shape<D, NT>::STATS + 16 + 4 * (batch + 1);
}

// Byte of 16-byte chunk c of token r in a slab: the chunks are permuted inside
// each 128-byte line so that the eight lanes of a phase meet eight banks
// groups, both where lanes take a token's four chunks (K) and where they take
// one chunk of every other token (V).
template <int D>
__device__ __forceinline__ int slab_at(int r, int c) {
  if (D == 128) return r * 128 + ((c ^ (((r >> 1) & 3) << 1) ^ ((r & 1) << 2)) << 4);
  const int line = r >> 1;
  return line * 128 + ((((r & 1) << 2 | c) ^ ((line & 3) << 1)) << 4);
}

// ---- one unit's pass ---------------------------------------------------------
// A warp takes 16 tokens of each tile.  Tokens are the rows of both products
// (S^T = K Q^T, O^T = V^T P^T), 8 queries their columns, so a kv head's group
// of queries fills one m16n8k16 column block, and a lane's 16 bytes of a K row
// or of a V row are its operand without any exchange: the products' inner
// index may be permuted as long as both operands are.
template <typename T, int FMT, int D, int NT>
struct Pass {
  static constexpr int KS = D / 16;          // k-steps of the first product, m-tiles of the second
  float o[KS][NT][4];                        // dims 2 mt, 2 mt + 1 of the lane's D / 8, queries 2 tig, 2 tig + 1
  float ml[NT][2], mv[NT][2], l[NT][2];
  float cq[NT][2];                           // sigma log2(e) of the query (and its power of two)
  int end[NT][2];                            // positions that it sees
  int min_end;
  uint32_t qf[NT][KS][2];
  int lane, gid, tig, warp;

  __device__ void start(const Q8AttendArgs& a, int row, int kvh, int r0) {
#pragma unroll
    for (int m = 0; m < KS; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][t][e] = 0.f;
    const int len = a.lens[row], nr = a.n_rows ? a.n_rows[row] : a.n;
    min_end = len - nr + 1 + r0 / a.G;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float up = a.scale_log2;
      load_q<true>(a, row, kvh, r0, t, qf[t], up);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        ml[t][j] = mv[t][j] = kLowest;
        l[t][j] = 0.f;
        cq[t][j] = __shfl_sync(~0u, up, 4 * (2 * tig + j));
        end[t][j] = len - nr + 1 + (r0 + 8 * t + 2 * tig + j) / a.G;
      }
    }
  }

  // The B operand of query 8 t + gid.  AS_HALF: fp16 whatever the type; a bf16
  // query is scaled by the power of two that brings its largest element into
  // [1, 2), and `up` takes that factor back.
  template <bool AS_HALF>
  __device__ void load_q(const Q8AttendArgs& a, int row, int kvh, int r0, int t, uint32_t (&f)[KS][2], float& up) {
    const int r = r0 + 8 * t + gid;
    const bool on = r < a.n * a.G;
    const int i = on ? r / a.G : 0, h = on ? r % a.G : 0;
    const T* q = static_cast<const T*>(a.q) + row * a.row_stride + i * a.token_stride +
                 (int64_t)(kvh * a.G + h) * a.head_stride;
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint4 v = on ? *reinterpret_cast<const uint4*>(q + 64 * j + 16 * tig + 8 * x) : make_uint4(0, 0, 0, 0);
        f[4 * j + 2 * x][0] = v.x, f[4 * j + 2 * x][1] = v.y;
        f[4 * j + 2 * x + 1][0] = v.z, f[4 * j + 2 * x + 1][1] = v.w;
      }
    if (AS_HALF && Pair16<T>::kWide) {
      uint32_t mx = 0;
#pragma unroll
      for (int s = 0; s < KS; ++s) mx = __vmaxu2(mx, __vmaxu2(f[s][0] & 0x7fff7fffu, f[s][1] & 0x7fff7fffu));
      mx = max(mx & 0xffffu, mx >> 16);
      mx = max(mx, __shfl_xor_sync(~0u, mx, 1));
      mx = max(mx, __shfl_xor_sync(~0u, mx, 2));
      int e = (int)(mx >> 7) - 127;                        // of the largest element
      e = mx >= 0x7f80u ? 0 : max(e, -126);                // NaN and infinities pass as they are
      const float down = __uint_as_float((uint32_t)(127 - min(e, 126)) << 23);
      up *= __uint_as_float((uint32_t)(127 + min(e, 126)) << 23);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 w = unpack16<T>(f[s][x]);
          f[s][x] = pack16<__half>(w.x * down, w.y * down);
        }
    }
  }

  // Weights of 16 tokens from their logits, c_p = x_p / f.  VIS: positions
  // first + gid (+ 8) may be behind a query's end, or bad (bits of `bad`).
  // Returns the numerator's weights in `w` (denominators are added here).
  template <bool VIS>
  __device__ __forceinline__ void weights(const float (&s)[NT][4], const float (&f)[NT][2], float lsv, int first,
                                          uint32_t bad, float (&w)[NT][4]) {
    float pl[NT][4];
    float top_l = kLowest, top_v = kLowest;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = e & 1;
        pl[t][e] = fmaf(s[t][e], f[t][j], -ml[t][j]);
        w[t][e] = fmaf(s[t][e], f[t][j], lsv - mv[t][j]);
        const bool vis = !VIS || first + gid + 8 * (e >> 1) < end[t][j];
        if (vis) top_l = fmaxf(top_l, pl[t][e]), top_v = fmaxf(top_v, w[t][e]);
      }
    if (__any_sync(~0u, top_l > kLazy || top_v > kLazy + kShift)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x0 = s[t][j] * f[t][j], x1 = s[t][j + 2] * f[t][j];
          if (VIS) {
            if (first + gid >= end[t][j]) x0 = kLowest;
            if (first + gid + 8 >= end[t][j]) x1 = kLowest;
          }
          float mx = fmaxf(x0, x1);
#pragma unroll
          for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
          const float nl = fmaxf(ml[t][j], mx), nv = mx > kLowest ? fmaxf(mv[t][j], mx + lsv - kShift) : mv[t][j];
          l[t][j] *= ex2(ml[t][j] - nl);
          const float c = ex2(mv[t][j] - nv);
          ml[t][j] = nl;
          mv[t][j] = nv;
#pragma unroll
          for (int m = 0; m < KS; ++m) o[m][t][j] *= c, o[m][t][j + 2] *= c;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pl[t][e] = fmaf(s[t][e], f[t][e & 1], -ml[t][e & 1]);
          w[t][e] = fmaf(s[t][e], f[t][e & 1], lsv - mv[t][e & 1]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float p = ex2(pl[t][e]);
        w[t][e] = ex2(w[t][e]);
        if (VIS) {
          const bool vis = first + gid + 8 * (e >> 1) < end[t][e & 1];
          const bool nan = bad >> (gid + 8 * (e >> 1)) & 1;
          p = !vis ? 0.f : nan ? NAN : p;
          w[t][e] = !vis ? 0.f : nan ? NAN : w[t][e];
        }
        l[t][e & 1] += p;
      }
  }

  // 16 tokens of a whole block from the ring stage at `st`, scales behind it.
  template <bool VIS>
  __device__ __forceinline__ void codes(uint32_t st, int first) {
    constexpr int SLAB = Shape<D, NT>::SLAB;
    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
    const float sk = lds32f(st + 2 * SLAB), sv = lds32f(st + 2 * SLAB + 4);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const uint4 ka = lds128(st + slab_at<D>(gid, tig + 4 * j)), kb = lds128(st + slab_at<D>(gid + 8, tig + 4 * j));
      const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t a0, a1, a2, a3;
        codes_to_half4<FMT>(wa[x], a0, a2);
        codes_to_half4<FMT>(wb[x], a1, a3);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(s[t], a0, a1, a2, a3, qf[t][4 * j + x][0], qf[t][4 * j + x][1], __half());
      }
    }
    float f[NT][2], w[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) f[t][0] = sk * cq[t][0], f[t][1] = sk * cq[t][1];
    weights<VIS>(s, f, lg2(sv), first, 0u, w);
    uint32_t b[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      b[t][0] = movmatrix(pack16<__half>(w[t][0], w[t][1]));
      b[t][1] = movmatrix(pack16<__half>(w[t][2], w[t][3]));
    }
    uint32_t v[4][D / 32];                                 // tokens 2 tig, 2 tig + 1, + 8, + 9
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 2 * tig + (i & 1) + 8 * (i >> 1);
      if (D == 128) {
        const uint4 x = lds128(st + SLAB + slab_at<D>(r, gid));
        v[i][0] = x.x, v[i][1] = x.y, v[i][D / 32 - 2] = x.z, v[i][D / 32 - 1] = x.w;
      } else {
        const uint2 x = lds64(st + SLAB + slab_at<D>(r, gid >> 1) + 8 * (gid & 1));
        v[i][0] = x.x, v[i][1] = x.y;
      }
    }
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t lo = __byte_perm(v[0][x], v[1][x], y ? 0x7362 : 0x5140);
        const uint32_t hi = __byte_perm(v[2][x], v[3][x], y ? 0x7362 : 0x5140);
        uint32_t a0, a1, a2, a3;
        codes_to_half4<FMT>(lo, a0, a1);
        codes_to_half4<FMT>(hi, a2, a3);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(o[2 * x + y][t], a0, a1, a2, a3, b[t][0], b[t][1], __half());
      }
  }

  // The warp's 16 tokens of the open block, from the 16-bit ring.  Its products
  // take the cache's own type, exactly; bf16 weights go in as two bf16 parts.
  __device__ void open(const Q8AttendArgs& a, int row, int kvh, int r0, int whole) {
    const int cnt = a.lens[row] - whole * kQ8Block - 16 * warp;  // tokens of this warp
    if (cnt <= 0) return;
    const size_t unit = (size_t)row * a.c.num_kv_heads + kvh;
    const size_t base = (unit * kQ8Ring + (whole & 1) * kQ8Block + 16 * warp) * D;
    const T *kr = static_cast<const T*>(a.c.k_recent) + base, *vr = static_cast<const T*>(a.c.v_recent) + base;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint32_t bad = 0;
    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
    uint32_t k[2][KS][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint4 w = gid + 8 * i < cnt ? *reinterpret_cast<const uint4*>(kr + (gid + 8 * i) * D + 64 * j + 16 * tig + 8 * x) : zero;
          k[i][4 * j + 2 * x][0] = w.x, k[i][4 * j + 2 * x][1] = w.y;
          k[i][4 * j + 2 * x + 1][0] = w.z, k[i][4 * j + 2 * x + 1][1] = w.w;
          if (pair_bad<T>(w.x) || pair_bad<T>(w.y) || pair_bad<T>(w.z) || pair_bad<T>(w.w)) bad |= 1u << (gid + 8 * i);
        }
    uint32_t v[4][KS];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 2 * tig + (i & 1) + 8 * (i >> 1);
#pragma unroll
      for (int x = 0; x < KS / 4; ++x) {
        const uint4 w = r < cnt ? *reinterpret_cast<const uint4*>(vr + r * D + D / 8 * gid + 8 * x) : zero;
        v[i][4 * x] = w.x, v[i][4 * x + 1] = w.y, v[i][4 * x + 2] = w.z, v[i][4 * x + 3] = w.w;
        if (pair_bad<T>(w.x) || pair_bad<T>(w.y) || pair_bad<T>(w.z) || pair_bad<T>(w.w)) bad |= 1u << r;
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t raw[KS][2];
      float unused = 0.f;
      if (Pair16<T>::kWide) load_q<false>(a, row, kvh, r0, t, raw, unused);
#pragma unroll
      for (int x = 0; x < KS; ++x)
        mma16816(s[t], k[0][x][0], k[1][x][0], k[0][x][1], k[1][x][1], Pair16<T>::kWide ? raw[x][0] : qf[t][x][0],
                 Pair16<T>::kWide ? raw[x][1] : qf[t][x][1], T());
    }
    bad = __reduce_or_sync(~0u, bad);
    if (bad) {                                             // 0 x NaN would reach queries that do not see the token
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (bad >> (2 * tig + (i & 1) + 8 * (i >> 1)) & 1)
#pragma unroll
          for (int x = 0; x < KS; ++x) v[i][x] = 0;
    }
    float f[NT][2], w[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) f[t][0] = f[t][1] = a.scale_log2;
    weights<true>(s, f, 0.f, whole * kQ8Block + 16 * warp, bad, w);
#pragma unroll
    for (int part = 0; part < (Pair16<T>::kWide ? 2 : 1); ++part) {
      uint32_t b[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t pk = pack16<T>(w[t][2 * e], w[t][2 * e + 1]);
          b[t][e] = movmatrix(pk);
          const float2 r = unpack16<T>(pk);
          w[t][2 * e] -= r.x, w[t][2 * e + 1] -= r.y;
        }
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const uint32_t a0 = __byte_perm(v[0][x], v[1][x], 0x5410), a1 = __byte_perm(v[0][x], v[1][x], 0x7632);
        const uint32_t a2 = __byte_perm(v[2][x], v[3][x], 0x5410), a3 = __byte_perm(v[2][x], v[3][x], 0x7632);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(o[x][t], a0, a1, a2, a3, b[t][0], b[t][1], T());
      }
    }
  }

  // Joins the four warps' results into warp 0's registers (o, ml, mv, l).
  __device__ void join(float* area, float* stats) {
    constexpr int ROWS = Shape<D, NT>::ROWS, OROW = Shape<D, NT>::OROW;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[t][j] += __shfl_xor_sync(~0u, l[t][j], d);
        if (gid == 0) {
          float* p = stats + (warp * ROWS + 8 * t + 2 * tig + j) * 4;
          p[0] = ml[t][j], p[1] = mv[t][j], p[2] = l[t][j];
        }
      }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float gl = kLowest, gv = kLowest, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* p = stats + (w * ROWS + 8 * t + 2 * tig + j) * 4;
          gl = fmaxf(gl, p[0]), gv = fmaxf(gv, p[1]);
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* p = stats + (w * ROWS + 8 * t + 2 * tig + j) * 4;
          sum += p[2] * ex2(p[0] - gl);
        }
        const float c = ex2(mv[t][j] - gv);
#pragma unroll
        for (int m = 0; m < KS; ++m) o[m][t][j] *= c, o[m][t][j + 2] *= c;
        ml[t][j] = gl, mv[t][j] = gv, l[t][j] = sum;
      }
#pragma unroll
    for (int half = 2; half >= 1; half /= 2) {
      if (warp >= half && warp < 2 * half) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int m = 0; m < KS; ++m)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              *reinterpret_cast<float2*>(area + ((warp - half) * ROWS + 8 * t + 2 * tig + j) * OROW + D / 8 * gid + 2 * m) =
                  make_float2(o[m][t][j], o[m][t][j + 2]);
      }
      __syncthreads();
      if (warp < half) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int m = 0; m < KS; ++m)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 x = *reinterpret_cast<const float2*>(area + (warp * ROWS + 8 * t + 2 * tig + j) * OROW + D / 8 * gid + 2 * m);
              o[m][t][j] += x.x, o[m][t][j + 2] += x.y;
            }
      }
      __syncthreads();
    }
  }
};

__device__ __forceinline__ float result(float o, float ml, float mv, float l) {
  return l == 0.f ? 0.f : o * (ex2(mv - ml) / l);
}

template <typename T, int FMT, int D, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NT)) q8_attend_kernel(const Q8AttendArgs a) {
  using S = Shape<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  float* area = reinterpret_cast<float*>(smem + S::RING);
  float* stats = reinterpret_cast<float*>(smem + S::RING + S::JOIN);
  uint32_t* sums = reinterpret_cast<uint32_t*>(smem + S::RING + S::JOIN + S::STATS);
  uint32_t* pre = sums + 4;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int groups = (a.n * a.G + S::ROWS - 1) / S::ROWS, subs = a.c.num_kv_heads * groups;
  plan_rows(a, subs, pre, sums);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.c.batch; b += kThreads)
      if (!row_valid(a, a.lens[b], a.n_rows ? a.n_rows[b] : a.n)) atomicOr(a.c.status, kQ8StatusInvalid);
  const uint32_t tiles = pre[a.c.batch], ctas = plan_ctas(tiles, gridDim.x);
  if (blockIdx.x >= ctas) return;
  const uint32_t t0 = cta_start(blockIdx.x, tiles, ctas), t1 = cta_start(blockIdx.x + 1, tiles, ctas);

  Pass<T, FMT, D, NT> ps;
  ps.lane = threadIdx.x % 32, ps.warp = threadIdx.x / 32;
  ps.gid = ps.lane / 4, ps.tig = ps.lane % 4;
  const uint32_t ring = smem_u32(smem) + ps.warp * kStages * S::STAGE;
  // The warp's 16 tokens of the run's next whole block go to a stage of the warp's ring (open blocks are
  // read where they are used): 16-byte copies from kp, vp, and the two scales.
  Walk get;
  const uint8_t *kp = nullptr, *vp = nullptr;
  const float* sp = nullptr;
  int more = 0;                                            // whole blocks to fetch from kp, vp on
  auto aim = [&](bool on) {
    for (; on; on = get.next(a, pre, subs)) {
      more = min(get.end, get.whole) - get.begin;
      if (more <= 0) continue;
      const size_t unit = (size_t)get.row * a.c.num_kv_heads + get.sub / groups;
      const size_t at = (unit * a.c.capacity + (size_t)get.begin * kQ8Block + 16 * ps.warp) * D + 16 * ps.lane;
      kp = static_cast<const uint8_t*>(a.c.k_codes) + at;
      vp = static_cast<const uint8_t*>(a.c.v_codes) + at;
      sp = (ps.lane ? a.c.v_scales : a.c.k_scales) + unit * (a.c.capacity / kQ8Block) + get.begin;
      return;
    }
    more = 0;
  };
  uint32_t dst[S::SLAB / 512];
#pragma unroll
  for (int i = 0; i < S::SLAB / 512; ++i) {
    const int x = i * 32 + ps.lane;
    dst[i] = slab_at<D>(x / (D / 16), x % (D / 16));
  }
  auto fetch = [&](uint32_t st) {
    if (more > 0) {
#pragma unroll
      for (int i = 0; i < S::SLAB / 512; ++i) {
        cp_async16(st + dst[i], kp + 512 * i);
        cp_async16(st + S::SLAB + dst[i], vp + 512 * i);
      }
      if (ps.lane < 2) cp_async4(st + 2 * S::SLAB + 4 * ps.lane, sp);
      kp += kQ8Block * D, vp += kQ8Block * D, ++sp;
      if (--more == 0) aim(get.next(a, pre, subs));
    }
    cp_commit();
  };
  Walk use;
  bool on = use.first(a, pre, subs, t0, t1);
  get = use;
  aim(on);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(ring + i * S::STAGE);

  uint32_t st = ring, ahead = ring + (kStages - 1) * S::STAGE;
  for (; on; on = use.next(a, pre, subs)) {
    const int kvh = use.sub / groups, r0 = use.sub % groups * S::ROWS;
    ps.start(a, use.row, kvh, r0);
    const int blocks = min(use.end, use.whole);
    for (int tile = use.begin; tile < blocks; ++tile) {
      fetch(ahead);
      cp_wait<kStages - 1>();
      __syncwarp();
      const int first = tile * kQ8Block + 16 * ps.warp;
      if ((tile + 1) * kQ8Block <= ps.min_end) ps.template codes<false>(st, first);
      else ps.template codes<true>(st, first);
      __syncwarp();                                        // every lane has read before the stage is filled again
      ahead = st;
      st = st == ring + (kStages - 1) * S::STAGE ? ring : st + S::STAGE;
    }
    if (use.end > use.whole) ps.open(a, use.row, kvh, r0, use.whole);
    ps.join(area, stats);
    if (ps.warp == 0) {
      const bool all = use.begin == 0 && use.end == use.tiles;
      // its second result where the unit begins inside the run: of two units that the run shares, one does
      const uint32_t unit0 = pre[use.row] + (uint32_t)use.sub * (kUnitCost + use.tiles) + kUnitCost;
      float* part = reinterpret_cast<float*>(a.scratch) + ((size_t)blockIdx.x * 2 + (t0 < unit0)) * S::ROWS * S::OROW;
      const int nr = a.n_rows ? a.n_rows[use.row] : a.n;
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = 8 * q + 2 * ps.tig + j, i = (r0 + r) / a.G, h = (r0 + r) % a.G;
          if (i >= nr) continue;
          if (all) {
            T* out = static_cast<T*>(a.out) + (((size_t)use.row * a.n + i) * a.Hq + kvh * a.G + h) * D + D / 8 * ps.gid;
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
              reinterpret_cast<uint32_t*>(out)[m] =
                  pack16<T>(result(ps.o[m][q][j], ps.ml[q][j], ps.mv[q][j], ps.l[q][j]),
                            result(ps.o[m][q][j + 2], ps.ml[q][j], ps.mv[q][j], ps.l[q][j]));
          } else {
            float* p = part + r * S::OROW;
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
              *reinterpret_cast<float2*>(p + D / 8 * ps.gid + 2 * m) = make_float2(ps.o[m][q][j], ps.o[m][q][j + 2]);
            if (ps.gid == 0) *reinterpret_cast<float4*>(p + D) = make_float4(ps.ml[q][j], ps.mv[q][j], ps.l[q][j], 0.f);
          }
        }
    }
  }
}

// Joins the partial results of units that several CTAs share, one block per
// (unit, query row), and writes what no CTA had work for: zeros for rows
// without tokens, NaN for rows whose length is refused.  It is bound by the
// latency of its loads: the warps take the results in turn, a warp 32 of them
// at a time, each lane first one result's references and sum, then all lanes
// D / 32 dims of every result, the loads of eight together.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads) q8_join_kernel(const Q8AttendArgs a, uint32_t grid) {
  using S = Shape<D, NT>;
  constexpr int E = D / 32;
  extern __shared__ uint32_t pre[];
  __shared__ uint32_t sums[kWarps];
  __shared__ float wm[kWarps][3], wo[kWarps][D];
  const int R = a.n * a.G, groups = (R + S::ROWS - 1) / S::ROWS, subs = a.c.num_kv_heads * groups;
  const int row = blockIdx.y, kvh = blockIdx.x / R, r = blockIdx.x % R, i = r / a.G;
  plan_rows(a, subs, pre, sums);
  const int len = a.lens[row], nr = a.n_rows ? a.n_rows[row] : a.n;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool valid = row_valid(a, len, nr);
  if (valid && i >= nr) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  T* out = static_cast<T*>(a.out) + (((size_t)row * a.n + i) * a.Hq + kvh * a.G + r % a.G) * D;
  if (!valid || len == 0) {
    if (threadIdx.x < D) out[threadIdx.x] = valid ? (T)0.f : (T)__uint_as_float(0x7fffffffu);
    return;
  }
  const uint32_t places = pre[a.c.batch], ctas = plan_ctas(places, grid), unit = (pre[row + 1] - pre[row]) / subs;
  const uint32_t first = pre[row] + (uint32_t)(kvh * groups + r / S::ROWS) * unit + kUnitCost;
  const uint32_t c0 = cta_of(first, places, ctas), c1 = cta_of(first + unit - kUnitCost - 1, places, ctas);
  if (c0 == c1) return;
  // CTA c's first result, or its second where the unit begins inside its run
  const uint32_t slot0 = cta_start(c0, places, ctas) < first;
  const float* part = reinterpret_cast<const float*>(a.scratch) + (size_t)(r % S::ROWS) * S::OROW;
  float gl = kLowest, gv = kLowest, sum = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (uint32_t b = c0 + warp; b <= c1; b += 32 * kWarps) {
    const uint32_t c = b + kWarps * lane;                  // this lane's CTA
    const int n = (int)min(32u, (c1 - b) / kWarps + 1);
    float ml = kLowest, mv = kLowest, l = 0.f;
    if (lane < n) {
      const float4 x = *reinterpret_cast<const float4*>(part + (size_t)(c * 2 + (c == c0 ? slot0 : 0)) * S::ROWS * S::OROW + D);
      ml = x.x, mv = x.y, l = x.z;
    }
    float nl = fmaxf(gl, ml), nv = fmaxf(gv, mv);
#pragma unroll
    for (int d = 16; d; d /= 2) nl = fmaxf(nl, __shfl_xor_sync(~0u, nl, d)), nv = fmaxf(nv, __shfl_xor_sync(~0u, nv, d));
    l *= ex2(ml - nl);
#pragma unroll
    for (int d = 16; d; d /= 2) l += __shfl_xor_sync(~0u, l, d);
    sum = sum * ex2(gl - nl) + l;
    const float keep = ex2(gv - nv), w = ex2(mv - nv);
    gl = nl, gv = nv;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
    for (int x0 = 0; x0 < n; x0 += 8) {
      float p[8][E];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint32_t cx = min(b + kWarps * (x0 + x), c1 - (c1 - b) % kWarps);
        const float* src = part + (size_t)(cx * 2 + (cx == c0 ? slot0 : 0)) * S::ROWS * S::OROW + E * lane;
        if (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          p[x][0] = v.x, p[x][1] = v.y, p[x][E - 2] = v.z, p[x][E - 1] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          p[x][0] = v.x, p[x][1] = v.y;
        }
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float wx = __shfl_sync(~0u, w, x0 + x);
        if (x0 + x < n)
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = fmaf(wx, p[x][e], o[e]);
      }
    }
  }
  if (lane == 0) wm[warp][0] = gl, wm[warp][1] = gv, wm[warp][2] = sum;
#pragma unroll
  for (int e = 0; e < E; ++e) wo[warp][E * lane + e] = o[e];
  __syncthreads();
  if (threadIdx.x >= D) return;
  gl = gv = kLowest, sum = 0.f;
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) gl = fmaxf(gl, wm[w][0]), gv = fmaxf(gv, wm[w][1]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    sum += wm[w][2] * ex2(wm[w][0] - gl);
    t += wo[w][threadIdx.x] * ex2(wm[w][1] - gv);
  }
  out[threadIdx.x] = (T)result(t, gl, gv, sum);
}

// Query rows of one pass: 8 where a unit has no more, else 16.
int pick_nt(int rows) { return rows <= 8 ? 1 : 2; }

uint32_t grid_of(const tq_q8_cache& c, int Hq, int n, int num_sms) {
  const int rows = n * (Hq / c.num_kv_heads), nt = pick_nt(rows);
  const int64_t tiles = (int64_t)c.batch * c.num_kv_heads * ((rows + 8 * nt - 1) / (8 * nt)) *
                        (c.capacity / kQ8Block + kUnitCost);
  const int64_t most = (int64_t)num_sms * ctas_per_sm(c.head_dim, nt), want = (tiles + kMinTiles - 1) / kMinTiles;
  return (uint32_t)(want < most ? want : most);
}

template <typename T, int FMT, int D, int NT>
cudaError_t launch(const Q8AttendArgs& a, uint32_t grid, cudaStream_t s) {
  const int smem = smem_bytes<D, NT>(a.c.batch);
  auto kernel = q8_attend_kernel<T, FMT, D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // a programmatic dependent: it waits for the attention kernel before it reads its results
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.c.num_kv_heads * a.n * a.G), (unsigned)a.c.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 4 * (a.c.batch + 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q8_join_kernel<T, D, NT>, a, grid);
}

template <typename T, int FMT>
cudaError_t pick(const Q8AttendArgs& a, uint32_t grid, cudaStream_t s) {
  const bool one = pick_nt(a.n * a.G) == 1;
  if (a.c.head_dim == 64) return one ? launch<T, FMT, 64, 1>(a, grid, s) : launch<T, FMT, 64, 2>(a, grid, s);
  return one ? launch<T, FMT, 128, 1>(a, grid, s) : launch<T, FMT, 128, 2>(a, grid, s);
}

}  // namespace

size_t q8_attend_scratch(const tq_q8_cache& c, int Hq, int n, int num_sms) {
  const int rows = 8 * pick_nt(n * (Hq / c.num_kv_heads));
  return ((size_t)grid_of(c, Hq, n, num_sms) * 2 * rows * (c.head_dim + 4) * 4 + 255) / 256 * 256;
}

cudaError_t launch_q8_attend(const Q8AttendArgs& a, int num_sms, cudaStream_t s) {
  const uint32_t grid = grid_of(a.c, a.Hq, a.n, num_sms);
  const bool i8 = a.c.format == TQ_Q8_INT8;
  if (a.c.dtype == TQ_DTYPE_FP16)
    return i8 ? pick<__half, TQ_Q8_INT8>(a, grid, s) : pick<__half, TQ_Q8_E4M3>(a, grid, s);
  return i8 ? pick<__nv_bfloat16, TQ_Q8_INT8>(a, grid, s) : pick<__nv_bfloat16, TQ_Q8_E4M3>(a, grid, s);
}

}  // namespace tq
