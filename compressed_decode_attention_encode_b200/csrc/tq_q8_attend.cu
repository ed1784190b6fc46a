// Attention over the 8-bit cache (include/tq.h has the contract).
//
// For a query q of a row's (row, kv head) unit, with a block's scales s_k, s_v
// and codes c:
//   x_p = sigma log2(e) s_k <q, c_k>,   o = sum_p 2^x_p s_v c_v / sum_p 2^x_p
// in one pass, with two running references: ml of x for the denominator, and
// ml + dv of x + log2 s_v for the numerator, whose weights
// 2^((x - ml) + (log2 s_v - dv)) take the place of an fp16 operand without a
// multiplication by s_v.  dv is kept as a difference because a sum x + log2 s_v
// is rounded at x: at logits of 10^5 it left half a percent of error.  Codes
// and fp16 values are exact operands, sums and references float32.  Weights
// enter the second product in parts that leave float32's own precision: two of
// fp16 (2^-22), in a bf16 cache's open block three of bf16 (2^-24).  With one
// fp16 part, which saved up to 13 %, the error beside an fp16 result's own
// rounding was 1.6 times as large where many tokens of either sign weigh
// alike, and one bf16 result in a hundred was rounded to the neighbour.
//
// The work is the batch's tiles (a unit's whole blocks of 64 tokens, then its
// open block), flattened and cut into equal runs, one per CTA, so that rows of
// any length share the card; every CTA finds its run from the lengths alone
// (they are device memory).  Each unit has unit_cost places before its first
// tile, which stand for what a pass costs besides its tiles (its queries'
// latency, the open block's, the join of the warps).  A unit inside one CTA's
// run is finished there; the others leave partial results that a second
// kernel joins in a fixed order.
//
// One query per row is bound by the fetch of the codes: 8 rows of 32768 tokens
// (32/8 heads of 128, e4m3, fp16) take 90 us on the device, 6.0 TB/s, and the
// kernel without its arithmetic as long (100 us in loops of a fifth of a second
// and more, graphs and calls alike).  One row of 131583 (int8, bf16) takes 56.2
// us, its fetch alone 49.4; 33 ragged rows (e4m3, bf16) 45.5 and 39.0.  Several
// queries are bound by the chain of dependent instructions at 8 warps per SM: 5
// in each of 16 ragged rows up to 4109 tokens take 27.9 us, the fetch alone
// 15.5, where the bytes would take 7.6.
#include <atomic>
#include <cmath>
#include <mutex>

#include "tq_q8.cuh"

namespace tq {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
// Stages of a warp's ring.  Two keep 48 KB per SM on their way; with three 8 rows of 32K tokens take 99 us instead of
// 90, 33 ragged rows 52 instead of 45, and 8 queries in 16 rows of 4096 76.5 instead of 77.8.
constexpr int kStages = 2;
constexpr float kLowest = -3.0e38f;          // ml before its first token
constexpr float kShift = 7.f;                // numerator weights are 2^7 at their reference (dv holds it less 7),
constexpr float kNothing = -1000.f;          // in place of log2 s_v where the codes are zeros: moves no reference
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
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
// Result = numerator x both factors, with the numerator's reference gv (relative
// to the denominator's), whose power of two alone may be no float32.  A
// denominator of zero has no token behind it, or only logits of -inf, which is
// no number.
struct Factors {
  float a, b;
  __device__ __forceinline__ Factors(float gv, float sum, bool sees) {
    a = ex2(0.5f * gv), b = sum == 0.f ? (sees ? NAN : 0.f) : a / sum;
  }
  __device__ __forceinline__ float operator()(float t) const { return t * a * b; }
};
template <typename T>
__device__ __forceinline__ bool quad_bad(const uint4& v) {
  return pair_bad<T>(v.x) || pair_bad<T>(v.y) || pair_bad<T>(v.z) || pair_bad<T>(v.w);
}

// ---- the plan: which tiles a CTA takes -------------------------------------
__device__ __forceinline__ bool row_valid(const Q8AttendArgs& a, int len, int nr) {
  return len >= 0 && len <= a.c.capacity && nr >= 0 && nr <= a.n;
}
// What a unit costs besides its tiles, in tiles.  Measured, one query each (NT = 1) with 4, 6, 8 and 12: 33 ragged rows
// up to 9001 tokens (bf16) 50.2, 45.1, 45.3 and 46.6 us; 64 up to 4000 46.1, 43.4, 46.1 and 49.1; 16 rows of 8192 with
// 64 query heads 52.7, 53.0, 55.5 and 54.5; 16 rows of 4096 (fp16) 31.8, 32.8, 33.9 and 35.4.  5 queries in each of 16
// ragged rows (NT = 3, heavier tiles) with 2, 3, 4 and 8: 33.0, 29.0, 27.9 and 30.4; 8 of them in rows of 4096 alike
// with 2 to 4 (77.8), 81.3 with 8.
constexpr int unit_cost(int nt) { return nt == 1 ? 6 : 4; }
// In shared memory: places before each row [batch + 1], lengths [batch] (0 where a row has no work).
struct Plan {
  uint32_t* pre;
  int* len;
};
__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t y = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += y;
  }
  return v;
}
// Places before each row (a unit's places x units of a row).
__device__ __forceinline__ void plan_rows(const Q8AttendArgs& a, int subs, int cost, const Plan& p, uint32_t* warp_sums) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  auto places = [&](int b) {
    if (b >= a.c.batch) return 0u;
    const int len = a.lens[b], nr = a.n_rows ? a.n_rows[b] : a.n;
    const bool on = row_valid(a, len, nr) && nr > 0 && len > 0;
    p.len[b] = on ? len : 0;
    return on ? (uint32_t)(cost + (len + kQ8Block - 1) / kQ8Block) * subs : 0u;
  };
  if (a.c.batch <= 32) {                   // every warp for itself: all write the same values
    const uint32_t v = places(lane), s = warp_scan(v);
    if (lane < a.c.batch) p.pre[lane] = s - v;
    if (lane == 31) p.pre[a.c.batch] = s;
    __syncwarp();
    return;
  }
  uint32_t total = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.c.batch; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const uint32_t v = places(b), s = warp_scan(v);
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    uint32_t before = total;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_sums[w];
      total += warp_sums[w];
    }
    if (b < a.c.batch) p.pre[b] = before + s - v;
    __syncthreads();
  }
  if (threadIdx.x == 0) p.pre[a.c.batch] = total;
  __syncthreads();
}
// A run has one place at least: with few, short rows the tiles' latency is what counts (a row of 1536 tokens with 4
// kv heads: 6.4 us with one place a CTA; an earlier build 6.7, and 7.3 with two, 8.3 with four).
__device__ __forceinline__ uint32_t plan_ctas(uint32_t places, uint32_t grid) { return places < grid ? places : grid; }
// Runs of places / ctas places, one more in the first ones.
struct Runs {
  uint32_t len, more, ctas;
  __device__ __forceinline__ Runs(uint32_t places, uint32_t grid) {
    ctas = plan_ctas(places, grid);
    len = ctas ? places / ctas : 0;
    more = places - len * ctas;
  }
  __device__ __forceinline__ uint32_t start(uint32_t c) const { return c * len + min(c, more); }
  // The CTA whose run holds place t.
  __device__ __forceinline__ uint32_t of(uint32_t t) const {
    const uint32_t longer = more * (len + 1);
    return t < longer ? t / (len + 1) : more + (t - longer) / len;
  }
};

// A CTA's run, segment by segment: a segment is the run's tiles [begin, end) of one unit (kv head x query
// group of a row), never empty.  Kept in shared memory, one for what a warp computes and one, ahead of it,
// for what it fetches, so that the code that moves them is there once: a pass's straight code runs once per
// unit, and its instruction fetches cost more than its instructions do.
struct Walk {
  int row, sub;
  uint32_t left;                           // places of the run behind this segment
  int whole, tiles, begin, end;            // of the unit: whole blocks, tiles; of the segment: tiles
};
// To the next segment; begin == end at the end of the run.  The warp's lanes write the same values.
__device__ __noinline__ void walk_next(Walk* w, Plan p, int subs, int cost) {
  Walk x = *w;
  do {
    if (x.left == 0) {
      x.begin = x.end = 0;
      break;
    }
    if (++x.sub == subs) {
      x.sub = 0;
      do ++x.row;
      while (p.pre[x.row + 1] == p.pre[x.row]);
      const int len = p.len[x.row];
      x.whole = len / kQ8Block;
      x.tiles = x.whole + (len % kQ8Block != 0);
    }
    const uint32_t take = min(x.left, (uint32_t)(cost + x.tiles));
    x.begin = 0;
    x.end = (int)take - cost;
    x.left -= take;
  } while (x.end <= x.begin);
  __syncwarp();
  *w = x;
  __syncwarp();
}
__device__ __forceinline__ Walk walk_first(const Plan& p, int batch, int subs, int cost, uint32_t t0, uint32_t t1) {
  Walk x;
  // the last row with pre[row] <= t0: of every 32nd, then of 32 (at most 1024 rows)
  const int lane = threadIdx.x % 32;
  int lo = 0;
  if (batch > 32) lo = 32 * (__popc(__ballot_sync(~0u, 32 * lane < batch && p.pre[min(32 * lane, batch)] <= t0)) - 1);
  lo += __popc(__ballot_sync(~0u, lo + lane < batch && p.pre[min(lo + lane, batch)] <= t0)) - 1;
  x.row = lo;
  const int len = p.len[lo];
  x.whole = len / kQ8Block;
  x.tiles = x.whole + (len % kQ8Block != 0);
  const uint32_t off = t0 - p.pre[lo], places = cost + x.tiles;
  x.sub = off / places;
  const uint32_t pos = off - x.sub * places, take = min(t1 - t0, places - pos);
  x.begin = max((int)pos - cost, 0);
  x.end = (int)(pos + take) - cost;   // <= begin: a run that begins with places alone
  x.left = t1 - t0 - take;
  return x;
}

template <int D, int NT>
struct Shape {
  static constexpr int COST = unit_cost(NT);
  static constexpr int ROWS = 8 * NT;                      // query rows of a unit's pass
  static constexpr int SLAB = 16 * D;                      // bytes of 16 tokens' codes
  static constexpr int STAGE = 2 * SLAB + 16;              // K, V, scales
  static constexpr int RING = kWarps * kStages * STAGE;
  static constexpr int OROW = D + 4;                       // a row of partial results: o, ml, dv, l
  static constexpr int JOIN = kWarps * ROWS * OROW * 4;
  static constexpr int WALK = kWarps * 2 * (int)sizeof(Walk);
  static constexpr bool QS = NT > 1;                       // queries in shared memory, not in registers
  static_assert(NT <= kWarps);                             // a warp brings eight of them
  static constexpr int Q = QS ? NT * (D / 16) * 256 + ROWS * 4 : 0;
};
// CTAs per SM: what registers and shared memory allow, at spills of 40 bytes a thread at most (bf16, d = 128, NT = 1).
// Two queries' passes of d = 64 with three instead of two: 19.5 us instead of 20.2 for 8 rows of 8192; NT = 1 of
// d = 128 with four instead of three spills, 151 us instead of 90 for 8 rows of 32768.
constexpr int ctas_per_sm(int d, int nt) { return nt == 1 ? (d == 128 ? 3 : 4) : nt == 2 && d == 64 ? 3 : 2; }
template <int D, int NT>
int smem_bytes(int batch) {
  using S = Shape<D, NT>;
  return S::RING + S::JOIN + S::WALK + S::Q + 16 + 4 * (2 * batch + 1);
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
  using S = Shape<D, NT>;
  static constexpr int KS = D / 16;          // k-steps of the first product, m-tiles of the second
  static constexpr int PARTS = 2, OPEN_PARTS = Pair16<T>::kWide ? 3 : 2;   // of a weight: for whole blocks, for the open one
  float o[KS][NT][4];                        // dims 2 mt, 2 mt + 1 of the lane's D / 8, queries 2 tig, 2 tig + 1
  float ml[NT][2], dv[NT][2], l[NT][2];
  float cq[NT][2];                           // sigma log2(e) of the query (and its power of two)
  uint32_t qf[S::QS ? 1 : NT][KS][2];        // the queries' operand, or its place in shared memory
  uint2* qs;
  float* qup;
  int base, r0;                              // query row r of the pass sees positions below base + (r0 + r) / G
  uint32_t inv_g;                            // 2^16 / G, rounded up: (r inv_g) >> 16 is r / G for r < 2^11
  int lane, gid, tig, warp;

  // Query row r of a unit (r = token G + head); rows behind the last one repeat it and are not stored.
  __device__ __forceinline__ const T* q_row(const Q8AttendArgs& a, int row, int kvh, int r) {
    r = min(r, a.n * a.G - 1);
    const int i = (int)((uint32_t)r * inv_g >> 16);
    return static_cast<const T*>(a.q) + row * a.row_stride + i * a.token_stride +
           (int64_t)(kvh * a.G + r - i * a.G) * a.head_stride;
  }

  // Column 8 t + gid of the queries' operand, as it is.
  __device__ __forceinline__ void load_q(const Q8AttendArgs& a, int row, int kvh, int t, uint32_t (&f)[KS][2]) {
    const T* q = q_row(a, row, kvh, r0 + 8 * t + gid) + 16 * tig;
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint4 v = *reinterpret_cast<const uint4*>(q + 64 * j + 8 * x);
        f[4 * j + 2 * x][0] = v.x, f[4 * j + 2 * x][1] = v.y;
        f[4 * j + 2 * x + 1][0] = v.z, f[4 * j + 2 * x + 1][1] = v.w;
      }
  }
  // ... in fp16: a bf16 query is scaled by the power of two that brings its
  // largest element into [2^14, 2^15), so that elements down to 2^-31 of it are
  // exact and those below lose at most 2^-40 of it; returns sigma log2(e) by
  // that power.  (With the largest element in [1, 2) these were 2^-17 and
  // 2^-25, which showed where the largest elements meet keys of zero.)
  __device__ __forceinline__ float half_q(const Q8AttendArgs& a, uint32_t (&f)[KS][2]) {
    if (!Pair16<T>::kWide) return a.scale_log2;
    uint32_t mx = 0;
#pragma unroll
    for (int s = 0; s < KS; ++s) mx = __vmaxu2(mx, __vmaxu2(f[s][0] & 0x7fff7fffu, f[s][1] & 0x7fff7fffu));
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(~0u, mx, 1));
    mx = max(mx, __shfl_xor_sync(~0u, mx, 2));
    const int e = mx >= 0x7f80u ? 0 : max((int)(mx >> 7) - 127 - 14, -126);   // NaN and infinities pass as they are
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float2 w = unpack16<T>(f[s][x]);
        f[s][x] = pack16<__half>(w.x * down, w.y * down);
      }
    return a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
  }

  // The first half of a pass's start: the loads of its queries, before any fetch that they would wait behind.
  __device__ __forceinline__ void load(const Q8AttendArgs& a, int row, int kvh, int first_row) {
    r0 = first_row;
    if (!S::QS || warp < NT) load_q(a, row, kvh, S::QS ? warp : 0, qf[0]);
  }
  __device__ __forceinline__ void start(const Q8AttendArgs& a, int row, int kvh, int len) {
#pragma unroll
    for (int m = 0; m < KS; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][t][e] = 0.f;
    base = len - (a.n_rows ? a.n_rows[row] : a.n) + 1;
    if (S::QS) {
      // warp t brings columns 8 t .. 8 t + 7, for all
      if (warp < NT) {
        const float up = half_q(a, qf[0]);
#pragma unroll
        for (int s = 0; s < KS; ++s) qs[(warp * KS + s) * 32 + lane] = make_uint2(qf[0][s][0], qf[0][s][1]);
        if (tig == 0) qup[8 * warp + gid] = up;
      }
      __syncthreads();
    }
    const float up = S::QS ? 0.f : half_q(a, qf[0]);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        ml[t][j] = kLowest;
        dv[t][j] = l[t][j] = 0.f;
        cq[t][j] = !Pair16<T>::kWide ? a.scale_log2 : S::QS ? qup[8 * t + 2 * tig + j] : __shfl_sync(~0u, up, 4 * (2 * tig + j));
      }
  }
  __device__ __forceinline__ uint2 q_at(int t, int s) {
    return S::QS ? qs[(t * KS + s) * 32 + lane] : make_uint2(qf[0][s][0], qf[0][s][1]);
  }
  __device__ __forceinline__ int end_of(int t, int j) {
    return base + (int)((uint32_t)(r0 + 8 * t + 2 * tig + j) * inv_g >> 16);
  }

  // Weights of 16 tokens from their logits x = s f: denominators are added up
  // here, the numerators' are returned in x.  `mask`: a token at position
  // first + gid (+ 8) counts only before a query's end.
  __device__ __forceinline__ void weights(float (&x)[NT][4], const float (&f)[NT][2], float lsv, int first, bool mask) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[t][e] *= f[t][e & 1];
    if (mask) {
      const bool nan = isnan(lsv);                         // of the block: for the queries that see it
      if (nan) lsv = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[t][e] = first + gid + 8 * (e >> 1) >= end_of(t, e & 1) ? -INFINITY : nan ? NAN : x[t][e];
    }
    float over = -INFINITY;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float y = fmaxf(x[t][j], x[t][j + 2]) - ml[t][j];
        over = fmaxf(over, fmaxf(y, y + (lsv - dv[t][j] - kShift)));
      }
    if (__any_sync(~0u, over > kLazy)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float m = fmaxf(x[t][j], x[t][j + 2]);
#pragma unroll
          for (int d = 4; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
          const float nl = fmaxf(ml[t][j], m), down = ml[t][j] - nl;
          const float old = dv[t][j] + down, nv = fmaxf(old, (m - nl) + (lsv - kShift));
          l[t][j] *= ex2(down);
          const float c = ex2(old - nv);
          ml[t][j] = nl, dv[t][j] = nv;
#pragma unroll
          for (int k = 0; k < KS; ++k) o[k][t][j] *= c, o[k][t][j + 2] *= c;
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float y = x[t][e] - ml[t][e & 1];
        l[t][e & 1] += ex2(y);
        x[t][e] = ex2(y + (lsv - dv[t][e & 1]));
      }
  }

  // The next 16-bit part of the weights as the second product's operand; what
  // it leaves stays in w.
  template <typename P>
  __device__ __forceinline__ void split(float (&w)[NT][4], uint32_t (&b)[NT][2]) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t pk = pack16<P>(w[t][2 * e], w[t][2 * e + 1]);
        b[t][e] = movmatrix(pk);
        const float2 r = unpack16<P>(pk);
        w[t][2 * e] -= r.x, w[t][2 * e + 1] -= r.y;
      }
  }

  // The warp's 16 tokens of a tile: of a whole block, from the ring stage at
  // `st` with the scales behind it, or of the open block, from the 16-bit
  // ring in global memory.  The open block's products take the cache's own
  // type, exactly, and the weights in parts of it.
  __device__ __forceinline__ void tile(const Q8AttendArgs& a, const uint8_t* st, int tile, bool open, int row, int kvh,
                                       int len) {
    constexpr int SLAB = S::SLAB;
    const int first = tile * kQ8Block + 16 * warp, cnt = len - first;
    if (cnt <= 0) return;                                  // behind the open block's tokens
    float s[NT][4], f[NT][2], lsv = 0.f;
    uint32_t bad = 0;                                      // the open block's tokens with a NaN or an infinity
    uint4 vo[4][KS / 4];                                   // its values
    float up = 1.f;                                        // bf16: what its weights are short of
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
    if (!open) {
      const float sk = *reinterpret_cast<const float*>(st + 2 * SLAB);
      const float sv = *reinterpret_cast<const float*>(st + 2 * SLAB + 4);
      lsv = lg2(sv);
      if (sv == 1.f) {
        // A block of zeros has this scale.  Its tokens add nothing to the numerator, and its reference would leave
        // the weights of later blocks with small values below what fp16 holds.
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < SLAB / 512; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(st + SLAB + 512 * i + 16 * lane);
          any |= v.x | v.y | v.z | v.w;
        }
        if (FMT == TQ_Q8_E4M3) any &= 0x7f7f7f7fu;         // -0 is a zero
        if (!__any_sync(~0u, any)) lsv = kNothing;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) f[t][0] = sk * cq[t][0], f[t][1] = sk * cq[t][1];
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const uint4 ka = *reinterpret_cast<const uint4*>(st + slab_at<D>(gid, tig + 4 * j));
        const uint4 kb = *reinterpret_cast<const uint4*>(st + slab_at<D>(gid + 8, tig + 4 * j));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t a0, a1, a2, a3;
          codes_to_half4<FMT>(word(ka, x), a0, a2);
          codes_to_half4<FMT>(word(kb, x), a1, a3);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint2 b = q_at(t, 4 * j + x);
            mma16816(s[t], a0, a1, a2, a3, b.x, b.y, __half());
          }
        }
      }
    } else {
      const size_t ring = (((size_t)row * a.c.num_kv_heads + kvh) * kQ8Ring + first % kQ8Ring) * D;
      const T* vr = static_cast<const T*>(a.c.v_recent) + ring + D / 8 * gid;
      const T* kr = static_cast<const T*>(a.c.k_recent) + ring + 16 * tig;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * tig + (i & 1) + 8 * (i >> 1);
#pragma unroll
        for (int x = 0; x < KS / 4; ++x) {
          vo[i][x] = r < cnt ? *reinterpret_cast<const uint4*>(vr + r * D + 8 * x) : make_uint4(0, 0, 0, 0);
          if (quad_bad<T>(vo[i][x])) bad |= 1u << r;
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) f[t][0] = f[t][1] = a.scale_log2;
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint4 k[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = gid + 8 * i;
            k[i] = r < cnt ? *reinterpret_cast<const uint4*>(kr + r * D + 64 * j + 8 * x) : make_uint4(0, 0, 0, 0);
            if (quad_bad<T>(k[i])) bad |= 1u << r;
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint2 b0 = q_at(t, 4 * j + 2 * x), b1 = q_at(t, 4 * j + 2 * x + 1);
            if (Pair16<T>::kWide) {                        // the raw query: cached by the first load of it
              const uint4 v = *reinterpret_cast<const uint4*>(q_row(a, row, kvh, r0 + 8 * t + gid) + 64 * j + 16 * tig + 8 * x);
              b0 = make_uint2(v.x, v.y), b1 = make_uint2(v.z, v.w);
            }
            mma16816(s[t], k[0].x, k[1].x, k[0].y, k[1].y, b0.x, b0.y, T());
            mma16816(s[t], k[0].z, k[1].z, k[0].w, k[1].w, b1.x, b1.y, T());
          }
        }
      if (Pair16<T>::kWide) {
        // The open block's values stand for themselves, at a scale of 1; bf16 ones may be so small, or zeros, that the
        // reference of that scale would leave what the whole blocks gave below float32.  So the reference takes the
        // power of two of the largest, and the weights that power back.
        __nv_bfloat162 m2 = __floats2bfloat162_rn(0.f, 0.f);  // NaN drops out; infinities count as 1 and more
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < KS; ++x) {
            const uint32_t v = word(vo[i][x / 4], x % 4);
            m2 = __hmax2(m2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v)));
          }
        uint32_t mx = *reinterpret_cast<const uint32_t*>(&m2);
        mx = __reduce_max_sync(~0u, max(mx & 0xffffu, mx >> 16));
        const int k = min(max(127 - (int)(mx >> 7), 0), 100);   // 0 for values of 1 and more
        lsv = mx == 0 ? kNothing : (float)-k;
        up = __uint_as_float((uint32_t)(127 + k) << 23);
      }
    }
    weights(s, f, lsv, first, open || (tile + 1) * kQ8Block > base + (int)((uint32_t)r0 * inv_g >> 16));
    if (!open) {
      uint32_t b[PARTS][NT][2];
#pragma unroll
      for (int part = 0; part < PARTS; ++part) split<__half>(s, b[part]);
      uint32_t v[4][D / 32];                               // tokens 2 tig, 2 tig + 1, + 8, + 9
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * tig + (i & 1) + 8 * (i >> 1);
        if (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(st + SLAB + slab_at<D>(r, gid));
          v[i][0] = x.x, v[i][1] = x.y, v[i][D / 32 - 2] = x.z, v[i][D / 32 - 1] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(st + SLAB + slab_at<D>(r, gid >> 1) + 8 * (gid & 1));
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
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
              mma16816(o[2 * x + y][t], a0, a1, a2, a3, b[part][t][0], b[part][t][1], __half());
        }
    } else {
      bad = __reduce_or_sync(~0u, bad);
      if (bad) {
        // NaN for the queries that see the token; 0 x NaN would reach the others, so its values go
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (bad >> (2 * tig + (i & 1) + 8 * (i >> 1)) & 1)
#pragma unroll
            for (int x = 0; x < KS / 4; ++x) vo[i][x] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((bad >> (gid + 8 * (e >> 1)) & 1) && first + gid + 8 * (e >> 1) < end_of(t, e & 1)) s[t][e] = NAN;
      }
      if (Pair16<T>::kWide)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][e] *= up;
#pragma unroll
      for (int part = 0; part < OPEN_PARTS; ++part) {
        uint32_t b[NT][2];
        split<T>(s, b);
#pragma unroll
        for (int x = 0; x < KS; ++x) {
          const uint32_t v0 = word(vo[0][x / 4], x % 4), v1 = word(vo[1][x / 4], x % 4);
          const uint32_t v2 = word(vo[2][x / 4], x % 4), v3 = word(vo[3][x / 4], x % 4);
          const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632);
          const uint32_t a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816(o[x][t], a0, a1, a2, a3, b[t][0], b[t][1], T());
        }
      }
    }
  }

  // The warp's results into its rows of the join area.
  __device__ __forceinline__ void leave(float* area) {
    constexpr int ROWS = Shape<D, NT>::ROWS, OROW = Shape<D, NT>::OROW;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float* p = area + (warp * ROWS + 8 * t + 2 * tig + j) * OROW;
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[t][j] += __shfl_xor_sync(~0u, l[t][j], d);
        if (gid == 0) p[D] = ml[t][j], p[D + 1] = dv[t][j], p[D + 2] = l[t][j];
#pragma unroll
        for (int m = 0; m < KS; m += 2)
          *reinterpret_cast<float4*>(p + D / 8 * gid + 2 * m) =
              make_float4(o[m][t][j], o[m][t][j + 2], o[m + 1][t][j], o[m + 1][t][j + 2]);
      }
  }
};

template <typename T, int FMT, int D, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NT)) q8_attend_kernel(const Q8AttendArgs a) {
  using S = Shape<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  float* area = reinterpret_cast<float*>(smem + S::RING);
  Walk* walks = reinterpret_cast<Walk*>(smem + S::RING + S::JOIN);
  uint8_t* qmem = smem + S::RING + S::JOIN + S::WALK;
  uint32_t* sums = reinterpret_cast<uint32_t*>(qmem + S::Q);
  const Plan plan{sums + 4, reinterpret_cast<int*>(sums + 4 + a.c.batch + 1)};
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join's blocks, as this grid leaves room
  const int groups = (a.n * a.G + S::ROWS - 1) / S::ROWS, subs = a.c.num_kv_heads * groups;
  plan_rows(a, subs, S::COST, plan, sums);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.c.batch; b += kThreads)
      if (!row_valid(a, a.lens[b], a.n_rows ? a.n_rows[b] : a.n)) atomicOr(a.c.status, kQ8StatusInvalid);
  const Runs runs(plan.pre[a.c.batch], gridDim.x);
  if (blockIdx.x >= runs.ctas) return;
  const uint32_t t0 = runs.start(blockIdx.x), t1 = runs.start(blockIdx.x + 1);
  // unit of the row -> kv head (its query group is what is left)
  auto head_of = [&](int sub) { return groups == 1 ? sub : sub / groups; };

  Pass<T, FMT, D, NT> ps;
  ps.lane = threadIdx.x % 32, ps.warp = threadIdx.x / 32;
  ps.gid = ps.lane / 4, ps.tig = ps.lane % 4;
  ps.qs = reinterpret_cast<uint2*>(qmem), ps.qup = reinterpret_cast<float*>(qmem + S::Q - S::ROWS * 4);
  ps.inv_g = (65536u + a.G - 1) / a.G;
  Walk *get = walks + 2 * ps.warp, *use = get + 1;
  *get = walk_first(plan, a.c.batch, subs, S::COST, t0, t1);
  __syncwarp();
  if (get->end <= get->begin) walk_next(get, plan, subs, S::COST);
  *use = *get;
  __syncwarp();

  // The warp's 16 tokens of the run's next whole block go to a stage of the warp's ring (open blocks are
  // read where they are used): 16-byte copies from kp, vp, and the two scales.
  const uint8_t *kp = nullptr, *vp = nullptr;
  const float* sp = nullptr;
  int more = 0;                                            // whole blocks to fetch from kp, vp on
  uint32_t dst[S::SLAB / 512];
#pragma unroll
  for (int i = 0; i < S::SLAB / 512; ++i) {
    const int x = i * 32 + ps.lane;
    dst[i] = slab_at<D>(x / (D / 16), x % (D / 16));
  }
  const uint32_t ring0 = smem_u32(smem) + ps.warp * kStages * S::STAGE;
  bool fresh = true;                                       // `get` is at a segment that kp, vp have not begun
  auto fetch = [&](int stage) {
    while (more == 0 && get->begin < get->end) {
      const bool first = fresh;
      if (!first) walk_next(get, plan, subs, S::COST);
      fresh = false;
      more = max(min(get->end, get->whole) - get->begin, 0);
      const int kvh = head_of(get->sub);
      const size_t unit = (size_t)get->row * a.c.num_kv_heads + kvh;
      const size_t at = (unit * a.c.capacity + (size_t)get->begin * kQ8Block + 16 * ps.warp) * D + 16 * ps.lane;
      kp = static_cast<const uint8_t*>(a.c.k_codes) + at;
      vp = static_cast<const uint8_t*>(a.c.v_codes) + at;
      sp = (ps.lane ? a.c.v_scales : a.c.k_scales) + unit * (a.c.capacity / kQ8Block) + get->begin;
      // What the pass reads outside the ring, into L2: behind the fetches in flight it would wait for them all.
      if (ps.lane < S::ROWS && !first)                     // (the first pass has its queries' loads behind it)
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          prefetch_l2(ps.q_row(a, get->row, kvh, (get->sub - kvh * groups) * S::ROWS + ps.lane) + 64 * i);
      const int cnt = plan.len[get->row] - get->whole * kQ8Block - 16 * ps.warp;
      if (get->end > get->whole && cnt > 0) {
        const size_t open = (unit * kQ8Ring + (get->whole & 1) * kQ8Block + 16 * ps.warp) * D;
        for (int i = ps.lane; i < min(cnt, 16) * (D / 64); i += 32) {
          prefetch_l2(static_cast<const T*>(a.c.k_recent) + open + 64 * i);
          prefetch_l2(static_cast<const T*>(a.c.v_recent) + open + 64 * i);
        }
      }
    }
    if (more > 0) {
      const uint32_t st = ring0 + stage * S::STAGE;
#pragma unroll
      for (int i = 0; i < S::SLAB / 512; ++i) {
        cp_async16(st + dst[i], kp + 512 * i);
        cp_async16(st + S::SLAB + dst[i], vp + 512 * i);
      }
      if (ps.lane < 2) cp_async4(st + 2 * S::SLAB + 4 * ps.lane, sp);
      kp += kQ8Block * D, vp += kQ8Block * D, ++sp;
      --more;
    }
    cp_commit();
  };

  // `lag` fetches run ahead before the first tile is used.
  int stage = 0, ahead = 0, lag = kStages - 1;
#pragma unroll 1
  while (use->begin < use->end) {
    const int row = use->row, kvh = head_of(use->sub), r0 = (use->sub - kvh * groups) * S::ROWS, len = plan.len[row];
    const int begin = use->begin, end = use->end, whole = use->whole;
    bool started = false;
    ps.load(a, row, kvh, r0);
#pragma unroll 1
    for (int tile = begin; tile < end;) {
      const bool open = tile >= whole;
      if (!open || lag > 0) {
        fetch(ahead);
        ahead = ahead + 1 == kStages ? 0 : ahead + 1;
        if (lag > 0) {
          --lag;
          continue;
        }
      }
      if (!started) ps.start(a, row, kvh, len), started = true;
      cp_wait<kStages - 1>();
      __syncwarp();
      ps.tile(a, smem + (ps.warp * kStages + stage) * S::STAGE, tile, open, row, kvh, len);
      __syncwarp();                                        // every lane has read before the stage is filled again
      if (!open) stage = stage + 1 == kStages ? 0 : stage + 1;
      ++tile;
    }
    ps.leave(area);
    __syncthreads();
    // all threads: the four warps' rows together, four dims of a row each
    const bool all = begin == 0 && end == use->tiles;
    // the run's second result where the unit begins inside it: of two units that a run has parts of, one does
    const uint32_t place0 = plan.pre[row] + (uint32_t)use->sub * (S::COST + use->tiles) + S::COST;
    float* part = reinterpret_cast<float*>(a.scratch) + ((size_t)blockIdx.x * 2 + (t0 < place0)) * S::ROWS * S::OROW;
    const int rows = min(S::ROWS, (a.n_rows ? a.n_rows[row] : a.n) * a.G - r0);
#pragma unroll 1
    for (int x = threadIdx.x; x < rows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), d = x % (D / 4) * 4;
      const float* p = area + r * S::OROW;
      float gl = kLowest, gv = -INFINITY, sum = 0.f;
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) gl = fmaxf(gl, p[w * S::ROWS * S::OROW + D]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        gv = fmaxf(gv, p[w * S::ROWS * S::OROW + D + 1] + (p[w * S::ROWS * S::OROW + D] - gl));
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* pw = p + w * S::ROWS * S::OROW;
        const float down = pw[D] - gl;
        sum += pw[D + 2] * ex2(down);
        const float c = ex2(pw[D + 1] + down - gv);
        const float4 v = *reinterpret_cast<const float4*>(pw + d);
        t.x += v.x * c, t.y += v.y * c, t.z += v.z * c, t.w += v.w * c;
      }
      if (all) {
        const int i = (int)((uint32_t)(r0 + r) * ps.inv_g >> 16), h = kvh * a.G + (r0 + r) - i * a.G;
        T* out = static_cast<T*>(a.out) + (((size_t)row * a.n + i) * a.Hq + h) * D + d;
        const Factors c(gv, sum, ps.base + i > 0);
        *reinterpret_cast<uint2*>(out) = make_uint2(pack16<T>(c(t.x), c(t.y)), pack16<T>(c(t.z), c(t.w)));
      } else {
        *reinterpret_cast<float4*>(part + r * S::OROW + d) = t;
        if (d == 0) *reinterpret_cast<float4*>(part + r * S::OROW + D) = make_float4(gl, gv, sum, 0.f);
      }
    }
    walk_next(use, plan, subs, S::COST);
    __syncthreads();
  }
}

// Joins the partial results of units that several CTAs share, WPR warps per
// (unit, query row), and writes what no CTA had work for: zeros for rows
// without tokens, NaN for rows whose length is refused.  It is bound by the
// latency of its loads: a row's warps take the results in turn, a warp 32 of
// them at a time, each lane first one result's references and sum, then all
// lanes D / 32 dims of every result, the loads of eight together.
template <typename T, int D, int NT, int WPR>
__global__ void __launch_bounds__(kThreads) q8_join_kernel(const Q8AttendArgs a, uint32_t grid) {
  using S = Shape<D, NT>;
  constexpr int E = D / 32;
  extern __shared__ uint32_t pre[];
  const Plan plan{pre, reinterpret_cast<int*>(pre + a.c.batch + 1)};
  __shared__ uint32_t sums[kWarps];
  __shared__ float wm[kWarps][3], wo[kWarps][D];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, part_of = warp % WPR;
  const int R = a.n * a.G, groups = (R + S::ROWS - 1) / S::ROWS, subs = a.c.num_kv_heads * groups;
  const int ur = (int)blockIdx.x * (kWarps / WPR) + warp / WPR;   // query row among the batch row's units
  const int row = blockIdx.y, kvh = ur / R, r = ur % R, i = r / a.G;
  plan_rows(a, subs, S::COST, plan, sums);
  const int len = a.lens[row], nr = a.n_rows ? a.n_rows[row] : a.n;
  const bool valid = row_valid(a, len, nr);
  const Runs runs(plan.pre[a.c.batch], grid);
  const uint32_t unit = S::COST + (len + kQ8Block - 1) / kQ8Block;
  const uint32_t first = plan.pre[row] + (uint32_t)(kvh * groups + r / S::ROWS) * unit + S::COST;
  uint32_t c0 = 0, c1 = 0;
  if (valid && len > 0 && nr > 0 && kvh < a.c.num_kv_heads) c0 = runs.of(first), c1 = runs.of(first + unit - S::COST - 1);
  // CTA c's first result, or its second where the unit begins inside its run
  const uint32_t slot0 = runs.start(c0) < first;
  wait_for_stream();                                       // until here nothing of the attention kernel is read
  if (kvh >= a.c.num_kv_heads || (valid && i >= nr)) return;      // all warps of a row alike
  T* out = static_cast<T*>(a.out) + (((size_t)row * a.n + i) * a.Hq + kvh * a.G + r % a.G) * D;
  if (!valid || len == 0) {
    for (int d = part_of * 32 + lane; d < D; d += 32 * WPR) out[d] = valid ? (T)0.f : (T)__uint_as_float(0x7fffffffu);
    return;
  }
  if (c0 == c1) return;
  const bool sees = len - nr + 1 + i > 0;
  const float* part = reinterpret_cast<const float*>(a.scratch) + (size_t)(r % S::ROWS) * S::OROW;
  float gl = kLowest, gv = -INFINITY, sum = 0.f, o[E];      // gv relative to gl
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (uint32_t b = c0 + part_of; b <= c1; b += 32 * WPR) {
    const uint32_t c = b + WPR * lane;                     // this lane's CTA
    const int n = (int)min(32u, (c1 - b) / WPR + 1);
    float ml = kLowest, dv = -INFINITY, l = 0.f;
    if (lane < n) {
      const float4 x = *reinterpret_cast<const float4*>(part + (size_t)(c * 2 + (c == c0 ? slot0 : 0)) * S::ROWS * S::OROW + D);
      ml = x.x, dv = x.y, l = x.z;
    }
    float nl = fmaxf(gl, ml);
#pragma unroll
    for (int d = 16; d; d /= 2) nl = fmaxf(nl, __shfl_xor_sync(~0u, nl, d));
    l *= ex2(ml - nl);
    gv += gl - nl, dv += ml - nl;
    float nv = fmaxf(gv, dv);
#pragma unroll
    for (int d = 16; d; d /= 2) l += __shfl_xor_sync(~0u, l, d), nv = fmaxf(nv, __shfl_xor_sync(~0u, nv, d));
    sum = sum * ex2(gl - nl) + l;
    const float keep = ex2(gv - nv), w = ex2(dv - nv);
    gl = nl, gv = nv;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
    for (int x0 = 0; x0 < n; x0 += 8) {
      float p[8][E];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint32_t cx = min(b + WPR * (x0 + x), c1 - (c1 - b) % WPR);
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
  if (WPR == 1) {
    const Factors c(gv, sum, sees);
#pragma unroll
    for (int e = 0; e < E; e += 2) reinterpret_cast<uint32_t*>(out)[(E * lane + e) / 2] = pack16<T>(c(o[e]), c(o[e + 1]));
    return;
  }
  if (lane == 0) wm[warp][0] = gl, wm[warp][1] = gv, wm[warp][2] = sum;
#pragma unroll
  for (int e = 0; e < E; ++e) wo[warp][E * lane + e] = o[e];
  __syncthreads();                                         // WPR is kWarps: one row a block
  if (threadIdx.x >= D) return;
  gl = kLowest, gv = -INFINITY, sum = 0.f;
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) gl = fmaxf(gl, wm[w][0]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) gv = fmaxf(gv, wm[w][1] + (wm[w][0] - gl));
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float down = wm[w][0] - gl;
    sum += wm[w][2] * ex2(down);
    t += wo[w][threadIdx.x] * ex2(wm[w][1] + down - gv);
  }
  out[threadIdx.x] = (T)Factors(gv, sum, sees)(t);
}

// A unit's query rows are cut into passes of up to 24, as even as eights allow.  24 rows are what the registers hold
// (251 to 255 of them, up to 28 bytes spilled for bf16 of d = 128); passes of up to 32 spill more.  16 rows of 4096
// tokens (32 / 8 heads of 128): 8 queries take 77.8 us (int8, fp16) and 70.0 (e4m3, bf16) so, 80.1 and 112 with 32 rows;
// 64 queries 456 us, 521 with 32 and 553 with 16.
int pick_nt(int rows) {
  const int eights = (rows + 7) / 8, passes = (eights + 2) / 3;
  return (eights + passes - 1) / passes;
}

int groups_of(const tq_q8_cache& c, int Hq, int n) {
  const int rows = n * (Hq / c.num_kv_heads), nt = pick_nt(rows);
  return (rows + 8 * nt - 1) / (8 * nt);
}

uint32_t grid_of(const tq_q8_cache& c, int Hq, int n, int num_sms) {
  const int nt = pick_nt(n * (Hq / c.num_kv_heads));
  const int64_t places = (int64_t)c.batch * c.num_kv_heads * groups_of(c, Hq, n) * (c.capacity / kQ8Block + unit_cost(nt));
  const int64_t most = (int64_t)num_sms * ctas_per_sm(c.head_dim, nt);
  return (uint32_t)(places < most ? places : most);
}

template <typename T, int FMT, int D, int NT>
cudaError_t launch(const Q8AttendArgs& a, uint32_t grid, cudaStream_t s) {
  auto kernel = q8_attend_kernel<T, FMT, D, NT>;
  // once per device: the shared memory that the largest batch takes
  static std::atomic<uint64_t> set{0};
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev % 64);
  if (!(set.load(std::memory_order_relaxed) & bit) || dev >= 64) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D, NT>(kQ8MaxRows));
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  e = launch_dependent(kernel, dim3(grid), kThreads, smem_bytes<D, NT>(a.c.batch), s, a);
  if (e != cudaSuccess) return e;
  // A warp per query row where units have some 16 partial results at most, else four.  One and four warps: 5 queries in
  // 16 ragged rows 27.9 and 32.1 us, 256 rows of 512 tokens 67.7 and 80.0, 16 rows of 4096 33.8 and 34.3; 4 rows of 8192
  // 21.8 and 21.5; one row of 8192 14.9 and 11.6, of 131583 59.5 and 55.9.
  const int rows = a.c.num_kv_heads * a.n * a.G, units = a.c.batch * a.c.num_kv_heads * groups_of(a.c, a.Hq, a.n);
  const int join_smem = 4 * (2 * a.c.batch + 1);
  if ((int64_t)units * 16 >= grid)
    return launch_dependent(q8_join_kernel<T, D, NT, 1>, dim3((unsigned)((rows + kWarps - 1) / kWarps), (unsigned)a.c.batch),
                            kThreads, join_smem, s, a, grid);
  return launch_dependent(q8_join_kernel<T, D, NT, kWarps>, dim3((unsigned)rows, (unsigned)a.c.batch), kThreads, join_smem,
                          s, a, grid);
}

template <typename T, int FMT, int D>
cudaError_t pick(const Q8AttendArgs& a, uint32_t grid, cudaStream_t s) {
  switch (pick_nt(a.n * a.G)) {
    case 1: return launch<T, FMT, D, 1>(a, grid, s);
    case 2: return launch<T, FMT, D, 2>(a, grid, s);
    default: return launch<T, FMT, D, 3>(a, grid, s);
  }
}

template <typename T, int FMT>
cudaError_t pick(const Q8AttendArgs& a, uint32_t grid, cudaStream_t s) {
  return a.c.head_dim == 64 ? pick<T, FMT, 64>(a, grid, s) : pick<T, FMT, 128>(a, grid, s);
}

}  // namespace

size_t q8_attend_scratch(const tq_q8_cache& c, int Hq, int n, int num_sms) {
  const size_t rows = 8 * (size_t)pick_nt(n * (Hq / c.num_kv_heads));
  return ((size_t)grid_of(c, Hq, n, num_sms) * 2 * rows * (c.head_dim + 4) * 4 + 255) / 256 * 256;
}

cudaError_t launch_q8_attend(const Q8AttendArgs& a, int num_sms, cudaStream_t s) {
  const uint32_t grid = grid_of(a.c, a.Hq, a.n, num_sms);
  // A call's two launches follow one another: between them another thread's call on the stream would overwrite
  // the partial results, where both take the same scratch (others need not wait).
  static std::mutex launches[64];
  const std::lock_guard<std::mutex> hold(launches[(uintptr_t)a.scratch / 256 % 64]);
  const bool i8 = a.c.format == TQ_Q8_INT8;
  if (a.c.dtype == TQ_DTYPE_FP16)
    return i8 ? pick<__half, TQ_Q8_INT8>(a, grid, s) : pick<__half, TQ_Q8_E4M3>(a, grid, s);
  return i8 ? pick<__nv_bfloat16, TQ_Q8_INT8>(a, grid, s) : pick<__nv_bfloat16, TQ_Q8_E4M3>(a, grid, s);
}

}  // namespace tq
