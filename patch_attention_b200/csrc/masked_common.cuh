// masked_common.cuh -- what the forward and backward kernels of masked attention share: which
// keys a query row sees, how its scores are capped and biased, and small warp helpers.
#pragma once

#include <cuda_bf16.h>

#include "pf_internal.h"
#include "sm100_ptx.cuh"

namespace pf {
namespace masked {

using namespace ptx;

constexpr int kRows = 128;              // rows of a query tile and of a key tile
constexpr int kChunkBytes = 128 * 128;  // 128 rows x 64 bf16 columns (one 128-byte swizzle span)
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum : unsigned { kWdLoad = 1u, kWdMma = 2u, kWdSoftmax = 4u, kWdEpilogue = 8u, kWdScrub = 32u };

template <int D>
struct Dims {
  static constexpr int kChunks = (D + 63) / 64;     // 64-column chunks per row
  static constexpr int kMmaN = (D + 15) / 16 * 16;  // head_dim padded to 16 (72 -> 80)
  static constexpr int kTileBytes = kChunks * kChunkBytes;
};

// Whether the phase of `bar` with the given parity has completed; does not wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// One lane of a converged warp.  Unlike a test of the lane number it tells the compiler that the
// code behind it is one thread's, so that the operands of TMA and MMA instructions are computed
// in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void raise_abort(volatile int* abort, unsigned* watchdog, unsigned code) {
  *abort = 1;
  atomicOr(watchdog, code);
}

// Start-address field of a matrix descriptor.  In a cluster a shared address carries the CTA's
// rank above its offset, which must not reach the descriptor's next field.
__device__ __forceinline__ uint32_t desc_start(uint32_t addr) { return (addr >> 4) & 0x3FFFu; }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);  // .x (low half) = lo
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Maximum of three that is NaN if any of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Maximum of 64 values: 8 independent chains, then a tree.  A NaN among them wins, so that a
// row with a NaN score becomes NaN as a whole.
__device__ __forceinline__ float row_max64(const uint32_t (&s)[64]) {
  float mv[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) mv[k] = __uint_as_float(s[k]);
#pragma unroll
  for (int k = 8; k < 56; k += 2)
    mv[(k >> 1) & 7] = max3_nan(mv[(k >> 1) & 7], __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
#pragma unroll
  for (int k = 0; k < 4; ++k) mv[k] = max3_nan(mv[k], mv[k + 4], __uint_as_float(s[56 + k]));
  mv[0] = max3_nan(mv[0], __uint_as_float(s[60]), __uint_as_float(s[61]));
  mv[1] = max3_nan(mv[1], __uint_as_float(s[62]), __uint_as_float(s[63]));
  return max3_nan(mv[0], mv[1], max3_nan(mv[2], mv[3], mv[3]));
}

// Barrier among `count` threads that ANDs a predicate over them.
__device__ __forceinline__ bool named_bar_and(int id, int count, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

// ------------------------------------------------------------------ masks

// The last key that a query row may see by position (its own position under the causal mask,
// or the prefix where that reaches further; a prefix below zero is none); -1: no key.  Rows stand
// at query + n_k - n_q.
__device__ __forceinline__ int key_limit(const MaskParams& m, int query, int prefix) {
  const int last = m.n_k - 1;
  if (!m.causal) return last;
  const int at = query + (m.n_k - m.n_q);
  return max(min(max(at, max(prefix, 0) - 1), last), -1);
}

// Bit k set: key base + k is at most `limit` (64 keys).
__device__ __forceinline__ uint64_t limit_bits(int limit, int base) {
  const int n = limit - base + 1;  // keys of the 64 that count
  return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
}

// Bit k set: element k of the 64 ids held by the warp (id0: k = lane, id1: k = lane + 32) equals
// this lane's `mine` and is a document (>= 0).  One round of votes per distinct id in the warp:
// neighbouring rows nearly always share one.
__device__ __forceinline__ uint64_t document_bits(int mine, int id0, int id1) {
  uint64_t bits = 0;
  unsigned todo = __ballot_sync(0xffffffffu, mine >= 0);
  while (todo != 0) {
    const int id = __shfl_sync(0xffffffffu, mine, __ffs(todo) - 1);
    const uint64_t hit = static_cast<uint64_t>(__ballot_sync(0xffffffffu, id0 == id)) |
                         static_cast<uint64_t>(__ballot_sync(0xffffffffu, id1 == id)) << 32;
    if (mine == id) bits = hit;
    todo &= ~__ballot_sync(0xffffffffu, mine == id);
  }
  return bits;
}

// Smallest and largest document of 1 to 128 ids (negative ones left out), and whether any id was
// negative.  Whole-warp; hi < 0: no document.  The ids are loaded first, so that several ranges
// can be in flight; past the end the last id is taken again.
struct DocRange {
  unsigned lo;
  int hi;
  bool gaps;
};
struct DocIds {
  int id[4];
  __device__ __forceinline__ void load(const int* ids, int count, int lane) {
#pragma unroll
    for (int x = 0; x < 4; ++x) id[x] = __ldg(ids + min(x * 32 + lane, count - 1));
  }
  __device__ __forceinline__ DocRange range() const {
    // as unsigned numbers the negative ids are the largest
    const unsigned u[4] = {static_cast<unsigned>(id[0]), static_cast<unsigned>(id[1]), static_cast<unsigned>(id[2]),
                           static_cast<unsigned>(id[3])};
    DocRange r;
    r.lo = __reduce_min_sync(0xffffffffu, min(min(u[0], u[1]), min(u[2], u[3])));
    r.hi = __reduce_max_sync(0xffffffffu, max(max(id[0], id[1]), max(id[2], id[3])));
    r.gaps = __any_sync(0xffffffffu, (id[0] | id[1] | id[2] | id[3]) < 0);
    return r;
  }
};
__device__ __forceinline__ DocRange doc_range(const int* ids, int count, int lane) {
  DocIds d;
  d.load(ids, count, lane);
  return d.range();
}

// Whether a tile of rows and a tile of keys can hide something from each other:
// 0 no pair in common, 1 some pairs, 2 every pair.
__device__ __forceinline__ int doc_class(const DocRange& a, const DocRange& b) {
  if (a.hi < 0 || b.hi < 0 || static_cast<unsigned>(a.hi) < b.lo || static_cast<unsigned>(b.hi) < a.lo) return 0;
  return a.lo == b.lo && a.hi == b.hi && a.lo == static_cast<unsigned>(a.hi) && !a.gaps && !b.gaps ? 2 : 1;
}

// Classes of tiles [j0, j1) of ids (`count` of them from the start) against NQ ranges, 2 bits each,
// into cls[j - j0]; the first and the last tile that any of them sees into range[0], range[1]
// (shared; range[0] > range[1]: none).  By all warps of the block, followed by a barrier.  All of a
// warp's loads are in flight at once: a pass over the ids of every tile costs every CTA about
// one memory latency.
template <int NQ, int WARPS>
__device__ __forceinline__ void class_tiles(const int* ids, int count, int j0, int j1, const DocRange (&q)[NQ],
                                            uint8_t* cls, int* range, int warp, int lane) {
  constexpr int kAtOnce = 8;
  int first = INT32_MAX, last = -1;
  for (int j = j0 + warp; j < j1; j += WARPS * kAtOnce) {
    DocIds d[kAtOnce];
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      const int jx = min(j + x * WARPS, j1 - 1);
      d[x].load(ids + static_cast<long long>(jx) * kRows, min(kRows, count - jx * kRows), lane);
    }
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      const int jx = j + x * WARPS;
      const DocRange r = d[x].range();
      int c = doc_class(q[0], r);
      if (NQ == 2) c |= doc_class(q[NQ - 1], r) << 2;
      if (jx < j1) {
        if (lane == 0) cls[jx - j0] = static_cast<uint8_t>(c);
        if (c != 0) {
          first = min(first, jx);
          last = jx;
        }
      }
    }
  }
  if (lane == 0 && last >= 0) {
    atomicMin(range, first);
    atomicMax(range + 1, last);
  }
}

// ------------------------------------------------------------------ scores

// A raw product q.k to a score in log2 units: capped, then lowered by the distance.
//   cap:  cap tanh(y), y = scale qk / cap.  Where |y| is at most 1/2 (scores up to half the cap),
//         tanh comes from y (a0 + a1 y^2 + a2 y^4 + a3 y^6), fitted for least relative error
//         (5.6e-7, Lawson's iteratively reweighted least squares), on pairs on the FMA pipe; else
//         from 1 - 2 / (1 + exp(2 y)) on the special-function unit, whose absolute error is
//         about 2^-22.  So a capped score is off by about 2^-20 of itself, however large the cap
//         (the fit for least absolute error, 1.3e-7, was off by 2.3e-6 of a score far below the cap).
//         The form goes by the element alone: a warp only skips the second one where none of its
//         elements needs it, so a row's bits depend neither on its neighbours nor on what hidden
//         keys and unwritten rows hold.
//   bias: -slope |position - key|.  With e = (first column's distance, signed), the 64 columns
//         are at |e + k|; where every row of the warp lies on one side of them that is linear in
//         k, and the row's part goes into the exponential's reference.
// (One special-function result per element for the softmax and two for the exact tanh: they
// bound a capped tile of 128 x 128 at three times 1024 cycles, the polynomial at about 1100.)
constexpr float kTanh0 = 0.999999464f, kTanh1 = -0.333263189f, kTanh2 = 0.131903037f, kTanh3 = -0.044402387f;

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Largest |s| of N values (a NaN wins).
template <int N>
__device__ __forceinline__ float abs_max(const uint32_t (&s)[N]) {
  float mv[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < N; k += 2)
    asm("max.NaN.abs.f32 %0, %1, %2, %3;"
        : "=f"(mv[(k >> 1) & 3])
        : "f"(mv[(k >> 1) & 3]), "f"(__uint_as_float(s[k])), "f"(__uint_as_float(s[k + 1])));
  return max3_nan(mv[0], mv[1], max3_nan(mv[2], mv[3], mv[3]));
}

// Raw products to factor tanh(scale qk / cap), in place.  The polynomial's steps are the same, rounding for
// rounding, on pairs and one by one; one by one where both forms are needed (2 x 16 heads x 4216 of 72
// with cap, bias and prefix, scores beyond half the cap in most warps: 389 us, on pairs 430).  The
// factor's products stand in both branches: shared, they cost the first 5% (283 for 271 us).
template <int N>
__device__ __forceinline__ void tanh_scores(uint32_t (&s)[N], const MaskParams& m, float factor) {
  if (__all_sync(0xffffffffu, abs_max<N>(s) <= m.cap_half)) {
    const float t0 = kTanh0 * factor, t1 = kTanh1 * factor, t2 = kTanh2 * factor, t3 = kTanh3 * factor;
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const float2 y = __fmul2_rn(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), both(m.cap_in));
      const float2 z = __fmul2_rn(y, y);
      float2 p = __ffma2_rn(z, both(t3), both(t2));
      p = __ffma2_rn(p, z, both(t1));
      p = __fmul2_rn(__ffma2_rn(p, z, both(t0)), y);
      s[k] = __float_as_uint(p.x);
      s[k + 1] = __float_as_uint(p.y);
    }
  } else {
    const float t0 = kTanh0 * factor, t1 = kTanh1 * factor, t2 = kTanh2 * factor, t3 = kTanh3 * factor;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float raw = __uint_as_float(s[k]);
      const float y = __fmul_rn(raw, m.cap_in), z = __fmul_rn(y, y);
      const float p = __fmul_rn(__fmaf_rn(__fmaf_rn(__fmaf_rn(z, t3, t2), z, t1), z, t0), y);
      const float e = fmaf(-2.f * factor, rcp(ex2(raw * (2.f * kLog2e * m.cap_in)) + 1.f), factor);
      s[k] = __float_as_uint(fabsf(raw) <= m.cap_half ? p : e);
    }
  }
}

// Adds the bias to N scores: the columns' distances are |e + k|.  Returns what is still to be
// added to every score of the row (0 where a row lies inside the columns), in log2 units; the
// scores are in units of `unit` of those.
template <int N>
__device__ __forceinline__ float add_bias(uint32_t (&s)[N], float slope_log2, float unit, int e) {
  const float slope = slope_log2 / unit;
  const bool right = __all_sync(0xffffffffu, e >= 0), left = __all_sync(0xffffffffu, e + N - 1 <= 0);
  if (right || left) {
    const float b = right ? -slope : slope;
#pragma unroll
    for (int k = 0; k < N; ++k)  // one FMA with an immediate; on pairs the columns would be moved to registers first
      s[k] = __float_as_uint(fmaf(b, static_cast<float>(k), __uint_as_float(s[k])));
    return (right ? -slope_log2 : slope_log2) * static_cast<float>(e);
  }
#pragma unroll
  for (int k = 0; k < N; ++k)
    s[k] = __float_as_uint(fmaf(-slope, fabsf(static_cast<float>(e) + static_cast<float>(k)), __uint_as_float(s[k])));
  return 0.f;
}

// factor * s, on pairs, in place.
template <int N>
__device__ __forceinline__ void scale_scores(uint32_t (&s)[N], float factor) {
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    const float2 v = __fmul2_rn(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), both(factor));
    s[k] = __float_as_uint(v.x);
    s[k + 1] = __float_as_uint(v.y);
  }
}

}  // namespace masked
}  // namespace pf
