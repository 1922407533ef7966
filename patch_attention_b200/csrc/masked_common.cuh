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
// or the prefix where that reaches further); -1: none.  Rows stand at query + n_k - n_q.
__device__ __forceinline__ int key_limit(const MaskParams& m, int query, int prefix) {
  const int last = m.n_k - 1;
  if (!m.causal) return last;
  const int at = query + (m.n_k - m.n_q);
  return max(min(max(at, prefix - 1), last), -1);
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

// Smallest and largest document of a run of ids (negative ones left out), and whether any
// id was negative.  Whole-warp; lo > hi: no document.
struct DocRange {
  int lo, hi;
  bool gaps;
};
__device__ __forceinline__ DocRange doc_range(const int* ids, int first, int count, int lane) {
  int lo = INT32_MAX, hi = -1;
  bool gaps = false;
  for (int i = lane; i < count; i += 32) {
    const int id = __ldg(ids + first + i);
    if (id < 0) {
      gaps = true;
    } else {
      lo = min(lo, id);
      hi = max(hi, id);
    }
  }
  DocRange r;
  r.lo = __reduce_min_sync(0xffffffffu, lo);
  r.hi = __reduce_max_sync(0xffffffffu, hi);
  r.gaps = __any_sync(0xffffffffu, gaps);
  return r;
}

// Whether a tile of rows and a tile of keys can hide something from each other:
// 0 no pair in common, 1 some pairs, 2 every pair.
__device__ __forceinline__ int doc_class(const DocRange& a, const DocRange& b) {
  if (a.lo > a.hi || b.lo > b.hi || a.hi < b.lo || b.hi < a.lo) return 0;
  return a.lo == a.hi && b.lo == b.hi && a.lo == b.lo && !a.gaps && !b.gaps ? 2 : 1;
}

// ------------------------------------------------------------------ scores

// A raw product q.k to a score in log2 units: capped, then lowered by the distance.
//   cap:  cap tanh(scale qk / cap) = cap - 2 cap / (1 + exp(2 scale qk / cap)), whose absolute
//         error (about 2^-22 cap) is what the exponential afterwards feels
//   bias: -slope |position - key|
__device__ __forceinline__ float cap_score(float s, const MaskParams& m) {
  const float e = ex2(s * m.cap_in);
  return fmaf(-2.f * m.cap_log2, rcp(e + 1.f), m.cap_log2);
}

}  // namespace masked
}  // namespace pf
