// layernorm.cu -- layer normalisation with an affine or a per-group modulation, forward and
// backward.
//
//   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), x^ = (x - m) r
//   y = x^ (w_g + w0) + b_g              g: the row's group (its sample, or the one affine)
//   a = dy (w_g + w0);  dx = r (a - mean(a) - x^ mean(a x^))
//   dw_g = sum over the group's rows of dy x^,  db_g = sum of dy
//
// Both directions are HBM bound: forward reads x and writes y, backward reads x and dy and
// writes dx.  A row of up to 2048 elements belongs to one warp, so that it needs no barrier and
// its fixed cost (two shuffle trees) is spread over up to 64 elements per lane; wider rows belong
// to a block of up to 16 warps.  Where a warp has several rows of a group, the group's
// parameters are converted to fp32 once, into shared memory.  The forward pass reads a row into
// registers once.  The backward pass keeps the weight-gradient sums of a lane's columns in registers, and the
// next row of x and dy is copied into shared memory (each lane its own elements, so no barrier)
// while the current one is worked on.  Arithmetic is on pairs (two fp32 lanes per instruction):
// element by element, instruction issue was the bound (25 instructions per element forward),
// as it was with bounds checks on every access: the elements per lane are the least multiple of 8
// that covers the row, so only a lane's last 8 are checked.
// The variance is taken around means: a warp's around its own; in wider rows the warps' (mean, sum
// of squares) are then combined.
//
// Measured on a B200 (a copy of the same tensor in brackets): 2 x 16384 x 1536 bf16 modulated,
// forward 38 us, 5.2 TB/s (35 us); 4 x 4096 x 1152 bf16 forward 15.0 us (12.6), backward 31.5 us;
// fp32 8192 x 1152 14.9 and 29.3 us, 8191 x 1153, whose rows start on no 16-byte boundary, 19.0 and
// 53 us (elements are copied to shared memory one by one, and the row's chain of them is the bound).
// The backward pass holds two rows' sums per column, so few warps fit an SM: 2 x 16384 x 1536 60 us.
//
// The backward pass writes one fp32 partial row of the weight gradients per block; a second
// kernel adds the partials in a fixed order, so equal inputs give equal bits.

#include <mutex>

#include "block_ops.cuh"

namespace pf {
namespace {

using namespace blk;

struct LnParams {
  const void* x;
  const void* dy;      // backward
  void* y;             // forward: y; backward: dx
  const void* weight;  // may be null: a factor of 1
  const void* bias;    // may be null
  float* mean;         // forward: may be null; backward: inputs
  float* rstd;
  float* part;         // backward: [group][part][2][channels] partial sums, or null
  long long rows, rows_per_group, weight_stride, bias_stride;
  int channels, parts;
  int warps;           // warps per row
  int stages;          // backward: rows of shared memory per warp, 2 (or 1 where 2 do not fit)
  int wide;            // the parameters are fp32 (else the type of x)
  float w0, eps;
};

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <typename T>
__device__ __forceinline__ float2 pair_of(const T* v) {
  return make_float2(to_f<T>(v[0]), to_f<T>(v[1]));
}
template <>
__device__ __forceinline__ float2 pair_of<__nv_bfloat16>(const __nv_bfloat16* v) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(v);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 pair_of<__half>(const __half* v) {
  return __half22float2(*reinterpret_cast<const __half2*>(v));
}
template <typename T>
__device__ __forceinline__ void put_pair(T* to, float2 f) {
  to[0] = from_f<T>(f.x);
  to[1] = from_f<T>(f.y);
}
template <>
__device__ __forceinline__ void put_pair<__nv_bfloat16>(__nv_bfloat16* to, float2 f) {
  *reinterpret_cast<__nv_bfloat162*>(to) = __floats2bfloat162_rn(f.x, f.y);
}
template <>
__device__ __forceinline__ void put_pair<__half>(__half* to, float2 f) {
  *reinterpret_cast<__half2*>(to) = __floats2half2_rn(f.x, f.y);
}

// A lane's columns: unit i (VEC consecutive elements) of EPT / VEC starts at column(i).
template <int VEC>
struct Place {
  int first;
  __device__ __forceinline__ int column(int i) const { return first + i * 32 * VEC; }
};

template <typename T, int VEC>
using Unit = Vec<T, VEC>;

// How the elements of a lane are walked: K steps, each of P pairs -- one unit, or for VEC = 1 the
// two units 2k and 2k + 1.
template <int VEC, int EPT>
struct Walk {
  static constexpr int P = VEC == 1 ? 1 : VEC / 2;
  static constexpr int K = EPT / 2 / P;
  static constexpr int kPerStep = VEC == 1 ? 2 : 1;
  // Whether unit i may lie past the row's end; CHECK: every unit may.
  template <bool CHECK>
  static __device__ __forceinline__ bool in(int i, const Place<VEC>& at, int n) {
    return (!CHECK && (i + 1) * VEC <= EPT - 8) || at.column(i) < n;
  }
};

// The lane's parameters of step k as pairs, from global memory.
template <typename T, int VEC, int N>
__device__ __forceinline__ void direct_params(float2 (&f)[N], const void* base, long long row, float plus, float none,
                                              int k, const LnParams& p, const Place<VEC>& at) {
  if constexpr (VEC == 1) {
    float v[2] = {none, none};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = at.column(2 * k + u);
      if (base != nullptr && c < p.channels) {
        float x[1];
        load_param<T, 1>(base, row + c, p.wide, x);
        v[u] = x[0] + plus;
      }
    }
    f[0] = make_float2(v[0], v[1]);
  } else if (base == nullptr) {
#pragma unroll
    for (int u = 0; u < VEC / 2; ++u) f[u] = both(none);
  } else if (p.wide) {
    float v[VEC];
    load_param<T, VEC>(base, row + at.column(k), true, v);
#pragma unroll
    for (int u = 0; u < VEC / 2; ++u) f[u] = add2(make_float2(v[2 * u], v[2 * u + 1]), both(plus));
  } else {
    const Unit<T, VEC> v = load_vec<T, VEC>(static_cast<const T*>(base) + row + at.column(k));
#pragma unroll
    for (int u = 0; u < VEC / 2; ++u) f[u] = add2(pair_of<T>(v.v + 2 * u), both(plus));
  }
}

// A group's parameters in shared memory as fp32, so laid out that the lanes of a warp read
// their 16-byte quarters side by side: [unit][quad of the unit][lane][4] (VEC = 1: in order).
template <typename T, int VEC>
__device__ __forceinline__ void stage_params(float* to, const void* base, long long row, float plus, float none,
                                             const LnParams& p) {
#pragma unroll 2
  for (int u = threadIdx.x; u * VEC < p.channels; u += blockDim.x) {
    float v[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = none;
    if (base != nullptr) {
      load_param<T, VEC>(base, row + u * VEC, p.wide, v);
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[k] += plus;
    }
#pragma unroll
    for (int k = 0; k < VEC; k += 4) {
      if constexpr (VEC == 1)
        to[u] = v[0];
      else
        *reinterpret_cast<float4*>(to + ((u / 32 * (VEC / 4) + k / 4) * 32 + u % 32) * 4) =
            make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
    }
  }
}
// A group's 16-bit parameters in shared memory, in order; 0 where there are none.
template <typename T, int VEC>
__device__ __forceinline__ void copy_params(T* to, const void* base, long long row, int channels) {
#pragma unroll 2
  for (int c = threadIdx.x * VEC; c < channels; c += blockDim.x * VEC) {
    Unit<T, VEC> v = {};
    if (base != nullptr) v = load_vec<T, VEC>(static_cast<const T*>(base) + row + c);
    *reinterpret_cast<Unit<T, VEC>*>(to + c) = v;
  }
}
template <int VEC, int N>
__device__ __forceinline__ void staged_params(float2 (&f)[N], const float* from, int k, int lane, const Place<VEC>& at,
                                              int n) {
  if constexpr (VEC == 1) {
    f[0].x = from[at.column(2 * k)];
    f[0].y = at.column(2 * k + 1) < n ? from[at.column(2 * k + 1)] : 0.f;
  } else {
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) {
      const float4 v = *reinterpret_cast<const float4*>(from + ((k * (VEC / 4) + q) * 32 + lane) * 4);
      f[2 * q] = make_float2(v.x, v.y);
      f[2 * q + 1] = make_float2(v.z, v.w);
    }
  }
}
// Two values summed over the row's warps.  Consecutive calls alternate between two buffers, so
// one barrier each is enough.
struct Exchange {
  float2 (*slots)[16];  // [parity][warp]
  int parity = 0;
  __device__ __forceinline__ const float2* publish(float2 v, int warp, int lane) {
    float2* mine = slots[parity];
    parity ^= 1;
    if (lane == 0) mine[warp] = v;
    __syncthreads();
    return mine;
  }
};

// KIND 0: a warp takes one row, parameters from global memory (few rows: least latency).
// KIND 1: a block of four warps walks rows of one group, its parameters in shared memory.
// KIND 2: a block of up to 16 warps takes one row.
// KIND 3: as 1, with 16-bit parameters left as they are in shared memory: as fp32 their reads took
//         70% of L1's rate (2 x 16384 x 1536 modulated: 46.0 us, as they are 44.5).
template <typename T, int VEC, int EPT, int KIND>
__global__ void __launch_bounds__(KIND == 2 ? 512 : 128) ln_fwd_kernel(const __grid_constant__ LnParams p) {
  using Wk = Walk<VEC, EPT>;
  constexpr bool WIDE = KIND == 2, WALK = KIND == 1 || KIND == 3;
  __shared__ float2 slots[2][16];
  __shared__ __align__(16) float staged[KIND == 1 ? 2 * 32 * EPT : KIND == 3 ? 32 * EPT : 4];
  T* narrow = reinterpret_cast<T*>(staged);  // KIND 3: weights, then biases
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = p.channels;
  long long row, end, g;
  int step = 1;
  if constexpr (WALK) {
    g = blockIdx.x / p.parts;
    const int part = static_cast<int>(blockIdx.x % p.parts);
    row = g * p.rows_per_group + p.rows_per_group * part / p.parts + warp;
    end = g * p.rows_per_group + p.rows_per_group * (part + 1) / p.parts;
    step = 4;
  } else {
    row = KIND == 2 ? blockIdx.x : static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp;
    if (row >= p.rows) return;
    end = row + 1;
    g = static_cast<unsigned>(row) / static_cast<unsigned>(p.rows_per_group);  // both fit 31 bits
  }
  const int first = WIDE ? warp * 32 * EPT : 0;  // this warp's columns
  const float mine = static_cast<float>(min(max(n - first, 0), 32 * EPT));
  const float inv_mine = mine > 0.f ? 1.f / mine : 0.f, inv_n = 1.f / static_cast<float>(n);
  const Place<VEC> at = {first + lane * VEC};
  const float plus = p.weight != nullptr ? p.w0 : 1.f;
  Unit<T, VEC> raw[EPT / VEC];
  auto fetch = [&](long long r) {
    const T* x = static_cast<const T*>(p.x) + r * n;
#pragma unroll
    for (int i = 0; i < EPT / VEC; ++i)
      if (Wk::template in<WIDE>(i, at, n)) raw[i] = load_vec<T, VEC>(x + at.column(i));
  };
  if (row < end) fetch(row);
  if constexpr (WALK) {
    if constexpr (KIND == 1) {
      stage_params<T, VEC>(staged, p.weight, g * p.weight_stride, p.w0, 1.f, p);
      stage_params<T, VEC>(staged + 32 * EPT, p.bias, g * p.bias_stride, 0.f, 0.f, p);
    } else {
      copy_params<T, VEC>(narrow, p.weight, g * p.weight_stride, p.channels);
      copy_params<T, VEC>(narrow + 32 * EPT, p.bias, g * p.bias_stride, p.channels);
    }
    __syncthreads();
  }
  for (; row < end; row += step) {
    float2 f[EPT / 2];
    float2 s2 = both(0.f);
#pragma unroll
    for (int k = 0; k < Wk::K; ++k) {
      if constexpr (VEC == 1) {
        f[k].x = Wk::template in<WIDE>(2 * k, at, n) ? to_f<T>(raw[2 * k].v[0]) : 0.f;
        f[k].y = Wk::template in<WIDE>(2 * k + 1, at, n) ? to_f<T>(raw[2 * k + 1].v[0]) : 0.f;
        s2 = add2(s2, f[k]);
      } else if (Wk::template in<WIDE>(k, at, n)) {
#pragma unroll
        for (int u = 0; u < Wk::P; ++u) {
          f[k * Wk::P + u] = pair_of<T>(raw[k].v + 2 * u);
          s2 = add2(s2, f[k * Wk::P + u]);
        }
      }
    }
    if (WALK && row + step < end) fetch(row + step);  // while this row is reduced
    float mean = warp_sum(s2.x + s2.y) * inv_mine;
    float2 q2 = both(0.f);
#pragma unroll
    for (int k = 0; k < Wk::K; ++k) {
      if constexpr (VEC == 1) {
        float2 d = add2(f[k], both(-mean));
        if (!Wk::template in<WIDE>(2 * k, at, n)) d.x = 0.f;
        if (!Wk::template in<WIDE>(2 * k + 1, at, n)) d.y = 0.f;
        q2 = fma2(d, d, q2);
      } else if (Wk::template in<WIDE>(k, at, n)) {
#pragma unroll
        for (int u = 0; u < Wk::P; ++u) {
          const float2 d = add2(f[k * Wk::P + u], both(-mean));
          q2 = fma2(d, d, q2);
        }
      }
    }
    float sq = warp_sum(q2.x + q2.y);
    if constexpr (WIDE) {
      Exchange ex{slots};
      const float2* all = ex.publish(make_float2(mean, sq), warp, lane);
      float m = 0.f, c = 0.f;
      for (int k = 0; k < p.warps; ++k) m = fmaf(static_cast<float>(min(n - k * 32 * EPT, 32 * EPT)), all[k].x, m);
      m *= inv_n;
      for (int k = 0; k < p.warps; ++k) {
        const float d = all[k].x - m;
        c += fmaf(static_cast<float>(min(n - k * 32 * EPT, 32 * EPT)) * d, d, all[k].y);
      }
      mean = m;
      sq = c;
    }
    const float rstd = rsqrtf(fmaf(sq, inv_n, p.eps));
    if (lane == 0 && (!WIDE || warp == 0)) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + row * n;
#pragma unroll
    for (int k = 0; k < Wk::K; ++k) {
      if (!Wk::template in<WIDE>(Wk::kPerStep * k, at, n)) continue;
      float2 w[Wk::P], b[Wk::P];
      if constexpr (KIND == 1) {
        staged_params<VEC>(w, staged, k, lane, at, n);
        staged_params<VEC>(b, staged + 32 * EPT, k, lane, at, n);
      } else if constexpr (KIND == 3) {
        const Unit<T, VEC> wv = *reinterpret_cast<const Unit<T, VEC>*>(narrow + at.column(k));
        const Unit<T, VEC> bv = *reinterpret_cast<const Unit<T, VEC>*>(narrow + 32 * EPT + at.column(k));
#pragma unroll
        for (int u = 0; u < Wk::P; ++u) {
          w[u] = add2(pair_of<T>(wv.v + 2 * u), both(plus));
          b[u] = pair_of<T>(bv.v + 2 * u);
        }
      } else {
        direct_params<T, VEC>(w, p.weight, g * p.weight_stride, p.w0, 1.f, k, p, at);
        direct_params<T, VEC>(b, p.bias, g * p.bias_stride, 0.f, 0.f, k, p, at);
      }
      Unit<T, VEC> o;
#pragma unroll
      for (int u = 0; u < Wk::P; ++u) {
        const float2 v = fma2(mul2(add2(f[k * Wk::P + u], both(-mean)), both(rstd)), w[u], b[u]);
        if constexpr (VEC == 1) {
          y[at.column(2 * k)] = from_f<T>(v.x);
          if (Wk::template in<WIDE>(2 * k + 1, at, n)) y[at.column(2 * k + 1)] = from_f<T>(v.y);
        } else {
          put_pair<T>(o.v + 2 * u, v);
        }
      }
      if constexpr (VEC > 1) store_vec<T, VEC>(y + at.column(k), o);
    }
  }
}

template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES) : "memory");
}

constexpr int kBwdTeams = 4;  // rows in flight per block where a warp takes a row

// Shared bytes: `stages` rows of (x, dy) units per warp, reused for the sums of a block's teams,
// and (where a warp takes a row) the group's weights.
// Single 16-bit elements are not staged: a copy into shared memory is at least 4 bytes.
constexpr size_t kBwdSmem = 200 * 1024;
template <typename T, int VEC, int EPT, bool WIDE>
size_t bwd_smem(int warps, int stages) {
  const size_t row = sizeof(T) * VEC < 4 ? 0 : 2 * EPT * 32 * sizeof(T);
  const size_t ring = (WIDE ? warps : kBwdTeams) * stages * row;
  const size_t sums = WIDE ? 0 : 2 * 32 * EPT * sizeof(float);
  return (WIDE ? 0 : 32 * EPT * sizeof(float)) + (ring > sums ? ring : sums);
}

template <typename T, int VEC, int EPT, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 512 : 128, WIDE ? 1 : EPT <= 16 ? 5 : EPT <= 24 ? 4 : EPT <= 32 ? 3 : 2)
ln_bwd_kernel(const __grid_constant__ LnParams p) {
  using Wk = Walk<VEC, EPT>;
  // else elements are read from global memory, and again in the second pass over the row
  constexpr bool kRing = sizeof(T) * VEC >= 4;
  constexpr int kUnits = EPT / VEC;
  extern __shared__ __align__(16) uint8_t shared[];
  float* staged = reinterpret_cast<float*>(shared);
  uint8_t* dyn = shared + (WIDE ? 0 : 32 * EPT * sizeof(float));
  __shared__ float2 slots[2][16];
  // only for the reduction: other programmatic dependents may read their inputs as soon as they start
  if (p.part != nullptr) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Exchange ex{slots};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = p.channels;
  const Place<VEC> at = {(WIDE ? warp * 32 * EPT : 0) + lane * VEC};
  const long long g = blockIdx.x / p.parts;
  const int part = static_cast<int>(blockIdx.x % p.parts);
  const long long lo = g * p.rows_per_group + p.rows_per_group * part / p.parts;
  const long long hi = g * p.rows_per_group + p.rows_per_group * (part + 1) / p.parts;
  constexpr int kStep = WIDE ? 1 : kBwdTeams;
  const float inv_n = 1.f / static_cast<float>(n);
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  // this lane's slots: [stage][x, dy][unit], a unit's lanes side by side
  Unit<T, VEC>* ring = reinterpret_cast<Unit<T, VEC>*>(dyn) + warp * p.stages * 2 * kUnits * 32 + lane;
  auto slot = [&](int stage, int which, int i) { return ring + ((stage * 2 + which) * kUnits + i) * 32; };
  auto fetch = [&](long long row, int stage) {
    if constexpr (kRing) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
        if (Wk::template in<WIDE>(i, at, n)) {
          copy_async<sizeof(T) * VEC>(slot(stage, 0, i), x + row * n + at.column(i));
          copy_async<sizeof(T) * VEC>(slot(stage, 1, i), dy + row * n + at.column(i));
        }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  float2 aw[EPT / 2], ab[EPT / 2];
#pragma unroll
  for (int k = 0; k < EPT / 2; ++k) aw[k] = ab[k] = both(0.f);
  long long row = lo + (WIDE ? 0 : warp);
  float mean = 0.f, rstd = 0.f;
  if (row < hi) {
    fetch(row, 0);
    mean = p.mean[row];
    rstd = p.rstd[row];
  }
  if constexpr (!WIDE) {
    stage_params<T, VEC>(staged, p.weight, g * p.weight_stride, p.w0, 1.f, p);
    __syncthreads();
  }
  auto weights = [&](float2(&w)[Wk::P], int k) {
    if constexpr (WIDE)
      direct_params<T, VEC>(w, p.weight, g * p.weight_stride, p.w0, 1.f, k, p, at);
    else
      staged_params<VEC>(w, staged, k, lane, at, n);
  };
  if (row < hi) {
    const int flip = p.stages - 1;
    for (int stage = 0;; stage ^= flip) {
      const bool more = row + kStep < hi;
      float next_mean = 0.f, next_rstd = 0.f;
      if (more) {
        if (flip) fetch(row + kStep, stage ^ 1);
        next_mean = p.mean[row + kStep];
        next_rstd = p.rstd[row + kStep];
      }
      if constexpr (kRing) {
        // this lane's own copies: nothing to synchronise
        if (more && flip)
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
          asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      // pairs of the row's x (which = 0) or dy (1) in step k, a second element past the end as 0
      auto get = [&](int which, int k, float2(&f)[Wk::P]) {
        if constexpr (VEC == 1) {
          const T* src = which ? dy : x;
          f[0].x = to_f<T>(kRing ? slot(stage, which, 2 * k)->v[0] : src[row * n + at.column(2 * k)]);
          f[0].y = 0.f;
          if (Wk::template in<WIDE>(2 * k + 1, at, n))
            f[0].y = to_f<T>(kRing ? slot(stage, which, 2 * k + 1)->v[0] : src[row * n + at.column(2 * k + 1)]);
        } else {
          const Unit<T, VEC> v = *slot(stage, which, k);
#pragma unroll
          for (int u = 0; u < Wk::P; ++u) f[u] = pair_of<T>(v.v + 2 * u);
        }
      };
      const float2 shift = both(-mean * rstd);
      float2 s2 = both(0.f), q2 = both(0.f);
#pragma unroll
      for (int k = 0; k < Wk::K; ++k) {
        if (!Wk::template in<WIDE>(Wk::kPerStep * k, at, n)) continue;
        float2 xv[Wk::P], dv[Wk::P], w[Wk::P];
        get(0, k, xv);
        get(1, k, dv);
        weights(w, k);
#pragma unroll
        for (int u = 0; u < Wk::P; ++u) {
          const int e = k * Wk::P + u;
          const float2 xh = fma2(xv[u], both(rstd), shift);
          aw[e] = fma2(dv[u], xh, aw[e]);
          ab[e] = add2(ab[e], dv[u]);
          const float2 a = mul2(dv[u], w[u]);
          s2 = add2(s2, a);
          q2 = fma2(a, xh, q2);
        }
      }
      float sa = warp_sum(s2.x + s2.y), sx = warp_sum(q2.x + q2.y);
      if constexpr (WIDE) {
        const float2* all = ex.publish(make_float2(sa, sx), warp, lane);
        sa = sx = 0.f;
        for (int k = 0; k < p.warps; ++k) {
          sa += all[k].x;
          sx += all[k].y;
        }
      }
      const float2 c0 = both(-rstd * sa * inv_n), c1 = both(-rstd * sx * inv_n);
      T* out = static_cast<T*>(p.y) + row * n;
#pragma unroll
      for (int k = 0; k < Wk::K; ++k) {
        if (!Wk::template in<WIDE>(Wk::kPerStep * k, at, n)) continue;
        float2 xv[Wk::P], dv[Wk::P], w[Wk::P];
        get(0, k, xv);
        get(1, k, dv);
        weights(w, k);
        Unit<T, VEC> o;
#pragma unroll
        for (int u = 0; u < Wk::P; ++u) {
          const float2 xh = fma2(xv[u], both(rstd), shift);
          const float2 v = fma2(xh, c1, fma2(mul2(dv[u], w[u]), both(rstd), c0));
          if constexpr (VEC == 1) {
            out[at.column(2 * k)] = from_f<T>(v.x);
            if (Wk::template in<WIDE>(2 * k + 1, at, n)) out[at.column(2 * k + 1)] = from_f<T>(v.y);
          } else {
            put_pair<T>(o.v + 2 * u, v);
          }
        }
        if constexpr (VEC > 1) store_vec<T, VEC>(out + at.column(k), o);
      }
      if (!more) break;
      row += kStep;
      mean = next_mean;
      rstd = next_rstd;
      if (!flip) fetch(row, 0);
    }
  }
  if (p.part == nullptr) return;
  // the block's partial: teams add in order, so the result does not depend on timing
  float* out = p.part + (g * p.parts + part) * 2 * n;
  float* comb = reinterpret_cast<float*>(dyn);  // [2][32 EPT], quads laid out as the staged weights
  __syncthreads();
  for (int t = 0; t < kStep; ++t) {
    if (WIDE || warp == t) {
      const bool last = t + 1 == kStep;
#pragma unroll
      for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int e = 0; e < EPT; e += VEC == 1 ? 1 : 4) {
          const float2* sum = which ? ab : aw;
          if constexpr (VEC == 1) {
            const int c = at.column(e);
            if (c >= n) continue;
            float v = e & 1 ? sum[e / 2].y : sum[e / 2].x;
            if (t > 0) v += comb[which * 32 * EPT + e * 32 + lane];
            if (last)
              out[which * n + c] = v;
            else
              comb[which * 32 * EPT + e * 32 + lane] = v;
          } else {
            const int c = at.column(e / VEC) + e % VEC;
            if (c >= n) continue;
            float4 v = make_float4(sum[e / 2].x, sum[e / 2].y, sum[e / 2 + 1].x, sum[e / 2 + 1].y);
            float4* mine = reinterpret_cast<float4*>(comb + which * 32 * EPT) + e / 4 * 32 + lane;
            if (t > 0) v = make_float4(v.x + mine->x, v.y + mine->y, v.z + mine->z, v.w + mine->w);
            *(last ? reinterpret_cast<float4*>(out + which * n + c) : mine) = v;
          }
        }
    }
    if (!WIDE) __syncthreads();
  }
}

// 32 columns x 8 part lanes per block: lane y adds parts y, y + 8, ... in order, then the 8
// sums are added in order.
constexpr int kRedLanes = 8;
__global__ void __launch_bounds__(32 * kRedLanes) reduce_parts_kernel(const float* __restrict__ part, int parts,
                                                                      int cols, void* out0, void* out1,
                                                                      int out_dtype) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tiles = (cols + 31) / 32;
  const int which = blockIdx.x / tiles % 2;
  const long long g = blockIdx.x / tiles / 2;
  const int c = (blockIdx.x % tiles) * 32 + threadIdx.x;
  void* out = which ? out1 : out0;
  if (out == nullptr) return;
  float s = 0.f;
  if (c < cols) {
    const float* p = part + (g * parts * 2 + which) * cols + c;
#pragma unroll 8
    for (int i = threadIdx.y; i < parts; i += kRedLanes) s += p[static_cast<long long>(i) * 2 * cols];
  }
  __shared__ float red[kRedLanes][32];
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= cols) return;
#pragma unroll
  for (int i = 1; i < kRedLanes; ++i) s += red[i][threadIdx.x];
  const long long at = g * cols + c;
  if (out_dtype == PF_F32)
    static_cast<float*>(out)[at] = s;
  else if (out_dtype == PF_F16)
    static_cast<__half*>(out)[at] = __float2half_rn(s);
  else
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(s);
}

constexpr int kSms = 148;
constexpr int kMostParts = kSms * 8;
constexpr int kFwdBlocks = 5;  // blocks of four warps per SM of the forward kernel that walks rows

// Resident blocks per SM of a backward kernel with rows of `warps` warps, looked up once.
template <typename T, int VEC, int EPT, bool WIDE>
cudaError_t bwd_blocks(size_t smem, int warps, int* blocks) {
  auto kernel = ln_bwd_kernel<T, VEC, EPT, WIDE>;
  static std::mutex mu;
  static int known[64][17] = {};  // [device ordinal][warps]
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  int& k = known[dev][warps];
  if (k == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdSmem);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k, kernel, 32 * (WIDE ? warps : kBwdTeams), smem);
    if (e != cudaSuccess) return e;
    if (k < 1) return cudaErrorInvalidConfiguration;
  }
  *blocks = k;
  return cudaSuccess;
}

template <typename T, int VEC, int EPT, bool WIDE>
cudaError_t launch_cut(LnParams& p, long long groups, bool bwd, cudaStream_t stream) {
  if (bwd) {
    const int threads = 32 * (WIDE ? p.warps : kBwdTeams);
    p.stages = bwd_smem<T, VEC, EPT, WIDE>(p.warps, 2) <= kBwdSmem ? 2 : 1;
    const size_t smem = bwd_smem<T, VEC, EPT, WIDE>(p.warps, p.stages);
    int blocks = 0;
    const cudaError_t e = bwd_blocks<T, VEC, EPT, WIDE>(smem, p.warps, &blocks);
    if (e != cudaSuccess) return e;
    // as many parts as are resident at once over all groups
    const long long parts = static_cast<long long>(kSms) * blocks / groups;
    if (parts < p.parts) p.parts = parts < 1 ? 1 : static_cast<int>(parts);
    ln_bwd_kernel<T, VEC, EPT, WIDE><<<static_cast<unsigned>(groups * p.parts), threads, smem, stream>>>(p);
    return cudaGetLastError();
  }
  if (!WIDE && p.rows >= kSms * kFwdBlocks * 8 && p.rows_per_group >= 16) {
    // As many blocks as are resident, or up to four times that, of sixteen rows at least: short
    // blocks even out the SMs' different speeds (2 x 16384 x 1536: 43.8 us in one round,
    // 38.5 in four), long ones read the parameters less often (4 x 4096 x 1152: 15.9 and 17.3 us).
    const long long rounds = p.rows >= kSms * kFwdBlocks * 32 ? 4 : 1;
    const long long parts = kSms * kFwdBlocks * rounds / groups, most = p.rows_per_group / 16;
    p.parts = static_cast<int>(parts < 1 ? 1 : parts < most ? parts : most);
    const unsigned grid = static_cast<unsigned>(groups * p.parts);
    if (VEC == 8 && !p.wide)
      ln_fwd_kernel<T, VEC, EPT, WIDE ? 2 : VEC == 8 ? 3 : 1><<<grid, 128, 0, stream>>>(p);
    else
      ln_fwd_kernel<T, VEC, EPT, WIDE ? 2 : 1><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
  }
  // one warp per block while that still leaves SMs without work, else four
  const int rows = WIDE || p.rows <= kSms * 8 ? 1 : 4;
  ln_fwd_kernel<T, VEC, EPT, WIDE ? 2 : 0><<<static_cast<unsigned>((p.rows + rows - 1) / rows),
                                             32 * (WIDE ? p.warps : rows), 0, stream>>>(p);
  return cudaGetLastError();
}

// Elements per lane: the least multiple of 8 that covers the row with one warp; rows that
// would take more than 64 take 32 per lane of several warps.
template <typename T, int VEC>
cudaError_t launch_width(LnParams& p, long long groups, bool bwd, cudaStream_t stream) {
  const int per_lane = (p.channels + 31) / 32;
  p.warps = 1;
  if (per_lane <= 8) return launch_cut<T, VEC, 8, false>(p, groups, bwd, stream);
  if (per_lane <= 16) return launch_cut<T, VEC, 16, false>(p, groups, bwd, stream);
  if (per_lane <= 24) return launch_cut<T, VEC, 24, false>(p, groups, bwd, stream);
  if (per_lane <= 32) return launch_cut<T, VEC, 32, false>(p, groups, bwd, stream);
  if (per_lane <= 40) return launch_cut<T, VEC, 40, false>(p, groups, bwd, stream);
  if (per_lane <= 48) return launch_cut<T, VEC, 48, false>(p, groups, bwd, stream);
  if (per_lane <= 56) return launch_cut<T, VEC, 56, false>(p, groups, bwd, stream);
  if (per_lane <= 64) return launch_cut<T, VEC, 64, false>(p, groups, bwd, stream);
  p.warps = (p.channels + 1023) / 1024;
  return launch_cut<T, VEC, 32, true>(p, groups, bwd, stream);
}

template <typename T>
cudaError_t launch_type(LnParams& p, long long groups, bool bwd, bool aligned, cudaStream_t stream) {
  constexpr int kVec = 16 / sizeof(T);
  return aligned ? launch_width<T, kVec>(p, groups, bwd, stream) : launch_width<T, 1>(p, groups, bwd, stream);
}

// 16-byte accesses need every row of x, dy, y and of the parameters to start on 16 bytes.
bool rows_aligned(const LnArgs& a) {
  const size_t e = a.dtype == PF_F32 ? 4 : 2, we = a.wdtype == PF_F32 ? 4 : 2;
  auto ok = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const bool many = a.groups > 1;
  return a.channels * e % 16 == 0 && (!many || (a.weight_stride * we % 16 == 0 && a.bias_stride * we % 16 == 0)) &&
         ok(a.x) && ok(a.dy) && ok(a.y) && ok(a.weight) && ok(a.bias);
}

// Launches; the backward pass lowers p.parts to what is resident at once.
cudaError_t dispatch(const LnArgs& a, LnParams& p, bool bwd, cudaStream_t stream) {
  const bool al = rows_aligned(a);
  switch (a.dtype) {
    case PF_BF16: return launch_type<__nv_bfloat16>(p, a.groups, bwd, al, stream);
    case PF_F16: return launch_type<__half>(p, a.groups, bwd, al, stream);
    default: return launch_type<float>(p, a.groups, bwd, al, stream);
  }
}

LnParams params_of(const LnArgs& a) {
  LnParams p = {};
  p.x = a.x;
  p.dy = a.dy;
  p.y = a.y;
  p.weight = a.weight;
  p.bias = a.bias;
  p.mean = a.mean;
  p.rstd = a.rstd;
  p.rows = a.groups * a.rows_per_group;
  p.rows_per_group = a.rows_per_group;
  p.weight_stride = a.weight_stride;
  p.bias_stride = a.bias_stride;
  p.channels = a.channels;
  p.wide = a.wdtype == PF_F32 && a.dtype != PF_F32;
  p.w0 = a.weight_offset;
  p.eps = a.eps;
  return p;
}

}  // namespace

// Most blocks per group of the backward pass: each of them has at least eight rows, so that a
// partial row is written once for many rows read.
int ln_bwd_parts(long long groups, long long rows_per_group) {
  long long parts = kMostParts / groups;
  if (parts > (rows_per_group + 7) / 8) parts = (rows_per_group + 7) / 8;
  return parts < 1 ? 1 : static_cast<int>(parts);
}

cudaError_t launch_layernorm(const LnArgs& a, cudaStream_t stream) {
  LnParams p = params_of(a);
  return p.rows == 0 ? cudaSuccess : dispatch(a, p, false, stream);
}

cudaError_t launch_layernorm_bwd(const LnArgs& a, void* dweight, void* dbias, float* part, cudaStream_t stream) {
  LnParams p = params_of(a);
  p.parts = p.rows == 0 ? 0 : ln_bwd_parts(a.groups, a.rows_per_group);
  const bool sums = dweight != nullptr || dbias != nullptr;
  p.part = sums ? part : nullptr;
  if (p.rows > 0) {
    const cudaError_t e = dispatch(a, p, true, stream);
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  return launch_reduce_parts(part, static_cast<int>(a.groups), p.parts, a.channels, dweight, dbias, a.wdtype, stream);
}

cudaError_t launch_reduce_parts(const float* part, int groups, int parts, int cols, void* out0, void* out1,
                                int out_dtype, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(groups) * 2 * ((cols + 31) / 32)));
  cfg.blockDim = dim3(32, kRedLanes);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, reduce_parts_kernel, part, parts, cols, out0, out1, out_dtype);
}

}  // namespace pf
