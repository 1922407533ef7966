// block_ops.cuh -- element types, vector loads and the partial-sum reduction shared by the
// layer-norm and the norm + rotary kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pf_internal.h"

namespace pf {
namespace blk {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// N consecutive elements, moved as one 4-, 8- or 16-byte access (or two 16-byte ones).
template <typename T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Vec {
  T v[N];
};

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T* p) {
  return *reinterpret_cast<const Vec<T, N>*>(p);
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, N>& v) {
  *reinterpret_cast<Vec<T, N>*>(p) = v;
}

// N consecutive parameters held as T or, when `wide`, as fp32.
template <typename T, int N>
__device__ __forceinline__ void load_param(const void* base, long long at, bool wide, float (&out)[N]) {
  if (wide) {
    const float* p = static_cast<const float*>(base) + at;
#pragma unroll
    for (int i = 0; i < N; i += (N < 4 ? N : 4)) {
      const auto x = load_vec<float, (N < 4 ? N : 4)>(p + i);
#pragma unroll
      for (int k = 0; k < (N < 4 ? N : 4); ++k) out[i + k] = x.v[k];
    }
  } else {
    const auto x = load_vec<T, N>(static_cast<const T*>(base) + at);
#pragma unroll
    for (int k = 0; k < N; ++k) out[k] = to_f<T>(x.v[k]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

}  // namespace blk

// out[which][g][c] = sum over parts of part[g][p][which][c] in part order groups, rounded once to the output
// type.  A null output is skipped.  Launched as a programmatic dependent of the kernel that
// writes the partials.
cudaError_t launch_reduce_parts(const float* part, int groups, int parts, int cols, void* out0, void* out1,
                                int out_dtype, cudaStream_t stream);

}  // namespace pf
