// layernorm.cu -- layer normalisation with an affine or a per-group modulation, forward and
// backward.
//
//   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), x^ = (x - m) r
//   y = x^ (w_g + w0) + b_g              g: the row's group (its sample, or the one affine)
//   a = dy (w_g + w0);  dx = r (a - mean(a) - x^ mean(a x^))
//   dw_g = sum over the group's rows of dy x^,  db_g = sum of dy
//
// Both directions are HBM bound: forward reads x and writes y, backward reads x and dy and
// writes dx.  A row is read once and stays in registers, so the variance is taken around the
// mean (two passes over registers, none over memory).  Rows up to 1536 elements belong to one
// warp (no block barrier; many rows in flight per SM); wider ones to a block of 128 or 512
// threads.  The backward pass keeps the weight-gradient sums of its columns in registers over
// a contiguous run of rows and writes one fp32 partial row per block; a second kernel adds
// the partials in a fixed order, so equal inputs give equal bits.

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
  int wide;            // the parameters are fp32 (else the type of x)
  float w0, eps;
};

// Sum of two values over a team: a warp, or the whole block (then `scratch` holds 2 x 16
// values per parity so that consecutive calls need one barrier each).
template <int TEAM>
__device__ __forceinline__ void team_sum2(float& a, float& b, float (*scratch)[2][16], int& parity) {
  a = warp_sum(a);
  b = warp_sum(b);
  if constexpr (TEAM > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
      scratch[parity][0][warp] = a;
      scratch[parity][1][warp] = b;
    }
    __syncthreads();
    a = lane < TEAM / 32 ? scratch[parity][0][lane] : 0.f;
    b = lane < TEAM / 32 ? scratch[parity][1][lane] : 0.f;
#pragma unroll
    for (int off = TEAM / 64; off > 0; off >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, off);
      b += __shfl_xor_sync(0xffffffffu, b, off);
    }
    a = __shfl_sync(0xffffffffu, a, 0);
    b = __shfl_sync(0xffffffffu, b, 0);
    parity ^= 1;
  }
}

template <typename T, int VEC, int TEAM, int EPT>
__global__ void __launch_bounds__(TEAM == 32 ? 128 : TEAM) ln_fwd_kernel(const __grid_constant__ LnParams p) {
  constexpr int NV = EPT / VEC;
  __shared__ float scratch[2][2][16];
  int parity = 0;
  const int t = TEAM == 32 ? threadIdx.x & 31 : threadIdx.x;
  const long long row = TEAM == 32 ? static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)
                                   : static_cast<long long>(blockIdx.x);
  if (row >= p.rows) return;  // whole teams leave
  const T* x = static_cast<const T*>(p.x) + row * p.channels;
  Vec<T, VEC> raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TEAM + t) * VEC;
    if (c < p.channels) raw[i] = load_vec<T, VEC>(x + c);
  }
  float s = 0.f, unused = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * TEAM + t) * VEC < p.channels) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) s += to_f<T>(raw[i].v[k]);
    }
  team_sum2<TEAM>(s, unused, scratch, parity);
  const float inv_n = 1.f / static_cast<float>(p.channels);
  const float mean = s * inv_n;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * TEAM + t) * VEC < p.channels) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float d = to_f<T>(raw[i].v[k]) - mean;
        ss = fmaf(d, d, ss);
      }
    }
  team_sum2<TEAM>(ss, unused, scratch, parity);
  const float rstd = rsqrtf(fmaf(ss, inv_n, p.eps));
  if (t == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
  const long long g = row / p.rows_per_group;
  T* y = static_cast<T*>(p.y) + row * p.channels;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TEAM + t) * VEC;
    if (c < p.channels) {
      float w[VEC], b[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        w[k] = 1.f;
        b[k] = 0.f;
      }
      if (p.weight != nullptr) {
        load_param<T, VEC>(p.weight, g * p.weight_stride + c, p.wide, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[k] += p.w0;
      }
      if (p.bias != nullptr) load_param<T, VEC>(p.bias, g * p.bias_stride + c, p.wide, b);
      Vec<T, VEC> o;
#pragma unroll
      for (int k = 0; k < VEC; ++k) o.v[k] = from_f<T>(fmaf((to_f<T>(raw[i].v[k]) - mean) * rstd, w[k], b[k]));
      store_vec<T, VEC>(y + c, o);
    }
  }
}

template <typename T, int VEC, int TEAM, int EPT>
__global__ void __launch_bounds__(TEAM == 32 ? 128 : TEAM) ln_bwd_kernel(const __grid_constant__ LnParams p) {
  constexpr int NV = EPT / VEC;
  constexpr int TEAMS = TEAM == 32 ? 4 : 1;
  __shared__ float scratch[2][2][16];
  __shared__ float comb[TEAM == 32 ? 2 * 32 * EPT : 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int parity = 0;
  const int t = TEAM == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int team = TEAM == 32 ? threadIdx.x >> 5 : 0;
  const long long g = blockIdx.x / p.parts;
  const int part = static_cast<int>(blockIdx.x % p.parts);
  const long long lo = g * p.rows_per_group + p.rows_per_group * part / p.parts;
  const long long hi = g * p.rows_per_group + p.rows_per_group * (part + 1) / p.parts;
  const float inv_n = 1.f / static_cast<float>(p.channels);
  float aw[EPT], ab[EPT];
#pragma unroll
  for (int k = 0; k < EPT; ++k) aw[k] = ab[k] = 0.f;
  for (long long row = lo + team; row < hi; row += TEAMS) {
    const T* x = static_cast<const T*>(p.x) + row * p.channels;
    const T* dy = static_cast<const T*>(p.dy) + row * p.channels;
    Vec<T, VEC> rx[NV], rd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TEAM + t) * VEC;
      if (c < p.channels) {
        rx[i] = load_vec<T, VEC>(x + c);
        rd[i] = load_vec<T, VEC>(dy + c);
      }
    }
    const float mean = p.mean[row], rstd = p.rstd[row];
    float sa = 0.f, sx = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TEAM + t) * VEC;
      if (c < p.channels) {
        float w[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[k] = 1.f;
        if (p.weight != nullptr) {
          load_param<T, VEC>(p.weight, g * p.weight_stride + c, p.wide, w);
#pragma unroll
          for (int k = 0; k < VEC; ++k) w[k] += p.w0;
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float d = to_f<T>(rd[i].v[k]);
          const float xh = (to_f<T>(rx[i].v[k]) - mean) * rstd;
          aw[i * VEC + k] = fmaf(d, xh, aw[i * VEC + k]);
          ab[i * VEC + k] += d;
          const float a = d * w[k];
          sa += a;
          sx = fmaf(a, xh, sx);
        }
      }
    }
    team_sum2<TEAM>(sa, sx, scratch, parity);
    sa *= inv_n;
    sx *= inv_n;
    T* dx = static_cast<T*>(p.y) + row * p.channels;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TEAM + t) * VEC;
      if (c < p.channels) {
        float w[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[k] = 1.f;
        if (p.weight != nullptr) {
          load_param<T, VEC>(p.weight, g * p.weight_stride + c, p.wide, w);
#pragma unroll
          for (int k = 0; k < VEC; ++k) w[k] += p.w0;
        }
        Vec<T, VEC> o;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float xh = (to_f<T>(rx[i].v[k]) - mean) * rstd;
          o.v[k] = from_f<T>(rstd * (to_f<T>(rd[i].v[k]) * w[k] - sa - xh * sx));
        }
        store_vec<T, VEC>(dx + c, o);
      }
    }
  }
  if (p.part == nullptr) return;
  // the block's partial: teams add in order, so the result does not depend on timing
  float* out = p.part + (g * p.parts + part) * 2 * p.channels;
  if constexpr (TEAM == 32) {
    for (int w = 0; w < TEAMS; ++w) {
      if (team == w) {
#pragma unroll
        for (int k = 0; k < EPT; ++k) {
          float* a = comb + k * 32 + t;
          float* b = a + 32 * EPT;
          *a = w == 0 ? aw[k] : *a + aw[k];
          *b = w == 0 ? ab[k] : *b + ab[k];
        }
      }
      __syncthreads();
    }
    for (int e = threadIdx.x; e < 2 * p.channels; e += 128) {
      const int which = e >= p.channels, c = e - which * p.channels;
      const int vec = c / VEC, k = c % VEC;  // column c: lane vec % 32, slot (vec / 32) VEC + k
      out[e] = comb[which * 32 * EPT + ((vec / 32) * VEC + k) * 32 + vec % 32];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const int c = (i * TEAM + t) * VEC + k;
        if (c < p.channels) {
          out[c] = aw[i * VEC + k];
          out[p.channels + c] = ab[i * VEC + k];
        }
      }
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

template <typename T, int VEC, int TEAM, int EPT>
cudaError_t launch_team(const LnParams& p, long long groups, bool bwd, cudaStream_t stream) {
  if (bwd) {
    ln_bwd_kernel<T, VEC, TEAM, EPT>
        <<<static_cast<unsigned>(groups * p.parts), TEAM == 32 ? 128 : TEAM, 0, stream>>>(p);
  } else if (TEAM == 32) {
    // one warp per block while that still leaves SMs without work, else four
    const int warps = p.rows <= 148 * 8 ? 1 : 4;
    ln_fwd_kernel<T, VEC, TEAM, EPT>
        <<<static_cast<unsigned>((p.rows + warps - 1) / warps), 32 * warps, 0, stream>>>(p);
  } else {
    ln_fwd_kernel<T, VEC, TEAM, EPT><<<static_cast<unsigned>(p.rows), TEAM, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t launch_width(const LnParams& p, long long groups, bool bwd, cudaStream_t stream) {
  const int c = p.channels;
  if (c <= 32 * 8) return launch_team<T, VEC, 32, 8>(p, groups, bwd, stream);
  if (c <= 32 * 16) return launch_team<T, VEC, 32, 16>(p, groups, bwd, stream);
  if (c <= 32 * 32) return launch_team<T, VEC, 32, 32>(p, groups, bwd, stream);
  if (c <= 32 * 48) return launch_team<T, VEC, 32, 48>(p, groups, bwd, stream);
  if (c <= 128 * 16) return launch_team<T, VEC, 128, 16>(p, groups, bwd, stream);
  if (c <= 128 * 32) return launch_team<T, VEC, 128, 32>(p, groups, bwd, stream);
  if (c <= 512 * 16) return launch_team<T, VEC, 512, 16>(p, groups, bwd, stream);
  return launch_team<T, VEC, 512, 32>(p, groups, bwd, stream);
}

template <typename T>
cudaError_t launch_type(const LnParams& p, long long groups, bool bwd, bool aligned, cudaStream_t stream) {
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

cudaError_t dispatch(const LnArgs& a, const LnParams& p, bool bwd, cudaStream_t stream) {
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

// Blocks per group of the backward pass: enough for four blocks per SM over all groups, but
// at least eight rows each, so that a partial row is written once for many rows read.
int ln_bwd_parts(long long groups, long long rows_per_group) {
  long long parts = (148 * 4) / groups;
  if (parts > (rows_per_group + 7) / 8) parts = (rows_per_group + 7) / 8;
  return parts < 1 ? 1 : static_cast<int>(parts);
}

cudaError_t launch_layernorm(const LnArgs& a, cudaStream_t stream) {
  const LnParams p = params_of(a);
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
