// qk_norm_rope.cu -- per-head RMS normalisation of queries and keys followed by a rotary
// embedding over several position axes, forward and backward.
//
//   z = x r g,  r = 1 / sqrt(mean(x^2) + eps)   (or z = x without the norm)
//   pair i of axis a (e0, e1):  y[e0] = z[e0] c - z[e1] s,  y[e1] = z[e0] s + z[e1] c
//   c, s = cos, sin of pos[token][a] theta_a^(-2 i / w_a)
//   backward: dz turns dy by the opposite angle;  dg = sum dz x r
//             dx = r (dz g - x^ mean(dz g x^)),  x^ = x r
//
// HBM bound: every element is read once and written once (backward: two reads, one write).
// A lane owns four pairs of a vector, so a pair's elements meet in one lane's registers for
// either pairing: one 16-byte access for interleaved pairs (e1 = e0 + 1), two 8-byte ones for
// half-split pairs (e1 = e0 + w_a / 2).  The four angles of a lane are the same for every
// head of a token: a warp takes one token (or a share of its heads) and computes them once.
// Angles are taken in turns, pos * (theta^(-2i/w) / 2 pi) in 64 bits, and only their fraction
// is rounded to 32 bits, so far positions lose nothing.
//
// The backward pass keeps the gain-gradient sums of a lane's elements in registers over the
// tokens of its warp; blocks write fp32 partials that a second kernel adds in a fixed order.

#include "block_ops.cuh"

namespace pf {
namespace {

using namespace blk;

constexpr int kWarps = 8;

struct RopeParams {
  const void* x[2];   // q, k: forward input, backward saved input (null without norm)
  const void* dy[2];  // backward: gradients of the rotated output
  void* y[2];         // forward: output; backward: dx
  const void* gain[2];
  long long xs[2][3], ds[2][3], ys[2][3];  // element strides: batch, token, head
  const float* pos;   // [tokens][n_axes] (pos_batch apart per batch element)
  long long pos_batch;
  float* part;        // backward: [block][2][head_dim], or null
  long long items;    // batch * tokens * splits
  int tokens, n_axes, heads[2], head_dim, splits;
  float eps;          // 0: no norm
  RopeTable tab;
};

// A lane's four pairs: where they lie and how far they turn per unit of position.
struct Pairs {
  float c[4], s[4];
  bool turn[4];
};

// Elements of a lane's pairs, first[k] and second[k], as PV consecutive ones per access.
// INTER: pair k is elements (e + 2 k, e + 2 k + 1) of one 8-element run.
template <typename T, bool INTER, int PV>
__device__ __forceinline__ void load8(const T* p, const int (&e0)[4], const int (&e1)[4], float (&a)[4], float (&b)[4]) {
  if constexpr (INTER) {
    const auto v = load_vec<T, 8>(p + e0[0]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = to_f<T>(v.v[2 * k]);
      b[k] = to_f<T>(v.v[2 * k + 1]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; k += PV) {
      const auto u = load_vec<T, PV>(p + e0[k]);
      const auto v = load_vec<T, PV>(p + e1[k]);
#pragma unroll
      for (int j = 0; j < PV; ++j) {
        a[k + j] = to_f<T>(u.v[j]);
        b[k + j] = to_f<T>(v.v[j]);
      }
    }
  }
}

template <typename T, bool INTER, int PV>
__device__ __forceinline__ void store8(T* p, const int (&e0)[4], const int (&e1)[4], const float (&a)[4], const float (&b)[4]) {
  if constexpr (INTER) {
    Vec<T, 8> v;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v.v[2 * k] = from_f<T>(a[k]);
      v.v[2 * k + 1] = from_f<T>(b[k]);
    }
    store_vec<T, 8>(p + e0[0], v);
  } else {
#pragma unroll
    for (int k = 0; k < 4; k += PV) {
      Vec<T, PV> u, v;
#pragma unroll
      for (int j = 0; j < PV; ++j) {
        u.v[j] = from_f<T>(a[k + j]);
        v.v[j] = from_f<T>(b[k + j]);
      }
      store_vec<T, PV>(p + e0[k], u);
      store_vec<T, PV>(p + e1[k], v);
    }
  }
}

__device__ __forceinline__ void token_angles(const RopeParams& p, int lane_pair0, const float* pos, Pairs& pr) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = lane_pair0 + k;
    const int axis = p.tab.axis[i];
    pr.turn[k] = axis < p.n_axes;  // pairs past the axes are copied
    pr.c[k] = 1.f;
    pr.s[k] = 0.f;
    if (pr.turn[k]) {
      const double turns = static_cast<double>(__ldg(pos + axis)) * p.tab.turns[i];
      sincospif(2.f * static_cast<float>(turns - rint(turns)), &pr.s[k], &pr.c[k]);
    }
  }
}

template <int SEG>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int off = SEG / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The heads of a warp's item are walked 32 / SEG at a time, kUnroll steps of loads in flight.
template <typename T, bool INTER, int PV, int SEG>
__global__ void __launch_bounds__(32 * kWarps) rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPer = 32 / SEG;
  constexpr int kUnroll = 4;
  const int lane = threadIdx.x & 31, sub = lane / SEG, chunk = lane % SEG;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (item >= p.items) return;  // whole warps leave
  const int split = static_cast<int>(item % p.splits);
  const long long bt = item / p.splits;
  const long long b = bt / p.tokens, tok = bt % p.tokens;
  const bool active = chunk * 8 < p.head_dim;
  const int i0 = active ? chunk * 4 : 0;
  int e0[4], e1[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    e0[k] = p.tab.e0[i0 + k];
    e1[k] = p.tab.e1[i0 + k];
  }
  const int n = p.heads[0] + p.heads[1];
  const int h_lo = n * split / p.splits, h_hi = n * (split + 1) / p.splits;
  float ga[2][4], gb[2][4];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
#pragma unroll
    for (int k = 0; k < 4; ++k) ga[w][k] = gb[w][k] = 1.f;
    if (p.gain[w] != nullptr) load8<T, INTER, PV>(static_cast<const T*>(p.gain[w]), e0, e1, ga[w], gb[w]);
  }
  Pairs pr;
  bool angles = false;
  const float inv_d = 1.f / static_cast<float>(p.head_dim);
  for (int h0 = h_lo; h0 < h_hi; h0 += kPer * kUnroll) {
    float a[kUnroll][4], c[kUnroll][4];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kPer + sub;
      const int w = h >= p.heads[0];
#pragma unroll
      for (int k = 0; k < 4; ++k) a[u][k] = c[u][k] = 0.f;
      if (active && h < h_hi)
        load8<T, INTER, PV>(static_cast<const T*>(p.x[w]) + b * p.xs[w][0] + tok * p.xs[w][1] +
                                (h - w * p.heads[0]) * p.xs[w][2],
                            e0, e1, a[u], c[u]);
    }
    if (!angles) {  // behind the first loads
      token_angles(p, i0, p.pos + b * p.pos_batch + tok * p.n_axes, pr);
      angles = true;
    }
    float r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) r[u] = 1.f;
    if (p.eps > 0.f) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = fmaf(a[u][k], a[u][k], fmaf(c[u][k], c[u][k], ss));
        r[u] = rsqrtf(fmaf(seg_sum<SEG>(ss), inv_d, p.eps));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kPer + sub;
      const int w = h >= p.heads[0];
      if (!active || h >= h_hi) continue;
      float ya[4], yb[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float za = a[u][k] * r[u] * (w ? ga[1][k] : ga[0][k]);
        const float zb = c[u][k] * r[u] * (w ? gb[1][k] : gb[0][k]);
        ya[k] = pr.turn[k] ? za * pr.c[k] - zb * pr.s[k] : za;
        yb[k] = pr.turn[k] ? za * pr.s[k] + zb * pr.c[k] : zb;
      }
      store8<T, INTER, PV>(static_cast<T*>(p.y[w]) + b * p.ys[w][0] + tok * p.ys[w][1] +
                               (h - w * p.heads[0]) * p.ys[w][2],
                           e0, e1, ya, yb);
    }
  }
}

template <typename T, bool INTER, int PV, int SEG>
__global__ void __launch_bounds__(32 * kWarps) rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPer = 32 / SEG;
  constexpr int kUnroll = 2;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float red[2][256];
  const int lane = threadIdx.x & 31, sub = lane / SEG, chunk = lane % SEG, warp = threadIdx.x >> 5;
  const bool active = chunk * 8 < p.head_dim;
  const int i0 = active ? chunk * 4 : 0;
  int e0[4], e1[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    e0[k] = p.tab.e0[i0 + k];
    e1[k] = p.tab.e1[i0 + k];
  }
  float ga[2][4], gb[2][4], sa[2][4], sb[2][4];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      ga[w][k] = gb[w][k] = 1.f;
      sa[w][k] = sb[w][k] = 0.f;
    }
    if (p.gain[w] != nullptr) load8<T, INTER, PV>(static_cast<const T*>(p.gain[w]), e0, e1, ga[w], gb[w]);
  }
  const int n = p.heads[0] + p.heads[1];
  const float inv_d = 1.f / static_cast<float>(p.head_dim);
  const bool norm = p.eps > 0.f;
  const long long stride = static_cast<long long>(gridDim.x) * kWarps;
  for (long long item = static_cast<long long>(blockIdx.x) * kWarps + warp; item < p.items; item += stride) {
    const int split = static_cast<int>(item % p.splits);
    const long long bt = item / p.splits;
    const long long b = bt / p.tokens, tok = bt % p.tokens;
    const int h_lo = n * split / p.splits, h_hi = n * (split + 1) / p.splits;
    Pairs pr;
    token_angles(p, i0, p.pos + b * p.pos_batch + tok * p.n_axes, pr);
    for (int h0 = h_lo; h0 < h_hi; h0 += kPer * kUnroll) {
      float a[kUnroll][4], c[kUnroll][4], da[kUnroll][4], db[kUnroll][4];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * kPer + sub;
        const int w = h >= p.heads[0];
        const long long hh = h - w * p.heads[0];
#pragma unroll
        for (int k = 0; k < 4; ++k) a[u][k] = c[u][k] = da[u][k] = db[u][k] = 0.f;
        if (active && h < h_hi) {
          load8<T, INTER, PV>(static_cast<const T*>(p.dy[w]) + b * p.ds[w][0] + tok * p.ds[w][1] + hh * p.ds[w][2],
                              e0, e1, da[u], db[u]);
          if (norm)
            load8<T, INTER, PV>(static_cast<const T*>(p.x[w]) + b * p.xs[w][0] + tok * p.xs[w][1] + hh * p.xs[w][2],
                                e0, e1, a[u], c[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * kPer + sub;
        const int w = h >= p.heads[0];
        float za[4], zb[4], ss = 0.f, sx = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          za[k] = pr.turn[k] ? da[u][k] * pr.c[k] + db[u][k] * pr.s[k] : da[u][k];
          zb[k] = pr.turn[k] ? db[u][k] * pr.c[k] - da[u][k] * pr.s[k] : db[u][k];
        }
        if (norm) {
          float ta[4], tb[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            ta[k] = za[k] * (w ? ga[1][k] : ga[0][k]);
            tb[k] = zb[k] * (w ? gb[1][k] : gb[0][k]);
            ss = fmaf(a[u][k], a[u][k], fmaf(c[u][k], c[u][k], ss));
            sx = fmaf(ta[k], a[u][k], fmaf(tb[k], c[u][k], sx));
          }
          ss = seg_sum<SEG>(ss);
          sx = seg_sum<SEG>(sx);
          const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
          const float m = r * r * sx * inv_d;  // r mean(a x^) = r^2 mean(a x): times x, then r
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float xa = a[u][k] * r, xb = c[u][k] * r;
            // an absent head has dz = x = 0 and adds nothing
            if (w) {
              sa[1][k] = fmaf(za[k], xa, sa[1][k]);
              sb[1][k] = fmaf(zb[k], xb, sb[1][k]);
            } else {
              sa[0][k] = fmaf(za[k], xa, sa[0][k]);
              sb[0][k] = fmaf(zb[k], xb, sb[0][k]);
            }
            za[k] = r * (ta[k] - a[u][k] * m);
            zb[k] = r * (tb[k] - c[u][k] * m);
          }
        }
        if (active && h < h_hi)
          store8<T, INTER, PV>(static_cast<T*>(p.y[w]) + b * p.ys[w][0] + tok * p.ys[w][1] +
                                   (h - w * p.heads[0]) * p.ys[w][2],
                               e0, e1, za, zb);
      }
    }
  }
  if (p.part == nullptr) return;
  // the warp's sub-vectors, then the block's warps in order
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int off = 16; off >= SEG; off >>= 1) {
        sa[w][k] += __shfl_xor_sync(0xffffffffu, sa[w][k], off);
        sb[w][k] += __shfl_xor_sync(0xffffffffu, sb[w][k], off);
      }
    }
  for (int wi = 0; wi < kWarps; ++wi) {
    if (warp == wi && sub == 0 && active) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          red[w][e0[k]] = wi == 0 ? sa[w][k] : red[w][e0[k]] + sa[w][k];
          red[w][e1[k]] = wi == 0 ? sb[w][k] : red[w][e1[k]] + sb[w][k];
        }
    }
    __syncthreads();
  }
  float* out = p.part + static_cast<long long>(blockIdx.x) * 2 * p.head_dim;
  for (int e = threadIdx.x; e < 2 * p.head_dim; e += 32 * kWarps)
    out[e] = red[e >= p.head_dim][e >= p.head_dim ? e - p.head_dim : e];
}

template <typename T, bool INTER, int PV, int SEG>
cudaError_t launch_kernel(const RopeParams& p, bool bwd, int blocks, cudaStream_t stream) {
  if (bwd)
    rope_bwd_kernel<T, INTER, PV, SEG><<<blocks, 32 * kWarps, 0, stream>>>(p);
  else
    rope_fwd_kernel<T, INTER, PV, SEG><<<blocks, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, bool INTER, int PV>
cudaError_t launch_seg(const RopeParams& p, bool bwd, int blocks, cudaStream_t stream) {
  const int chunks = p.head_dim / 8;
  if (chunks <= 4) return launch_kernel<T, INTER, PV, 4>(p, bwd, blocks, stream);
  if (chunks <= 8) return launch_kernel<T, INTER, PV, 8>(p, bwd, blocks, stream);
  if (chunks <= 16) return launch_kernel<T, INTER, PV, 16>(p, bwd, blocks, stream);
  return launch_kernel<T, INTER, PV, 32>(p, bwd, blocks, stream);
}

template <typename T>
cudaError_t launch_type(const RopeParams& p, bool inter, bool bwd, int blocks, cudaStream_t stream) {
  if (inter) return launch_seg<T, true, 4>(p, bwd, blocks, stream);
  // half-split pairs: 4, 2 or 1 consecutive elements of a lane's pairs lie side by side,
  // aligned, when every section's half is a multiple of that
  if (p.tab.half_align % 4 == 0) return launch_seg<T, false, 4>(p, bwd, blocks, stream);
  if (p.tab.half_align % 2 == 0) return launch_seg<T, false, 2>(p, bwd, blocks, stream);
  return launch_seg<T, false, 1>(p, bwd, blocks, stream);
}

cudaError_t dispatch(const RopeArgs& a, const RopeParams& p, bool bwd, int blocks, cudaStream_t stream) {
  switch (a.dtype) {
    case PF_BF16: return launch_type<__nv_bfloat16>(p, a.interleaved, bwd, blocks, stream);
    case PF_F16: return launch_type<__half>(p, a.interleaved, bwd, blocks, stream);
    default: return launch_type<float>(p, a.interleaved, bwd, blocks, stream);
  }
}

// A warp takes a whole token, whose angles it then computes once, unless the tokens are too
// few to give every SM sixteen warps; then a token's heads are shared out.
int head_splits(long long tokens, int heads, int per_step) {
  const long long want = (148 * 16 + tokens - 1) / tokens;
  const long long most = (heads + per_step - 1) / per_step;
  return static_cast<int>(want < most ? want : most);
}

RopeParams params_of(const RopeArgs& a) {
  RopeParams p = {};
  for (int w = 0; w < 2; ++w) {
    p.x[w] = a.x[w];
    p.dy[w] = a.dy[w];
    p.y[w] = a.y[w];
    p.gain[w] = a.gain[w];
    for (int i = 0; i < 3; ++i) {
      p.xs[w][i] = a.xs[w][i];
      p.ds[w][i] = a.ds[w][i];
      p.ys[w][i] = a.ys[w][i];
    }
    p.heads[w] = a.heads[w];
  }
  p.pos = a.pos;
  p.pos_batch = a.pos_batch;
  p.tokens = a.tokens;
  p.n_axes = a.n_axes;
  p.head_dim = a.head_dim;
  p.eps = a.eps;
  p.tab = a.tab;
  const int chunks = a.head_dim / 8;
  const int per_step = chunks <= 4 ? 8 : chunks <= 8 ? 4 : chunks <= 16 ? 2 : 1;
  const long long toks = static_cast<long long>(a.batch) * a.tokens;
  p.splits = toks > 0 ? head_splits(toks, a.heads[0] + a.heads[1], per_step) : 1;
  p.items = toks * p.splits;
  return p;
}

}  // namespace

// Blocks of the backward pass: at most three per SM, each warp walking several tokens, so
// that few partial gain gradients are written.
int rope_bwd_blocks(const RopeArgs& a) {
  const long long items = params_of(a).items;
  const long long blocks = (items + kWarps - 1) / kWarps;
  return static_cast<int>(blocks < 148 * 3 ? blocks : 148 * 3);
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t stream) {
  const RopeParams p = params_of(a);
  if (p.items == 0) return cudaSuccess;
  return dispatch(a, p, false, static_cast<int>((p.items + kWarps - 1) / kWarps), stream);
}

cudaError_t launch_qk_norm_rope_bwd(const RopeArgs& a, void* dgain_q, void* dgain_k, float* part, cudaStream_t stream) {
  RopeParams p = params_of(a);
  const bool sums = dgain_q != nullptr || dgain_k != nullptr;
  p.part = sums ? part : nullptr;
  const int blocks = rope_bwd_blocks(a);
  if (blocks > 0) {
    const cudaError_t e = dispatch(a, p, true, blocks, stream);
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  return launch_reduce_parts(part, 1, blocks, a.head_dim, dgain_q, dgain_k, a.dtype, stream);
}

}  // namespace pf
