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
// half-split pairs (e1 = e0 + w_a / 2).  A block takes 1 to 8 tokens; its threads first compute the
// tokens' cosines and sines once, into shared memory (behind the first loads), then each warp
// walks its share of a token's heads, 32 / SEG vectors at a time with kUnroll steps of loads in
// flight.  Angles are taken in turns, pos * (theta^(-2i/w) / 2 pi) in 64 bits, and only their
// fraction is rounded to 32 bits, so far positions lose nothing.
//
// The backward pass keeps the gain-gradient sums of a lane's elements in registers while its
// block walks tokens; blocks write fp32 partials that a second kernel adds in a fixed order.

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
  int total;          // batch * tokens
  int tokens, n_axes, heads[2], head_dim;
  int shares;         // warps of a block that share a token's heads: 1, 2, 4 or 8
  float eps;          // 0: no norm
  RopeTable tab;
};

// A lane's eight elements as read: one run (INTER) or PV-element pieces of both halves.
template <typename T, bool INTER, int PV>
struct Raw {
  Vec<T, INTER ? 8 : PV> v[INTER ? 1 : 8 / PV];

  __device__ __forceinline__ void load(const T* p, const int (&e0)[4], const int (&e1)[4]) {
    if constexpr (INTER) {
      v[0] = load_vec<T, 8>(p + e0[0]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; k += PV) {
        v[k / PV] = load_vec<T, PV>(p + e0[k]);
        v[4 / PV + k / PV] = load_vec<T, PV>(p + e1[k]);
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (INTER ? 1 : 8 / PV); ++i)
#pragma unroll
      for (int k = 0; k < (INTER ? 8 : PV); ++k) v[i].v[k] = from_f<T>(0.f);
  }
  __device__ __forceinline__ void store(T* p, const int (&e0)[4], const int (&e1)[4]) const {
    if constexpr (INTER) {
      store_vec<T, 8>(p + e0[0], v[0]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; k += PV) {
        store_vec<T, PV>(p + e0[k], v[k / PV]);
        store_vec<T, PV>(p + e1[k], v[4 / PV + k / PV]);
      }
    }
  }
  // first and second elements of the four pairs
  __device__ __forceinline__ void get(float (&a)[4], float (&b)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = to_f<T>(INTER ? v[0].v[2 * k] : v[k / PV].v[k % PV]);
      b[k] = to_f<T>(INTER ? v[0].v[2 * k + 1] : v[4 / PV + k / PV].v[k % PV]);
    }
  }
  __device__ __forceinline__ void put(const float (&a)[4], const float (&b)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      (INTER ? v[0].v[2 * k] : v[k / PV].v[k % PV]) = from_f<T>(a[k]);
      (INTER ? v[0].v[2 * k + 1] : v[4 / PV + k / PV].v[k % PV]) = from_f<T>(b[k]);
    }
  }
};

// cos and sin of every pair of the block's tokens, [token of the block][pair].
__device__ __forceinline__ void fill_angles(const RopeParams& p, float2* cs, unsigned first, int count) {
  const int pairs = p.head_dim / 2;
  for (int i = threadIdx.x; i < count * pairs; i += 32 * kWarps) {
    const int t = i / pairs, k = i - t * pairs;
    const unsigned bt = first + t;
    if (bt >= static_cast<unsigned>(p.total)) break;
    const unsigned b = bt / static_cast<unsigned>(p.tokens), tok = bt - b * static_cast<unsigned>(p.tokens);
    const int axis = p.tab.axis[k];
    float c = 1.f, s = 0.f;
    if (axis < p.n_axes) {
      const float at = __ldg(p.pos + b * p.pos_batch + static_cast<long long>(tok) * p.n_axes + axis);
      const double turns = static_cast<double>(at) * p.tab.turns[k];
      sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
    }
    cs[t * 128 + k] = make_float2(c, s);
  }
}

template <int SEG>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int off = SEG / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// This warp's token and heads of a block's tokens.
struct Item {
  unsigned b, tok;
  int slot, lo, hi;  // token of the block; heads [lo, hi) of q's and k's together
  bool on;
  __device__ Item(const RopeParams& p, unsigned first, int warp, int split, int splits) {
    slot = warp / p.shares;
    const unsigned bt = first + slot;
    on = bt < static_cast<unsigned>(p.total);
    b = bt / static_cast<unsigned>(p.tokens);
    tok = bt - b * static_cast<unsigned>(p.tokens);
    const int n = p.heads[0] + p.heads[1], share = split * p.shares + warp % p.shares, all = splits * p.shares;
    lo = static_cast<int>(static_cast<long long>(n) * share / all);
    hi = static_cast<int>(static_cast<long long>(n) * (share + 1) / all);
  }
};

// A lane's place in a vector.
struct Lane {
  int sub, e0[4], e1[4], pair0;
  bool active;
  unsigned turn;  // bit k: pair k turns (pairs past the axes are copied)
  template <int SEG>
  static __device__ __forceinline__ Lane make(const RopeParams& p) {
    Lane l;
    const int lane = threadIdx.x & 31, chunk = lane % SEG;
    l.sub = lane / SEG;
    l.active = chunk * 8 < p.head_dim;
    l.pair0 = l.active ? chunk * 4 : 0;
    l.turn = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      l.e0[k] = p.tab.e0[l.pair0 + k];
      l.e1[k] = p.tab.e1[l.pair0 + k];
      l.turn |= (p.tab.axis[l.pair0 + k] < p.n_axes ? 1u : 0u) << k;
    }
    return l;
  }
};

template <typename T, bool INTER, int PV, int SEG>
__global__ void __launch_bounds__(32 * kWarps) rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPer = 32 / SEG;
  constexpr int kUnroll = 4;
  __shared__ float2 cs[kWarps * 128];
  const Lane ln = Lane::make<SEG>(p);
  const int per_block = kWarps / p.shares;
  const unsigned first = blockIdx.x * static_cast<unsigned>(per_block);
  const Item it(p, first, threadIdx.x >> 5, blockIdx.y, gridDim.y);
  const float inv_d = 1.f / static_cast<float>(p.head_dim);
  const bool norm = p.eps > 0.f;
  bool filled = false;
  float c[4], s[4];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int lo = w ? max(it.lo - p.heads[0], 0) : it.lo, hi = w ? it.hi - p.heads[0] : min(it.hi, p.heads[0]);
    if (w == 1 && (!it.on || lo >= hi)) break;
    const bool any = it.on && lo < hi;
    const T* x = static_cast<const T*>(p.x[w]) + it.b * p.xs[w][0] + it.tok * p.xs[w][1];
    T* y = static_cast<T*>(p.y[w]) + it.b * p.ys[w][0] + it.tok * p.ys[w][1];
    float ga[4], gb[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) ga[k] = gb[k] = 1.f;
    if (any && p.gain[w] != nullptr) {
      Raw<T, INTER, PV> g;
      g.load(static_cast<const T*>(p.gain[w]), ln.e0, ln.e1);
      g.get(ga, gb);
    }
    for (int h0 = lo; h0 < hi || !filled; h0 += kPer * kUnroll) {
      Raw<T, INTER, PV> raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * kPer + ln.sub;
        if (any && ln.active && h < hi)
          raw[u].load(x + h * p.xs[w][2], ln.e0, ln.e1);
        else
          raw[u].zero();
      }
      if (!filled) {
        fill_angles(p, cs, first, per_block);
        __syncthreads();
        filled = true;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = cs[it.slot * 128 + ln.pair0 + k];
          c[k] = v.x;
          s[k] = v.y;
        }
      }
      float a[kUnroll][4], b[kUnroll][4], r[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        raw[u].get(a[u], b[u]);
        r[u] = 1.f;
      }
      if (norm) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          float ss = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) ss = fmaf(a[u][k], a[u][k], fmaf(b[u][k], b[u][k], ss));
          r[u] = rsqrtf(fmaf(seg_sum<SEG>(ss), inv_d, p.eps));
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * kPer + ln.sub;
        float ya[4], yb[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float za = a[u][k] * (r[u] * ga[k]), zb = b[u][k] * (r[u] * gb[k]);
          const bool turn = ln.turn >> k & 1u;
          ya[k] = turn ? za * c[k] - zb * s[k] : za;
          yb[k] = turn ? za * s[k] + zb * c[k] : zb;
        }
        raw[u].put(ya, yb);
        if (any && ln.active && h < hi) raw[u].store(y + h * p.ys[w][2], ln.e0, ln.e1);
      }
    }
  }
}

template <typename T, bool INTER, int PV, int SEG>
__global__ void __launch_bounds__(32 * kWarps, 2) rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPer = 32 / SEG;
  constexpr int kUnroll = 2;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float2 cs[2][kWarps * 128];
  __shared__ float red[2][256];
  const Lane ln = Lane::make<SEG>(p);
  const int warp = threadIdx.x >> 5;
  const int per_block = kWarps / p.shares;
  float sa[2][4], sb[2][4];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int k = 0; k < 4; ++k) sa[w][k] = sb[w][k] = 0.f;
  const float inv_d = 1.f / static_cast<float>(p.head_dim);
  const bool norm = p.eps > 0.f;
  const unsigned stride = gridDim.x * static_cast<unsigned>(per_block);
  int buf = 0;
  for (unsigned first = blockIdx.x * static_cast<unsigned>(per_block); first < static_cast<unsigned>(p.total);
       first += stride, buf ^= 1) {
    const Item it(p, first, warp, 0, 1);
    bool filled = false;
    float c[4], s[4];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int lo = w ? max(it.lo - p.heads[0], 0) : it.lo, hi = w ? it.hi - p.heads[0] : min(it.hi, p.heads[0]);
      if (w == 1 && (!it.on || lo >= hi)) break;
      const bool any = it.on && lo < hi;
      const T* x = static_cast<const T*>(p.x[w]) + it.b * p.xs[w][0] + it.tok * p.xs[w][1];
      const T* d = static_cast<const T*>(p.dy[w]) + it.b * p.ds[w][0] + it.tok * p.ds[w][1];
      T* y = static_cast<T*>(p.y[w]) + it.b * p.ys[w][0] + it.tok * p.ys[w][1];
      float ga[4], gb[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) ga[k] = gb[k] = 1.f;
      if (any && p.gain[w] != nullptr) {
        Raw<T, INTER, PV> g;
        g.load(static_cast<const T*>(p.gain[w]), ln.e0, ln.e1);
        g.get(ga, gb);
      }
      for (int h0 = lo; h0 < hi || !filled; h0 += kPer * kUnroll) {
        Raw<T, INTER, PV> rd[kUnroll], rx[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int h = h0 + u * kPer + ln.sub;
          rd[u].zero();
          rx[u].zero();
          if (any && ln.active && h < hi) {
            rd[u].load(d + h * p.ds[w][2], ln.e0, ln.e1);
            if (norm) rx[u].load(x + h * p.xs[w][2], ln.e0, ln.e1);
          }
        }
        if (!filled) {
          // two tables in turn: the barrier of the next tokens also covers this one's readers
          fill_angles(p, cs[buf], first, per_block);
          __syncthreads();
          filled = true;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = cs[buf][it.slot * 128 + ln.pair0 + k];
            c[k] = v.x;
            s[k] = v.y;
          }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int h = h0 + u * kPer + ln.sub;
          float da[4], db[4], za[4], zb[4];
          rd[u].get(da, db);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool turn = ln.turn >> k & 1u;
            za[k] = turn ? da[k] * c[k] + db[k] * s[k] : da[k];
            zb[k] = turn ? db[k] * c[k] - da[k] * s[k] : db[k];
          }
          if (norm) {
            float a[4], b[4], ta[4], tb[4], ss = 0.f, sx = 0.f;
            rx[u].get(a, b);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              ta[k] = za[k] * ga[k];
              tb[k] = zb[k] * gb[k];
              ss = fmaf(a[k], a[k], fmaf(b[k], b[k], ss));
              sx = fmaf(ta[k], a[k], fmaf(tb[k], b[k], sx));
            }
            ss = seg_sum<SEG>(ss);
            sx = seg_sum<SEG>(sx);
            const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
            const float m = r * r * sx * inv_d;  // r mean(a x^) = r^2 mean(a x): times x, then r
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // an absent head has dz = x = 0 and adds nothing
              sa[w][k] = fmaf(za[k], a[k] * r, sa[w][k]);
              sb[w][k] = fmaf(zb[k], b[k] * r, sb[w][k]);
              za[k] = r * (ta[k] - a[k] * m);
              zb[k] = r * (tb[k] - b[k] * m);
            }
          }
          if (any && ln.active && h < hi) {
            rd[u].put(za, zb);
            rd[u].store(y + h * p.ys[w][2], ln.e0, ln.e1);
          }
        }
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
    if (warp == wi && ln.sub == 0 && ln.active) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          red[w][ln.e0[k]] = wi == 0 ? sa[w][k] : red[w][ln.e0[k]] + sa[w][k];
          red[w][ln.e1[k]] = wi == 0 ? sb[w][k] : red[w][ln.e1[k]] + sb[w][k];
        }
    }
    __syncthreads();
  }
  float* out = p.part + static_cast<long long>(blockIdx.x) * 2 * p.head_dim;
  for (int e = threadIdx.x; e < 2 * p.head_dim; e += 32 * kWarps)
    out[e] = red[e >= p.head_dim][e >= p.head_dim ? e - p.head_dim : e];
}

template <typename T, bool INTER, int PV, int SEG>
cudaError_t launch_kernel(const RopeParams& p, bool bwd, dim3 blocks, cudaStream_t stream) {
  if (bwd)
    rope_bwd_kernel<T, INTER, PV, SEG><<<blocks, 32 * kWarps, 0, stream>>>(p);
  else
    rope_fwd_kernel<T, INTER, PV, SEG><<<blocks, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, bool INTER, int PV>
cudaError_t launch_seg(const RopeParams& p, bool bwd, dim3 blocks, cudaStream_t stream) {
  const int chunks = p.head_dim / 8;
  if (chunks <= 4) return launch_kernel<T, INTER, PV, 4>(p, bwd, blocks, stream);
  if (chunks <= 8) return launch_kernel<T, INTER, PV, 8>(p, bwd, blocks, stream);
  if (chunks <= 16) return launch_kernel<T, INTER, PV, 16>(p, bwd, blocks, stream);
  return launch_kernel<T, INTER, PV, 32>(p, bwd, blocks, stream);
}

template <typename T>
cudaError_t launch_type(const RopeParams& p, bool inter, bool bwd, dim3 blocks, cudaStream_t stream) {
  if (inter) return launch_seg<T, true, 4>(p, bwd, blocks, stream);
  // half-split pairs: 4, 2 or 1 consecutive elements of a lane's pairs lie side by side,
  // aligned, when every section's half is a multiple of that
  if (p.tab.half_align % 4 == 0) return launch_seg<T, false, 4>(p, bwd, blocks, stream);
  if (p.tab.half_align % 2 == 0) return launch_seg<T, false, 2>(p, bwd, blocks, stream);
  return launch_seg<T, false, 1>(p, bwd, blocks, stream);
}

cudaError_t dispatch(const RopeArgs& a, const RopeParams& p, bool bwd, dim3 blocks, cudaStream_t stream) {
  switch (a.dtype) {
    case PF_BF16: return launch_type<__nv_bfloat16>(p, a.interleaved, bwd, blocks, stream);
    case PF_F16: return launch_type<__half>(p, a.interleaved, bwd, blocks, stream);
    default: return launch_type<float>(p, a.interleaved, bwd, blocks, stream);
  }
}

// How a call's tokens and heads are laid over blocks: `shares` warps per token so that the
// tokens give every SM sixteen warps or more, and, where eight are not enough, the heads of a
// token over `splits` blocks (forward only).
struct Grid {
  int shares, splits, blocks;
};
Grid grid_of(const RopeParams& p, bool bwd) {
  const int chunks = p.head_dim / 8;
  const int per_step = chunks <= 4 ? 8 : chunks <= 8 ? 4 : chunks <= 16 ? 2 : 1;  // vectors of a warp at once
  const long long steps = (p.heads[0] + p.heads[1] + per_step - 1) / per_step;    // most warps with work
  const long long want = (148 * 16 + p.total - 1) / p.total;
  Grid g = {1, 1, 0};
  while (g.shares < 8 && g.shares < want && g.shares < steps) g.shares *= 2;
  if (!bwd && g.shares == 8) {
    const long long more = want < steps ? want : steps;
    g.splits = static_cast<int>((more + 7) / 8);
  }
  const int per_block = kWarps / g.shares;
  g.blocks = (p.total + per_block - 1) / per_block;
  // backward: two blocks per SM walk the tokens, so that few partial gain gradients are written
  if (bwd && g.blocks > 148 * 2) g.blocks = 148 * 2;
  return g;
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
  p.total = a.batch * a.tokens;  // at most 2^31 - 1, checked
  p.tokens = a.tokens;
  p.n_axes = a.n_axes;
  p.head_dim = a.head_dim;
  p.eps = a.eps;
  p.tab = a.tab;
  return p;
}

}  // namespace

// Blocks of the backward pass, each writing one partial row of gain gradients.
int rope_bwd_blocks(const RopeArgs& a) {
  const RopeParams p = params_of(a);
  return p.total == 0 ? 0 : grid_of(p, true).blocks;
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t stream) {
  RopeParams p = params_of(a);
  if (p.total == 0) return cudaSuccess;
  const Grid g = grid_of(p, false);
  p.shares = g.shares;
  return dispatch(a, p, false, dim3(static_cast<unsigned>(g.blocks), static_cast<unsigned>(g.splits)), stream);
}

cudaError_t launch_qk_norm_rope_bwd(const RopeArgs& a, void* dgain_q, void* dgain_k, float* part, cudaStream_t stream) {
  RopeParams p = params_of(a);
  const bool sums = dgain_q != nullptr || dgain_k != nullptr;
  p.part = sums ? part : nullptr;
  Grid g = {1, 1, 0};
  if (p.total > 0) {
    g = grid_of(p, true);
    p.shares = g.shares;
    const cudaError_t e = dispatch(a, p, true, dim3(static_cast<unsigned>(g.blocks)), stream);
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  return launch_reduce_parts(part, 1, g.blocks, a.head_dim, dgain_q, dgain_k, a.dtype, stream);
}

}  // namespace pf
