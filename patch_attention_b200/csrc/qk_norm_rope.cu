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
// half-split pairs (e1 = e0 + w_a / 2).  A block takes 1 to 4 tokens; its threads first compute the
// tokens' cosines and sines once, into shared memory, then each warp walks its share of a
// token's heads, 32 / SEG vectors a step, several steps' loads in flight.  Angles are taken in turns,
// pos * (theta^(-2i/w) / 2 pi) in 64 bits, and only their fraction is rounded to 32 bits, so far
// positions lose nothing.
// Measured on a B200: 4096 x (24 + 24) x 128 bf16 forward 25.5 us, 4.0 TB/s, backward 51 us; 16384 x
// (24 + 24) x 64 forward 42 us (neighbouring pairs) and 44 us (split halves), 4.6 to 4.8 TB/s,
// backward 82 and 105 us.  What is left of HBM's rate goes to the start of each block (its angles)
// and to instruction issue (61% of the slots), and in the backward pass to the registers of two tensors' vectors and the gains' sums.
//
// The backward pass keeps the gain-gradient sums of a lane's elements in registers while its
// block walks tokens; blocks write fp32 partials that a second kernel adds in a fixed order.

#include <type_traits>

#include "block_ops.cuh"

namespace pf {
namespace {

using namespace blk;

constexpr int kWarps = 4;

struct RopeParams {  // (pointers and strides of q, k)
  const void* x[2];   // forward input, backward saved input (null without norm)
  const void* dy[2];  // backward: gradients of the rotated output
  void* y[2];         // forward: output; backward: dx
  const void* gain[2];
  long long xs[2][3], ds[2][3], ys[2][3];  // element strides: batch, token, head
  const float* pos;   // [tokens][n_axes] (pos_batch apart per batch element)
  long long pos_batch;
  float* part;        // backward: [block][2][head_dim], or null
  int total;          // batch * tokens
  int tokens, n_axes, heads[2], head_dim;
  int shares;         // warps of a block that share a token's heads: 1, 2 or 4
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
  __device__ __forceinline__ T first(int k) const { return INTER ? v[0].v[2 * k] : v[k / PV].v[k % PV]; }
  __device__ __forceinline__ T second(int k) const {
    return INTER ? v[0].v[2 * k + 1] : v[4 / PV + k / PV].v[k % PV];
  }
  // first (a) and second (b) elements of pairs 0, 1 and 2, 3
  __device__ __forceinline__ void get(float2 (&a)[2], float2 (&b)[2]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      a[j] = make_float2(to_f<T>(first(2 * j)), to_f<T>(first(2 * j + 1)));
      b[j] = make_float2(to_f<T>(second(2 * j)), to_f<T>(second(2 * j + 1)));
    }
  }
  __device__ __forceinline__ void put(const float2 (&a)[2], const float2 (&b)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (INTER) {
        put2(v[0].v + 4 * j, a[j].x, b[j].x);
        put2(v[0].v + 4 * j + 2, a[j].y, b[j].y);
      } else if constexpr (PV >= 2) {
        put2(v[2 * j / PV].v + 2 * j % PV, a[j].x, a[j].y);
        put2(v[4 / PV + 2 * j / PV].v + 2 * j % PV, b[j].x, b[j].y);
      } else {
        v[2 * j].v[0] = from_f<T>(a[j].x);
        v[2 * j + 1].v[0] = from_f<T>(a[j].y);
        v[4 + 2 * j].v[0] = from_f<T>(b[j].x);
        v[5 + 2 * j].v[0] = from_f<T>(b[j].y);
      }
    }
  }
  static __device__ __forceinline__ void put2(T* to, float x, float y) {
    if constexpr (sizeof(T) == 4) {
      to[0] = x;
      to[1] = y;
    } else if constexpr (std::is_same<T, __half>::value) {
      *reinterpret_cast<__half2*>(to) = __floats2half2_rn(x, y);
    } else {
      *reinterpret_cast<__nv_bfloat162*>(to) = __floats2bfloat162_rn(x, y);
    }
  }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 neg(float2 v) { return make_float2(-v.x, -v.y); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
// a where the bits of pairs 2 j and 2 j + 1 are set, else b
__device__ __forceinline__ float2 pick(unsigned bits, int j, float2 a, float2 b) {
  return make_float2(bits >> (2 * j) & 1u ? a.x : b.x, bits >> (2 * j + 1) & 1u ? a.y : b.y);
}

// cos and sin of a lane's four pairs.
__device__ __forceinline__ void read_angles(const float2* at, float2 (&c)[2], float2 (&s)[2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 u = at[2 * j], v = at[2 * j + 1];
    c[j] = make_float2(u.x, v.x);
    s[j] = make_float2(u.y, v.y);
  }
}

template <int SEG>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int off = SEG / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A lane's place in a vector: its pairs' elements (three table words, four pairs each).
struct Lane {
  int sub, e0[4], e1[4], pair0;
  bool active;
  unsigned turn;  // bit k: pair k turns (pairs past the axes are copied)
  template <bool INTER, int SEG>
  static __device__ __forceinline__ Lane make(const RopeParams& p) {
    Lane l;
    const int lane = threadIdx.x & 31, chunk = lane % SEG;
    l.sub = lane / SEG;
    l.active = chunk * 8 < p.head_dim;
    l.pair0 = l.active ? chunk * 4 : 0;
    const uint32_t ax = *reinterpret_cast<const uint32_t*>(p.tab.axis + l.pair0);
    const uint32_t w0 = INTER ? 0u : *reinterpret_cast<const uint32_t*>(p.tab.e0 + l.pair0);
    const uint32_t w1 = INTER ? 0u : *reinterpret_cast<const uint32_t*>(p.tab.e1 + l.pair0);
    l.turn = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      l.e0[k] = INTER ? 2 * (l.pair0 + k) : static_cast<int>(w0 >> (8 * k) & 255u);
      l.e1[k] = INTER ? 2 * (l.pair0 + k) + 1 : static_cast<int>(w1 >> (8 * k) & 255u);
      l.turn |= (static_cast<int>(ax >> (8 * k) & 255u) < p.n_axes ? 1u : 0u) << k;
    }
    return l;
  }
};

// This warp's token and its share of the token's heads.
struct Item {
  unsigned b, tok;
  int slot, share;   // token of the block, share of the token within the block
  int lo[2], hi[2];  // heads of q, k
  bool on;
  __device__ Item(const RopeParams& p, unsigned first, int warp, int split, int splits) {
    slot = warp / p.shares;
    share = warp - slot * p.shares;
    const unsigned bt = first + slot;
    on = bt < static_cast<unsigned>(p.total);
    b = bt / static_cast<unsigned>(p.tokens);
    tok = bt - b * static_cast<unsigned>(p.tokens);
    const int n = p.heads[0] + p.heads[1], at = split * p.shares + share, all = splits * p.shares;
    const int each = n / all, more = n - each * all;  // the first `more` shares take one head more
    const int from = at * each + min(at, more), to = on ? from + each + (at < more ? 1 : 0) : from;
    lo[0] = min(from, p.heads[0]);
    hi[0] = min(to, p.heads[0]);
    lo[1] = max(from - p.heads[0], 0);
    hi[1] = max(to - p.heads[0], 0);
  }
  // cos and sin of the token's pairs into `cs`, by the warps that share the token
  __device__ __forceinline__ void fill_angles(const RopeParams& p, float2* cs) const {
    if (!on) return;
    for (int k = (threadIdx.x & 31) + 32 * share; k < p.head_dim / 2; k += 32 * p.shares) {
      const int axis = p.tab.axis[k];
      float c = 1.f, s = 0.f;
      if (axis < p.n_axes) {
        const float at = __ldg(p.pos + b * p.pos_batch + static_cast<long long>(tok) * p.n_axes + axis);
        const double turns = static_cast<double>(at) * p.tab.turns[k];
        sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
      }
      cs[slot * 128 + k] = make_float2(c, s);
    }
  }
  // this lane's first vector of operand w of a tensor, and the distance between its vectors
  template <typename T, int PER>
  __device__ __forceinline__ T* start(const void* base, const long long (&st)[3], int w, const Lane& ln, long long& step) const {
    step = st[2] * PER;
    return static_cast<T*>(const_cast<void*>(base)) + b * st[0] + tok * st[1] + (lo[w] + ln.sub) * st[2];
  }
};

template <typename T, bool INTER, int PV>
__device__ __forceinline__ void load_gain(const void* g, const Lane& ln, float2 (&ga)[2], float2 (&gb)[2]) {
  ga[0] = ga[1] = gb[0] = gb[1] = both(1.f);
  if (g != nullptr) {
    Raw<T, INTER, PV> r;
    r.load(static_cast<const T*>(g), ln.e0, ln.e1);
    r.get(ga, gb);
  }
}

// FULL: every pair turns.
template <typename T, bool INTER, int PV, int SEG, bool FULL>
__global__ void __launch_bounds__(32 * kWarps, INTER ? 7 : 0) rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPer = 32 / SEG;
  constexpr int kSteps = 4;
  __shared__ float2 cs[kWarps * 128];
  const Lane ln = Lane::make<INTER, SEG>(p);
  const Item it(p, blockIdx.x * static_cast<unsigned>(kWarps / p.shares), threadIdx.x >> 5, blockIdx.y, gridDim.y);
  const float inv_d = 1.f / static_cast<float>(p.head_dim);
  const bool norm = p.eps > 0.f;
  // kSteps vectors of x, of which this lane has `left`
  Raw<T, INTER, PV> raw[kSteps];
  auto fetch = [&](const T*& x, long long step, int left) {
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      raw[u].zero();
      if (u * kPer < left) raw[u].load(x, ln.e0, ln.e1);
      x += step;
    }
  };
  // Pairs of neighbours: the first vectors are on their way while the angles are computed (4096 x 24
  // x 128: 27.7 to 25.8 us; the pieces of split halves need too many registers for that: 44.7 and
  // 48.7 us at 16384 x 24 x 64).
  const int w0 = !INTER ? 2 : it.lo[0] < it.hi[0] ? 0 : 1;
  if (INTER && it.lo[w0 & 1] < it.hi[w0 & 1]) {
    long long xstep;
    const T* x = it.start<T, kPer>(p.x[w0 & 1], p.xs[w0 & 1], w0 & 1, ln, xstep);
    fetch(x, xstep, ln.active ? it.hi[w0 & 1] - it.lo[w0 & 1] - ln.sub : 0);
  }
  it.fill_angles(p, cs);
  __syncthreads();
  float2 c[2], s[2];
  read_angles(cs + it.slot * 128 + ln.pair0, c, s);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (it.lo[w] >= it.hi[w]) continue;
    float2 ga[2], gb[2];
    load_gain<T, INTER, PV>(p.gain[w], ln, ga, gb);
    long long xstep, ystep;
    const T* x = it.start<T, kPer>(p.x[w], p.xs[w], w, ln, xstep);
    bool here = INTER && w == w0;  // the first vectors
    if (here) x += kSteps * xstep;
    T* y = it.start<T, kPer>(p.y[w], p.ys[w], w, ln, ystep);
    // vectors of this lane left (none for a lane past the vector's end)
    int left = ln.active ? it.hi[w] - it.lo[w] - ln.sub : 0;
    for (int steps = (it.hi[w] - it.lo[w] + kPer - 1) / kPer; steps > 0; steps -= kSteps) {
      if (!here) fetch(x, xstep, left);
      here = false;
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        if (u >= steps) break;  // the whole warp
        float2 a[2], b[2], ya[2], yb[2];
        raw[u].get(a, b);
        float2 r = both(1.f);
        if (norm) {
          const float2 q = fma2(a[0], a[0], fma2(b[0], b[0], fma2(a[1], a[1], mul2(b[1], b[1]))));
          r = both(rsqrtf(fmaf(seg_sum<SEG>(q.x + q.y), inv_d, p.eps)));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          a[j] = mul2(a[j], mul2(r, ga[j]));
          b[j] = mul2(b[j], mul2(r, gb[j]));
          ya[j] = fma2(a[j], c[j], mul2(b[j], neg(s[j])));
          yb[j] = fma2(a[j], s[j], mul2(b[j], c[j]));
          if (!FULL) {
            ya[j] = pick(ln.turn, j, ya[j], a[j]);
            yb[j] = pick(ln.turn, j, yb[j], b[j]);
          }
        }
        raw[u].put(ya, yb);
        if (u * kPer < left) raw[u].store(y, ln.e0, ln.e1);
        y += ystep;
      }
      left -= kPer * kSteps;
    }
  }
}

template <typename T, bool INTER, int PV, int SEG, bool FULL>
__global__ void __launch_bounds__(32 * kWarps, 4) rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPer = 32 / SEG;
  constexpr int kSteps = 2;
  // only for the reduction: other programmatic dependents may read their inputs as soon as they start
  if (p.part != nullptr) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float2 cs[2][kWarps * 128];
  __shared__ float red[2][256];
  const Lane ln = Lane::make<INTER, SEG>(p);
  const int warp = threadIdx.x >> 5;
  float2 sa[2][2], sb[2][2];  // gain gradients of q, k
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int j = 0; j < 2; ++j) sa[w][j] = sb[w][j] = both(0.f);
  const float inv_d = 1.f / static_cast<float>(p.head_dim);
  const bool norm = p.eps > 0.f;
  const unsigned per_block = static_cast<unsigned>(kWarps / p.shares), stride = gridDim.x * per_block;
  int buf = 0;
  for (unsigned first = blockIdx.x * per_block; first < static_cast<unsigned>(p.total); first += stride, buf ^= 1) {
    const Item it(p, first, warp, 0, 1);
    // two tables in turn: the barrier of the next tokens also covers this one's readers
    it.fill_angles(p, cs[buf]);
    __syncthreads();
    float2 c[2], s[2];
    read_angles(cs[buf] + it.slot * 128 + ln.pair0, c, s);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (it.lo[w] >= it.hi[w]) continue;
      float2 ga[2], gb[2];
      load_gain<T, INTER, PV>(p.gain[w], ln, ga, gb);
      long long xstep = 0, dstep, ystep;
      const T* x = norm ? it.start<T, kPer>(p.x[w], p.xs[w], w, ln, xstep) : nullptr;
      const T* d = it.start<T, kPer>(p.dy[w], p.ds[w], w, ln, dstep);
      T* y = it.start<T, kPer>(p.y[w], p.ys[w], w, ln, ystep);
      int left = ln.active ? it.hi[w] - it.lo[w] - ln.sub : 0;
      for (int steps = (it.hi[w] - it.lo[w] + kPer - 1) / kPer; steps > 0; steps -= kSteps) {
        Raw<T, INTER, PV> rd[kSteps], rx[kSteps];
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          rd[u].zero();
          rx[u].zero();
          if (u * kPer < left) {
            rd[u].load(d, ln.e0, ln.e1);
            if (norm) rx[u].load(x, ln.e0, ln.e1);
          }
          d += dstep;
          x += xstep;
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          if (u >= steps) break;  // the whole warp
          float2 da[2], db[2], za[2], zb[2];
          rd[u].get(da, db);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            za[j] = fma2(da[j], c[j], mul2(db[j], s[j]));
            zb[j] = fma2(db[j], c[j], mul2(da[j], neg(s[j])));
            if (!FULL) {
              za[j] = pick(ln.turn, j, za[j], da[j]);
              zb[j] = pick(ln.turn, j, zb[j], db[j]);
            }
          }
          if (norm) {
            float2 a[2], b[2], ta[2], tb[2];
            rx[u].get(a, b);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              ta[j] = mul2(za[j], ga[j]);
              tb[j] = mul2(zb[j], gb[j]);
            }
            const float2 qs = fma2(a[0], a[0], fma2(b[0], b[0], fma2(a[1], a[1], mul2(b[1], b[1]))));
            const float2 qx = fma2(ta[0], a[0], fma2(tb[0], b[0], fma2(ta[1], a[1], mul2(tb[1], b[1]))));
            const float ss = seg_sum<SEG>(qs.x + qs.y), sx = seg_sum<SEG>(qx.x + qx.y);
            const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
            const float2 r2 = both(r), m = both(-r * r * sx * inv_d);  // r mean(a x^) = r^2 mean(a x): times x, then r
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // an absent head has dz = x = 0 and adds nothing
              sa[w][j] = fma2(za[j], mul2(a[j], r2), sa[w][j]);
              sb[w][j] = fma2(zb[j], mul2(b[j], r2), sb[w][j]);
              za[j] = mul2(r2, fma2(a[j], m, ta[j]));
              zb[j] = mul2(r2, fma2(b[j], m, tb[j]));
            }
          }
          if (u * kPer < left) {
            rd[u].put(za, zb);
            rd[u].store(y, ln.e0, ln.e1);
          }
          y += ystep;
        }
        left -= kPer * kSteps;
      }
    }
  }
  if (p.part == nullptr) return;
  // the warp's sub-vectors, then the block's warps in order
  float v[2][2][4];  // [q, k][first, second][pair]
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[w][0][k] = k & 1 ? sa[w][k / 2].y : sa[w][k / 2].x;
      v[w][1][k] = k & 1 ? sb[w][k / 2].y : sb[w][k / 2].x;
#pragma unroll
      for (int off = 16; off >= SEG; off >>= 1) {
        v[w][0][k] += __shfl_xor_sync(0xffffffffu, v[w][0][k], off);
        v[w][1][k] += __shfl_xor_sync(0xffffffffu, v[w][1][k], off);
      }
    }
  for (int wi = 0; wi < kWarps; ++wi) {
    if (warp == wi && ln.sub == 0 && ln.active) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          red[w][ln.e0[k]] = wi == 0 ? v[w][0][k] : red[w][ln.e0[k]] + v[w][0][k];
          red[w][ln.e1[k]] = wi == 0 ? v[w][1][k] : red[w][ln.e1[k]] + v[w][1][k];
        }
    }
    __syncthreads();
  }
  float* out = p.part + static_cast<long long>(blockIdx.x) * 2 * p.head_dim;
  for (int e = threadIdx.x; e < 2 * p.head_dim; e += 32 * kWarps)
    out[e] = red[e >= p.head_dim][e >= p.head_dim ? e - p.head_dim : e];
}

template <typename T, bool INTER, int PV, int SEG, bool FULL>
cudaError_t launch_full(const RopeParams& p, bool bwd, dim3 blocks, cudaStream_t stream) {
  if (bwd)
    rope_bwd_kernel<T, INTER, PV, SEG, FULL><<<blocks, 32 * kWarps, 0, stream>>>(p);
  else
    rope_fwd_kernel<T, INTER, PV, SEG, FULL><<<blocks, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, bool INTER, int PV, int SEG>
cudaError_t launch_kernel(const RopeParams& p, bool bwd, dim3 blocks, cudaStream_t stream) {
  // the last pair turns: all do, as the sections come first
  if (p.tab.axis[p.head_dim / 2 - 1] < p.n_axes) return launch_full<T, INTER, PV, SEG, true>(p, bwd, blocks, stream);
  return launch_full<T, INTER, PV, SEG, false>(p, bwd, blocks, stream);
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
// tokens give every SM 64 warps (several rounds of what is resident: a short last round costs
// little), and, where kWarps are not enough, the heads of a
// token over `splits` blocks (forward only).
struct Grid {
  int shares, splits, blocks;
};
Grid grid_of(const RopeParams& p, bool bwd) {
  const int chunks = p.head_dim / 8;
  const int per_step = chunks <= 4 ? 8 : chunks <= 8 ? 4 : chunks <= 16 ? 2 : 1;  // vectors of a warp at once
  const long long steps = (p.heads[0] + p.heads[1] + per_step - 1) / per_step;    // most warps with work
  const long long total = p.total;  // up to 2^31 - 1: sums in 64 bits
  const long long want = (148 * 64 + total - 1) / total;
  Grid g = {1, 1, 0};
  while (g.shares < kWarps && g.shares < want && g.shares < steps) g.shares *= 2;
  if (!bwd && g.shares == kWarps) {
    const long long more = want < steps ? want : steps;
    g.splits = static_cast<int>((more + kWarps - 1) / kWarps);
  }
  const int per_block = kWarps / g.shares;
  g.blocks = static_cast<int>((total + per_block - 1) / per_block);
  // backward: the blocks that are resident at once walk the tokens, so that few partial gain
  // gradients are written
  if (bwd && g.blocks > 148 * 4) g.blocks = 148 * 4;
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
