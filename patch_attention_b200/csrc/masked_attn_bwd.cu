// masked_attn_bwd.cu -- gradients of the masked attention of masked_attn.cu for sm_100a.
//
//   p_ij = exp(s_ij - lse_i) over the visible keys, delta_i = sum_d o_id do_id
//   ds_ij = p_ij (do_i.v_j - delta_i) (1 - tanh^2)      (the last factor with a cap)
//   dv_j = sum_i p_ij do_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j
//   (dk and dv also sum over the query heads that share the key head)
//
// A small kernel computes delta.  Then one kernel template runs twice, once per side whose rows
// stay: for 128 keys (their K and V tiles stay in shared memory, the Q and dO tiles of every query
// head of the key head stream past; dK and dV accumulate in TMEM) and for 128 queries (Q and dO
// stay, K and V stream; dQ accumulates).  Nothing is added through memory, so there are no atomics
// and the sums have one order.  The price is that s and do.v are computed twice: 7 matrix products
// instead of 5.
//
// With X1, X2 the staying and Y1, Y2 the streaming tiles, for each 64-row half h of a Y tile:
//   S_h = X1 Y1_h^T, dP_h = X2 Y2_h^T into TMEM; a softmax warpgroup (one thread per staying row) turns
//   them into P_h and dS_h, written back over them as bf16;  accV += P_h Y2_h (keys stay only),
//   accK += dS_h Y1_h with P_h, dS_h as the TMEM operand and Y as an MN-major operand from shared memory.
// One warpgroup works on each half, so the tensor core runs the products of one half while the other
// is exponentiated.  P and dS are rounded to bf16, the operand type; everything else is fp32.
//
// Streaming rows whose product with a zero probability must not be NaN -- queries that see nothing
// (lse = -inf), keys that no query of the tile sees -- are zeroed in shared memory first.

#include <mutex>

#include "masked_common.cuh"

namespace pf {
namespace {

using namespace masked;

constexpr int kThreads = 384;  // warps 0-3, 4-7: softmax of half 0, 1; then MMA, TMA, helper
constexpr int kWarpMma = 8;
constexpr int kWarpLoad = 9;
constexpr int kWarpHelp = 10;
constexpr uint32_t kColDp = 128;    // S_h at 64 h, dP_h at 128 + 64 h
constexpr uint32_t kColAccK = 256;  // dK or dQ
constexpr uint32_t kColAccV = 384;  // dV

template <int D>
constexpr int kStages = D <= 64 ? 4 : 2;  // (Y1, Y2) pairs in flight

template <int D>
constexpr int smem_bytes(int cls_bytes) {
  return 1024 + (2 + 2 * kStages<D>)*Dims<D>::kTileBytes + kStages<D> * kRows * 8 + 256 + cls_bytes;
}

// KEYS: keys stay (dK, dV), else queries stay (dQ).  MOD: scores are capped or biased.
template <int D, bool KEYS, bool MOD>
__global__ void __launch_bounds__(kThreads, 1) masked_bwd_kernel(const __grid_constant__ MaskedBwdParams p) {
  using Dm = Dims<D>;
  constexpr int S = kStages<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sX = smem;                       // X1, X2
  uint8_t* sY = smem + 2 * Dm::kTileBytes;  // [stage] Y1, Y2
  float* stat = reinterpret_cast<float*>(sY + 2 * S * Dm::kTileBytes);  // [stage] -lse[128] (log2), -delta[128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(stat + S * 2 * kRows);
  uint64_t* x_full = bars;
  uint64_t* y_full = bars + 1;
  uint64_t* y_empty = y_full + S;
  uint64_t* y_ok = y_empty + S;
  uint64_t* s_full = y_ok + S;    // [h]
  uint64_t* dp_full = s_full + 2;
  uint64_t* pt_full = dp_full + 2;
  uint64_t* ds_full = pt_full + 2;
  uint64_t* acc_full = ds_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* cls = reinterpret_cast<uint8_t*>(bars) + 256;
  __shared__ int seen_tiles[2];  // first and last streaming tile with a document of this CTA's

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const MaskParams& mk = p.m;
  const int share = p.heads_q / p.heads_kv;
  const int x_tiles = ((KEYS ? mk.n_k : mk.n_q) + kRows - 1) / kRows;
  const int y_tiles = ((KEYS ? mk.n_q : mk.n_k) + kRows - 1) / kRows;
  int idx = static_cast<int>(blockIdx.x);
  int xt = idx % x_tiles;
  idx /= x_tiles;
  if (!KEYS && mk.causal) xt = x_tiles - 1 - xt;  // the last queries see the most keys: they start first
  const int heads = KEYS ? p.heads_kv : p.heads_q;
  const int x_head = idx % heads;
  const int b = idx / heads;
  const int rounds = KEYS ? share : 1;  // query heads that stream past
  const int y_head = KEYS ? x_head * share : x_head / share;
  const int x0 = xt * kRows;
  const int prefix = mk.prefix != nullptr ? __ldg(mk.prefix + b) : 0;
  const int off = mk.n_k - mk.n_q;
  const long long bq = static_cast<long long>(b) * mk.n_q, bk = static_cast<long long>(b) * mk.n_k;
  const bool docs = mk.doc_q != nullptr;

  if (threadIdx.x == 0) {
    seen_tiles[0] = INT32_MAX;
    seen_tiles[1] = -1;
    mbar_init(smem_u32(x_full), 1);
    for (int st = 0; st < S; ++st) {
      mbar_init(smem_u32(y_full + st), 1);
      mbar_init(smem_u32(y_empty + st), 1);
      mbar_init(smem_u32(y_ok + st), 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(smem_u32(s_full + h), 1);
      mbar_init(smem_u32(dp_full + h), 1);
      mbar_init(smem_u32(pt_full + h), 4);
      mbar_init(smem_u32(ds_full + h), 4);
    }
    mbar_init(smem_u32(acc_full), 1);
    *abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kWarpLoad && lane == 0) {
    prefetch_tmap(&p.tm_x1);
    prefetch_tmap(&p.tm_x2);
    if (y_tiles > 0) {
      prefetch_tmap(&p.tm_y1);
      prefetch_tmap(&p.tm_y2);
    }
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (docs) {
    const DocRange mine[1] = {doc_range((KEYS ? mk.doc_k + bk : mk.doc_q + bq) + x0,
                                        min(kRows, (KEYS ? mk.n_k : mk.n_q) - x0), lane)};
    __syncthreads();  // seen_tiles is set
    class_tiles<1, kThreads / 32>(KEYS ? mk.doc_q + bq : mk.doc_k + bk, KEYS ? mk.n_q : mk.n_k, 0, y_tiles, mine, cls,
                                  seen_tiles, warp, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // how this CTA's rows and streaming tile j see each other: 0 not at all, 1 in part, 2 entirely
  auto see = [&](int j) {
    const int q_first = KEYS ? j * kRows : x0, k_first = KEYS ? x0 : j * kRows;
    const int lo = key_limit(mk, q_first, prefix);
    const int hi = key_limit(mk, min(q_first + kRows, mk.n_q) - 1, prefix);
    if (k_first > hi) return 0;
    const int c = k_first + kRows - 1 <= lo ? 2 : 1;
    return docs ? min(c, static_cast<int>(cls[j])) : c;
  };
  // streaming tiles [y_lo, y_hi) are walked head by head; `next` finds the first one seen from
  // (g, j) on
  int y_lo = 0, y_hi = y_tiles;
  if (mk.causal) {
    if (!KEYS)  // the furthest key of the last query
      y_hi = min(y_hi, (key_limit(mk, min(x0 + kRows, mk.n_q) - 1, prefix) + kRows) / kRows);
    else if (x0 >= prefix)  // the first query at or behind the first key
      y_lo = max(x0 - off, 0) / kRows;
  }
  if (docs) {
    y_hi = min(y_hi, seen_tiles[1] + 1);
    y_lo = max(y_lo, min(seen_tiles[0], y_hi));
  }
  auto next = [&](int& g, int& j) {
    for (; g < rounds; ++g, j = y_lo)
      for (; j < y_hi; ++j)
        if (see(j) != 0) return true;
    return false;
  };

  if (warp >= 8) {
    if (warp == kWarpLoad) {
      // ------------------------------------------------------------ TMA producer
      if (elect_one()) {
        int g = 0, j = y_lo, i = 0;
        bool ok = true;
        bool more = next(g, j);
        if (more) {  // nothing to do without a tile
          const uint32_t xb = smem_u32(x_full);
          mbar_arrive_expect_tx(xb, 2 * Dm::kTileBytes);
          for (int c = 0; c < Dm::kChunks; ++c) {
            tma_load_4d(smem_u32(sX + c * kChunkBytes), &p.tm_x1, c * 64, x_head, x0, b, xb);
            tma_load_4d(smem_u32(sX + Dm::kTileBytes + c * kChunkBytes), &p.tm_x2, c * 64, x_head, x0, b, xb);
          }
        }
        const bool any = more;
        for (; more && ok; ++j, more = next(g, j), ++i) {
          const int st = i % S;
          if (!(ok = mbar_wait(smem_u32(y_empty + st), ((i / S) & 1) ^ 1, abort, kWaitNs))) break;
          const uint32_t yb = smem_u32(y_full + st);
          mbar_arrive_expect_tx(yb, 2 * Dm::kTileBytes);
          for (int c = 0; c < Dm::kChunks; ++c) {
            uint8_t* y = sY + 2 * st * Dm::kTileBytes + c * kChunkBytes;
            tma_load_4d(smem_u32(y), &p.tm_y1, c * 64, y_head + g, j * kRows, b, yb);
            tma_load_4d(smem_u32(y + Dm::kTileBytes), &p.tm_y2, c * 64, y_head + g, j * kRows, b, yb);
          }
        }
        if (!ok) raise_abort(abort, p.watchdog, kWdLoad);
        // drain: every issued copy must land before the CTA exits
        if (any) mbar_wait(smem_u32(x_full), 0, nullptr, kWaitNs);
        for (int k = i > S ? i - S : 0; k < i; ++k)
          mbar_wait(smem_u32(y_full + k % S), (k / S) & 1, nullptr, kWaitNs);
      }
    } else if (warp == kWarpMma) {
      // ------------------------------------------------------------ MMA issuer
      if (elect_one()) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(128, 64, 0);           // N = 64 streaming rows
        constexpr uint32_t idesc_acc = idesc_bf16_f32(128, Dm::kMmaN, 1);  // N = head_dim (padded)
        const uint32_t x_lo = desc_start(smem_u32(sX)) | desc_lbo_bits(16);
        const uint32_t yk_lo = desc_start(smem_u32(sY)) | desc_lbo_bits(16);
        const uint32_t yn_lo = desc_start(smem_u32(sY)) | desc_lbo_bits(kChunkBytes);
        // which = 0: S_h = X1 Y1_h^T, 1: dP_h = X2 Y2_h^T
        auto product = [=](int which, int h, int st) {
          const uint32_t a0 = x_lo + static_cast<uint32_t>((which * Dm::kTileBytes) >> 4);
          const uint32_t b0 = yk_lo + static_cast<uint32_t>(((2 * st + which) * Dm::kTileBytes + h * 8192) >> 4);
          const uint32_t d = tmem + which * kColDp + h * 64;
#pragma unroll
          for (int kk = 0; kk < Dm::kMmaN / 16; ++kk) {
            const uint32_t o = static_cast<uint32_t>(((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4);
            mma_ss(d, smem_desc_lo(a0 + o), smem_desc_lo(b0 + o), idesc_s, kk > 0);
          }
        };
        // which = 0: accK += dS_h Y1_h, 1: accV += P_h Y2_h
        auto accumulate = [=](int which, int h, int st, bool acc) {
          const uint32_t b0 = yn_lo + static_cast<uint32_t>(((2 * st + which) * Dm::kTileBytes + h * 8192) >> 4);
          const uint32_t d = tmem + (which ? kColAccV : kColAccK);
          const uint32_t a = tmem + (which ? 0 : kColDp) + h * 64;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(d, a + kk * 8, smem_desc_lo(b0 + static_cast<uint32_t>((kk * 2048) >> 4)), idesc_acc, acc || kk > 0);
        };
        int g = 0, j = y_lo, i = 0;
        bool ok = true;
        bool more = next(g, j);
        if (more) {
          ok = mbar_wait(smem_u32(x_full), 0, abort, kWaitNs) && mbar_wait(smem_u32(y_ok), 0, abort, kWaitNs);
          if (ok) {
            tc_fence_after();
            for (int h = 0; h < 2; ++h) {
              product(0, h, 0);
              mma_commit(smem_u32(s_full + h));
              product(1, h, 0);
              mma_commit(smem_u32(dp_full + h));
            }
          }
        }
        while (more && ok) {
          ++j;
          more = next(g, j);
          const int st = i % S, sn = (i + 1) % S;
          for (int h = 0; h < 2 && ok; ++h) {
            if (KEYS) {
              if (!(ok = mbar_wait(smem_u32(pt_full + h), i & 1, abort, kWaitNs))) break;
              tc_fence_after();
              accumulate(1, h, st, i > 0 || h > 0);
            }
            if (!(ok = mbar_wait(smem_u32(ds_full + h), i & 1, abort, kWaitNs))) break;
            tc_fence_after();
            accumulate(0, h, st, i > 0 || h > 0);
            if (more) {
              if (h == 0 && !(ok = mbar_wait(smem_u32(y_ok + sn), ((i + 1) / S) & 1, abort, kWaitNs))) break;
              tc_fence_after();
              product(0, h, sn);
              mma_commit(smem_u32(s_full + h));
              product(1, h, sn);
              mma_commit(smem_u32(dp_full + h));
            }
          }
          if (!ok) break;
          mma_commit(smem_u32(y_empty + st));
          ++i;
        }
        if (!ok) raise_abort(abort, p.watchdog, kWdMma);
        // every MMA of this thread: the accumulators are complete, and TMEM may be released
        mma_commit(smem_u32(acc_full));
        mbar_wait(smem_u32(acc_full), 0, nullptr, kWaitNs);
      }
    } else if (warp == kWarpHelp) {
      // ------------------------------------------------------------ row statistics, unseen rows to zero
      // queries stay: the queries of this lane, their documents and limits
      int my_doc[4], my_lim[4];
      int reach_all = -1;
      if (!KEYS) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int query = x0 + x * 32 + lane;
          const bool on = query < mk.n_q;
          my_doc[x] = on && docs ? __ldg(mk.doc_q + bq + query) : -1;
          my_lim[x] = on ? key_limit(mk, query, prefix) : -1;
          reach_all = max(reach_all, my_lim[x]);
        }
        reach_all = __reduce_max_sync(0xffffffffu, reach_all);
      }
      int g = 0, j = y_lo, i = 0;
      bool ok = true;
      for (bool more = next(g, j); more; ++j, more = next(g, j), ++i) {
        const int st = i % S;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(y_empty + st), ((i / S) & 1) ^ 1, abort, kWaitNs));
        if (!ok) break;
        bool unseen[4];
        if (KEYS) {
          const long long row = (static_cast<long long>(b) * p.heads_q + y_head + g) * mk.n_q;
          float* out = stat + st * 2 * kRows;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int query = j * kRows + x * 32 + lane;
            const float l = query < mk.n_q ? __ldg(p.lse + row + query) : -INFINITY;
            unseen[x] = l == -INFINITY;
            // a query that sees nothing: exp2(s - inf) = 0
            out[x * 32 + lane] = unseen[x] ? -INFINITY : -l * kLog2e;
            out[kRows + x * 32 + lane] = unseen[x] ? 0.f : -__ldg(p.delta + row + query);
          }
        } else {
          const bool partly = see(j) == 1;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = j * kRows + x * 32 + lane;
            unseen[x] = false;
            if (partly) {
              unseen[x] = key > reach_all;
              if (docs) {
                // the furthest key that a query of this key's document sees, one id at a time
                const int id = key < mk.n_k ? __ldg(mk.doc_k + bk + key) : -1;
                int reach = -1;
                unsigned todo = __ballot_sync(0xffffffffu, id >= 0);
                while (todo != 0) {
                  const int d = __shfl_sync(0xffffffffu, id, __ffs(todo) - 1);
                  int far = -1;
#pragma unroll
                  for (int y = 0; y < 4; ++y)
                    if (my_doc[y] == d) far = max(far, my_lim[y]);
                  far = __reduce_max_sync(0xffffffffu, far);
                  if (id == d) reach = far;
                  todo &= ~__ballot_sync(0xffffffffu, id == d);
                }
                unseen[x] = key > reach;
              }
            }
          }
        }
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(y_full + st), (i / S) & 1, abort, kWaitNs));
        if (!ok) break;
        bool wrote = false;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (unseen[x]) {
            wrote = true;
            uint4* r = reinterpret_cast<uint4*>(sY + 2 * st * Dm::kTileBytes + (x * 32 + lane) * 128);
#pragma unroll
            for (int c = 0; c < 2 * Dm::kChunks; ++c)
#pragma unroll
              for (int e = 0; e < 8; ++e) r[c * (kChunkBytes / 16) + e] = make_uint4(0, 0, 0, 0);
          }
        }
        if (wrote) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(y_ok + st));
      }
      if (!ok && lane == 0) raise_abort(abort, p.watchdog, kWdScrub);
    }
  } else {
    // ------------------------------------------------------------ softmax of half h, then an accumulator
    const int h = warp >> 2;
    const int wq = warp & 3;
    const int row = x0 + wq * 32 + lane;  // this thread's key or query
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + h * 64;
    const uint32_t tP = tS + kColDp;
    const bool in_range = row < (KEYS ? mk.n_k : mk.n_q);
    const int doc = docs && in_range ? __ldg((KEYS ? mk.doc_k + bk : mk.doc_q + bq) + row) : -1;
    const int* ids = KEYS ? mk.doc_q + bq : mk.doc_k + bk;
    const int y_rows = KEYS ? mk.n_q : mk.n_k;
    const int limit = !KEYS && in_range ? key_limit(mk, row, prefix) : -1;
    float neg_lse = -INFINITY, neg_delta = 0.f;  // queries stay: this row's
    if (!KEYS && in_range) {
      const long long at = (static_cast<long long>(b) * p.heads_q + x_head) * mk.n_q + row;
      const float l = __ldg(p.lse + at);
      if (l != -INFINITY) {
        neg_lse = -l * kLog2e;
        neg_delta = -__ldg(p.delta + at);
      }
    }
    float slope = 0.f;
    bool ok = true;
    int g = 0, j = y_lo, i = 0, slope_of = -1;
    for (bool more = next(g, j); more && ok; ++j, more = next(g, j), ++i) {
      const int st = i % S;
      const int base = j * kRows + h * 64;
      uint64_t bits = ~0ull;
      const bool partly = see(j) == 1;
      if (partly) {
        if (KEYS) {
          // queries from row - off on see this key; all of them where it lies in the prefix
          if (!in_range)
            bits = 0;
          else if (mk.causal && row >= prefix)
            bits = ~limit_bits(row - off - 1, base);
        } else {
          bits = limit_bits(limit, base);
        }
        if (docs) {
          const int id0 = base + lane < y_rows ? __ldg(ids + base + lane) : -1;
          const int id1 = base + 32 + lane < y_rows ? __ldg(ids + base + 32 + lane) : -1;
          bits &= document_bits(doc, id0, id1);
        }
      }
      if (MOD && mk.slopes != nullptr && slope_of != g) {
        slope = __ldg(mk.slopes + (KEYS ? y_head + g : x_head)) * kLog2e;
        slope_of = g;
      }
      if (KEYS) ok = mbar_wait(smem_u32(y_ok + st), (i / S) & 1, abort, kWaitNs);  // the statistics
      ok = ok && mbar_wait(smem_u32(s_full + h), i & 1, abort, kWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const float* st_lse = stat + st * 2 * kRows + h * 64;
      float2 pd[32];  // p, times 1 - tanh^2 with a cap
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t s[32], pk[16];
        tmem_ld32(tS + c0, s);
        tmem_wait_ld();
        reg_fence<32>(s);
        float rest = 0.f;
        float2 damp[16];
        if constexpr (MOD) {
          if (mk.cap_log2 > 0.f) {
            tanh_scores<32>(s, mk);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 t = make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]));
              damp[k] = __ffma2_rn(make_float2(-t.x, -t.y), t, both(1.f));
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) damp[k] = both(1.f);
          }
          scale_scores<32>(s, mk.cap_log2 > 0.f ? mk.cap_log2 : mk.scale_log2);
          if (mk.slopes != nullptr) rest = add_bias<32>(s, slope, base + c0 + (KEYS ? off - row : -off - row));
        }
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          float2 ref[2] = {both(neg_lse), both(neg_lse)};
          if (KEYS) {
            const float4 l = *reinterpret_cast<const float4*>(st_lse + c0 + 2 * k);
            ref[0] = make_float2(l.x, l.y);
            ref[1] = make_float2(l.z, l.w);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float2 x = make_float2(__uint_as_float(s[2 * (k + u)]), __uint_as_float(s[2 * (k + u) + 1]));
            const float2 y = MOD ? __fadd2_rn(__fadd2_rn(x, both(rest)), ref[u]) : __ffma2_rn(x, both(mk.scale_log2), ref[u]);
            pd[c0 / 2 + k + u] = make_float2(ex2(y.x), ex2(y.y));
          }
        }
        if (partly) {
          const uint32_t mask = static_cast<uint32_t>(bits >> c0);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            if (!(mask >> (2 * k) & 1u)) pd[c0 / 2 + k].x = 0.f;
            if (!(mask >> (2 * k + 1) & 1u)) pd[c0 / 2 + k].y = 0.f;
          }
        }
        if (KEYS) {
#pragma unroll
          for (int k = 0; k < 16; ++k) pk[k] = pack2(pd[c0 / 2 + k].x, pd[c0 / 2 + k].y);
          tmem_st16(tS + c0 / 2, pk);
        }
        if constexpr (MOD) {
#pragma unroll
          for (int k = 0; k < 16; ++k) pd[c0 / 2 + k] = __fmul2_rn(pd[c0 / 2 + k], damp[k]);
        }
      }
      if (KEYS) {
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(pt_full + h));
      }
      ok = mbar_wait(smem_u32(dp_full + h), i & 1, abort, kWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t dp[32], pk[16];
        tmem_ld32(tP + c0, dp);
        tmem_wait_ld();
        reg_fence<32>(dp);
        float2 e[16];
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          float2 ref[2] = {both(neg_delta), both(neg_delta)};
          if (KEYS) {
            const float4 l = *reinterpret_cast<const float4*>(st_lse + kRows + c0 + 2 * k);
            ref[0] = make_float2(l.x, l.y);
            ref[1] = make_float2(l.z, l.w);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float2 x = make_float2(__uint_as_float(dp[2 * (k + u)]), __uint_as_float(dp[2 * (k + u) + 1]));
            e[k + u] = __fmul2_rn(pd[c0 / 2 + k + u], __fadd2_rn(x, ref[u]));
          }
        }
        if (partly) {  // also where a hidden value makes dp NaN
          const uint32_t mask = static_cast<uint32_t>(bits >> c0);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            if (!(mask >> (2 * k) & 1u)) e[k].x = 0.f;
            if (!(mask >> (2 * k + 1) & 1u)) e[k].y = 0.f;
          }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) pk[k] = pack2(e[k].x, e[k].y);
        tmem_st16(tP + c0 / 2, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(ds_full + h));
    }
    if (!ok && lane == 0) raise_abort(abort, p.watchdog, kWdSoftmax);
    bool ok_o = ok && mbar_wait(smem_u32(acc_full), 0, abort, kWaitNs);
    ok_o = __all_sync(0xffffffffu, ok_o);
    if (!ok_o) {
      if (ok && lane == 0) raise_abort(abort, p.watchdog, kWdEpilogue);
    } else {
      tc_fence_after();
      // keys stay: half 0 writes dV, half 1 dK; queries stay: each half some columns of dQ
      constexpr int kParts = Dm::kMmaN / 16;
      const int lo = KEYS || h == 0 ? 0 : (kParts + 1) / 2, hi = KEYS || h == 1 ? kParts : (kParts + 1) / 2;
      const uint32_t acc = tmem + lane_off + (KEYS && h == 0 ? kColAccV : kColAccK);
      const float f = KEYS && h == 0 ? 1.f : p.scale;
      uint16_t* dst = KEYS ? (h == 0 ? p.dv : p.dk) + ((bk + row) * p.heads_kv + x_head) * D
                           : p.dq + ((bq + row) * p.heads_q + x_head) * D;
      for (int c = lo; c < hi; ++c) {
        uint32_t o[16];
        tmem_ld16(acc + c * 16, o);
        tmem_wait_ld();
        reg_fence<16>(o);
        float v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = i == 0 ? 0.f : __uint_as_float(o[k]) * f;
        if (in_range) {
#pragma unroll
          for (int k = 0; k < 16; k += 8)
            if (c * 16 + k < D)
              *reinterpret_cast<uint4*>(dst + c * 16 + k) = make_uint4(pack2(v[k], v[k + 1]), pack2(v[k + 2], v[k + 3]),
                                                                       pack2(v[k + 4], v[k + 5]), pack2(v[k + 6], v[k + 7]));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// delta[b][h][i] = sum_d o do, one head vector per LANES lanes of 8 elements each.
template <int D>
__global__ void __launch_bounds__(256) delta_kernel(const uint4* __restrict__ o, const uint4* __restrict__ dout,
                                                    float* __restrict__ delta, int n_q, int heads, long long vectors) {
  constexpr int kLanes = D <= 64 ? 8 : 16;
  const long long at = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / kLanes;
  const int c = threadIdx.x % kLanes;
  float s = 0.f;
  if (at < vectors && c < D / 8) {
    const uint4 a = o[at * (D / 8) + c], e = dout[at * (D / 8) + c];
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s = fmaf(__uint_as_float(x[k] << 16), __uint_as_float(y[k] << 16), s);
      s = fmaf(__uint_as_float(x[k] & 0xffff0000u), __uint_as_float(y[k] & 0xffff0000u), s);
    }
  }
#pragma unroll
  for (int m = kLanes / 2; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  if (at < vectors && c == 0) {
    const long long h = at % heads, row = at / heads;  // row = b n_q + i
    delta[(row / n_q * heads + h) * n_q + row % n_q] = s;
  }
}

template <int D, bool KEYS, bool MOD>
cudaError_t launch(const MaskedBwdParams& p, cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;  // bit per device ordinal
  constexpr int kMaxSmem = smem_bytes<D>(kMaskedDocTiles);
  static_assert(kMaxSmem <= 232448, "shared memory of one CTA");
  auto kernel = masked_bwd_kernel<D, KEYS, MOD>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(done >> dev & 1)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
      if (e != cudaSuccess) return e;
      done |= 1ull << dev;
    }
  }
  const int x_tiles = ((KEYS ? p.m.n_k : p.m.n_q) + kRows - 1) / kRows;
  const int y_tiles = ((KEYS ? p.m.n_q : p.m.n_k) + kRows - 1) / kRows;
  const unsigned grid = static_cast<unsigned>(p.batch) * (KEYS ? p.heads_kv : p.heads_q) * x_tiles;
  if (grid == 0) return cudaSuccess;
  kernel<<<grid, kThreads, smem_bytes<D>(p.m.doc_q != nullptr ? (y_tiles + 15) / 16 * 16 : 0), stream>>>(p);
  return cudaGetLastError();
}

template <int D, bool MOD>
cudaError_t launch_dim(MaskedBwdParams& p, const CUtensorMap (&maps)[4], cudaStream_t stream) {
  const long long vectors = static_cast<long long>(p.batch) * p.m.n_q * p.heads_q;
  if (vectors > 0) {
    const long long blocks = (vectors * (D <= 64 ? 8 : 16) + 255) / 256;
    delta_kernel<D><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        reinterpret_cast<const uint4*>(p.o), reinterpret_cast<const uint4*>(p.dout), p.delta, p.m.n_q, p.heads_q, vectors);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  p.tm_x1 = maps[1];  // K, V stay; Q, dO stream
  p.tm_x2 = maps[2];
  p.tm_y1 = maps[0];
  p.tm_y2 = maps[3];
  const cudaError_t e = launch<D, true, MOD>(p, stream);
  if (e != cudaSuccess) return e;
  p.tm_x1 = maps[0];  // Q, dO stay; K, V stream
  p.tm_x2 = maps[3];
  p.tm_y1 = maps[1];
  p.tm_y2 = maps[2];
  return launch<D, false, MOD>(p, stream);
}

}  // namespace

cudaError_t launch_masked_bwd(MaskedBwdParams& p, const CUtensorMap (&maps)[4], cudaStream_t stream) {
  const bool mod = p.m.cap_log2 > 0.f || p.m.slopes != nullptr;
  switch (p.head_dim) {
    case 64: return mod ? launch_dim<64, true>(p, maps, stream) : launch_dim<64, false>(p, maps, stream);
    case 72: return mod ? launch_dim<72, true>(p, maps, stream) : launch_dim<72, false>(p, maps, stream);
    case 128: return mod ? launch_dim<128, true>(p, maps, stream) : launch_dim<128, false>(p, maps, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pf
