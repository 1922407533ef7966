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
// With X1, X2 the staying and Y1, Y2 the streaming tiles (128 rows each):
//   S = X1 Y1^T, dP = X2 Y2^T into TMEM; two softmax warpgroups, each for 64 of the streaming rows (one
//   thread per staying row), turn them into P and dS, both written back over dP as bf16;
//   accV += P Y2 (keys stay only), accK += dS Y1 with P, dS as the TMEM operand and Y as an MN-major
//   operand from shared memory.
// S's columns are free as soon as they are in registers, so the next tile's S is computed under this
// one's exponentials, and dV, dK and the next dP under the next exponentials: with P written over S
// a chain ran through all four products (5600 cycles per tile at head_dim 128).  An MMA costs about
// 80 cycles or its 128 x N x 16 share of the tensor rate, whichever is more, so S and dP are made 128
// columns wide (64 at N = 128) and not per warpgroup (84 measured at N = 64, where 32 would do).  The
// two halves of a streaming tile are loaded and freed apart: two whole tiles fill the shared
// memory at head_dim 128, and half a tile's start is gained for the loads.  P and dS are rounded to
// bf16, the operand type, and delta is summed from the bf16 o that the forward call wrote;
// everything else is fp32.  So dq and dk are off by 1.45 times as much as with all three in fp32 where
// a query sees 32 keys or more, by 2.4 times at two keys, where do.v and delta nearly cancel.
//
// What bounds it, measured on a B200: the chain of a tile through the softmax warps (per 128 x 128
// tile 2000 to 2900 cycles at head_dim 64, 3000 to 4100 at 128, where the loads also come late; the
// exponentials are 1024 of them).  24 heads x 16538 x 16538: 7.50 ms at head_dim 64, 11.7 ms at 128
// (560 and 720 TFLOP/s of the five products' work); 4216 tokens in two documents, 24 / 8 heads of
// 128: 622 us.  The grid of dQ starts while that of dK, dV still runs and fills the SMs that its
// last CTAs leave idle: one after the other the same call took 775 us.
//
// Streaming rows whose product with a zero probability must not be NaN -- queries that see nothing
// (lse = -inf), keys that no query of the tile sees -- are zeroed in shared memory first.

#include <algorithm>
#include <mutex>

#include "masked_common.cuh"

namespace pf {
namespace {

using namespace masked;

constexpr int kThreads = 384;  // warps 0-3, 4-7: softmax of half 0, 1; then MMA, TMA, helper
constexpr int kUnit = 64;      // rows of half a streaming tile
constexpr int kWarpMma = 8;
constexpr int kWarpLoad = 9;
constexpr int kWarpHelp = 10;
constexpr uint32_t kColDp = 128;    // warpgroup h: S at 64 h, dP at 128 + 64 h (then dS, P: 32 columns each)
constexpr uint32_t kColAccK = 256;  // dK or dQ
constexpr uint32_t kColAccV = 384;  // dV

template <int D>
constexpr int kStages = D <= 64 ? 4 : 2;  // streaming tiles (Y1, Y2) in flight

template <int D>
constexpr int smem_bytes(int cls_bytes) {
  return 1024 + (2 + 2 * kStages<D>)*Dims<D>::kTileBytes + kStages<D> * (kRows * 8 + 16) + 512 + cls_bytes;
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
  constexpr int R = 2 * S;  // half tiles in flight: stage i / 2, half i % 2
  uint8_t* sY = smem + 2 * Dm::kTileBytes;  // [stage] Y1, Y2
  float* stat = reinterpret_cast<float*>(sY + 2 * S * Dm::kTileBytes);  // [half tile] -lse[64] (log2), -delta[64]
  // [stage] the tile's place among the streaming tiles (-1: none is left), its query head among
  // those that stream, and how it is seen (1 in part, 2 entirely): written by the helper
  int4* info = reinterpret_cast<int4*>(stat + R * 2 * kUnit);
  uint64_t* bars = reinterpret_cast<uint64_t*>(info + S);
  uint64_t* x_full = bars;
  uint64_t* y_full = bars + 1;
  uint64_t* y_empty = y_full + R;  // [half tile], as y_full, y_ok
  uint64_t* y_ok = y_empty + R;
  uint64_t* s_full = y_ok + R;
  uint64_t* dp_full = s_full + 1;
  uint64_t* s_free = dp_full + 1;  // [warpgroup] its S is in registers
  uint64_t* ds_full = s_free + 2;  // [warpgroup] its P and dS are written
  uint64_t* acc_full = ds_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* cls = reinterpret_cast<uint8_t*>(bars) + 512;
  __shared__ int seen_tiles[2];  // first and last streaming tile with a document of this CTA's

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const MaskParams& mk = p.m;
  const int share = p.heads_q / p.heads_kv;
  const int x_tiles = ((KEYS ? mk.n_k : mk.n_q) + kRows - 1) / kRows;
  const int y_tiles = ((KEYS ? mk.n_q : mk.n_k) + kRows - 1) / kRows;
  int idx = static_cast<int>(blockIdx.x);
  const int heads = KEYS ? p.heads_kv : p.heads_q;
  int xt = p.heads_first ? idx / (heads * p.batch) : idx % x_tiles;
  idx = p.heads_first ? idx % (heads * p.batch) : idx / x_tiles;
  if (!KEYS && mk.causal) xt = x_tiles - 1 - xt;  // the last queries see the most keys: they start first
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
    for (int r = 0; r < R; ++r) {
      mbar_init(smem_u32(y_full + r), 1);
      mbar_init(smem_u32(y_empty + r), 1);
      mbar_init(smem_u32(y_ok + r), 1);
    }
    mbar_init(smem_u32(s_full), 1);
    mbar_init(smem_u32(dp_full), 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(smem_u32(s_free + h), 4);
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
  if (KEYS) {
    // delta comes from the grid before this one.  With it complete the grid of the queries may
    // start where this one leaves SMs idle: they have no results in common.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (p.overlap) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }

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
  // Y1 (which = 0) or Y2 of half tile r: chunk c's 64 rows are at + c * kChunkBytes
  auto half_tile = [&](int r, int which) { return sY + (r & ~1) * Dm::kTileBytes + which * Dm::kTileBytes + (r & 1) * kUnit * 128; };

  if (warp >= 8) {
    if (warp == kWarpLoad) {
      // ------------------------------------------------------------ TMA producer
      if (elect_one()) {
        int g = 0, j = y_lo, i = 0;  // i: half tiles
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
        for (; more && ok; ++j, more = next(g, j))
          for (int h = 0; h < 2; ++h, ++i) {
            const int r = i % R;
            if (!(ok = mbar_wait(smem_u32(y_empty + r), ((i / R) & 1) ^ 1, abort, kWaitNs))) break;
            const uint32_t yb = smem_u32(y_full + r);
            mbar_arrive_expect_tx(yb, Dm::kTileBytes);
            for (int which = 0; which < 2; ++which)
              for (int c = 0; c < Dm::kChunks; ++c)
                tma_load_4d(smem_u32(half_tile(r, which) + c * kChunkBytes), which ? &p.tm_y2 : &p.tm_y1, c * 64, y_head + g,
                            j * kRows + h * kUnit, b, yb);
          }
        if (!ok) raise_abort(abort, p.watchdog, kWdLoad);
        // drain: every issued copy must land before the CTA exits
        if (any) mbar_wait(smem_u32(x_full), 0, nullptr, kWaitNs);
        for (int k = i > R ? i - R : 0; k < i; ++k)
          mbar_wait(smem_u32(y_full + k % R), (k / R) & 1, nullptr, kWaitNs);
      }
    } else if (warp == kWarpMma) {
      // ------------------------------------------------------------ MMA issuer
      if (elect_one()) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, 0);          // N = 128 streaming rows
        constexpr uint32_t idesc_acc = idesc_bf16_f32(128, Dm::kMmaN, 1);  // N = head_dim (padded)
        const uint32_t x_lo = desc_start(smem_u32(sX)) | desc_lbo_bits(16);
        const uint32_t yk_lo = desc_start(smem_u32(sY)) | desc_lbo_bits(16);
        const uint32_t yn_lo = desc_start(smem_u32(sY)) | desc_lbo_bits(kChunkBytes);
        // tile i, which = 0: S = X1 Y1^T, 1: dP = X2 Y2^T
        auto product = [=](int which, int i) {
          const uint32_t a0 = x_lo + static_cast<uint32_t>((which * Dm::kTileBytes) >> 4);
          const uint32_t b0 = yk_lo + static_cast<uint32_t>(((2 * (i % S) + which) * Dm::kTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < Dm::kMmaN / 16; ++kk) {
            const uint32_t o = static_cast<uint32_t>(((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4);
            mma_ss(tmem + which * kColDp, smem_desc_lo(a0 + o), smem_desc_lo(b0 + o), idesc_s, kk > 0);
          }
          mma_commit(smem_u32(which ? dp_full : s_full));
        };
        // half h of tile i, which = 0: accK += dS Y1, 1: accV += P Y2
        auto accumulate = [=](int which, int h, int i) {
          const uint32_t b0 = yn_lo + static_cast<uint32_t>(((2 * (i % S) + which) * Dm::kTileBytes + h * kUnit * 128) >> 4);
          const uint32_t d = tmem + (which ? kColAccV : kColAccK);
          const uint32_t a = tmem + kColDp + h * 64 + which * 32;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(d, a + kk * 8, smem_desc_lo(b0 + static_cast<uint32_t>((kk * 2048) >> 4)), idesc_acc,
                   i > 0 || h > 0 || kk > 0);
        };
        // Tile i's dV, dK and tile i + 1's S are issued as they become possible, in either order: with
        // two tiles in shared memory the next one's rows may come late, and dV, dK free the rows of
        // the one after.
        bool ok = mbar_wait(smem_u32(y_ok + 1), 0, abort, kWaitNs);
        const bool more = ok && info[0].x >= 0;
        if (more) {
          ok = mbar_wait(smem_u32(x_full), 0, abort, kWaitNs);
          if (ok) {
            tc_fence_after();
            product(0, 0);
            product(1, 0);
          }
        }
        for (int i = 0; more && ok; ++i) {
          const int n = 2 * (i + 1) + 1;  // the next tile's second half
          const uint32_t full = (n / R) & 1, turn = i & 1;
          bool begun = false, last = false;
          int done = 0;  // halves accumulated
          uint64_t t0 = 0;
          while (!(begun || last) || done < 2) {
            bool progress = false;
            if (!begun && !last && mbar_test(smem_u32(y_ok + n % R), full)) {
              if (info[(i + 1) % S].x < 0) {
                last = progress = true;
              } else if (mbar_test(smem_u32(s_free), turn) && mbar_test(smem_u32(s_free + 1), turn)) {
                tc_fence_after();
                product(0, i + 1);
                begun = progress = true;
              }
            }
            if (done < 2 && mbar_test(smem_u32(ds_full + done), turn)) {
              tc_fence_after();
              accumulate(0, done, i);
              if (KEYS) accumulate(1, done, i);
              mma_commit(smem_u32(y_empty + (2 * i + done) % R));
              ++done;
              progress = true;
            }
            if (progress) {
              t0 = 0;
            } else if (t0 == 0) {
              t0 = globaltimer_ns();
            } else if (*abort || globaltimer_ns() - t0 > kWaitNs) {
              ok = false;
              break;
            }
          }
          if (!ok || last) break;
          product(1, i + 1);
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
      // keys stay: the statistics of a half tile's queries, loaded one half tile ahead
      float l[2], dl[2];
      auto fetch = [&](int g, int j, int h) {
        const long long row = (static_cast<long long>(b) * p.heads_q + y_head + g) * mk.n_q;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int query = j * kRows + h * kUnit + x * 32 + lane;
          l[x] = query < mk.n_q ? __ldg(p.lse + row + query) : -INFINITY;
          dl[x] = query < mk.n_q ? __ldg(p.delta + row + query) : 0.f;
        }
      };
      int g = 0, j = y_lo, i = 0;  // i: half tiles
      bool ok = true;
      bool more = next(g, j);
      int kind = more ? see(j) : 0;
      if (KEYS && more) fetch(g, j, 0);
      while (more && ok) {
        const int here = j, head = g, seen = kind;
        const bool partly = !KEYS && seen == 1;
        for (int h = 0; h < 2; ++h, ++i) {
          const int r = i % R;
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(y_empty + r), ((i / R) & 1) ^ 1, abort, kWaitNs));
          if (!ok) break;
          bool unseen[2] = {false, false};
          if (KEYS) {
            float* out = stat + r * 2 * kUnit;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              unseen[x] = l[x] == -INFINITY;
              // a query that sees nothing: exp2(s - inf) = 0
              out[x * 32 + lane] = unseen[x] ? -INFINITY : -l[x] * kLog2e;
              out[kUnit + x * 32 + lane] = unseen[x] ? 0.f : -dl[x];
            }
          }
          if (h == 1) {
            // (both warpgroups are done with the stage's last tile once its second half is free)
            if (lane == 0) info[(i / 2) % S] = make_int4(here, head, seen, 0);
            ++j;
            more = next(g, j);
            kind = more ? see(j) : 0;
          }
          if (KEYS && more) fetch(g, j, h ^ 1);
          if (partly) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int key = here * kRows + h * kUnit + x * 32 + lane;
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
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(y_full + r), (i / R) & 1, abort, kWaitNs));
          if (!ok) break;
          if (__any_sync(0xffffffffu, unseen[0] || unseen[1])) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!unseen[x]) continue;
#pragma unroll
              for (int c = 0; c < 2 * Dm::kChunks; ++c) {
                uint4* to = reinterpret_cast<uint4*>(half_tile(r, c & 1) + (c >> 1) * kChunkBytes + (x * 32 + lane) * 128);
#pragma unroll
                for (int e = 0; e < 8; ++e) to[e] = make_uint4(0, 0, 0, 0);
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(y_ok + r));
        }
      }
      if (ok) {  // no tile is left
        const int r = (i + 1) % R;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(y_empty + r), (((i + 1) / R) & 1) ^ 1, abort, kWaitNs));
        if (ok && lane == 0) {
          info[(i / 2) % S] = make_int4(-1, 0, 0, 0);
          mbar_arrive(smem_u32(y_ok + r));
        }
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
    int i = 0, slope_of = -1;
    for (;; ++i) {
      const int r = (2 * i + h) % R;
      // the tile's place (and the statistics of both halves) come with its second half
      ok = mbar_wait(smem_u32(y_ok + (2 * i + 1) % R), ((2 * i + 1) / R) & 1, abort, kWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int4 tile = info[i % S];
      if (tile.x < 0) break;
      const int g = tile.y, base = tile.x * kRows + h * kUnit;
      uint64_t bits = ~0ull;
      const bool partly = tile.z == 1;
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
      ok = mbar_wait(smem_u32(s_full), i & 1, abort, kWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const float* neg = stat + r * 2 * kUnit;  // the columns' -lse, then -delta
      float2 pd[32];    // p, times 1 - tanh^2 with a cap
      uint32_t pk[32];  // p as bf16
      {
        uint32_t s[64];
        tmem_ld32(tS, s);
        tmem_ld32(tS + 32, s + 32);
        tmem_wait_ld();
        reg_fence<64>(s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(s_free + h));
        float rest = 0.f;
        if constexpr (MOD) {
          if (mk.cap_log2 > 0.f) {
            tanh_scores<64>(s, mk, 1.f);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float2 t = make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]));
              pd[k] = __ffma2_rn(make_float2(-t.x, -t.y), t, both(1.f));
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) pd[k] = both(1.f);
          }
          scale_scores<64>(s, mk.cap_log2 > 0.f ? mk.cap_log2 : mk.scale_log2);
          if (mk.slopes != nullptr) rest = add_bias<64>(s, slope, 1.f, base + (KEYS ? off - row : -off - row));
        }
        if (partly) {
          const uint32_t lo = static_cast<uint32_t>(bits), hi = static_cast<uint32_t>(bits >> 32);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (!(lo >> k & 1u)) s[k] = __float_as_uint(-INFINITY);
            if (!(hi >> k & 1u)) s[k + 32] = __float_as_uint(-INFINITY);
          }
          if constexpr (MOD) {  // the cap's factor of a hidden score may be NaN
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if (!(bits >> (2 * k) & 1ull)) pd[k].x = 0.f;
              if (!(bits >> (2 * k + 1) & 1ull)) pd[k].y = 0.f;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          float2 ref[2] = {both(neg_lse), both(neg_lse)};
          if (KEYS) {
            const float4 l = *reinterpret_cast<const float4*>(neg + 2 * k);
            ref[0] = make_float2(l.x, l.y);
            ref[1] = make_float2(l.z, l.w);
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const float2 x = make_float2(__uint_as_float(s[2 * (k + v)]), __uint_as_float(s[2 * (k + v) + 1]));
            const float2 y = MOD ? __fadd2_rn(__fadd2_rn(x, both(rest)), ref[v]) : __ffma2_rn(x, both(mk.scale_log2), ref[v]);
            const float2 e = make_float2(ex2(y.x), ex2(y.y));
            if (KEYS) pk[k + v] = pack2(e.x, e.y);
            pd[k + v] = MOD ? __fmul2_rn(pd[k + v], e) : e;
          }
        }
      }
      ok = mbar_wait(smem_u32(dp_full), i & 1, abort, kWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t dp[32], ds[16];
        tmem_ld32(tP + c0, dp);
        tmem_wait_ld();
        reg_fence<32>(dp);
        if (partly) {  // a hidden value may make dp NaN: p = 0 there would not be enough
          const uint32_t mask = static_cast<uint32_t>(bits >> c0);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!(mask >> k & 1u)) dp[k] = 0u;
        }
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          float2 ref[2] = {both(neg_delta), both(neg_delta)};
          if (KEYS) {
            const float4 l = *reinterpret_cast<const float4*>(neg + kUnit + c0 + 2 * k);
            ref[0] = make_float2(l.x, l.y);
            ref[1] = make_float2(l.z, l.w);
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const float2 x = make_float2(__uint_as_float(dp[2 * (k + v)]), __uint_as_float(dp[2 * (k + v) + 1]));
            const float2 e = __fmul2_rn(pd[c0 / 2 + k + v], __fadd2_rn(x, ref[v]));
            ds[k + v] = pack2(e.x, e.y);
          }
        }
        tmem_st16(tP + c0 / 2, ds);  // below the columns still to be read
      }
      if (KEYS) tmem_st32(tP + 32, pk);
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
  // what follows in the stream waits for this grid alone: it ends after the keys' grid
  if (!KEYS && blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D>(p.m.doc_q != nullptr ? (y_tiles + 15) / 16 * 16 : 0);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, bool MOD>
cudaError_t launch_dim(MaskedBwdParams& p, const CUtensorMap (&maps)[2][4], cudaStream_t stream) {
  // The longest CTAs of a causal mask first over all heads while two tensors of the longer side take
  // less than half of L2, beside the other side's (2 x 16 x 1100 of 72, 10 MB: 78 us, head by head 88; 39 MB: even;
  // 24 x 16538 of 64, 101 MB: 4.05 and 3.88 ms)
  const double rows = std::max(static_cast<double>(p.heads_q) * p.m.n_q, static_cast<double>(p.heads_kv) * p.m.n_k);
  p.heads_first = p.m.causal && 4.0 * p.batch * D * rows <= 64e6;
  const long long vectors = static_cast<long long>(p.batch) * p.m.n_q * p.heads_q;
  if (vectors > 0) {
    const long long blocks = (vectors * (D <= 64 ? 8 : 16) + 255) / 256;
    delta_kernel<D><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        reinterpret_cast<const uint4*>(p.o), reinterpret_cast<const uint4*>(p.dout), p.delta, p.m.n_q, p.heads_q, vectors);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  p.tm_x1 = maps[0][1];  // K, V stay; Q, dO stream
  p.tm_x2 = maps[0][2];
  p.tm_y1 = maps[1][0];
  p.tm_y2 = maps[1][3];
  // each starts under the one before: dK, dV's prologue under delta's end, dQ in the SMs that dK, dV
  // leaves idle (see the kernel for what they wait for)
  p.overlap = p.m.n_k > 0 && vectors > 0;
  const cudaError_t e = launch<D, true, MOD>(p, stream);
  if (e != cudaSuccess) return e;
  p.tm_x1 = maps[0][0];  // Q, dO stay; K, V stream
  p.tm_x2 = maps[0][3];
  p.tm_y1 = maps[1][1];
  p.tm_y2 = maps[1][2];
  return launch<D, false, MOD>(p, stream);
}

}  // namespace

cudaError_t launch_masked_bwd(MaskedBwdParams& p, const CUtensorMap (&maps)[2][4], cudaStream_t stream) {
  const bool mod = p.m.cap_log2 > 0.f || p.m.slopes != nullptr;
  switch (p.head_dim) {
    case 64: return mod ? launch_dim<64, true>(p, maps, stream) : launch_dim<64, false>(p, maps, stream);
    case 72: return mod ? launch_dim<72, true>(p, maps, stream) : launch_dim<72, false>(p, maps, stream);
    case 128: return mod ? launch_dim<128, true>(p, maps, stream) : launch_dim<128, false>(p, maps, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pf
