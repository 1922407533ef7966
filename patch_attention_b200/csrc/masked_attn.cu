// masked_attn.cu -- attention over capped, biased and masked scores for sm_100a.
//
//   s_ij = scale q_i.k_j, then cap tanh(s / cap), then - slope |p_i - j|,  p_i = i + n_k - n_q
//   key j is visible to query i if (not causal, or j <= p_i, or j < prefix) and, with documents,
//   doc_q[i] = doc_k[j] >= 0
//   o_i = sum_j softmax_j(s_ij) v_j over the visible keys; a query that sees none gives 0
// P is rounded to bf16, the type that the matrix product takes; sums, maxima and O are fp32.
//
// One CTA handles NQ (1 or 2) tiles of 128 query rows against a run of 128-key tiles, by the
// split-tile scheme of the patch attention: each key tile is two 64-key halves with their own
// score columns in TMEM, so the tensor core runs PV and the next QK of one half while the
// softmax threads (one per row) exponentiate the other; P goes back to TMEM over S as bf16 and
// O accumulates there.  Key tiles are classed against the query tile from their positions and
// documents: tiles that nobody sees are neither loaded nor multiplied, tiles that everybody sees
// skip the masks, and only the rest pay for 64-bit row masks.
//
// Few queries against many keys (a single new token): the query heads that share a key head are
// packed into one tile (their rows are one TMA box), so keys and values are read once; and the
// keys are split over a cluster of up to 8 CTAs that merge their (O, m, l) through distributed
// shared memory -- no workspace, no counters, and the same order of sums every time.
//
// What bounds it, measured on a B200: at head_dim 128 the tensor core (24 heads x 16538 x 16538:
// 2.56 to 2.81 ms by the power left, 1200 to 1310 TFLOP/s); at head_dim 64 the softmax warps, two
// per scheduler in step with each other -- of 1600 cycles per 128 x 128 tile 1024 are the
// special-function unit's, the rest is the maximum, the TMEM copies and the hand-over (2.32 ms,
// 725 TFLOP/s; three packed documents 1.17 ms).  A cap adds 1000 cycles per tile and a bias 800
// (2 x 16 x 4216, head_dim 72, causal: 142 us without, 271 us with cap, bias and prefix by itself and
// 296 among other calls, 389 where scores pass half the cap).  Documents that end inside tiles
// cost the query tiles that meet two of them the keys of both.  One token against 8 x 16538 keys
// (24 / 8 heads of 128): 108 us by itself, 116 among other calls, 5.0 and 4.7 TB/s of K and V.
//
// A value row that no query of the CTA sees may hold anything (padding, unwritten cache rows):
// its products with the zero probabilities would still be NaN, so a warp zeroes such rows in
// shared memory before the MMA reads them.
//
// Every wait is bounded; on expiry the role records itself in the device status word, raises the
// CTA's abort flag, drains what it has in flight and returns.

#include <mutex>

#include "masked_common.cuh"

namespace pf {
namespace {

using namespace masked;

constexpr int kThreads = 384;  // softmax warps 0-7, then MMA 0, TMA, scrub, MMA 1
// setmaxnreg shares, as launched: 384 threads x 168 registers = 128 x 120 + 256 x 192
constexpr uint32_t kRegsSoftmax = 192;
constexpr uint32_t kRegsOther = 120;
constexpr int kWarpMma = 8;
constexpr int kWarpLoad = 9;
constexpr int kWarpScrub = 10;
constexpr int kWarpMma2 = 11;
constexpr uint32_t kColO = 256;  // O_t at column 256 + 128 t, S_t at 128 t
constexpr int kMaxSplit = 8;

template <int D>
constexpr int kStages = D <= 64 ? 8 : 4;

template <int D, int NQ>
constexpr int smem_bytes(int cls_bytes) {
  return 1024 + (NQ + kStages<D>)*Dims<D>::kTileBytes + 512 + cls_bytes;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// This CTA's query rows, its key tiles [j0, j1) and how its query tiles see each of them.
template <int NQ>
struct Work {
  int b, head0, kv_head, q0;  // batch element, first query head, key head, first query
  int rows_per_tile;          // queries of a tile (128 / pack)
  int j0, j1;
  int lim_lo[NQ], lim_hi[NQ];  // key limits of the tile's first and last query; lim_hi -1: sees none
  const uint8_t* cls;          // documents' classes, 2 bits per query tile, from tile cls0 on; or null
  int cls0;

  // 0: no pair visible, 1: some, 2: every one
  __device__ __forceinline__ int of(int t, int j) const {
    const int k0 = j * kRows;
    if (k0 > (t == 0 ? lim_hi[0] : lim_hi[NQ - 1])) return 0;
    const int c = k0 + kRows - 1 <= (t == 0 ? lim_lo[0] : lim_lo[NQ - 1]) ? 2 : 1;
    return cls == nullptr ? c : min(c, (cls[j - cls0] >> (2 * t)) & 3);
  }
  __device__ __forceinline__ bool any(int j) const {
    bool r = of(0, j) != 0;
    if (NQ == 2) r = r || of(NQ - 1, j) != 0;
    return r;
  }
};

// MOD: scores are capped or biased.
template <int D, int NQ, bool MOD>
__global__ void __launch_bounds__(kThreads, 1) masked_fwd_kernel(const __grid_constant__ MaskedFwdParams p) {
  using Dm = Dims<D>;
  constexpr int S = kStages<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + NQ * Dm::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + S * Dm::kTileBytes);
  uint64_t* q_full = bars;
  uint64_t* kv_full = bars + 1;
  uint64_t* kv_empty = kv_full + S;
  uint64_t* v_ok = kv_empty + S;    // the scrub warp has seen the V tile
  uint64_t* s_full = v_ok + S;      // [2 t + h]
  uint64_t* p_full = s_full + 4;    // [2 t + h]
  uint64_t* pv_done = p_full + 4;   // [2 t + h]
  uint64_t* o_full = pv_done + 4;   // [t]
  uint64_t* mma_done = o_full + 2;  // [t]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 2);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* cls = reinterpret_cast<uint8_t*>(bars) + 512;
  __shared__ int seen_tiles[2];  // first and last key tile with a document of this CTA's

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const MaskParams& mk = p.m;
  Work<NQ> w;
  const int part = p.n_split > 1 ? static_cast<int>(cluster_rank()) : 0;
  {
    int idx = static_cast<int>(blockIdx.x) / p.n_split;
    const int heads = p.pack > 1 ? p.heads_kv : p.heads_q;
    const int grp = p.heads_first ? idx / (heads * p.batch) : idx % p.n_groups;
    idx = p.heads_first ? idx % (heads * p.batch) : idx / p.n_groups;
    const int hd = idx % heads;
    w.b = idx / heads;
    const int share = p.heads_q / p.heads_kv;
    w.head0 = p.pack > 1 ? hd * share : hd;
    w.kv_head = p.pack > 1 ? hd : hd / share;
    w.rows_per_tile = kRows / p.pack;
    // the last queries of a causal mask see the most keys: they start first
    w.q0 = (mk.causal ? p.n_groups - 1 - grp : grp) * NQ * w.rows_per_tile;
  }
  const int prefix = mk.prefix != nullptr ? __ldg(mk.prefix + w.b) : 0;
  DocRange qdoc[NQ];
  int lim_max = -1;
#pragma unroll
  for (int t = 0; t < NQ; ++t) {
    const int first = w.q0 + t * w.rows_per_tile;
    const int n = min(w.rows_per_tile, mk.n_q - first);
    w.lim_lo[t] = n > 0 ? key_limit(mk, first, prefix) : -1;
    w.lim_hi[t] = n > 0 ? key_limit(mk, first + n - 1, prefix) : -1;
    if (mk.doc_q != nullptr) {
      qdoc[t] = {0u, -1, true};
      if (n > 0) qdoc[t] = doc_range(mk.doc_q + static_cast<long long>(w.b) * mk.n_q + first, n, lane);
      if (qdoc[t].hi < 0) w.lim_hi[t] = -1;
    }
    lim_max = max(lim_max, w.lim_hi[t]);
  }
  const int n_tiles = (lim_max + kRows) / kRows;  // key tiles with something visible by position
  w.j0 = static_cast<int>(static_cast<long long>(n_tiles) * part / p.n_split);
  w.j1 = static_cast<int>(static_cast<long long>(n_tiles) * (part + 1) / p.n_split);
  w.cls = mk.doc_q != nullptr ? cls : nullptr;

  if (threadIdx.x == 0) {
    seen_tiles[0] = INT32_MAX;
    seen_tiles[1] = -1;
    mbar_init(smem_u32(q_full), 1);
    for (int st = 0; st < S; ++st) {
      mbar_init(smem_u32(kv_full + st), 1);
      mbar_init(smem_u32(kv_empty + st), NQ);
      mbar_init(smem_u32(v_ok + st), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(s_full + i), 1);
      mbar_init(smem_u32(p_full + i), 4);
      mbar_init(smem_u32(pv_done + i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(o_full + t), 1);
      mbar_init(smem_u32(mma_done + t), 1);
    }
    *abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kWarpLoad && lane == 0) {
    prefetch_tmap(&p.tm_q);
    if (mk.n_k > 0) {
      prefetch_tmap(&p.tm_k);
      prefetch_tmap(&p.tm_v);
    }
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (mk.doc_q != nullptr) {
    const int* ids = mk.doc_k + static_cast<long long>(w.b) * mk.n_k;
    __syncthreads();  // seen_tiles is set
    class_tiles<NQ, kThreads / 32>(ids, mk.n_k, w.j0, w.j1, qdoc, cls, seen_tiles, warp, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  w.cls0 = w.j0;
  if (mk.doc_q != nullptr) {  // only between the first and the last tile that shares a document
    w.j1 = min(w.j1, seen_tiles[1] + 1);
    w.j0 = min(seen_tiles[0], w.j1);
  }
  // V rows can only be unseen where something hides them
  const bool scrub = mk.causal || mk.doc_q != nullptr;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kWarpLoad) {
      // ------------------------------------------------------------ TMA producer
      if (elect_one()) {
        const uint32_t qbar = smem_u32(q_full);
        const uint32_t q_bytes = static_cast<uint32_t>(w.rows_per_tile * p.pack) * 128u * Dm::kChunks;
        mbar_arrive_expect_tx(qbar, NQ * q_bytes);
        for (int t = 0; t < NQ; ++t)
          for (int c = 0; c < Dm::kChunks; ++c)
            tma_load_4d(smem_u32(sQ + t * Dm::kTileBytes + c * kChunkBytes), &p.tm_q, c * 64, w.head0,
                        w.q0 + t * w.rows_per_tile, w.b, qbar);
        int i = 0;
        bool ok = true;
        for (int j = w.j0; j < w.j1 && ok; ++j) {
          if (!w.any(j)) continue;
          for (int kv = 0; kv < 2; ++kv, ++i) {
            const int st = i % S;
            if (!mbar_wait(smem_u32(kv_empty + st), ((i / S) & 1) ^ 1, abort, kWaitNs)) {
              ok = false;
              break;
            }
            const uint32_t fb = smem_u32(kv_full + st);
            mbar_arrive_expect_tx(fb, Dm::kTileBytes);
            for (int c = 0; c < Dm::kChunks; ++c)
              tma_load_4d(smem_u32(sKV + st * Dm::kTileBytes + c * kChunkBytes), kv ? &p.tm_v : &p.tm_k, c * 64,
                          w.kv_head, j * kRows, w.b, fb);
          }
        }
        if (!ok) raise_abort(abort, p.watchdog, kWdLoad);
        // drain: every issued copy must land before the CTA exits
        mbar_wait(qbar, 0, nullptr, kWaitNs);
        for (int k = i > S ? i - S : 0; k < i; ++k)
          mbar_wait(smem_u32(kv_full + (k % S)), (k / S) & 1, nullptr, kWaitNs);
      }
    } else if (warp == kWarpMma || (NQ == 2 && warp == kWarpMma2)) {
      // ------------------------------------------------------------ MMA issuer of query tile t
      if (elect_one()) {
        const int t = warp == kWarpMma ? 0 : 1;
        constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 64, 0);         // N = 64 keys
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, Dm::kMmaN, 1);  // N = head_dim (padded)
        const uint32_t q_lo = desc_start(smem_u32(sQ) + t * Dm::kTileBytes) | desc_lbo_bits(16);
        const uint32_t k_lo = desc_start(smem_u32(sKV)) | desc_lbo_bits(16);
        const uint32_t v_lo = desc_start(smem_u32(sKV)) | desc_lbo_bits(kChunkBytes);
        auto issue_qk = [=](int h, int st) {
          const uint32_t b0 = k_lo + static_cast<uint32_t>((st * Dm::kTileBytes + h * 8192) >> 4);
          const uint32_t d = tmem + t * 128 + h * 64;
#pragma unroll
          for (int kk = 0; kk < Dm::kMmaN / 16; ++kk) {
            const uint32_t off = static_cast<uint32_t>(((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4);
            mma_ss(d, smem_desc_lo(q_lo + off), smem_desc_lo(b0 + off), idesc_qk, kk > 0);
          }
        };
        auto issue_pv = [=](int h, int st, bool acc) {
          const uint32_t v0 = v_lo + static_cast<uint32_t>((st * Dm::kTileBytes + h * 8192) >> 4);
          const uint32_t d = tmem + kColO + t * 128;
          const uint32_t a = tmem + t * 128 + h * 64;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(d, a + kk * 8, smem_desc_lo(v0 + static_cast<uint32_t>((kk * 2048) >> 4)), idesc_pv,
                   acc || kk > 0);
        };
        uint64_t* v_bar = scrub ? v_ok : kv_full;

        bool ok = mbar_wait(smem_u32(q_full), 0, abort, kWaitNs);
        bool pending = false;  // the current tile's QK is already issued
        int i = 0, n = 0;      // loads taken (K, V of every tile of the CTA); own tiles
        int j = w.j0;
        while (j < w.j1 && !w.any(j)) ++j;
        while (j < w.j1 && ok) {
          int jn = j + 1;
          while (jn < w.j1 && !w.any(jn)) ++jn;
          const int sK = i % S, pK = (i / S) & 1, sV = (i + 1) % S, pV = ((i + 1) / S) & 1;
          const int sN = (i + 2) % S, pN = ((i + 2) / S) & 1;
          if (w.of(t, j) == 0) {
            // the other query tile's: hand the stages back once they are this use's
            if (!(ok = mbar_wait(smem_u32(kv_full + sK), pK, abort, kWaitNs))) break;
            mbar_arrive(smem_u32(kv_empty + sK));
            if (!(ok = mbar_wait(smem_u32(v_bar + sV), pV, abort, kWaitNs))) break;
            mbar_arrive(smem_u32(kv_empty + sV));
          } else {
            if (!pending) {
              if (!(ok = mbar_wait(smem_u32(kv_full + sK), pK, abort, kWaitNs))) break;
              tc_fence_after();
              issue_qk(0, sK);
              mma_commit(smem_u32(s_full + 2 * t));
              issue_qk(1, sK);
              mma_commit(smem_u32(s_full + 2 * t + 1));
              mma_commit(smem_u32(kv_empty + sK));
            }
            pending = jn < w.j1 && w.of(t, jn) != 0;
            if (!(ok = mbar_wait(smem_u32(v_bar + sV), pV, abort, kWaitNs))) break;
            if (pending && !(ok = mbar_wait(smem_u32(kv_full + sN), pN, abort, kWaitNs))) break;
            for (int h = 0; h < 2; ++h) {
              if (!(ok = mbar_wait(smem_u32(p_full + 2 * t + h), n & 1, abort, kWaitNs))) break;
              tc_fence_after();
              issue_pv(h, sV, n > 0 || h > 0);
              mma_commit(smem_u32(pv_done + 2 * t + h));
              if (pending) {
                issue_qk(h, sN);
                mma_commit(smem_u32(s_full + 2 * t + h));
              }
            }
            if (!ok) break;
            mma_commit(smem_u32(kv_empty + sV));
            if (pending) mma_commit(smem_u32(kv_empty + sN));
            ++n;
          }
          i += 2;
          j = jn;
        }
        if (ok) mma_commit(smem_u32(o_full + t));
        if (!ok) raise_abort(abort, p.watchdog, kWdMma);
        // drain every MMA issued by this thread before TMEM is released
        mma_commit(smem_u32(mma_done + t));
        mbar_wait(smem_u32(mma_done + t), 0, nullptr, kWaitNs);
      }
    } else if (warp == kWarpScrub && scrub) {
      // ------------------------------------------------------------ unseen V rows to zero
      const int* ids = mk.doc_k + static_cast<long long>(w.b) * mk.n_k;
      // with documents: this lane's queries, their documents and key limits
      constexpr int kMine = NQ * (kRows / 32);
      int my_doc[kMine], my_lim[kMine];
      if (mk.doc_q != nullptr) {
#pragma unroll
        for (int x = 0; x < kMine; ++x) {
          const int r = (x % 4) * 32 + lane, query = w.q0 + (x / 4) * w.rows_per_tile + r;
          const bool on = r < w.rows_per_tile && query < mk.n_q;
          my_doc[x] = on ? __ldg(mk.doc_q + static_cast<long long>(w.b) * mk.n_q + query) : -1;
          my_lim[x] = on ? key_limit(mk, query, prefix) : -1;
        }
      }
      int i = 1;
      bool ok = true;
      for (int j = w.j0; j < w.j1 && ok; ++j) {
        if (!w.any(j)) continue;
        const int st = i % S;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(kv_full + st), (i / S) & 1, abort, kWaitNs));
        if (!ok) break;
        bool part_seen = w.of(0, j) == 1;
        if (NQ == 2) part_seen = part_seen || w.of(NQ - 1, j) == 1;
        if (part_seen) {
#pragma unroll
          for (int r0 = 0; r0 < kRows; r0 += 32) {
            const int key = j * kRows + r0 + lane;
            bool seen = key <= lim_max;
            if (mk.doc_q != nullptr) {
              // the furthest key that a query of this key's document sees, one id at a time
              const int id = key < mk.n_k ? __ldg(ids + key) : -1;
              int reach = -1;
              unsigned todo = __ballot_sync(0xffffffffu, id >= 0);
              while (todo != 0) {
                const int d = __shfl_sync(0xffffffffu, id, __ffs(todo) - 1);
                int far = -1;
#pragma unroll
                for (int x = 0; x < kMine; ++x)
                  if (my_doc[x] == d) far = max(far, my_lim[x]);
                far = __reduce_max_sync(0xffffffffu, far);
                if (id == d) reach = far;
                todo &= ~__ballot_sync(0xffffffffu, id == d);
              }
              seen = key <= reach;
            }
            if (!seen) {
              uint4* row = reinterpret_cast<uint4*>(sKV + st * Dm::kTileBytes + (r0 + lane) * 128);
#pragma unroll
              for (int c = 0; c < Dm::kChunks; ++c)
#pragma unroll
                for (int x = 0; x < 8; ++x) row[c * (kChunkBytes / 16) + x] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(smem_u32(v_ok + st));
        i += 2;
      }
      if (!ok && lane == 0) raise_abort(abort, p.watchdog, kWdScrub);
    }
  } else if (warp < 4 * NQ) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------ softmax + epilogue
    const int t = warp >> 2;
    const int wq = warp & 3;
    const int rloc = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + t * 128;
    const uint32_t tO = tmem + lane_off + kColO + t * 128;
    // this row's query, head, limit and document
    const int query = w.q0 + t * w.rows_per_tile + rloc / p.pack;
    const int head = w.head0 + rloc % p.pack;
    const bool in_range = rloc < w.rows_per_tile * p.pack && query < mk.n_q;
    const int limit = in_range ? key_limit(mk, query, prefix) : -1;
    const int doc = in_range && mk.doc_q != nullptr ? __ldg(mk.doc_q + static_cast<long long>(w.b) * mk.n_q + query) : -1;
    const int* ids = mk.doc_k + static_cast<long long>(w.b) * mk.n_k;
    const float slope = MOD && mk.slopes != nullptr && in_range ? __ldg(mk.slopes + head) * kLog2e : 0.f;
    const int place = query + (mk.n_k - mk.n_q);
    // scores are c s + rest in log2 units; the cap leaves them there itself
    const float c = MOD && mk.cap_log2 > 0.f ? 1.f : mk.scale_log2;
    float m = -INFINITY;  // reference row maximum, in log2 units
    float l = 0.f;
    bool ok = true;
    int n = 0;
    for (int j = w.j0; j < w.j1 && ok; ++j) {
      const int kind = w.of(t, j);
      if (kind == 0) continue;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const int base = j * kRows + h * 64;
        int id0 = -1, id1 = -1;
        if (__builtin_expect(kind == 1, 0) && mk.doc_q != nullptr) {  // ahead of the wait
          if (base + lane < mk.n_k) id0 = __ldg(ids + base + lane);
          if (base + 32 + lane < mk.n_k) id1 = __ldg(ids + base + 32 + lane);
        }
        ok = mbar_wait(smem_u32(s_full + 2 * t + h), n & 1, abort, kWaitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[64];
        tmem_ld32(tS + h * 64, s);
        tmem_ld32(tS + h * 64 + 32, s + 32);
        tmem_wait_ld();
        reg_fence<64>(s);
        float rest = 0.f;  // to be added to every score of the row
        if constexpr (MOD) {
          if (mk.cap_log2 > 0.f) tanh_scores<64>(s, mk, mk.cap_log2);
          if (mk.slopes != nullptr) rest = add_bias<64>(s, slope, c, base - place);
        }
        if (__builtin_expect(kind == 1, 0)) {
          uint64_t bits = limit_bits(limit, base);
          if (mk.doc_q != nullptr) bits &= document_bits(doc, id0, id1);
          const uint32_t lo = static_cast<uint32_t>(bits), hi = static_cast<uint32_t>(bits >> 32);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (!(lo >> k & 1u)) s[k] = __float_as_uint(-INFINITY);
            if (!(hi >> k & 1u)) s[k + 32] = __float_as_uint(-INFINITY);
          }
        }
        const float mxs = MOD ? fmaf(row_max64(s), c, rest) : row_max64(s) * c;
        // O is rescaled only when the maximum grows by more than 2^8 (or is NaN): exact, as the
        // final O / l uses one reference for both
        const bool grow = in_range && !(mxs <= m + 8.f);
        const bool any_grow = __any_sync(0xffffffffu, grow);
        if (__builtin_expect(any_grow, 0)) {
          const float alpha = grow ? ex2(m - mxs) : 1.f;
          if (n > 0 || h > 0) {
            // O holds earlier PVs: this half's last one is complete (its scores are); wait for
            // the other half's
            const uint32_t par = h == 0 ? static_cast<uint32_t>((n - 1) & 1) : static_cast<uint32_t>(n & 1);
            ok = mbar_wait(smem_u32(pv_done + 2 * t + (h ^ 1)), par, abort, kWaitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < Dm::kMmaN; c0 += 16) {
              uint32_t o[16];
              tmem_ld16(tO + c0, o);
              tmem_wait_ld();
              reg_fence<16>(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st16(tO + c0, o);
            }
          }
          l *= alpha;
          // an infinite score makes the row NaN, as inf - inf would
          if (grow) m = mxs == INFINITY ? __int_as_float(0x7fffffff) : mxs;
        }
        const float ref = m == -INFINITY ? 0.f : m;  // nothing seen yet: every p is 0
        uint32_t pk[32];
        {
          const float2 cc = both(c), nm = both(rest - ref);
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                           make_float2(0.f, 0.f)};
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float2 raw = make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]));
            const float2 x = __ffma2_rn(raw, cc, nm);
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            acc[k & 3] = __fadd2_rn(acc[k & 3], e);
            pk[k] = pack2(e.x, e.y);  // bf16 probabilities: the MMA's operand type
          }
          const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
          l += a.x + a.y;
        }
        tmem_st32(tS + h * 64, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(p_full + 2 * t + h));
      }
      ++n;
    }
    if (!ok && lane == 0) raise_abort(abort, p.watchdog, kWdSoftmax);
    // (a tile without work has no O to wait for: the wait would last as long as the other tile's work)
    bool ok_o = ok && (n == 0 || mbar_wait(smem_u32(o_full + t), 0, abort, kWaitNs));
    ok_o = named_bar_and(1 + t, kRows, ok_o);
    if (!ok_o) {
      if (ok && lane == 0) raise_abort(abort, p.watchdog, kWdEpilogue);
    } else {
      tc_fence_after();
      const bool empty = m == -INFINITY;
      if (p.n_split == 1) {
        const float inv = empty ? 0.f : 1.f / l;
        const long long at = (static_cast<long long>(w.b) * mk.n_q + query) * p.heads_q + head;
        uint16_t* dst = p.o + at * D;
        if (in_range && p.lse != nullptr)
          p.lse[(static_cast<long long>(w.b) * p.heads_q + head) * mk.n_q + query] =
              empty ? -INFINITY : (m + log2f(l)) * kLn2;
#pragma unroll
        for (int c0 = 0; c0 < Dm::kMmaN; c0 += 16) {
          uint32_t o[16];
          tmem_ld16(tO + c0, o);
          tmem_wait_ld();
          reg_fence<16>(o);
          float f[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] = empty ? 0.f : __uint_as_float(o[k]) * inv;
          if (in_range) {
#pragma unroll
            for (int k = 0; k < 16; k += 8)
              if (c0 + k < D)
                *reinterpret_cast<uint4*>(dst + c0 + k) = make_uint4(pack2(f[k], f[k + 1]), pack2(f[k + 2], f[k + 3]),
                                                                     pack2(f[k + 4], f[k + 5]), pack2(f[k + 6], f[k + 7]));
          }
        }
      } else {
        // this part's row, for the cluster's merge (the K/V ring is free: every load and MMA is done)
        float* row = reinterpret_cast<float*>(sKV) + rloc * (D + 4);
#pragma unroll
        for (int c0 = 0; c0 < Dm::kMmaN; c0 += 16) {
          uint32_t o[16];
          tmem_ld16(tO + c0, o);
          tmem_wait_ld();
          reg_fence<16>(o);
          if (in_range) {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              if (c0 + k < D)
                *reinterpret_cast<float4*>(row + c0 + k) =
                    empty ? make_float4(0.f, 0.f, 0.f, 0.f)
                          : make_float4(__uint_as_float(o[k]), __uint_as_float(o[k + 1]), __uint_as_float(o[k + 2]),
                                        __uint_as_float(o[k + 3]));
          }
        }
        if (in_range) *reinterpret_cast<float2*>(row + D) = make_float2(m, l);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  }

  if (p.n_split > 1) {
    // Parts of one query tile, merged in part order: rows are dealt out to the CTAs, a thread
    // takes four columns of a row.  O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
    __syncwarp();
    cluster_sync();
    if (warp < 4 && !*abort) {
      constexpr int kQuads = D / 4;
      const int rows = min(w.rows_per_tile, mk.n_q - w.q0) * p.pack;
      const int mine = (rows - part + p.n_split - 1) / p.n_split;  // rows part, part + n_split, ...
      const uint32_t stage = smem_u32(sKV);
      for (int e = threadIdx.x; e < mine * kQuads; e += 128) {
        const int r = part + e / kQuads * p.n_split, c = e % kQuads * 4;
        float4 acc[kMaxSplit];
        float2 ml[kMaxSplit];
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k) {
          ml[k] = make_float2(-INFINITY, 0.f);
          acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < p.n_split) {
            const uint32_t a = map_rank(stage + static_cast<uint32_t>(r * (D + 4)) * 4u, k);
            ml[k] = ld_cluster2(a + D * 4);
            acc[k] = ld_cluster4(a + c * 4);
          }
        }
        // a part whose row is NaN (a NaN or infinite score) makes the whole row NaN, as in one part
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k) top = max3_nan(top, ml[k].x, ml[k].x);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        if (top != -INFINITY) {
#pragma unroll
          for (int k = 0; k < kMaxSplit; ++k) {
            const float f = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - top);
            l = fmaf(f, ml[k].y, l);
            o.x = fmaf(f, acc[k].x, o.x);
            o.y = fmaf(f, acc[k].y, o.y);
            o.z = fmaf(f, acc[k].z, o.z);
            o.w = fmaf(f, acc[k].w, o.w);
          }
          const float inv = 1.f / l;
          o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        }
        const int query = w.q0 + r / p.pack, head = w.head0 + r % p.pack;
        const long long at = (static_cast<long long>(w.b) * mk.n_q + query) * p.heads_q + head;
        *reinterpret_cast<uint2*>(p.o + at * D + c) = make_uint2(pack2(o.x, o.y), pack2(o.z, o.w));
        if (c == 0 && p.lse != nullptr)
          p.lse[(static_cast<long long>(w.b) * p.heads_q + head) * mk.n_q + query] =
              top == -INFINITY ? -INFINITY : (top + log2f(l)) * kLn2;
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another may read its part
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int NQ, bool MOD>
cudaError_t launch(const MaskedFwdParams& p, cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;  // bit per device ordinal
  constexpr int kMaxSmem = smem_bytes<D, NQ>(kMaskedDocTiles);
  static_assert(kMaxSmem <= 232448, "shared memory of one CTA");
  auto kernel = masked_fwd_kernel<D, NQ, MOD>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(done >> dev & 1)) {
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, kernel);
      if (e != cudaSuccess) return e;
      if (128 * static_cast<long>(kRegsOther) + 256 * static_cast<long>(kRegsSoftmax) >
          static_cast<long>(kThreads) * fa.numRegs)
        return cudaErrorNotSupported;  // the split would wait forever in setmaxnreg.inc
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
      if (e != cudaSuccess) return e;
      done |= 1ull << dev;
    }
  }
  const int heads = p.pack > 1 ? p.heads_kv : p.heads_q;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * heads * p.n_groups * p.n_split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D, NQ>(p.cls_bytes);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.n_split);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D>
cudaError_t launch_dim(const MaskedFwdParams& p, cudaStream_t stream) {
  const bool mod = p.m.cap_log2 > 0.f || p.m.slopes != nullptr;
  const int rows = kRows / p.pack;
  const bool two = p.n_groups < (p.m.n_q + rows - 1) / rows;
  if (two) return mod ? launch<D, 2, true>(p, stream) : launch<D, 2, false>(p, stream);
  return mod ? launch<D, 1, true>(p, stream) : launch<D, 1, false>(p, stream);
}

}  // namespace

void masked_fwd_plan(MaskedFwdParams& p, int n_sms) {
  const int share = p.heads_q / p.heads_kv;
  auto tiles = [](int n, int rows) { return (n + rows - 1) / rows; };
  // pack the query heads of a key head where that makes fewer tiles
  p.pack = 1;
  if (share > 1 && share <= kRows && tiles(p.m.n_q, kRows / share) < share * tiles(p.m.n_q, kRows)) p.pack = share;
  const int q_tiles = tiles(p.m.n_q, kRows / p.pack);
  const int heads = p.pack > 1 ? p.heads_kv : p.heads_q;
  const long long pairs = static_cast<long long>(p.batch) * heads * q_tiles;
  const int k_tiles = tiles(p.m.n_k, kRows);
  // One query tile per CTA and its keys split over a cluster while the tiles alone leave SMs
  // idle.  The cost of a split in key tiles: the rounds of CTAs times (a part's tiles and four
  // for its start and the merge).
  p.n_split = 1;
  if (pairs < n_sms) {
    double best = 0.0;
    for (int k = 1; k <= kMaxSplit && (k == 1 || k <= k_tiles); ++k) {
      const double rounds = static_cast<double>((pairs * k + n_sms - 1) / n_sms);
      const double cost = rounds * ((k_tiles + k - 1) / k + (k > 1 ? 4.0 : 3.0));
      if (k == 1 || cost < best) {
        best = cost;
        p.n_split = k;
      }
    }
  }
  // two query tiles per CTA share each key tile's load
  p.n_groups = p.n_split == 1 && q_tiles > 1 && pairs > n_sms ? (q_tiles + 1) / 2 : q_tiles;
  // The longest CTAs of a causal mask start first over all heads, so that the short ones fill the
  // last round of SMs (2 x 16 heads x 4216 of 72: 144 us, head by head 173; 24 x 16538 of 64: 1167
  // and 1264), while the keys and values of all heads fit in L2 (101 MB there; with 203 MB the two
  // are even, with 4 x 24 x 8269 of 128, 406 MB, they take 1695 and 1538 us).
  p.heads_first = p.m.causal && 4.0 * p.batch * p.heads_kv * p.m.n_k * p.head_dim <= 120e6;
  p.cls_bytes = p.m.doc_q != nullptr ? (k_tiles + 15) / 16 * 16 : 0;
}

cudaError_t launch_masked_fwd(const MaskedFwdParams& p, cudaStream_t stream) {
  switch (p.head_dim) {
    case 64: return launch_dim<64>(p, stream);
    case 72: return launch_dim<72>(p, stream);
    case 128: return launch_dim<128>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pf
