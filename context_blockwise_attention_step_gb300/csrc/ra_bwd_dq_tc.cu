// ra_bwd_dq_tc.cu — the dq half of the deterministic ring-attention backward (sm_103a).
//
// The fused backward adds every (K/V tile, query tile) contribution to dq with float
// reductions, whose order varies from run to run. For `deterministic` problems (nanotron
// how-to page, "Calling the Ring Attention Function Directly": the `deterministic` flag)
// dq is instead computed query-tile-major: one CTA owns a 128-row query tile of one rank
// and one query head and walks the ring like the forward — step s = 0..D-1 against K/V
// shard (r - s) mod D, and of each shard only the K/V tiles some row may see — with dq
// accumulated in TMEM in a fixed order ("Backward Pass and Gradient Accumulation": dq
// accumulates over the steps on its own rank). dk and dv come from the K/V-tile kernel
// without its dq part, which writes each K/V row from one CTA, so the whole backward is
// free of atomics. Per K/V tile:
//
//   S  = Q K^T                 tcgen05 (SS), TMEM (two buffers)
//   P  = 2^(S*scale*log2e - lse*log2e)   one thread per query row, masked by key counts
//   dP = dO V^T                tcgen05 (SS), TMEM
//   dS = P * (dP - delta)      bf16, written over the tile's S buffer (columns [32, 96))
//   dQ += dS K                 tcgen05 (TS: dS from TMEM, K MN-major), f32 in TMEM
//
// MMA order: S(0) dP(0) S(1) | dP(1) dQ(0) S(2) | dP(2) dQ(1) S(3) | ...: once dS(n) is
// written, dP(n+1) goes first, so the softmax threads compute dS(n+1) (into the other S
// buffer) while dQ(n) runs, and S(n+2) is ready while dS(n+1) is computed. K stays in
// shared memory from S(n) to dQ(n), which now trails dP(n+1): three K stages let the load
// of K(n+2) start before dQ(n) ends. Items (query tiles) come from a counter in the
// caller's workspace, passed from the producer thread to the other roles through a two-slot
// ring in shared memory. Warp roles (384 threads): warp 0 TMA producer, warp 1 TMEM
// allocator + MMA issuer, warps 4-7 and 8-11 the P / dS warpgroups (thread = query row;
// key columns 0-63 and 64-127; they also write dq).
//
// WIN (sliding window with always visible first tokens): the walk visits the K/V tiles that
// some row of the tile sees, as in the windowed forward. It is launched with the K/V pass and
// needs nothing of it, so it only waits for it at its own end.
// DELTA (windows of few keys): the walk without dQ; a row's two threads add their halves of
// sum_j P_j dP_j to the row's delta, which is 0 before.
#include <cuda_runtime.h>

#include "ra_internal.h"
#include "ra_plan.h"
#include "ra_ptx.cuh"
#include "ra_window.cuh"

namespace ra {

static __device__ unsigned int g_status_dq;

namespace {

constexpr int kDqThreads = 384;
// Of every 8 pairs of recomputed exponentials, this many are evaluated on the FMA pipe
// (exp2_poly2) and the rest on the MUFU unit.
#ifndef RA_DQ_POLY_PAIRS
#define RA_DQ_POLY_PAIRS 0
#endif
constexpr int kSubBytes = 128 * 128;
constexpr float kLog2e = 1.4426950408889634f;

template <int DH>
struct DqCfg {
  static constexpr int kSub = DH / 64;
  static constexpr int kTileBytes = 128 * DH * 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffDO = kTileBytes;
  static constexpr int kKStages = 3;  // K is held from S(n) to dQ(n), which trails dP(n+1)
  static constexpr int kOffK = 2 * kTileBytes;                // kKStages stages
  static constexpr int kOffV = kOffK + kKStages * kTileBytes; // 2 stages
  static constexpr int kOffBar = kOffV + 2 * kTileBytes;
  static constexpr int kSmemBytes = kOffBar + 256;
  static constexpr int kOffWin = kOffBar + 256;  // windowed: the item queue's slots
  static constexpr int kSmemWindow = kOffWin + 2 * sizeof(WinSlot);
  static constexpr int kKSteps = DH / 16;
  static constexpr uint32_t kTmemCols = 512;
  // TMEM columns: S0 | S1 | dP | dQ
  static constexpr uint32_t kColS0 = 0, kColS1 = 128, kColDP = 256, kColDQ = 384;
};

struct DqBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[3], k_empty[3], v_full[2], v_empty[2];
  uint64_t s_full[2], dp_full, ds_full[2], dq_done, dq_free;
  uint64_t drain;
  uint64_t item_full[2], item_empty[2];  // the CTA's item queue
  int item[2];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(DqBars) <= 256, "barrier block");
static_assert(DqCfg<128>::kSmemWindow <= 232448, "shared memory budget");

// Query-tile items: K/V heads outermost (CTAs that run together share K/V in L2), then
// the last query tile first (causal: it sees the most keys), then ranks, then the query
// heads of the group.
struct DqItem { int seq, h, r, qt; };

RA_HD int dq_items_of(const Plan& P, int L) { return ceil_div(L, kQTileRows) * plan_ranks(P) * P.hq; }

__device__ __forceinline__ DqItem decode_dq(const Plan& P, int w) {
  DqItem it;
  it.seq = find_seq(P, w);
  const SeqDesc& s = P.seq[it.seq];
  const int nqt = ceil_div(s.L, kQTileRows), nr = plan_ranks(P);
  int x = w - s.item_start;
  const int g = x % P.group;
  x /= P.group;
  it.r = P.rank_only >= 0 ? P.rank_only : x % nr;
  x /= nr;
  it.qt = nqt - 1 - x % nqt;
  const int hk = x / nqt;
  it.h = hk * P.group + g;
  return it;
}

__device__ __forceinline__ int dq_walk_tiles(const Plan& P, const DqItem& it, int L) {
  const int a_last = min(L, (it.qt + 1) * kQTileRows) - 1;
  int n = 0;
  for (int s = P.step_begin; s < P.step_end; ++s)
    n += kv_tiles_for(P, L, it.r, shard_at_step(P.D, it.r, s), a_last);
  return n;
}

// The CTA's item queue (two slots), as in the K/V-tile pass: the producer thread takes the
// next item from the shared counter (or by the static stride when there is none) and
// publishes it; the MMA thread and the softmax threads read it from the ring.
__device__ __forceinline__ int dq_item_publish(DqBars& sh, const Plan& P, int k,
                                               volatile int* abort_flag, uint64_t tmo,
                                               unsigned int* status) {
  const int slot = k & 1;
  if (!mbar_wait(&sh.item_empty[slot], ((k >> 1) & 1) ^ 1, abort_flag, tmo, status)) return -1;
  const int w = P.work_counter ? atomicAdd(P.work_counter, 1)
                               : static_cast<int>(blockIdx.x + static_cast<unsigned>(k) * gridDim.x);
  sh.item[slot] = w;
  mbar_arrive(&sh.item_full[slot]);
  return w;
}
__device__ __forceinline__ int dq_item_take(DqBars& sh, int k, volatile int* abort_flag,
                                            uint64_t tmo, unsigned int* status) {
  const int slot = k & 1;
  if (!mbar_wait(&sh.item_full[slot], (k >> 1) & 1, abort_flag, tmo, status)) return -1;
  const int w = *reinterpret_cast<volatile int*>(&sh.item[slot]);
  mbar_arrive(&sh.item_empty[slot]);
  return w;
}

// The windowed kernel's item queue, as in the windowed forward.
__device__ __forceinline__ int dq_window_publish(DqBars& sh, WinSlot* slots, const Plan& P, int k, int lane,
                                                 volatile int* abort_flag, uint64_t tmo,
                                                 unsigned int* status) {
  const int slot = k & 1;
  const bool ok = mbar_wait(&sh.item_empty[slot], ((k >> 1) & 1) ^ 1, abort_flag, tmo, status);
  if (!__all_sync(0xffffffffu, ok)) return -1;
  int w = 0;
  if (lane == 0)
    w = P.work_counter ? atomicAdd(P.work_counter, 1)
                       : static_cast<int>(blockIdx.x + static_cast<unsigned>(k) * gridDim.x);
  w = __shfl_sync(0xffffffffu, w, 0);
  if (w < P.n_items) {
    const DqItem it = decode_dq(P, w);
    const int a0 = it.qt * kQTileRows;
    fill_slot<false>(slots[slot], nullptr, P, it.seq, it.h, it.r, a0, min(P.seq[it.seq].L, a0 + kQTileRows) - 1);
  }
  if (lane == 0) {
    slots[slot].item = w;
    mbar_arrive(&sh.item_full[slot]);
  }
  return w;
}

template <int DH, bool WIN, bool DELTA = false>
__global__ void __launch_bounds__(kDqThreads, 1)
    ring_bwd_dq_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ CUtensorMap tmDO, const __grid_constant__ Plan P,
                          const float* __restrict__ lse, const float* __restrict__ delta,
                          void* __restrict__ dq) {
  using C = DqCfg<DH>;
  extern __shared__ __align__(1024) uint8_t smem[];
  DqBars& sh = *reinterpret_cast<DqBars*>(smem + C::kOffBar);
  WinSlot* slots = reinterpret_cast<WinSlot*>(smem + C::kOffWin);  // windowed only
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_status_dq, 2u);
    return;
  }
  volatile int* abort_flag = &sh.abort_flag;
  unsigned int* status = &g_status_dq;
  const uint64_t tmo = P.timeout_ns;

  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.ds_full[i], 256);
    }
    mbar_init(&sh.dp_full, 1);
    mbar_init(&sh.dq_done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.item_full[i], 1);
      mbar_init(&sh.item_empty[i], 1 + 256 + (WIN ? 1 : 0));  // windowed: the producer reads the slot too
    }
    mbar_init(&sh.dq_free, 256);
    mbar_init(&sh.drain, 1);
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmDO);
  }
  if (warp == 1) {
    tmem_alloc(&sh.tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if constexpr (WIN) {  // the whole warp walks, lane 0 issues
      uint32_t q_phase = 0;
      int kc = 0;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, tmo, status));
      };
      for (int kq = 0;; ++kq) {
        const int w = dq_window_publish(sh, slots, P, kq, lane, abort_flag, tmo, status);
        if (w < 0 || w >= P.n_items) break;
        const WinSlot& item = slots[kq & 1];
        if (!wait(&sh.q_empty, q_phase ^ 1)) break;
        q_phase ^= 1;
        if (lane == 0) {
          mbar_expect_tx(&sh.q_full, 2 * C::kTileBytes);
          for (int d = 0; d < C::kSub; ++d) {
            tma_load_3d(smem + C::kOffQ + d * kSubBytes, &tmQ, &sh.q_full, d * 64, item.h, item.row);
            tma_load_3d(smem + C::kOffDO + d * kSubBytes, &tmDO, &sh.q_full, d * 64, item.h, item.row);
          }
        }
        const int hk = item.h / P.group, nseg = item.nseg;
        const int row0 = item.row - item.a0 - item.r * P.shard_stride;  // of shard 0
        bool ok = true;
        for (int g = 0; g < nseg && ok; ++g) {
          const TileSet set = tiles_of(item.seg[g]);
          const int krow = row0 + item.seg[g].j * P.shard_stride, nb = tile_count(set);
          for (int i = 0; i < nb; ++i, ++kc) {
            const int row = krow + tile_at(set, i) * kKvTileRows;
            const int st = kc & 1, kst = kc % C::kKStages;
            if (!(ok = wait(&sh.k_empty[kst], ((kc / C::kKStages) & 1) ^ 1))) break;
            if (lane == 0) {
              mbar_expect_tx(&sh.k_full[kst], C::kTileBytes);
              for (int d = 0; d < C::kSub; ++d)
                tma_load_3d(smem + C::kOffK + kst * C::kTileBytes + d * kSubBytes, &tmK,
                            &sh.k_full[kst], d * 64, hk, row);
            }
            if (!(ok = wait(&sh.v_empty[st], ((kc >> 1) & 1) ^ 1))) break;
            if (lane == 0) {
              mbar_expect_tx(&sh.v_full[st], C::kTileBytes);
              for (int d = 0; d < C::kSub; ++d)
                tma_load_3d(smem + C::kOffV + st * C::kTileBytes + d * kSubBytes, &tmV,
                            &sh.v_full[st], d * 64, hk, row);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.item_empty[kq & 1]);
        if (!ok) break;
      }
    } else if (lane == 0) {
      uint32_t q_phase = 0;
      int kc = 0;
      for (int kq = 0;; ++kq) {
        const int w = dq_item_publish(sh, P, kq, abort_flag, tmo, status);
        if (w < 0 || w >= P.n_items) break;
        const DqItem it = decode_dq(P, w);
        const SeqDesc& sd = P.seq[it.seq];
        const int L = sd.L;
        const int N = dq_walk_tiles(P, it, L);
        if (N == 0) continue;
        if (!mbar_wait(&sh.q_empty, q_phase ^ 1, abort_flag, tmo, status)) break;
        q_phase ^= 1;
        mbar_expect_tx(&sh.q_full, 2 * C::kTileBytes);
        const int qrow = sd.row_off + it.r * P.shard_stride + it.qt * kQTileRows;
        for (int d = 0; d < C::kSub; ++d) {
          tma_load_3d(smem + C::kOffQ + d * kSubBytes, &tmQ, &sh.q_full, d * 64, it.h, qrow);
          tma_load_3d(smem + C::kOffDO + d * kSubBytes, &tmDO, &sh.q_full, d * 64, it.h, qrow);
        }
        const int hk = it.h / P.group;
        const int a_last = min(L, (it.qt + 1) * kQTileRows) - 1;
        bool ok = true;
        for (int s = P.step_begin; s < P.step_end && ok; ++s) {
          const int j = shard_at_step(P.D, it.r, s);
          const int nb = kv_tiles_for(P, L, it.r, j, a_last);
          const int krow = sd.row_off + j * P.shard_stride;
          for (int b = 0; b < nb; ++b, ++kc) {
            const int st = kc & 1;
            const uint32_t ph = (kc >> 1) & 1;
            const int kst = kc % C::kKStages;
            const uint32_t kph = (kc / C::kKStages) & 1;
            if (!(ok = mbar_wait(&sh.k_empty[kst], kph ^ 1, abort_flag, tmo, status))) break;
            mbar_expect_tx(&sh.k_full[kst], C::kTileBytes);
            for (int d = 0; d < C::kSub; ++d)
              tma_load_3d(smem + C::kOffK + kst * C::kTileBytes + d * kSubBytes, &tmK, &sh.k_full[kst],
                          d * 64, hk, krow + b * kKvTileRows);
            if (!(ok = mbar_wait(&sh.v_empty[st], ph ^ 1, abort_flag, tmo, status))) break;
            mbar_expect_tx(&sh.v_full[st], C::kTileBytes);
            for (int d = 0; d < C::kSub; ++d)
              tma_load_3d(smem + C::kOffV + st * C::kTileBytes + d * kSubBytes, &tmV, &sh.v_full[st],
                          d * 64, hk, krow + b * kKvTileRows);
          }
        }
        if (!ok) break;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t q_phase = 0, dqf_phase = 0;
      uint32_t ds_phase[2] = {0, 0};
      int kc = 0;
      const uint32_t idS = idesc_bf16_f32(128, 128, 0, 0);  // S, dP: A and B K-major
      const uint32_t idQ = idesc_bf16_f32(128, DH, 0, 1);   // dQ: A from TMEM, B MN-major
      const uint32_t sQ = smem_u32(smem + C::kOffQ), sDO = smem_u32(smem + C::kOffDO);
      const uint32_t sK = smem_u32(smem + C::kOffK), sV = smem_u32(smem + C::kOffV);
      bool ok = true;
      for (int kq = 0; ok; ++kq) {
        int w, N;
        if constexpr (WIN) {
          if (!(ok = mbar_wait(&sh.item_full[kq & 1], (kq >> 1) & 1, abort_flag, tmo, status))) break;
          w = slots[kq & 1].item;
          N = slots[kq & 1].tiles;
          mbar_arrive(&sh.item_empty[kq & 1]);
          if (w >= P.n_items) break;
        } else {
          w = dq_item_take(sh, kq, abort_flag, tmo, status);
          if (w < 0) ok = false;
          if (w < 0 || w >= P.n_items) break;
          const DqItem it = decode_dq(P, w);
          N = dq_walk_tiles(P, it, P.seq[it.seq].L);
        }
        if (N == 0) continue;
        if (!(ok = mbar_wait(&sh.q_full, q_phase, abort_flag, tmo, status))) break;
        q_phase ^= 1;
        tc_fence_after();
        auto issue_S = [&](int n) -> bool {
          const int c = kc + n, st = c % C::kKStages;
          if (!mbar_wait(&sh.k_full[st], (c / C::kKStages) & 1, abort_flag, tmo, status)) return false;
          tc_fence_after();
          const uint32_t ka = sK + st * C::kTileBytes;
#pragma unroll
          for (int k = 0; k < C::kKSteps; ++k) {
            const uint32_t off = (k >> 2) * kSubBytes + (k & 3) * 32;
            mma_ss(tmem + (n & 1 ? C::kColS1 : C::kColS0), sdesc_sw128(sQ + off, 16, 1024),
                   sdesc_sw128(ka + off, 16, 1024), idS, k > 0);
          }
          tc_commit(&sh.s_full[n & 1]);
          return true;
        };
        auto issue_dP = [&](int n) -> bool {
          const int c = kc + n, st = c & 1;
          if (!mbar_wait(&sh.v_full[st], (c >> 1) & 1, abort_flag, tmo, status)) return false;
          tc_fence_after();
          const uint32_t va = sV + st * C::kTileBytes;
#pragma unroll
          for (int k = 0; k < C::kKSteps; ++k) {
            const uint32_t off = (k >> 2) * kSubBytes + (k & 3) * 32;
            mma_ss(tmem + C::kColDP, sdesc_sw128(sDO + off, 16, 1024), sdesc_sw128(va + off, 16, 1024),
                   idS, k > 0);
          }
          tc_commit(&sh.dp_full);
          tc_commit(&sh.v_empty[st]);
          return true;
        };
        ok = issue_S(0) && issue_dP(0) && (N == 1 || issue_S(1));
        // the previous item's dq must be out of TMEM before the first dQ overwrites it
        if (ok) {
          ok = mbar_wait(&sh.dq_free, dqf_phase ^ 1, abort_flag, tmo, status);
          dqf_phase ^= 1;
          tc_fence_after();
        }
        for (int n = 0; n < N && ok; ++n) {
          const int c = kc + n, st = c % C::kKStages;
          if (!(ok = mbar_wait(&sh.ds_full[n & 1], ds_phase[n & 1], abort_flag, tmo, status))) break;
          ds_phase[n & 1] ^= 1;
          tc_fence_after();
          // dP(n+1) first: dP(n) has been read (ds_full), and dS(n+1) goes to the other S
          // buffer, so the softmax threads can compute it while dQ(n) runs
          if (n + 1 < N && !(ok = issue_dP(n + 1))) break;
          if constexpr (!DELTA) {
            const uint32_t ka = sK + st * C::kTileBytes;
            const uint32_t tds = tmem + (n & 1 ? C::kColS1 : C::kColS0) + 32;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ts(tmem + C::kColDQ, tds + 8 * k, sdesc_sw128(ka + k * 2048, kSubBytes, 1024), idQ,
                     (n > 0 || k > 0) ? 1u : 0u);
          }
          tc_commit(&sh.k_empty[st]);
          if (n + 2 < N) ok = issue_S(n + 2);
        }
        if (!ok) break;
        tc_commit(&sh.dq_done);
        tc_commit(&sh.q_empty);
        kc += N;
      }
      tc_commit(&sh.drain);
      mbar_wait(&sh.drain, 0, abort_flag, tmo, status);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ P / dS warpgroups
    const int wg = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;  // query row within the tile = TMEM lane
    const int c0 = wg * 64;               // this warpgroup's key columns
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float sl2 = P.scale_log2;
    const uint64_t sl2x2 = f2(sl2, sl2);
    uint32_t s_phase[2] = {0, 0}, dp_phase = 0, dd_phase = 0;
    for (int kq = 0;; ++kq) {
      const WinSlot* item = nullptr;  // windowed: in its slot until the item is done with
      DqItem it;
      int L, a;
      size_t qrow, li = 0;
      bool valid;
      if constexpr (WIN) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sh.item_full[kq & 1], (kq >> 1) & 1, abort_flag, tmo, status))) break;
        item = &slots[kq & 1];
        if (item->item >= P.n_items) break;
        it.h = item->h;
        it.r = item->r;
        L = item->L;
        a = item->a0 + row;
        valid = a < L;
        qrow = static_cast<size_t>(item->row + row);
        li = static_cast<size_t>(item->lse + row);
      } else {
        const int w = dq_item_take(sh, kq, abort_flag, tmo, status);
        if (w < 0 || w >= P.n_items) break;
        it = decode_dq(P, w);
        const SeqDesc& sd = P.seq[it.seq];
        L = sd.L;
        a = it.qt * kQTileRows + row;
        valid = a < L;
        qrow = static_cast<size_t>(sd.row_off + it.r * P.shard_stride + a);
        const int N = dq_walk_tiles(P, it, L);
        if (N == 0) {  // no key visible: dq = 0 (nothing to add for bwd_accum)
          if (valid && !P.bwd_accum) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(dq) + (qrow * P.hq + it.h) * DH;
#pragma unroll
            for (int c = wg * DH / 64; c < (wg + 1) * DH / 64; ++c) {
              uint4* d = reinterpret_cast<uint4*>(dst + c * 32);
#pragma unroll
              for (int q = 0; q < 4; ++q) d[q] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          continue;
        }
        if (valid)
          li = sd.lse_off + static_cast<size_t>(it.h) * P.lse_hstride +
               static_cast<size_t>(it.r) * P.shard_stride + a;
      }
      float nl = -INFINITY, dl = 0.f;
      int64_t pq = 0;
      if (valid) {
        const float l = lse[li];
        nl = l == -INFINITY ? -INFINITY : -l * kLog2e + (WIN ? kWeightShift : 0.f);
        if constexpr (!DELTA) dl = delta[li];
        pq = layout_pos(P.layout, P.D, L, it.r, a);
      }
      KeyLimit upto, before;  // windowed: the last key seen, the last one before the window
      if constexpr (WIN) {
        upto = key_limit_of(P, static_cast<int>(pq));
        before = key_limit_of(P, static_cast<int>(pq - P.window));
      }
      const uint64_t nl2 = f2(nl, nl), dl2 = f2(dl, dl);
      uint64_t row_sum = f2(0.f, 0.f);  // DELTA: of P dP
      const int a_last = WIN ? 0 : min(L, (it.qt + 1) * kQTileRows) - 1;
      int n = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool got = mbar_wait(bar, parity, abort_flag, tmo, status);
        return WIN ? __all_sync(0xffffffffu, got) : got;  // the windowed walk is the warp's
      };
      const int s_end = WIN ? item->nseg : P.step_end;
      for (int s = WIN ? 0 : P.step_begin; s < s_end && ok; ++s) {
        const int j = WIN ? item->seg[s].j : shard_at_step(P.D, it.r, s);
        TileSet set;
        if constexpr (WIN) set = tiles_of(item->seg[s]);
        const int nb = WIN ? tile_count(set) : kv_tiles_for(P, L, it.r, j, a_last);
        int lim, lo = 0, sk = 0;
        if constexpr (WIN) {  // of the shard's keys up to lim this row sees those before sk, and from lo on
          lim = valid ? limit_in(P, L, j, upto) : -1;
          lo = limit_in(P, L, j, before) + 1;
          sk = item->seg[s].sk;
        } else {
          lim = !valid ? -1 : (P.causal ? key_limit(P.layout, P.D, L, j, pq) : L - 1);
        }
        for (int i = 0; i < nb; ++i, ++n) {
          const int b = WIN ? tile_at(set, i) : i;
          const int buf = n & 1;
          const uint32_t tS = tmem + lane_off + (buf ? C::kColS1 : C::kColS0);
          int cnt = lim + 1 - b * kKvTileRows;  // visible keys of this tile (a prefix)
          cnt = cnt < 0 ? 0 : (cnt > kKvTileRows ? kKvTileRows : cnt);
          const int lo_t = WIN ? lo - b * kKvTileRows : 0, sk_t = WIN && b == 0 ? sk : 0;
          if (!(ok = wait(&sh.s_full[buf], s_phase[buf]))) break;
          s_phase[buf] ^= 1;
          tc_fence_after();
          uint32_t pp[32], sv2[2][32];
          bool some[2];  // windowed: the warp's rows see some key of the chunk
          tmem_ld32_nowait(tS + c0, sv2[0]);  // both chunks in flight, one wait
          tmem_ld32_nowait(tS + c0 + 32, sv2[1]);
          tmem_wait_ld();
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            const int cs = c0 + 32 * ch;
            const uint32_t (&sv)[32] = sv2[ch];
            const uint32_t vis = WIN ? visible_bits(cs, cnt, lo_t, sk_t) : 0u;
            if constexpr (WIN) {
              some[ch] = __any_sync(0xffffffffu, vis != 0);
              if (!some[ch]) continue;
            }
            const bool full = __all_sync(0xffffffffu, WIN ? vis == 0xffffffffu : cnt >= cs + 32);
            // staged: every FMA, then every exponential, then masking and packing
            uint64_t xv[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              xv[i] = fma2(f2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])), sl2x2, nl2);
            float ev[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 e = f2_split((i & 7) < RA_DQ_POLY_PAIRS ? exp2_poly2(xv[i]) : xv[i]);
              ev[2 * i] = (i & 7) < RA_DQ_POLY_PAIRS ? e.x : ex2(e.x);  // poly: x <= 0 if visible
              ev[2 * i + 1] = (i & 7) < RA_DQ_POLY_PAIRS ? e.y : ex2(e.y);
            }
            if (!full) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (WIN ? !((vis >> i) & 1u) : cs + i >= cnt) ev[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              pp[16 * ch + i] = WIN ? pack_f16x2(ev[2 * i], ev[2 * i + 1]) : pack_bf16x2(ev[2 * i], ev[2 * i + 1]);
          }
          if (!(ok = wait(&sh.dp_full, dp_phase))) break;
          dp_phase ^= 1;
          tc_fence_after();
          uint32_t dp2[2][32];
          tmem_ld32_nowait(tmem + lane_off + C::kColDP + c0, dp2[0]);
          tmem_ld32_nowait(tmem + lane_off + C::kColDP + c0 + 32, dp2[1]);
          tmem_wait_ld();
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            const uint32_t (&dp)[32] = dp2[ch];
            if constexpr (DELTA) {
              if (some[ch]) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  row_sum = fma2(f2(__uint_as_float(dp[2 * i]), __uint_as_float(dp[2 * i + 1])),
                                 f2_of_f16x2(pp[16 * ch + i]), row_sum);
              }
              continue;
            }
            uint32_t o[16];
            if (WIN && !some[ch]) {
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = 0;
              tmem_st16(tS + 32 + c0 / 2 + 16 * ch, o);
              continue;
            }
            uint64_t xv[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              xv[i] = sub2(f2(__uint_as_float(dp[2 * i]), __uint_as_float(dp[2 * i + 1])), dl2);
#pragma unroll
            for (int i = 0; i < 16; ++i) xv[i] = mul2(xv[i], WIN ? f2_of_f16x2(pp[16 * ch + i]) : f2_of_bf16x2(pp[16 * ch + i]));
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = bf16x2_of(xv[i]);
            // dS (bf16) into columns [32, 96) of this tile's S buffer (read into registers
            // above): the A operand of dQ += dS K
            tmem_st16(tS + 32 + c0 / 2 + 16 * ch, o);
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&sh.ds_full[buf]);
        }
      }
      if (!ok) break;
      // dq = scale * dQ (or dq += scale * dQ into float32 sums for bwd_accum, the per-step
      // block backward): warpgroup 0 takes columns [0, DH/2), warpgroup 1 the rest
      if (!wait(&sh.dq_done, dd_phase)) break;
      dd_phase ^= 1;
      tc_fence_after();
      if constexpr (DELTA) {  // two addends on 0: the same sum in either order
        const float2 half = f2_split(row_sum);
        if (valid) atomicAdd(static_cast<float*>(dq) + li, (half.x + half.y) * kWeightUnit);
        tc_fence_before();
        mbar_arrive(&sh.dq_free);
        mbar_arrive(&sh.item_empty[kq & 1]);
        continue;
      }
      const size_t qoff = (qrow * P.hq + it.h) * DH;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(dq) + qoff;
      float* dst_acc = static_cast<float*>(dq) + qoff;
      const float mul = P.scale * (WIN ? kWeightUnit : 1.f);
#pragma unroll
      for (int c = 0; c < DH / 64; ++c) {
        const int col = wg * (DH / 2) + 32 * c;
        uint32_t rr[32];
        tmem_ld32(tmem + lane_off + C::kColDQ + col, rr);
        if (valid && P.bwd_accum) {
          float4* d = reinterpret_cast<float4*>(dst_acc + col);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float4 u = d[q];
            u.x += __uint_as_float(rr[4 * q + 0]) * P.scale;
            u.y += __uint_as_float(rr[4 * q + 1]) * P.scale;
            u.z += __uint_as_float(rr[4 * q + 2]) * P.scale;
            u.w += __uint_as_float(rr[4 * q + 3]) * P.scale;
            d[q] = u;
          }
        } else if (valid) {
          uint4* d = reinterpret_cast<uint4*>(dst + col);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 u;
            u.x = pack_bf16x2(__uint_as_float(rr[8 * q + 0]) * mul, __uint_as_float(rr[8 * q + 1]) * mul);
            u.y = pack_bf16x2(__uint_as_float(rr[8 * q + 2]) * mul, __uint_as_float(rr[8 * q + 3]) * mul);
            u.z = pack_bf16x2(__uint_as_float(rr[8 * q + 4]) * mul, __uint_as_float(rr[8 * q + 5]) * mul);
            u.w = pack_bf16x2(__uint_as_float(rr[8 * q + 6]) * mul, __uint_as_float(rr[8 * q + 7]) * mul);
            d[q] = u;
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&sh.dq_free);
      if constexpr (WIN) mbar_arrive(&sh.item_empty[kq & 1]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if constexpr (WIN && !DELTA) wait_for_previous();  // what follows this kernel reads the K/V pass' sums too
}

template <int DH, bool WIN, bool DELTA = false>
cudaError_t launch_one(const Plan& P, const CUtensorMap& mq, const CUtensorMap& mk,
                       const CUtensorMap& mv, const CUtensorMap& mdo, const float* lse,
                       const float* delta, void* dq, int n_items, int n_sm, cudaStream_t st) {
  using C = DqCfg<DH>;
  auto kern = ring_bwd_dq_tc_kernel<DH, WIN, DELTA>;
  constexpr int smem = WIN ? C::kSmemWindow : C::kSmemBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = n_items < n_sm ? n_items : n_sm;
  if constexpr (WIN && !DELTA) {  // starts where the K/V pass leaves an SM free
    cudaLaunchAttribute early = {};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kDqThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, mdo, P, lse, delta, dq);
  }
  kern<<<grid, kDqThreads, smem, st>>>(mq, mk, mv, mdo, P, lse, delta, dq);
  return cudaGetLastError();
}

}  // namespace

namespace {

// The tensor maps and the plan of a pass over query tiles (its items renumbered), and its launch:
// launch(plan, maps of q, k, v, dout, SMs).
template <typename F>
cudaError_t over_query_tiles(const Plan& P0, int counter, const void* q, const void* k, const void* v,
                             const void* dout, F&& launch) {
  Plan P = P0;
  P.work_counter = P0.work_counter ? P0.work_counter + counter : nullptr;
  int items = 0;
  for (int i = 0; i < P.n_seqs; ++i) {
    P.seq[i].item_start = items;
    items += dq_items_of(P, P.seq[i].L);
  }
  P.n_items = items;
  if (items == 0) return cudaSuccess;
  CUtensorMap mq, mk, mv, mdo;
  cudaError_t e = make_token_tmap(&mq, q, P.n_rows, P.hq, P.head_dim);
  if (e == cudaSuccess) e = make_token_tmap(&mk, k, P.n_rows, P.hkv, P.head_dim);
  if (e == cudaSuccess) e = make_token_tmap(&mv, v, P.n_rows, P.hkv, P.head_dim);
  if (e == cudaSuccess) e = make_token_tmap(&mdo, dout, P.n_rows, P.hq, P.head_dim);
  if (e != cudaSuccess) return e;
  int dev = 0, n_sm = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  return launch(P, mq, mk, mv, mdo, n_sm);
}

}  // namespace

cudaError_t launch_bwd_dq_tc(const Plan& P0, const void* q, const void* k, const void* v,
                             const void* dout, const float* lse, const float* delta, void* dq,
                             cudaStream_t st) {
  // the second counter of the block
  return over_query_tiles(P0, 1, q, k, v, dout, [&](const Plan& P, auto& mq, auto& mk, auto& mv, auto& mdo, int n_sm) {
    if (P.window > 0)
      return P.head_dim == 128 ? launch_one<128, true>(P, mq, mk, mv, mdo, lse, delta, dq, P.n_items, n_sm, st)
                               : launch_one<64, true>(P, mq, mk, mv, mdo, lse, delta, dq, P.n_items, n_sm, st);
    return P.head_dim == 128 ? launch_one<128, false>(P, mq, mk, mv, mdo, lse, delta, dq, P.n_items, n_sm, st)
                             : launch_one<64, false>(P, mq, mk, mv, mdo, lse, delta, dq, P.n_items, n_sm, st);
  });
}

cudaError_t launch_window_delta_tc(const Plan& P0, const void* q, const void* k, const void* v, const void* dout,
                                   const float* lse, float* delta, cudaStream_t st) {
  return over_query_tiles(P0, 2, q, k, v, dout, [&](const Plan& P, auto& mq, auto& mk, auto& mv, auto& mdo, int n_sm) {
    return P.head_dim == 128
               ? launch_one<128, true, true>(P, mq, mk, mv, mdo, lse, nullptr, delta, P.n_items, n_sm, st)
               : launch_one<64, true, true>(P, mq, mk, mv, mdo, lse, nullptr, delta, P.n_items, n_sm, st);
  });
}

cudaError_t bwd_dq_status(unsigned int* value, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_status_dq, sizeof(unsigned int));
  if (e == cudaSuccess && reset) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_status_dq, &zero, sizeof(unsigned int));
  }
  return e;
}

}  // namespace ra
