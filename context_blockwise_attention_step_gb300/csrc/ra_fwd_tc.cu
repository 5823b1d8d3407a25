// ra_fwd_tc.cu — fused ring-attention forward on the 5th-generation tensor cores (sm_103a).
//
// One persistent CTA per SM takes work items (256 query rows of one rank and one query
// head) and walks the ring: for step s = begin..end-1 it reads the K/V shard
// j = (r - s) mod D (Ring Attention concept page, "Sequence sharding and the ring
// topology") and, of that shard, only the 128-row K/V tiles that some query of the block
// may see under the global-position causal rule ("Watch Out For"). For each tile:
//
//   S = Q K^T          tcgen05.mma, Q and K tiles TMA-loaded into 128B-swizzled smem,
//                      S (128 x 128 f32) accumulated in TMEM
//   online softmax     two threads per query row (64 columns each) read the S row from
//                      TMEM, mask the columns beyond the key count, update the running max
//                      m and denominator l, write P = 2^(S*scale*log2e - m) as bf16 back
//                      into TMEM over consumed S columns
//   O += P V           tcgen05.mma with A = P from TMEM, B = V tile (MN-major) from smem
//
// The running (m, l, O) persists across all tiles and all ring steps of the block, which
// is the log-sum-exp merge of update_out_and_lse (nanotron how-to page, "Numerically-
// Stable Output Fusion"; interview question page: rescale the old partial by
// exp(old_max - new_max)) fused into the tile loop. O is rescaled only when a row max grows
// by more than 2^8: with a stale reference value every exponent stays <= 2^8, and the final
// out = O / l and lse = m + log l are the same quantities (an exact identity, not an
// approximation). Finally out = O / l (bf16, or f32 for block outputs) and lse (natural
// log, f32) are written; a row that saw no key gets out = 0, lse = -inf.
//
// Warp roles (640 threads): warp 0 = TMA producer, warp 1 = TMEM allocator + MMA issuer,
// warps 4-11 = softmax of query tile 0, warps 12-19 = softmax of query tile 1. Each tile's
// rows are split between two warpgroups of 64 key columns, which exchange their partial
// row maxima every K/V tile and their partial sums at the end through shared memory; P
// goes to S columns [32, 96), each half on its own S columns. The two tiles ping-pong: the
// MMA order S0(n) S1(n) | O0(n) S0(n+1) O1(n) S1(n+1) | ... lets one tile's softmax run
// while the tensor core works on the other tile.
//
// WIN (sliding window with always visible first tokens): a block walks the K/V tiles that some
// of its rows sees through the window, and the first tile of the shards that hold sinks. The
// producer warp works these out ahead of time, one shard a lane, and leaves them with the item's
// other data in the item queue's slot, where the other roles read them until they are done; a
// K/V tile goes only to those of the block's two query tiles that see it, and 32 columns that no
// row of a warp sees are not worked out. What bounds it is what bounds the ring's forward, and the
// tiles' hidden parts: 65536 tokens in 16 sequences over 8 shards, 32/8 heads of 128, window 1024
// meet 1.97 times the visible pairs in whole tiles. 2.32 ms there (822 TFLOP/s of executed tiles),
// 44 us for 2 x 4096 tokens, 8 heads of 64, window 500, where 256 items make two rounds of 152 CTAs.
#include <cuda_runtime.h>

#include "ra_internal.h"
#include "ra_plan.h"
#include "ra_ptx.cuh"
#include "ra_window.cuh"

namespace ra {

static __device__ unsigned int g_status_fwd;

namespace {

constexpr int kFwdThreads = 640;  // 4 control warps + 4 softmax warpgroups (2 per query tile)
constexpr int kSubBytes = 128 * 128;  // 128 rows x 64 bf16: one 128B-swizzled sub-tile

template <int DH>
struct FwdCfg {
  static constexpr int kStages = DH == 128 ? 2 : 4;
  static constexpr int kSub = DH / 64;
  static constexpr int kTileBytes = 128 * DH * 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kSmemBytes = kOffV + kStages * kTileBytes + 1024;
  static constexpr int kKSteps = DH / 16;
  static constexpr uint32_t kTmemCols = 512;
  // TMEM columns: S0 | S1 | O0 | O1 (P of tile t overwrites the first 64 columns of S_t)
  __device__ static constexpr uint32_t col_s(int t) { return t ? 128u : 0u; }
  __device__ static constexpr uint32_t col_o(int t) { return t ? 256u + DH : 256u; }
};

struct FwdShared {
  uint64_t q_full, q_empty;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];
  uint64_t drain;
  uint64_t xmax_bar[2][2], xl_bar[2];  // half-row exchanges: [tile][slot], [tile]
  uint64_t item_full[2], item_empty[2];  // the CTA's item queue
  int item[2];
  uint32_t tmem_base;
  int abort_flag;
  float xmax[2][2][2][128];  // [tile][slot][half][row]: partial row maxima
  float xl[2][2][128];       // [tile][half][row]: partial row sums
};
// Windowed: the item queue's slots.
template <bool WIN>
struct FwdSlots {
  WinSlot slot[2];
  WinSeg half[2][2][kMaxWindowShards];  // [slot][query tile]: the tiles each query tile sees
  uint8_t flags[8];  // of the K/V tiles in flight: bit t: query tile t sees it; bit 2 + t: as its last
};
template <>
struct FwdSlots<false> {};

// Total K/V tiles a forward item walks, and its first/last valid query rows.
struct FwdWalk {
  int L, a0, a_last, N;
  bool two;
};

__device__ __forceinline__ FwdWalk fwd_walk(const Plan& P, const FwdItem& it) {
  FwdWalk w;
  w.L = P.seq[it.seq].L;
  w.a0 = it.blk * kFwdBlockRows;
  const int a_end = min(w.L, w.a0 + kFwdBlockRows);
  w.a_last = a_end - 1;
  w.two = (a_end - w.a0) > kQTileRows;
  w.N = 0;
  for (int s = P.step_begin; s < P.step_end; ++s)
    w.N += kv_tiles_for(P, w.L, it.r, shard_at_step(P.D, it.r, s), w.a_last);
  return w;
}

template <typename OutT>
__device__ __forceinline__ void store_row32(OutT* dst, const float (&v)[32]);

template <>
__device__ __forceinline__ void store_row32<__nv_bfloat16>(__nv_bfloat16* dst, const float (&v)[32]) {
  uint4* d = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint4 u;
    u.x = pack_bf16x2(v[8 * q + 0], v[8 * q + 1]);
    u.y = pack_bf16x2(v[8 * q + 2], v[8 * q + 3]);
    u.z = pack_bf16x2(v[8 * q + 4], v[8 * q + 5]);
    u.w = pack_bf16x2(v[8 * q + 6], v[8 * q + 7]);
    d[q] = u;
  }
}
template <>
__device__ __forceinline__ void store_row32<float>(float* dst, const float (&v)[32]) {
  float4* d = reinterpret_cast<float4*>(dst);
#pragma unroll
  for (int q = 0; q < 8; ++q) d[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
}

// The CTA's item queue (two slots): the producer thread takes the next item from the shared
// counter when the caller passed a workspace (a CTA that finishes early takes more items,
// in index order), else by the static stride, and publishes it; the MMA thread and the
// softmax threads read it from the ring. A value >= n_items ends the walk.
__device__ __forceinline__ int fwd_item_publish(FwdShared& sh, const Plan& P, int k,
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
__device__ __forceinline__ int fwd_item_take(FwdShared& sh, int k, volatile int* abort_flag,
                                             uint64_t tmo, unsigned int* status) {
  const int slot = k & 1;
  if (!mbar_wait(&sh.item_full[slot], (k >> 1) & 1, abort_flag, tmo, status)) return -1;
  const int w = *reinterpret_cast<volatile int*>(&sh.item[slot]);
  mbar_arrive(&sh.item_empty[slot]);
  return w;
}

// The windowed kernel's item queue: the producer warp takes the next item and fills in its slot;
// the other roles read it in place and release it when they have done with the item.
__device__ __forceinline__ int fwd_window_publish(FwdShared& sh, FwdSlots<true>& win, const Plan& P, int k, int lane,
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
    const FwdItem it = decode_fwd(P, w);
    const int a0 = it.blk * kFwdBlockRows;
    fill_slot<true>(win.slot[slot], win.half[slot][0], P, it.seq, it.h, it.r, a0, min(P.seq[it.seq].L, a0 + kFwdBlockRows) - 1);
  }
  if (lane == 0) {
    win.slot[slot].item = w;
    mbar_arrive(&sh.item_full[slot]);
  }
  return w;
}

template <int DH, typename OutT, bool WIN>
__global__ void __launch_bounds__(kFwdThreads, 1)
    ring_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Plan P,
                       OutT* __restrict__ out, float* __restrict__ lse) {
  using C = FwdCfg<DH>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ FwdShared sh;
  __shared__ FwdSlots<WIN> win;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sh.abort_flag;
  unsigned int* status = &g_status_fwd;
  const uint64_t tmo = P.timeout_ns;

  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_full[t], 256);
      mbar_init(&sh.o_done[t], 1);
      mbar_init(&sh.o_free[t], 256);
      mbar_init(&sh.xmax_bar[t][0], 256);
      mbar_init(&sh.xmax_bar[t][1], 256);
      mbar_init(&sh.xl_bar[t], 256);
    }
    mbar_init(&sh.drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.item_full[i], 1);
      // MMA thread and softmax warps; windowed also the producer, which reads the slot itself
      mbar_init(&sh.item_empty[i], (WIN ? 2 : 1) + (kFwdThreads - 128));
    }
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
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
      int kv_count = 0;
      uint32_t q_phase = 0;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, tmo, status));
      };
      for (int kq = 0;; ++kq) {
        const int w = fwd_window_publish(sh, win, P, kq, lane, abort_flag, tmo, status);
        if (w < 0 || w >= P.n_items) break;
        const WinSlot& item = win.slot[kq & 1];
        const bool two = item.a1 - item.a0 >= kQTileRows;
        if (!wait(&sh.q_empty, q_phase ^ 1)) break;
        q_phase ^= 1;
        if (lane == 0) {
          mbar_expect_tx(&sh.q_full, (two ? 2 : 1) * C::kTileBytes);
          for (int t = 0; t < (two ? 2 : 1); ++t)
            for (int d = 0; d < C::kSub; ++d)
              tma_load_3d(smem + C::kOffQ + t * C::kTileBytes + d * kSubBytes, &tmQ, &sh.q_full,
                          d * 64, item.h, item.row + t * kQTileRows);
        }
        const int hk = item.h / P.group, nseg = item.nseg;
        const int row0 = item.row - item.a0 - item.r * P.shard_stride;  // of shard 0
        int left[2] = {0, 0};  // K/V tiles that the query tiles have yet to see
        for (int g = 0; g < nseg; ++g)
          for (int t = 0; t < 2; ++t) left[t] += tile_count(tiles_of(win.half[kq & 1][t][g]));
        bool ok = true;
        for (int g = 0; g < nseg && ok; ++g) {
          const TileSet set = tiles_of(item.seg[g]);
          const TileSet half[2] = {tiles_of(win.half[kq & 1][0][g]), tiles_of(win.half[kq & 1][1][g])};
          const int krow = row0 + item.seg[g].j * P.shard_stride, nb = tile_count(set);
          for (int i = 0; i < nb; ++i, ++kv_count) {
            const int b = tile_at(set, i), row = krow + b * kKvTileRows;
            unsigned flags = 0;
            for (int t = 0; t < 2; ++t)
              if (has_tile(half[t], b)) flags |= (--left[t] == 0 ? 5u : 1u) << t;
            const int st = kv_count % C::kStages;
            const uint32_t ph = (kv_count / C::kStages) & 1;
            if (!(ok = wait(&sh.k_empty[st], ph ^ 1))) break;
            if (lane == 0) {
              win.flags[kv_count & 7] = static_cast<uint8_t>(flags);  // read after k_full
              mbar_expect_tx(&sh.k_full[st], C::kTileBytes);
              for (int d = 0; d < C::kSub; ++d)
                tma_load_3d(smem + C::kOffK + st * C::kTileBytes + d * kSubBytes, &tmK,
                            &sh.k_full[st], d * 64, hk, row);
            }
            if (!(ok = wait(&sh.v_empty[st], ph ^ 1))) break;
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
      int kv_count = 0;
      uint32_t q_phase = 0;
      for (int kq = 0;; ++kq) {
        const int w = fwd_item_publish(sh, P, kq, abort_flag, tmo, status);
        if (w < 0 || w >= P.n_items) break;
        const FwdItem it = decode_fwd(P, w);
        const FwdWalk wk = fwd_walk(P, it);
        if (wk.N == 0) continue;
        const SeqDesc& sd = P.seq[it.seq];
        if (!mbar_wait(&sh.q_empty, q_phase ^ 1, abort_flag, tmo, status)) goto producer_done;
        q_phase ^= 1;
        mbar_expect_tx(&sh.q_full, (wk.two ? 2 : 1) * C::kTileBytes);
        {
          const int qrow = sd.row_off + it.r * P.shard_stride + wk.a0;
          for (int t = 0; t < (wk.two ? 2 : 1); ++t)
            for (int d = 0; d < C::kSub; ++d)
              tma_load_3d(smem + C::kOffQ + t * C::kTileBytes + d * kSubBytes, &tmQ, &sh.q_full,
                          d * 64, it.h, qrow + t * kQTileRows);
        }
        const int hk = it.h / P.group;
        for (int s = P.step_begin; s < P.step_end; ++s) {
          const int j = shard_at_step(P.D, it.r, s);
          const int nb = kv_tiles_for(P, wk.L, it.r, j, wk.a_last);
          const int krow = sd.row_off + j * P.shard_stride;
          for (int b = 0; b < nb; ++b, ++kv_count) {
            const int st = kv_count % C::kStages;
            const uint32_t ph = (kv_count / C::kStages) & 1;
            if (!mbar_wait(&sh.k_empty[st], ph ^ 1, abort_flag, tmo, status)) goto producer_done;
            mbar_expect_tx(&sh.k_full[st], C::kTileBytes);
            for (int d = 0; d < C::kSub; ++d)
              tma_load_3d(smem + C::kOffK + st * C::kTileBytes + d * kSubBytes, &tmK,
                          &sh.k_full[st], d * 64, hk, krow + b * kKvTileRows);
            if (!mbar_wait(&sh.v_empty[st], ph ^ 1, abort_flag, tmo, status)) goto producer_done;
            mbar_expect_tx(&sh.v_full[st], C::kTileBytes);
            for (int d = 0; d < C::kSub; ++d)
              tma_load_3d(smem + C::kOffV + st * C::kTileBytes + d * kSubBytes, &tmV,
                          &sh.v_full[st], d * 64, hk, krow + b * kKvTileRows);
          }
        }
      }
    producer_done:;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int kv_count = 0;
      uint32_t q_phase = 0, p_phase[2] = {0, 0}, of_phase[2] = {0, 0};
      const uint32_t idS = idesc_bf16_f32(128, 128, 0, 0);
      const uint32_t idO = idesc_bf16_f32(128, DH, 0, 1);
      const uint32_t sQ = smem_u32(smem + C::kOffQ);
      const uint32_t sK = smem_u32(smem + C::kOffK);
      const uint32_t sV = smem_u32(smem + C::kOffV);
      bool ok = true;
      for (int kq = 0; ok; ++kq) {
        int w, N;
        bool two;
        if constexpr (WIN) {
          if (!(ok = mbar_wait(&sh.item_full[kq & 1], (kq >> 1) & 1, abort_flag, tmo, status))) break;
          const WinSlot& item = win.slot[kq & 1];
          w = item.item;
          N = item.tiles;
          two = item.a1 - item.a0 >= kQTileRows;
          mbar_arrive(&sh.item_empty[kq & 1]);
          if (w >= P.n_items) break;
        } else {
          w = fwd_item_take(sh, kq, abort_flag, tmo, status);
          if (w < 0) ok = false;
          if (w < 0 || w >= P.n_items) break;
          const FwdItem it = decode_fwd(P, w);
          const FwdWalk wk = fwd_walk(P, it);
          N = wk.N;
          two = wk.two;
        }
        if (N == 0) continue;
        const int nt = two ? 2 : 1;
        if (!(ok = mbar_wait(&sh.q_full, q_phase, abort_flag, tmo, status))) break;
        q_phase ^= 1;
        tc_fence_after();
        if constexpr (WIN) {
          // Tile n of the walk goes to the query tiles that see it: O_t(n-1), S_t(n) for t = 0, 1.
          unsigned prev = 0;
          bool first[2] = {true, true};
          for (int n = 0; n <= N && ok; ++n) {
            unsigned cur = 0;
            const int c = kv_count + n, st = c % C::kStages, pst = (c + C::kStages - 1) % C::kStages;
            for (int t = 0; t < 2 && ok; ++t) {
              if ((prev >> t) & 1u) {
                if (t == 0 || !(prev & 1u))
                  if (!(ok = mbar_wait(&sh.v_full[pst], ((c - 1) / C::kStages) & 1, abort_flag, tmo, status))) break;
                if (!(ok = mbar_wait(&sh.p_full[t], p_phase[t], abort_flag, tmo, status))) break;
                p_phase[t] ^= 1;
                if (first[t]) {
                  if (!(ok = mbar_wait(&sh.o_free[t], of_phase[t] ^ 1, abort_flag, tmo, status))) break;
                  of_phase[t] ^= 1;
                }
                tc_fence_after();
                const uint32_t va = sV + pst * C::kTileBytes;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  mma_ts(tmem + C::col_o(t), tmem + C::col_s(t) + 32 + 8 * k,
                         sdesc_sw128(va + k * 2048, kSubBytes, 1024), idO, (!first[t] || k > 0) ? 1u : 0u);
                first[t] = false;
                if ((prev >> (2 + t)) & 1u) tc_commit(&sh.o_done[t]);
                if (t == 1 || !(prev & 2u)) tc_commit(&sh.v_empty[pst]);
              }
              if (n == N) continue;
              if (t == 0) {
                if (!(ok = mbar_wait(&sh.k_full[st], (c / C::kStages) & 1, abort_flag, tmo, status))) break;
                tc_fence_after();
                cur = *reinterpret_cast<volatile uint8_t*>(&win.flags[c & 7]);
              }
              if ((cur >> t) & 1u) {
                const uint32_t qa = sQ + t * C::kTileBytes, ka = sK + st * C::kTileBytes;
#pragma unroll
                for (int k = 0; k < C::kKSteps; ++k) {
                  const uint32_t off = (k >> 2) * kSubBytes + (k & 3) * 32;
                  mma_ss(tmem + C::col_s(t), sdesc_sw128(qa + off, 16, 1024),
                         sdesc_sw128(ka + off, 16, 1024), idS, k > 0);
                }
                tc_commit(&sh.s_full[t]);
                if (t == 1 || !(cur & 2u)) tc_commit(&sh.k_empty[st]);
              }
            }
            prev = cur;
          }
          tc_commit(&sh.q_empty);
          kv_count += N;
          continue;
        }
        auto issue_S = [&](int t, int n) -> bool {
          const int c = kv_count + n;
          const int st = c % C::kStages;
          const uint32_t ph = (c / C::kStages) & 1;
          if (t == 0) {
            if (!mbar_wait(&sh.k_full[st], ph, abort_flag, tmo, status)) return false;
            tc_fence_after();
          }
          const uint32_t qa = sQ + t * C::kTileBytes, ka = sK + st * C::kTileBytes;
#pragma unroll
          for (int k = 0; k < C::kKSteps; ++k) {
            const uint32_t off = (k >> 2) * kSubBytes + (k & 3) * 32;
            mma_ss(tmem + C::col_s(t), sdesc_sw128(qa + off, 16, 1024),
                   sdesc_sw128(ka + off, 16, 1024), idS, k > 0);
          }
          tc_commit(&sh.s_full[t]);
          if (t == nt - 1) tc_commit(&sh.k_empty[st]);
          return true;
        };
        auto issue_O = [&](int t, int n) -> bool {
          const int c = kv_count + n;
          const int st = c % C::kStages;
          const uint32_t ph = (c / C::kStages) & 1;
          if (t == 0) {
            if (!mbar_wait(&sh.v_full[st], ph, abort_flag, tmo, status)) return false;
          }
          if (!mbar_wait(&sh.p_full[t], p_phase[t], abort_flag, tmo, status)) return false;
          p_phase[t] ^= 1;
          if (n == 0) {
            if (!mbar_wait(&sh.o_free[t], of_phase[t] ^ 1, abort_flag, tmo, status)) return false;
            of_phase[t] ^= 1;
          }
          tc_fence_after();
          const uint32_t va = sV + st * C::kTileBytes;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts(tmem + C::col_o(t), tmem + C::col_s(t) + 32 + 8 * k,
                   sdesc_sw128(va + k * 2048, kSubBytes, 1024), idO, (n > 0 || k > 0) ? 1u : 0u);
          if (n == N - 1) tc_commit(&sh.o_done[t]);
          if (t == nt - 1) tc_commit(&sh.v_empty[st]);
          return true;
        };
        ok = issue_S(0, 0) && (nt == 1 || issue_S(1, 0));
        for (int n = 0; n < N && ok; ++n) {
          ok = issue_O(0, n) && (n + 1 >= N || issue_S(0, n + 1));
          if (ok && nt == 2) ok = issue_O(1, n) && (n + 1 >= N || issue_S(1, n + 1));
        }
        tc_commit(&sh.q_empty);
        kv_count += N;
      }
      // let every MMA issued so far finish before TMEM is released
      tc_commit(&sh.drain);
      mbar_wait(&sh.drain, 0, abort_flag, tmo, status);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax + epilogue
    // Query tile t = (warp - 4) / 8; its rows are split in two halves of 64 key columns
    // (hf), each held by one warpgroup; the halves exchange partial maxima per tile and
    // partial sums at the end through shared memory (bounded mbarrier waits).
    const int t = (warp - 4) >> 3;
    const int hf = ((warp - 4) >> 2) & 1;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int c0 = hf * 64;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::col_s(t);
    const uint32_t tO = tmem + lane_off + C::col_o(t);
    const float sl2 = P.scale_log2;
    const uint64_t sl2x2 = f2(sl2, sl2);
    uint32_t s_phase = 0, od_phase = 0, xl_phase = 0;
    uint32_t xm_phase[2] = {0, 0};
    int xn = 0;  // max exchanges done (slot = xn & 1)
    for (int kq = 0;; ++kq) {
      const WinSlot* item = nullptr;  // windowed: in its slot until the item is done with
      FwdItem it;
      FwdWalk wk;
      if constexpr (WIN) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sh.item_full[kq & 1], (kq >> 1) & 1, abort_flag, tmo, status))) break;
        item = &win.slot[kq & 1];
        if (item->item >= P.n_items) break;
        wk.L = item->L;
        wk.a0 = item->a0;
        wk.two = item->a1 - item->a0 >= kQTileRows;
        it.r = item->r;
        if (t == 1 && !wk.two) {
          mbar_arrive(&sh.item_empty[kq & 1]);
          continue;
        }
      } else {
        const int w = fwd_item_take(sh, kq, abort_flag, tmo, status);
        if (w < 0 || w >= P.n_items) break;
        it = decode_fwd(P, w);
        wk = fwd_walk(P, it);
        if (t == 1 && !wk.two) continue;
      }
      const int a = wk.a0 + t * kQTileRows + row;
      const bool valid = a < wk.L;
      OutT* orow_ptr = nullptr;
      float* lse_ptr = nullptr;
      if constexpr (!WIN) {
        const SeqDesc& sd = P.seq[it.seq];
        const int orow = sd.row_off + it.r * P.shard_stride + a;
        orow_ptr = out + (static_cast<size_t>(orow) * P.hq + it.h) * DH;
        lse_ptr = lse + sd.lse_off + static_cast<size_t>(it.h) * P.lse_hstride +
                  static_cast<size_t>(it.r) * P.shard_stride + a;
        if (wk.N == 0) {  // a block with no visible key at these steps
          if (valid) {
            float z[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = 0.f;
#pragma unroll
            for (int c = 0; c < DH / 64; ++c) store_row32<OutT>(orow_ptr + hf * (DH / 2) + c * 32, z);
            if (hf == 0) *lse_ptr = -INFINITY;
          }
          continue;
        }
      }
      const int64_t pq = valid ? layout_pos(P.layout, P.D, wk.L, it.r, a) : 0;
      KeyLimit upto, before;  // windowed: the last key seen, the last one before the window
      if constexpr (WIN) {
        upto = key_limit_of(P, static_cast<int>(pq));
        before = key_limit_of(P, static_cast<int>(pq - P.window));
      }
      float m = -INFINITY, l = 0.f;
      int n = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool got = mbar_wait(bar, parity, abort_flag, tmo, status);
        return WIN ? __all_sync(0xffffffffu, got) : got;  // the windowed walk is the warp's, to its end
      };
      const int s_end = WIN ? item->nseg : P.step_end;
      for (int s = WIN ? 0 : P.step_begin; s < s_end && ok; ++s) {
        const int j = WIN ? item->seg[s].j : shard_at_step(P.D, it.r, s);
        TileSet set;
        if constexpr (WIN) set = tiles_of(win.half[kq & 1][t][s]);
        const int nb = WIN ? tile_count(set) : kv_tiles_for(P, wk.L, it.r, j, wk.a_last);
        int lim, lo = 0, sk = 0;
        if constexpr (WIN) {  // of the shard's keys up to lim this row sees those before sk, and from lo on
          lim = valid ? limit_in(P, wk.L, j, upto) : -1;
          lo = limit_in(P, wk.L, j, before) + 1;
          sk = item->seg[s].sk;
        } else {
          lim = !valid ? -1 : (P.causal ? key_limit(P.layout, P.D, wk.L, j, pq) : wk.L - 1);
        }
        for (int i = 0; i < nb; ++i, ++n) {
          const int b = WIN ? tile_at(set, i) : i;
          if (!(ok = wait(&sh.s_full[t], s_phase))) break;
          s_phase ^= 1;
          tc_fence_after();
          int cnt = lim + 1 - b * kKvTileRows;
          cnt = cnt < 0 ? 0 : (cnt > kKvTileRows ? kKvTileRows : cnt);
          const int lo_t = WIN ? lo - b * kKvTileRows : 0, sk_t = WIN && b == 0 ? sk : 0;
          const bool full =  // no mask needed
              __all_sync(0xffffffffu, cnt == kKvTileRows && (!WIN || lo_t <= sk_t));
          uint32_t vis[2];
          bool some[2], all[2];  // of a chunk: the warp's rows see some column, every column
          if constexpr (WIN) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              vis[h] = visible_bits(c0 + 32 * h, cnt, lo_t, sk_t);
              some[h] = __any_sync(0xffffffffu, vis[h] != 0);
              all[h] = __all_sync(0xffffffffu, vis[h] == 0xffffffffu);
            }
          }
          // pass 1: partial row max over this half's visible columns, then both halves'
          uint32_t r2[2][32];
          tmem_ld32_nowait(tS + c0, r2[0]);
          tmem_ld32_nowait(tS + c0 + 32, r2[1]);
          tmem_wait_ld();
          float mx;
          {  // four independent max chains (one chain of 32 dependent max ops is slow)
            float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (full) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  mq[2 * h] = max3(mq[2 * h], __uint_as_float(r2[h][i]), __uint_as_float(r2[h][i + 1]));
                  mq[2 * h + 1] =
                      max3(mq[2 * h + 1], __uint_as_float(r2[h][i + 2]), __uint_as_float(r2[h][i + 3]));
                }
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (WIN && !some[h]) continue;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const bool see = WIN ? (vis[h] >> i) & 1u : c0 + 32 * h + i < cnt;
                  const float v = see ? __uint_as_float(r2[h][i]) : -INFINITY;
                  mq[2 * h + (i & 1)] = fmaxf(mq[2 * h + (i & 1)], v);
                }
              }
            }
            mx = fmaxf(max3(mq[0], mq[1], mq[2]), mq[3]);
          }
          {
            const int slot = xn & 1;
            sh.xmax[t][slot][hf][row] = mx;
            mbar_arrive(&sh.xmax_bar[t][slot]);
            if (!(ok = wait(&sh.xmax_bar[t][slot], xm_phase[slot]))) break;
            xm_phase[slot] ^= 1;
            mx = fmaxf(mx, sh.xmax[t][slot][hf ^ 1][row]);
            ++xn;
          }
          mx *= sl2;
          const float m_new = fmaxf(m, mx);
          const bool grow = m_new > m + 8.f;  // also true for the first visible key
          const bool need = grow && n > 0 && m != -INFINITY;
          if (__any_sync(0xffffffffu, need)) {  // rescale this half's output columns
            const float alpha = need ? ex2(m - m_new) : 1.f;
#pragma unroll
            for (int c = 0; c < DH / 64; ++c) {
              uint32_t r[32];
              tmem_ld32(tO + hf * (DH / 2) + c * 32, r);
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
              tmem_st32(tO + hf * (DH / 2) + c * 32, r);
            }
            if (need) l *= alpha;
          }
          if (grow) m = m_new;
          const float mref = (m == -INFINITY) ? 0.f : m;
          // pass 2: P = 2^(S*scale*log2e - m) as bf16 pairs into S columns [32 + c0/2, +32),
          // inside this half's own S columns; both chunks are in registers before any P is
          // written.
          const uint64_t nm2 = f2(-mref, -mref);
          uint64_t l2 = f2(0.f, 0.f);
          uint32_t rr[2][32];
          tmem_ld32_nowait(tS + c0, rr[0]);
          tmem_ld32_nowait(tS + c0 + 32, rr[1]);
          tmem_wait_ld();
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            const int cs = c0 + 32 * ch;
            uint32_t (&r)[32] = rr[ch];
            uint32_t pk[16];
            if (WIN && !some[ch]) {
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[i] = 0;
              tmem_st16(tS + 32 + c0 / 2 + 16 * ch, pk);
              continue;
            }
            // staged: every FMA, then every exponential (independent, so they issue back to
            // back), then packing and two partial sums
            uint64_t xv[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              xv[i] = fma2(f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), sl2x2, nm2);
            float ev[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 e = f2_split(xv[i]);
              ev[2 * i] = ex2(e.x);
              ev[2 * i + 1] = ex2(e.y);
            }
            if (WIN ? !all[ch] : !full) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (WIN ? !((vis[ch] >> i) & 1u) : cs + i >= cnt) ev[i] = 0.f;
            }
            uint64_t la = f2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t p2 = f2(ev[2 * i], ev[2 * i + 1]);
              if (i & 1) la = add2(la, p2); else l2 = add2(l2, p2);
              pk[i] = bf16x2_of(p2);
            }
            l2 = add2(l2, la);
            tmem_st16(tS + 32 + c0 / 2 + 16 * ch, pk);
          }
          {
            const float2 ls = f2_split(l2);
            l += ls.x + ls.y;
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&sh.p_full[t]);
        }
      }
      if (!ok) break;
      // epilogue: both halves' sums, out = O / l for this half's columns, lse
      sh.xl[t][hf][row] = l;
      mbar_arrive(&sh.xl_bar[t]);
      if (!wait(&sh.xl_bar[t], xl_phase)) break;
      xl_phase ^= 1;
      l += sh.xl[t][hf ^ 1][row];
      if (!wait(&sh.o_done[t], od_phase)) break;
      od_phase ^= 1;
      tc_fence_after();
      const float inv_l = l > 0.f ? 1.f / l : 0.f;
      if constexpr (WIN) {
        orow_ptr = out + (static_cast<size_t>(item->row + t * kQTileRows + row) * P.hq + item->h) * DH;
        lse_ptr = lse + item->lse + t * kQTileRows + row;
      }
#pragma unroll
      for (int c = 0; c < DH / 64; ++c) {
        uint32_t r[32];
        tmem_ld32(tO + hf * (DH / 2) + c * 32, r);
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * inv_l;
        if (valid) store_row32<OutT>(orow_ptr + hf * (DH / 2) + c * 32, v);
      }
      if (valid && hf == 0) *lse_ptr = l > 0.f ? (m + lg2(l)) * 0.69314718055994531f : -INFINITY;
      tc_fence_before();
      mbar_arrive(&sh.o_free[t]);
      if constexpr (WIN) mbar_arrive(&sh.item_empty[kq & 1]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// One CTA waits on a barrier nothing completes, with a bounded wait (failure-path test).
__global__ void wait_timeout_kernel(uint64_t timeout_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_wait(&bar, 0, &abort_flag, timeout_ns, &g_status_fwd);
  __syncthreads();
}

// exp2_poly2 on n values (test hook for its error bound).
__global__ void exp2_poly_kernel(const float* __restrict__ x, float* __restrict__ y, int n) {
  const int i = 2 * (blockIdx.x * blockDim.x + threadIdx.x);
  if (i >= n) return;
  const float x1 = i + 1 < n ? x[i + 1] : 0.f;
  const float2 r = f2_split(exp2_poly2(f2(x[i], x1)));
  y[i] = r.x;
  if (i + 1 < n) y[i + 1] = r.y;
}

template <int DH, typename OutT, bool WIN>
cudaError_t launch_one(const Plan& P, const CUtensorMap& mq, const CUtensorMap& mk,
                       const CUtensorMap& mv, OutT* out, float* lse, int n_sm, cudaStream_t st) {
  using C = FwdCfg<DH>;
  auto kern = ring_fwd_tc_kernel<DH, OutT, WIN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int grid = P.n_items < n_sm ? P.n_items : n_sm;
  kern<<<grid, kFwdThreads, C::kSmemBytes, st>>>(mq, mk, mv, P, out, lse);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fwd_tc(const Plan& P, const void* q, const void* k, const void* v, void* out,
                          float* lse, cudaStream_t st) {
  if (P.n_items == 0) return cudaSuccess;
  CUtensorMap mq, mk, mv;
  cudaError_t e = make_token_tmap(&mq, q, P.n_rows, P.hq, P.head_dim);
  if (e == cudaSuccess) e = make_token_tmap(&mk, k, P.n_rows, P.hkv, P.head_dim);
  if (e == cudaSuccess) e = make_token_tmap(&mv, v, P.n_rows, P.hkv, P.head_dim);
  if (e != cudaSuccess) return e;
  int dev = 0, n_sm = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  using B = __nv_bfloat16;
  if (P.window > 0) {  // (block outputs, the float32 ones, have no window)
    B* o = static_cast<B*>(out);
    return P.head_dim == 128 ? launch_one<128, B, true>(P, mq, mk, mv, o, lse, n_sm, st)
                             : launch_one<64, B, true>(P, mq, mk, mv, o, lse, n_sm, st);
  }
  if (P.out_f32) {
    float* o = static_cast<float*>(out);
    return P.head_dim == 128 ? launch_one<128, float, false>(P, mq, mk, mv, o, lse, n_sm, st)
                             : launch_one<64, float, false>(P, mq, mk, mv, o, lse, n_sm, st);
  }
  B* o = static_cast<B*>(out);
  return P.head_dim == 128 ? launch_one<128, B, false>(P, mq, mk, mv, o, lse, n_sm, st)
                           : launch_one<64, B, false>(P, mq, mk, mv, o, lse, n_sm, st);
}

cudaError_t launch_exp2_poly(const float* x, float* y, int n, cudaStream_t st) {
  const int pairs = (n + 1) / 2;
  exp2_poly_kernel<<<(pairs + 255) / 256, 256, 0, st>>>(x, y, n);
  return cudaGetLastError();
}

cudaError_t launch_wait_timeout(uint64_t timeout_ns, cudaStream_t st) {
  wait_timeout_kernel<<<1, 32, 0, st>>>(timeout_ns);
  return cudaGetLastError();
}

cudaError_t fwd_status(unsigned int* value, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_status_fwd, sizeof(unsigned int));
  if (e == cudaSuccess && reset) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_status_fwd, &zero, sizeof(unsigned int));
  }
  return e;
}

}  // namespace ra
