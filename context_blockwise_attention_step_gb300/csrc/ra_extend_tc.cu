// ra_extend_tc.cu — attention of the new tokens of many sequences over a paged cache, bf16, on the
// 5th-generation tensor cores.
//
// A persistent CTA walks the pieces of its share (ra_extend.h): up to 256 rows, the new tokens of a
// sequence, or of all sequences of a group for the prefix that they share, times the query heads of
// a K/V head, against tiles of 128 keys.
//
//   S = Q K^T          tcgen05.mma; the rows of Q, (token, head) with the heads of a group next to
//                      each other, come by TMA, those of K and V page by page, in boxes of as many
//                      keys as divide a page and a tile
//   online softmax     a thread a row, whose 128 scores it holds in registers from one read of TMEM on; O
//                      rescaled only when a row's maximum grows by more than 2^8, as in the ring's
//                      forward; P = 2^(S scale log2 e - m) as bf16 into TMEM
//   O += P V           A = P from TMEM, V from shared memory
//
// Two teams of softmax warps, each with a score tile and an accumulator in TMEM, keep the tensor core
// busy in turn. A block of more than 128 rows gives each team its own query tile and both every key
// tile; of one of at most 128 rows the teams take the even and the odd key tiles, and join their sums
// in the end. So a block of few rows, whose time is its keys' bytes, has two tiles in flight too.
// A piece's result is final (out and lse), or a part for the join (ra_extend.cu): of a block that is
// cut between CTAs, or of a row that has a prefix's part as well.
//
// Keys that no row of a block sees are not read, and their values in a tile are made 0 before the
// product (what lies in a page behind a sequence's end may be NaN); their scores are masked.
//
// P enters its product as one bf16 number, as in the ring's forward: the weights' errors, of up to 2^-8 each, partly
// average out over the keys, and `out` is 0.0023 from the definition in relative L2, of which its own rounding is
// 0.0017. Where the rows are few and the keys' bytes count, P goes in as two bf16 numbers (2^-16; a second product
// with the same V), so that a step that is given shared prefixes is as exact as one that reads each sequence
// apart with the kernel for few rows or the decode attention: in decoding steps, for sequences of at most 16 rows a K/V
// head, and, in calls of no more than that a sequence on average, for prefixes of whose rows at least half are
// of such sequences. (64 sequences' last tokens behind 32768 shared keys 38 us with one number, 48 with two. For
// prefixes of many rows, which the products bound, one number: 16 questions of up to 300 tokens behind 16384, 8/8 heads
// of 64, 184 us, and 274 with two.)
//
// What bounds it: a chunk of 4096 tokens behind 28672 others, 32/8 heads of 128, 1347 us, 1.53 PFLOP/s, 0.81
// of the measured burst rate; the tensor pipe is active 66 % of the time, the softmax warps issue in 37 %
// of the cycles, and neither hides the hand-over of S and P between them. 16 questions of up to 500
// tokens behind 16384: 855 us, 0.75 (they leave half tiles). Where rows are few, a tile's latency counts: 64
// sequences' last tokens behind 32768 shared keys 48 us for 135 MB, 14 tiles a CTA and 10 us of start and end.
//
// Warp roles (384 threads, so that a thread may have 168 registers): 0 = TMA of Q and K (a lane a box), 3 =
// TMA of V, 1 = TMEM and MMA, 2 = the walk over the pieces, four ahead of the others, 4-7 and 8-11 = the
// softmax teams.
#include <type_traits>

#include "ra_extend.cuh"
#include "ra_window.cuh"

namespace ra {

static __device__ unsigned int g_status_tc[2];  // a wait that ran out; an index outside the cache

namespace {

constexpr int kThreads = 384;
constexpr int kSubBytes = 128 * 128;  // 128 rows x 64 bf16: one 128B-swizzled sub-tile
constexpr int kItems = 4;             // slots of the queue of pieces

template <int DH>
struct Cfg {
  static constexpr int kStages = DH == 128 ? 2 : 4;
  static constexpr int kSub = DH / 64;
  static constexpr int kTileBytes = 128 * DH * 2;
  static constexpr int kOffK = 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kSmemBytes = kOffV + kStages * kTileBytes + 1024;
  static constexpr int kKSteps = DH / 16;
  static constexpr uint32_t kTmemCols = 512;
  // TMEM columns: S0 | S1 | O0 | O1 (P of team t overwrites the first 64 columns of S_t, its second
  // numbers the others)
  __device__ static constexpr uint32_t col_s(int t) { return t ? 128u : 0u; }
  __device__ static constexpr uint32_t col_rest(int t) { return col_s(t) + 64u; }
  __device__ static constexpr uint32_t col_o(int t) { return t ? 256u + DH : 256u; }
};

struct Shared {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_part[2], p_full[2], o_done[2], o_free;  // p_part: three quarters of P
  uint64_t drain, sums_bar;
  uint64_t item_full[kItems], item_empty[kItems];
  ExtItem item[kItems];  // tiles 0: the end
  uint32_t tmem_base;
  int abort_flag;
  float sum[2][2][128], max[2][2][128];  // [item parity][team][row]: the rows' states, for the other team
};

__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
  return x != 0;
}

// What of key tile `tile` a block sees: keys [0, sinks) and [from, to) of the tile.
struct TileKeys {
  int sinks, from, to;
  __device__ __forceinline__ bool whole() const { return from <= sinks && to == 128; }
};
__device__ __forceinline__ TileKeys tile_keys(const ExtArgs& A, const ExtItem& it, int j) {
  const int tile = ext_tile(it.walk, j), k0 = tile * 128;
  TileKeys t;
  t.sinks = A.sh[kExtMany].window > 0 && tile == 0 ? min(A.sh[kExtMany].sinks, it.end) : 0;
  t.from = j < it.walk.ns ? 128 : max(0, it.low - k0);
  t.to = j < it.walk.ns ? 128 : min(128, it.end - k0);
  if (j < it.walk.ns) t.to = t.from = t.sinks;  // sinks only
  return t;
}

__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32(addr, r);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void store_cols(__nv_bfloat16* dst, const float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    reinterpret_cast<uint4*>(dst)[q] =
        make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                   pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
}
__device__ __forceinline__ void store_cols(float* dst, const float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) st_global_v8(dst + 8 * q, v + 8 * q);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// The loads of one key tile by the producer warp: lane i takes the boxes i, i + 32, ...
struct Boxes {
  static constexpr int MAX = 4;  // boxes of a lane (boxes of one key: 128)
  int page[MAX], slot[MAX];
  unsigned on;  // bit b: this lane's b-th box is loaded
  int count;    // boxes of the whole warp
};
__device__ __forceinline__ Boxes boxes_of(const ExtArgs& A, const ExtItem& it, int j, int lane) {
  const TileKeys t = tile_keys(A, it, j);
  const int k0 = ext_tile(it.walk, j) * 128, rows = A.box_rows, n = 128 / rows;
  Boxes b;
  b.on = 0;
  int mine = 0;
#pragma unroll
  for (int i = 0; i < Boxes::MAX; ++i) {
    const int box = lane + 32 * i, a = box * rows;
    b.page[i] = b.slot[i] = 0;
    if (box < n && (a < t.sinks || (a < t.to && a + rows > t.from))) {
      const int key = k0 + a, page = key / A.page_size;
      b.page[i] = ext_page(A, it.seq, page, g_status_tc + 1);
      b.slot[i] = key - page * A.page_size;
      b.on |= 1u << i;
      ++mine;
    }
  }
  b.count = __reduce_add_sync(0xffffffffu, mine);
  return b;
}
template <int DH>
__device__ __forceinline__ void load_boxes(const ExtArgs& A, const Boxes& b, const CUtensorMap* map, uint64_t* bar,
                                           uint8_t* dst, int hk, int lane) {
  const int rows = A.box_rows;
  if (lane == 0) mbar_expect_tx(bar, b.count * rows * DH * 2);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < Boxes::MAX; ++i) {
    if (!((b.on >> i) & 1u)) continue;
    int c[3];
#pragma unroll
    for (int d = 0; d < 3; ++d) c[d] = A.ord[0] == d ? hk : A.ord[1] == d ? b.slot[i] : b.page[i];
#pragma unroll
    for (int d = 0; d < DH / 64; ++d)
      tma_load_4d(dst + d * kSubBytes + (lane + 32 * i) * rows * 128, map, bar, d * 64, c[0], c[1], c[2]);
  }
}

// FINE: some pieces may want weights of two numbers. (This form is slower on pieces that do not: 16 questions of up to 500
// tokens behind 16384 keys, 32/8 heads of 128, 909 us and 925, 8/8 heads of 64 behind 32768 420 and 456.)
template <int DH, bool FINE>
__global__ void __launch_bounds__(kThreads, 1)
    extend_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ ExtArgs A) {
  using C = Cfg<DH>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (the same in a warp's lanes)
  volatile int* abort_flag = &sh.abort_flag;
  if (A.few_rows > 0) {  // the plan is there: a CTA without work has nothing to set up
    launch_dependents();
    if (!ext_acquire(A.head, A.timeout_ns, g_status_tc) ||
        A.starts[kExtMany][blockIdx.x].u0 == A.starts[kExtMany][blockIdx.x + 1].u0) {
      wait_for_previous();
      return;
    }
  }
  unsigned int* status = g_status_tc;
  const uint64_t tmo = A.timeout_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_part[i], 128);
      mbar_init(&sh.p_full[i], 128);
      mbar_init(&sh.o_done[i], 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_empty[i], 1);
    }
    mbar_init(&sh.o_free, 256);
    mbar_init(&sh.sums_bar, 256);
    mbar_init(&sh.drain, 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sh.item_full[i], 1);
      mbar_init(&sh.item_empty[i], 3 + 256);  // producers, MMA thread, softmax threads
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
  if (A.few_rows == 0) {
    wait_for_previous();
    launch_dependents();
  }
  const uint32_t tmem = sh.tmem_base;

  if (warp == 2) {
    // ------------------------------------------------------------------ the walk
    ExtCursor<kExtMany> cur;
    bool more = cur.begin(A, blockIdx.x);
    for (int kq = 0;; ++kq) {
      const int slot = kq % kItems;
      const bool ok = mbar_wait(&sh.item_empty[slot], ((kq / kItems) & 1) ^ 1, abort_flag, tmo, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      ExtItem it;
      it.tiles = 0;
      if (more) more = cur.next(A, it);
      if (!more) it.tiles = 0;
      if (lane == 0) {
        sh.item[slot] = it;
        mbar_arrive(&sh.item_full[slot]);
      }
      if (!more) break;
    }
  } else if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------------ TMA producers: Q and K, V
    int kv = 0, qt = 0;  // key tiles and query tiles so far
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, tmo, status));
    };
    bool ok = true;
    for (int kq = 0; ok; ++kq) {
      const int slot = kq % kItems;
      if (!wait(&sh.item_full[slot], (kq / kItems) & 1)) break;
      const ExtItem it = sh.item[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_empty[slot]);
      if (it.tiles == 0) break;
      for (int t = 0; warp == 0 && t < (it.two ? 2 : 1) && ok; ++t, ++qt) {
        const int qs = qt & 1;
        if (!(ok = wait(&sh.q_empty[qs], ((qt >> 1) & 1) ^ 1))) break;
        if (lane == 0) {
          mbar_expect_tx(&sh.q_full[qs], A.sh[kExtMany].half * A.hb * DH * 2);
          for (int d = 0; d < C::kSub; ++d)
            tma_load_4d(smem + qs * C::kTileBytes + d * kSubBytes, &tmQ, &sh.q_full[qs], d * 64, it.g0, it.hk,
                        it.tok0 + t * A.sh[kExtMany].half);
        }
      }
      if (!ok) break;
      uint64_t* full = warp == 0 ? sh.k_full : sh.v_full;
      uint64_t* empty = warp == 0 ? sh.k_empty : sh.v_empty;
      const CUtensorMap* map = warp == 0 ? &tmK : &tmV;
      uint8_t* ring = smem + (warp == 0 ? C::kOffK : C::kOffV);
      for (int j = it.j0; j < it.j0 + it.tiles; ++j, ++kv) {
        const Boxes b = boxes_of(A, it, j, lane);
        const int st = kv % C::kStages;
        if (!(ok = wait(&empty[st], ((kv / C::kStages) & 1) ^ 1))) break;
        load_boxes<DH>(A, b, map, &full[st], ring + st * C::kTileBytes, it.hk, lane);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    // The whole warp walks, with values that are the same in all lanes (they stay in uniform registers,
    // where the products want their descriptors), and one lane issues.
    const bool leader = elect_one();
    int kv = 0, qt = 0;
    uint32_t p_phase[2] = {0, 0}, of_phase = 0;
    const uint32_t idS = idesc_bf16_f32(128, 128, 0, 0);
    const uint32_t idO = idesc_bf16_f32(128, DH, 0, 1);
    const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dQ = sdesc_sw128(smem_u32(smem), 16, 1024), dK = sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024),
                   dV = sdesc_sw128(smem_u32(smem + C::kOffV), kSubBytes, 1024);
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, tmo, status));
    };
    bool ok = true;
    for (int kq = 0; ok; ++kq) {
      const int slot = kq % kItems;
      if (!(ok = wait(&sh.item_full[slot], (kq / kItems) & 1))) break;
      const int N = __shfl_sync(0xffffffffu, sh.item[slot].tiles, 0);
      const bool two = __shfl_sync(0xffffffffu, sh.item[slot].two, 0) != 0;
      const bool fine = FINE && __shfl_sync(0xffffffffu, sh.item[slot].fine, 0) != 0;
      if (leader) mbar_arrive(&sh.item_empty[slot]);
      if (N == 0) break;
      for (int t = 0; t < (two ? 2 : 1) && ok; ++t) ok = wait(&sh.q_full[(qt + t) & 1], ((qt + t) >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      auto products = [&](auto with_rest) {
        constexpr bool REST = decltype(with_rest)::value;
        // team t's k-th key tile is n; O_t(k-1) before S_t(k)
        const int count0 = two ? N : (N + 1) / 2, count1 = two ? N : N / 2;
        for (int k = 0; k <= count0 && ok; ++k) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int count = t ? count1 : count0;
            if (ok && k >= 1 && k - 1 < count) {
              const int n = two ? k - 1 : 2 * (k - 1) + t, c = kv + n, st = c % C::kStages;
              if (!two || t == 0) ok = wait(&sh.v_full[st], (c / C::kStages) & 1);
              ok = ok && wait(&sh.p_part[t], p_phase[t]);
              if (t == 0 && k == 1) {  // both accumulators have been read
                ok = ok && wait(&sh.o_free, of_phase ^ 1);
                of_phase ^= 1;
              }
              tc_fence_after();
              if (ok && leader) {
                const uint64_t dv = dV + st * (C::kTileBytes >> 4);
#pragma unroll
                for (int s = 0; s < 6; ++s)
                  mma_ts(base + C::col_o(t), base + C::col_s(t) + 8 * s, dv + s * (2048 >> 4), idO,
                         (k > 1 || s > 0) ? 1u : 0u);
                if constexpr (REST) {
#pragma unroll
                  for (int s = 0; s < 6; ++s)
                    mma_ts(base + C::col_o(t), base + C::col_rest(t) + 8 * s, dv + s * (2048 >> 4), idO, 1u);
                }
              }
              ok = ok && wait(&sh.p_full[t], p_phase[t]);
              p_phase[t] ^= 1;
              tc_fence_after();
              if (ok && leader) {
                const uint64_t dv = dV + st * (C::kTileBytes >> 4);
#pragma unroll
                for (int s = 6; s < 8; ++s)
                  mma_ts(base + C::col_o(t), base + C::col_s(t) + 8 * s, dv + s * (2048 >> 4), idO, 1u);
                if constexpr (REST) {
#pragma unroll
                  for (int s = 6; s < 8; ++s)
                    mma_ts(base + C::col_o(t), base + C::col_rest(t) + 8 * s, dv + s * (2048 >> 4), idO, 1u);
                }
                if (k == count) tc_commit(&sh.o_done[t]);
                if (!two || t == 1) tc_commit(&sh.v_empty[st]);
              }
            }
            if (ok && k < count) {
              const int n = two ? k : 2 * k + t, c = kv + n, st = c % C::kStages;
              if (!two || t == 0) ok = wait(&sh.k_full[st], (c / C::kStages) & 1);
              tc_fence_after();
              if (ok && leader) {
                const int qs = (qt + (two ? t : 0)) & 1;
                const uint64_t dq = dQ + qs * (C::kTileBytes >> 4), dk = dK + st * (C::kTileBytes >> 4);
#pragma unroll
                for (int s = 0; s < C::kKSteps; ++s) {
                  const int off = ((s >> 2) * kSubBytes + (s & 3) * 32) >> 4;
                  mma_ss(base + C::col_s(t), dq + off, dk + off, idS, s > 0);
                }
                tc_commit(&sh.s_full[t]);
                if (!two || t == 1) tc_commit(&sh.k_empty[st]);
                if (two ? k == N - 1 : n == N - 1) tc_commit(&sh.q_empty[qs]);
              }
            }
          }
        }
      };
      if constexpr (FINE) {
        if (fine) products(std::true_type{}); else products(std::false_type{});
      } else {
        products(std::false_type{});
      }
      kv += N;
      qt += two ? 2 : 1;
    }
    // let every MMA issued so far finish before TMEM is released
    if (leader) {
      tc_commit(&sh.drain);
      mbar_wait(&sh.drain, 0, abort_flag, tmo, status);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax + epilogue
    const int t = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::col_s(t);
    const uint32_t tO = tmem + lane_off + C::col_o(t);
    const float sl2 = A.scale_log2;
    const uint64_t sl2x2 = f2(sl2, sl2);
    const int tok = row / A.hb, head = row - tok * A.hb;  // of a query tile
    uint32_t tiles = 0;  // of this team so far: the phase of S
    uint32_t od1_phase = 0;
    int kv = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, tmo, status));
    };
    for (int kq = 0;; ++kq) {
      const int slot = kq % kItems;
      if (!wait(&sh.item_full[slot], (kq / kItems) & 1)) break;
      const ExtItem& it = sh.item[slot];
      const int N = it.tiles;
      if (N == 0) break;
      const bool two = it.two != 0;
      const int count0 = two ? N : (N + 1) / 2, count1 = two ? N : N / 2, mine = t ? count1 : count0;
      const int tk = tok + (two && t ? A.sh[kExtMany].half : 0);  // token of the block
      const bool valid = tok < A.sh[kExtMany].half && tk < it.ntok && head < it.heads;
      const bool idle = !__any_sync(0xffffffffu, valid);
      // keys lo .. hi - 1, and the first `sinks`. What a row that is none is given does not matter (no
      // row of a product depends on another): it sees everything, so that it asks for no mask.
      const int hi = !valid ? 0x7fffffff : it.shared ? it.end : it.base + tk + 1;
      const int lo = valid && A.sh[kExtMany].window > 0 ? max(0, hi - A.sh[kExtMany].window) : 0;
      // tiles full_from .. full_to - 1 are seen whole by every row of the warp
      const int full_from = (__reduce_max_sync(0xffffffffu, lo) + 127) >> 7, full_to = __reduce_min_sync(0xffffffffu, hi) >> 7;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int k = 0; k < mine; ++k) {
        const int n = two ? k : 2 * k + t, j = it.j0 + n, tile = ext_tile(it.walk, j), k0 = tile * 128;
        if (!(ok = wait(&sh.s_full[t], tiles & 1))) break;
        tc_fence_after();
        ++tiles;
        // values of keys that no row of the block sees: 0 (the other team's product with this tile
        // comes after this one's)
        if ((!two || t == 0) && (k0 < it.low || it.end - k0 < 128)) {
          const TileKeys seen = tile_keys(A, it, j);
          if (!seen.whole()) {
            const int c = kv + n, st = c % C::kStages;
            if (!(ok = wait(&sh.v_full[st], (c / C::kStages) & 1))) break;
            uint8_t* v = smem + C::kOffV + st * C::kTileBytes;
            if (row >= seen.sinks && (row < seen.from || row >= seen.to)) {
#pragma unroll
              for (int i = 0; i < DH / 8; ++i)  // 16-byte pieces of the row
                *reinterpret_cast<uint4*>(v + (i / 8) * kSubBytes + row * 128 + (i % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
        }
        uint64_t sum = f2(0.f, 0.f);
        if (!idle) {  // (the products of a warp without rows are not looked at)
          const bool full = tile >= full_from && tile < full_to;  // no mask needed
          uint32_t r[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_nowait(tS + 32 * c, r[c]);
          tmem_wait_ld();
          if (!full) {
            const int cnt = min(max(hi - k0, 0), 128), sk_t = A.sh[kExtMany].window > 0 && k0 == 0 ? A.sh[kExtMany].sinks : 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t vis = visible_bits(32 * c, cnt, lo - k0, sk_t);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((vis >> i) & 1u)) r[c][i] = 0xff800000u;  // -inf
            }
          }
          float mx;
          {  // independent chains (one chain of dependent max operations is slow)
            float mq[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              uint32_t (&v)[32] = r[q >> 1];
              const int i0 = (q & 1) * 16;
              mq[q] = fmaxf(__uint_as_float(v[i0]), __uint_as_float(v[i0 + 1]));
#pragma unroll
              for (int i = 2; i < 16; i += 2) mq[q] = max3(mq[q], __uint_as_float(v[i0 + i]), __uint_as_float(v[i0 + i + 1]));
            }
            mx = max3(max3(mq[0], mq[1], mq[2]), max3(mq[3], mq[4], mq[5]), fmaxf(mq[6], mq[7]));
          }
          mx *= sl2;
          const float m_new = fmaxf(m, mx);
          const bool grow = m_new > m + 8.f;  // also true for the first visible key
          const bool need = grow && k > 0 && m != -INFINITY;
          if (__any_sync(0xffffffffu, need)) {  // rescale the output so far
            const float alpha = need ? ex2(m - m_new) : 1.f;
#pragma unroll
            for (int c = 0; c < DH / 8; ++c) {  // (in pieces that leave the scores their registers)
              uint32_t o[8];
              tmem_ld8(tO + c * 8, o);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st8(tO + c * 8, o);
            }
            if (need) l *= alpha;
          }
          if (grow) m = m_new;
          const float mref = (m == -INFINITY) ? 0.f : m;
          // P = 2^(S*scale*log2e - m) as bf16 pairs over the first columns of S, 32 keys at a time: every FMA, then
          // every exponential, then packing and the sums
          const uint64_t nm2 = f2(-mref, -mref);
          uint64_t la = f2(0.f, 0.f), lb = f2(0.f, 0.f);
          auto weights = [&](auto with_rest) {
            constexpr bool REST = decltype(with_rest)::value;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint64_t xv[16];
#pragma unroll
              for (int i = 0; i < 16; ++i)
                xv[i] = fma2(f2(__uint_as_float(r[c][2 * i]), __uint_as_float(r[c][2 * i + 1])), sl2x2, nm2);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 e = f2_split(xv[i]);
                xv[i] = f2(ex2(e.x), ex2(e.y));
              }
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                if (i & 1) la = add2(la, xv[i]); else lb = add2(lb, xv[i]);
                pk[i] = bf16x2_of(xv[i]);
              }
              tmem_st16(tS + 16 * c, pk);
              if constexpr (REST) {  // what the rounding left
#pragma unroll
                for (int i = 0; i < 16; ++i) pk[i] = bf16x2_of(sub2(xv[i], f2_of_bf16x2(pk[i])));
                tmem_st16(tS + 64 + 16 * c, pk);
              }
              if (c == 2) {  // the product with these keys may begin (2 % of the whole)
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&sh.p_part[t]);
              }
            }
          };
          if constexpr (FINE) {
            if (it.fine) weights(std::true_type{}); else weights(std::false_type{});
          } else {
            weights(std::false_type{});
          }
          sum = add2(la, lb);
        } else {
          mbar_arrive(&sh.p_part[t]);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sh.p_full[t]);
        const float2 s2 = f2_split(sum);
        l += s2.x + s2.y;
      }
      if (!ok) break;
      kv += N;
      // epilogue: the rows' sums and maxima to everyone
      const int par = kq & 1;
      sh.sum[par][t][row] = l;
      sh.max[par][t][row] = m;
      mbar_arrive(&sh.sums_bar);
      if (!wait(&sh.sums_bar, par)) break;
      if (!wait(&sh.o_done[0], par)) break;
      if (count1 > 0) {
        if (!wait(&sh.o_done[1], od1_phase)) break;
        od1_phase ^= 1;
      }
      tc_fence_after();
      float M, L, f0 = 1.f, f1 = 0.f;
      if (two) {
        M = m;
        L = l;
      } else {
        const float m0 = sh.max[par][0][row], m1 = sh.max[par][1][row];
        M = fmaxf(m0, m1);
        const float ref = M == -INFINITY ? 0.f : M;
        f0 = ex2(m0 - ref);
        f1 = ex2(m1 - ref);
        L = f0 * sh.sum[par][0][row] + f1 * sh.sum[par][1][row];
      }
      const int dest = it.dest;
      const int64_t at = static_cast<int64_t>(it.tok0 + tk) * A.hq + it.hk * A.group + it.g0 + head;  // (token, head)
      const float inv = dest != kExtFinal ? 1.f : L > 0.f ? 1.f / L : 0.f;
      const int64_t to = dest == kExtFinal ? at
                         : dest == kExtRows ? static_cast<int64_t>(it.slot) * A.n_tokens * A.hq + at
                                            : static_cast<int64_t>(it.slot) * A.part[kExtMany].rows + tk * A.hb + head;
      float* fo = (dest == kExtRows ? A.row_o : A.part[kExtMany].o) + to * DH;
      __nv_bfloat16* bo = static_cast<__nv_bfloat16*>(A.out) + to * DH;
      const bool lead = two || t == 0;
      if (valid && lead) {
        if (dest == kExtFinal) A.lse[at] = L > 0.f ? (M + lg2(L)) * 0.69314718055994531f : -INFINITY;
        else (dest == kExtRows ? A.row_ml : A.part[kExtMany].ml)[to] = make_float2(M, L);
      }
      if (two) {
#pragma unroll
        for (int c = 0; c < DH / 32; ++c) {
          const int col = c * 32;
          float v[32];
          tmem_ld_cols(tO + col, v);
          if (valid) {
            if (dest == kExtFinal) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] *= inv;
              store_cols(bo + col, v);
            } else {
              store_cols(fo + col, v);
            }
          }
        }
      } else {
        // half the columns each
#pragma unroll
        for (int c = 0; c < DH / 64; ++c) {
          const int col = t * (DH / 2) + c * 32;
          float v[32];
          tmem_ld_cols(tmem + lane_off + C::col_o(0) + col, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= f0;
          if (count1 > 0) {
            float u[32];
            tmem_ld_cols(tmem + lane_off + C::col_o(1) + col, u);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += f1 * u[i];
          }
          if (valid) {
            if (dest == kExtFinal) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] *= inv;
              store_cols(bo + col, v);
            } else {
              store_cols(fo + col, v);
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&sh.o_free);
      mbar_arrive(&sh.item_empty[slot]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  wait_for_previous();  // what follows in the stream waits for this kernel alone
}

template <int DH, bool FINE>
cudaError_t launch(const ExtArgs& A, const ExtMaps& maps, cudaStream_t st) {
  using C = Cfg<DH>;
  auto kernel = extend_tc_kernel<DH, FINE>;
  static std::atomic<bool> done[kExtDevices];
  const cudaError_t e = ext_allow_smem(kernel, C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(A.part[kExtMany].most_ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps.q, maps.k, maps.v, A);
}

}  // namespace

// The map of q is [tokens, K/V heads, heads of a group, dh], of the pages [page, slot, head, dh] with
// the three outer dimensions in the order of their strides; a page's keys come in boxes of the largest
// power of two that divides it, at most a tile.
cudaError_t make_extend_maps(ExtMaps* maps, const ra_paged_cache* c, ExtArgs* A) {
  const uint64_t dh = A->dh, row = dh * 2;
  {
    const uint64_t dims[4] = {dh, static_cast<uint64_t>(A->group), static_cast<uint64_t>(A->hkv),
                              static_cast<uint64_t>(A->n_tokens)};
    const uint64_t strides[3] = {row, row * A->group, row * A->hq};
    const uint32_t box[4] = {64, static_cast<uint32_t>(A->hb), 1, static_cast<uint32_t>(A->sh[kExtMany].half)};
    const cudaError_t e = make_tmap_bf16(&maps->q, A->q, 4, dims, strides, box);
    if (e != cudaSuccess) return e;
  }
  const int low = c->page_size & -c->page_size;
  A->box_rows = low < 128 ? low : 128;
  struct Dim {
    uint64_t size, stride;
    int which;
  } d[3] = {{static_cast<uint64_t>(c->hkv), static_cast<uint64_t>(c->head_stride) * 2, 0},
            {static_cast<uint64_t>(c->page_size), static_cast<uint64_t>(c->slot_stride) * 2, 1},
            {static_cast<uint64_t>(c->n_pages), static_cast<uint64_t>(c->page_stride) * 2, 2}};
  for (Dim& x : d)
    if (x.size == 1) x.stride = row;  // never stepped over
  for (int i = 1; i < 3; ++i)
    for (int j = i; j > 0 && d[j].stride < d[j - 1].stride; --j) {
      const Dim x = d[j];
      d[j] = d[j - 1];
      d[j - 1] = x;
    }
  const uint64_t dims[4] = {dh, d[0].size, d[1].size, d[2].size};
  const uint64_t strides[3] = {d[0].stride, d[1].stride, d[2].stride};
  uint32_t box[4] = {64, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    A->ord[d[i].which] = i;
    if (d[i].which == 1) box[i + 1] = A->box_rows;
  }
  cudaError_t e = make_tmap_bf16(&maps->k, c->k_pages, 4, dims, strides, box);
  if (e == cudaSuccess) e = make_tmap_bf16(&maps->v, c->v_pages, 4, dims, strides, box);
  return e;
}

cudaError_t extend_tc_status(unsigned int value[2], bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_status_tc, sizeof g_status_tc);
  if (e == cudaSuccess && reset) {
    const unsigned int zero[2] = {0, 0};
    e = cudaMemcpyToSymbol(g_status_tc, zero, sizeof zero);
  }
  return e;
}

cudaError_t launch_extend_tc(const ExtArgs& A, const ExtMaps& maps, cudaStream_t st) {
  const bool fine = A.cu_new == nullptr || static_cast<int64_t>(A.n_tokens) * A.group <= static_cast<int64_t>(kExtFewRows) * A.n_seqs;
  if (A.dh == 128) return fine ? launch<128, true>(A, maps, st) : launch<128, false>(A, maps, st);
  return fine ? launch<64, true>(A, maps, st) : launch<64, false>(A, maps, st);
}

}  // namespace ra
