// ra_extend.cuh — what the kernels of ra_extend.cu and ra_extend_tc.cu share: the call's arguments,
// a CTA's walk over its share of the work, and where the parts of a cut block go.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "ra_extend.h"
#include "ra_internal.h"
#include "ra_ptx.cuh"

namespace ra {

constexpr int kExtSms = 152;
constexpr int kExtDevices = 64;  // whose properties and kernel attributes are looked up and set once

// What the planning kernel finds out, at the beginning of the workspace; the segments follow.
struct ExtHead {
  int64_t units[2];
  int32_t ctas[2], segs, own_blocks;
  uint32_t ready;  // set when the rest and the segments are there
};

// The kernels of a call and what they wait for. The planning kernel comes first. The kernel for few rows
// waits for its end, and only then lets the one for many rows start, which has the plan too, then, and
// need not wait for the other to end: it takes the SMs that the other leaves free. (The flag that it
// reads first orders its reads of the plan behind the plan's writes.) It ends after the other has
// ended, so that the join, which waits for its end, has both kernels' results. A kernel that is alone
// waits for the plan. So the plan is there when the join may start, too: it finds its blocks' parts while
// the last CTAs still work.
__device__ __forceinline__ void ext_publish(ExtHead* h) {
  __threadfence();
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(&h->ready), "r"(1u) : "memory");
}
// False if the plan does not come (the wait has a limit).
__device__ __forceinline__ bool ext_acquire(const ExtHead* h, uint64_t timeout_ns, unsigned int* status) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    uint32_t ready;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(ready) : "l"(&h->ready) : "memory");
    if (ready == 1u) return true;
    if (globaltimer_ns() - t0 > timeout_ns) {
      atomicOr(status, 1u);
      return false;
    }
  }
}
// The parts of the blocks of a class that are cut between CTAs: [CTA][2][rows], and [dh].
struct ExtParts {
  float* o;    // sums, not divided by l
  float2* ml;  // running max (log2), denominator
  int32_t rows, most_ctas;
};

struct ExtArgs {
  const void* q;
  const void* k_pages;
  const void* v_pages;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu_new;       // null: one new token of every sequence
  const int32_t* cu_groups;
  const int32_t* prefix_lens;
  int64_t table_stride, page_stride, slot_stride, head_stride;
  int32_t n_seqs, n_groups, n_tokens, max_pages, page_size, n_pages;
  int32_t hq, hkv, group, dh;
  int32_t hb, blocks_per_kv;   // query heads of a block (the last one may have fewer), blocks of a K/V head
  int32_t box_rows, ord[3];    // tensor-core kernel: keys of a copy; places of head, slot, page in the map
  ExtShape sh[2];              // of each class
  int32_t few_rows;            // most rows a K/V head of a segment of few rows; 0: that kernel does not run
  ExtParts part[2];
  float scale_log2;
  uint64_t timeout_ns;
  ExtHead* head;
  ExtSeg* segs;
  ExtStart* starts[2];         // of each class's most_ctas CTAs (u0 alone without work), and of one behind the last
  float* row_o;                // results like a part's, of whole blocks that are joined: [2][n_tokens][hq][dh]
  float2* row_ml;
  void* out;
  float* lse;
};

// Where a block's result goes.
enum : int { kExtFinal = 0, kExtPart = 1, kExtRows = 2 };

// A piece of a block: walk indexes j0 .. j0 + tiles - 1.
struct ExtItem {
  ExtWalk walk;
  int32_t tiles, j0;
  int32_t tok0, ntok, two;     // token row of the block's first row, tokens; more than `half`
  int32_t hk, g0, heads;       // K/V head, first query head of its group, heads
  int32_t base, shared;        // position of tok0; prefix: every row sees keys 0 .. end - 1
  int32_t fine;                // the weights as two bf16 numbers (tensor-core kernel)
  int32_t low, end;            // keys of the block: low .. end - 1, and with a window sinks
  int32_t seq, dest, slot;     // kExtPart: which part; kExtRows: 0 prefix, 1 own
};

// The walk of one warp over the pieces of a CTA's share (every lane holds the same state).
template <int CLS>
struct ExtCursor {
  int64_t u0, u1, base;
  ExtSeg g;
  int cta, seg, hk, hblk, blk, blocks;

  // False for a CTA without work.
  __device__ __forceinline__ bool begin(const ExtArgs& A, int which) {
    const ExtStart s = A.starts[CLS][which];
    cta = which;
    u0 = s.u0;
    u1 = A.starts[CLS][which + 1].u0;
    if (u0 == u1) return false;
    base = s.base;
    seg = s.seg;
    hk = s.hk;
    hblk = s.hblk;
    blk = s.blk;
    g = A.segs[seg];
    blocks = ext_blocks(A.sh[CLS], g.n);
    return true;
  }

  __device__ __forceinline__ bool next(const ExtArgs& A, ExtItem& it) {
    const ExtShape& sh = A.sh[CLS];
    while (base < u1) {
      const ExtWalk w = ext_walk(sh, g, blk);
      const int weight = ext_weight(sh, g, blk);
      const int j0 = ext_tile_from(sh, base, weight, w.count, u0);
      const int j1 = ext_tile_from(sh, base, weight, w.count, u1);
      if (j0 < j1) {
        const int a = blk * sh.bt;
        it.walk = w;
        it.j0 = j0;
        it.tiles = j1 - j0;
        it.tok0 = g.t0 + a;
        it.ntok = min(sh.bt, g.n - a);
        it.two = it.ntok > sh.half;
        it.hk = hk;
        it.g0 = hblk * A.hb;
        it.heads = min(A.hb, A.group - it.g0);
        it.shared = g.shared;
        it.fine = A.cu_new == nullptr || (g.shared ? g.shared == 2 : ext_few(g.n, A.group));
        it.base = g.base + a;
        it.low = g.shared ? 0 : static_cast<int>(ext_low(sh, g, blk));
        it.end = g.shared ? g.k1 : it.base + it.ntok;
        it.seq = g.seq;
        const bool whole = j0 == 0 && j1 == w.count, joined = g.shared || g.prefix >= 0;
        it.dest = !whole ? kExtPart : joined ? kExtRows : kExtFinal;
        it.slot = !whole ? cta * 2 + (j0 > 0 ? 0 : 1) : g.shared ? 0 : 1;
      }
      base += ext_units(sh, w.count, weight);
      if (++blk == blocks) {
        blk = 0;
        if (++hblk == A.blocks_per_kv) {
          hblk = 0;
          ++hk;
        }
        if (hk == A.hkv && base < u1) {
          hk = 0;
          do {  // (units are left, so there is one)
            g = A.segs[++seg];
          } while (g.units == 0 || g.cls != CLS);
          blocks = ext_blocks(sh, g.n);
        }
      }
      if (j0 < j1) return true;
    }
    return false;
  }
};

// Where page `page` of a sequence is (page 0 in place of one outside the cache, which is recorded).
__device__ __forceinline__ int ext_page(const ExtArgs& A, int seq, int page, unsigned int* status) {
  const int at = A.block_table[seq * A.table_stride + page];
  if (at >= 0 && at < A.n_pages) return at;
  atomicOr(status, 1u);
  return 0;
}

// Allows a kernel its dynamic shared memory, once on each device (`done`: a flag of the kernel's for each).
template <typename K>
cudaError_t ext_allow_smem(K kernel, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < kExtDevices && done[dev].load(std::memory_order_acquire))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < kExtDevices) done[dev].store(true, std::memory_order_release);
  return e;
}

// The tensor-core kernel: its tensor maps (they also fill in box_rows and ord), and its launch.
struct ExtMaps {
  CUtensorMap q, k, v;
};
cudaError_t make_extend_maps(ExtMaps* maps, const ra_paged_cache* c, ExtArgs* A);
cudaError_t launch_extend_tc(const ExtArgs& A, const ExtMaps& maps, cudaStream_t st);
cudaError_t extend_tc_status(unsigned int value[2], bool reset);  // as extend_status, of that kernel alone

// The kernel of the segments of few rows, bf16.
int extend_few_ctas(int head_dim);  // most CTAs
cudaError_t launch_extend_few(const ExtArgs& A, cudaStream_t st);
cudaError_t extend_few_status(unsigned int* value, bool reset);

}  // namespace ra
