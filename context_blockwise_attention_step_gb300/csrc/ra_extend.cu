// ra_extend.cu — attention of the new tokens of many sequences over a paged cache, with prefixes that
// groups of sequences share: the planning kernel, the float32 kernel, the join, and the call.
//
// Keys that many sequences share are read once for all of them: the rows of a group's sequences
// stand together in blocks against the prefix, and each sequence's rows against its own keys behind
// it. The two results of a row, and the parts of a block that is cut between CTAs, are joined by the
// log-sum-exp merge of the ring's blocks (nanotron how-to page, "Numerically-Stable Output Fusion"):
//
//   M = max m_i,  l = sum 2^(m_i - M) l_i,  out = sum 2^(m_i - M) o_i / l,  lse = (M + log2 l) ln 2
//
// Three launches, the second and the third while the one before still runs (programmatic dependent
// launch): the planning kernel reads the lengths and lists the segments (ra_extend.h); the main kernel
// (ra_extend_tc.cu for bf16) deals them out evenly to its CTAs; the join works on the blocks that need
// it. The host need not know a length.
#include <cuda_bf16.h>

#include <cmath>

#include "ra_extend.cuh"

namespace ra {

static __device__ unsigned int g_status_extend;  // an index outside the cache

namespace {

// ---------------------------------------------------------------- planning
constexpr int kPlanThreads = 1024;

struct Tokens {
  int t0, n, len;
  bool live, bad;  // has rows that see something; lengths that do not go together
};
__device__ __forceinline__ int bounded(int x, int hi) { return x < 0 ? 0 : x > hi ? hi : x; }
__device__ __forceinline__ Tokens tokens_of(const ExtArgs& A, int b) {
  Tokens t;
  t.bad = false;
  t.t0 = b;
  t.n = 1;
  if (A.cu_new != nullptr) {
    const int a = A.cu_new[b], e = A.cu_new[b + 1];
    t.t0 = bounded(a, A.n_tokens);
    t.n = bounded(e, A.n_tokens) - t.t0;
    if (t.n < 0) t.n = 0;
    t.bad = a != t.t0 || e != t.t0 + t.n;
  }
  t.len = A.seq_lens[b];
  const int64_t cap = static_cast<int64_t>(A.max_pages) * A.page_size;
  if (t.len < 0 || t.len > cap) {
    t.bad = true;
    t.len = t.len < 0 ? 0 : static_cast<int>(cap);
  }
  if (t.n > t.len && !(A.cu_new == nullptr && t.len == 0)) t.bad = t.bad || t.n > 0;
  t.live = t.n > 0 && t.n <= t.len;
  return t;
}

__global__ void __launch_bounds__(kPlanThreads) extend_plan(const __grid_constant__ ExtArgs A) {
  __shared__ int64_t scan_units[32];
  __shared__ int scan_blocks[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const ExtShape& s = A.sh;
  launch_dependents();
  // groups, a warp each: whether the prefix lies before every new token, and whether sharing it pays
  for (int g = warp; g < A.n_groups; g += 32) {
    const int b0 = bounded(A.cu_groups[g], A.n_seqs), b1 = bounded(A.cu_groups[g + 1], A.n_seqs);
    const int64_t cap = static_cast<int64_t>(A.max_pages) * A.page_size;
    int p = A.prefix_lens[g];
    if (p > cap) p = static_cast<int>(cap);
    const int tiles = p > 0 ? p >> s.shift : 0;
    int64_t apart = 0;
    int first = A.n_seqs, ok = 1;
    for (int b = b0 + lane; b < b1; b += 32) {
      const Tokens t = tokens_of(A, b);
      if (t.bad) ok = 0;
      if (!t.live) continue;
      if (t.len - t.n < tiles << s.shift) ok = 0;
      apart += ext_block_units(s, t.n);
      first = min(first, b);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) apart += __shfl_xor_sync(0xffffffffu, apart, o);
    first = __reduce_min_sync(0xffffffffu, first);
    ok = __reduce_min_sync(0xffffffffu, ok);
    if (lane == 0) {
      ExtSeg e = {};
      e.shared = 1;
      e.prefix = -1;
      e.k1 = tiles << s.shift;
      if (b0 < b1 && first < A.n_seqs && ok) {
        const Tokens a = tokens_of(A, b0), z = tokens_of(A, b1 - 1);
        const int n = z.t0 + z.n - a.t0;
        const int64_t together = ext_block_units(s, n);
        if (n > 0 && ext_worth_sharing(tiles, apart, together)) {
          e.t0 = a.t0;
          e.n = n;
          e.seq = first;
          e.units = together * tiles;
        }
      }
      A.segs[g] = e;
    }
  }
  __syncthreads();
  // all segments in order, a run of them for each thread
  const int segs = A.n_groups + A.n_seqs, pairs = A.hkv * A.blocks_per_kv;
  const int chunk = (segs + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(segs, tid * chunk), i1 = min(segs, i0 + chunk);
  int64_t units = 0;
  int blocks = 0;
  for (int i = i0; i < i1; ++i) {
    ExtSeg e = {};
    if (i < A.n_groups) {
      e = A.segs[i];
    } else {
      const int b = i - A.n_groups;
      const Tokens t = tokens_of(A, b);
      if (t.bad) atomicOr(&g_status_extend, 1u);
      e.t0 = t.t0;
      e.n = t.n;
      e.base = t.len - t.n;
      e.k1 = t.len;
      e.seq = b;
      e.prefix = -1;
      if (A.n_groups > 0 && t.live) {
        int lo = 0, hi = A.n_groups - 1;  // the last group that begins at b or before
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (A.cu_groups[mid] <= b) lo = mid; else hi = mid - 1;
        }
        if (A.cu_groups[lo] <= b && b < A.cu_groups[lo + 1] && A.segs[lo].units > 0) {
          e.prefix = lo;
          e.k0 = A.segs[lo].k1;
        }
      }
      if (t.live) e.units = ext_units_before(s, e, ext_blocks(s, t.n));
      e.blocks0 = blocks;
      blocks += ext_blocks(s, t.n);
    }
    e.unit0 = units;
    units += e.units * pairs;
    A.segs[i] = e;
  }
  int64_t x = units;
  int y = blocks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, x, o);
    const int c = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += a;
      y += c;
    }
  }
  if (lane == 31) {
    scan_units[warp] = x;
    scan_blocks[warp] = y;
  }
  __syncthreads();
  int64_t before = x - units, all = 0;
  int blocks_before = y - blocks, all_blocks = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) {
      before += scan_units[w];
      blocks_before += scan_blocks[w];
    }
    all += scan_units[w];
    all_blocks += scan_blocks[w];
  }
  for (int i = i0; i < i1; ++i) {
    A.segs[i].unit0 += before;
    A.segs[i].blocks0 += blocks_before;
  }
  if (tid == 0) {
    ExtHead h;
    h.units = all;
    h.ctas = ext_ctas(all, A.most_ctas, s.wide);
    h.segs = segs;
    h.own_blocks = all_blocks;
    h.pad = 0;
    *A.head = h;
  }
}

// ---------------------------------------------------------------- float32
// 64 rows against tiles of 64 keys on the CUDA cores, 256 threads: thread (y, x) works out the scores
// of rows 4y .. 4y+3 and keys x, x + 16, x + 32, x + 48, sixteen lanes have a row's scores, and of the
// result rows 4y .. and the columns 4x .. 4x+3, and 64 + 4x .. What bounds it: 2 dh FMAs a row and key
// and product; four FMAs a 16-byte word of shared memory.
constexpr int kSimtThreads = 256, kSimtRows = 64, kSimtKeys = 64;
__host__ __device__ constexpr int simt_pitch(int dh) { return (dh + 3) / 4 * 4 + 4; }
constexpr int simt_smem(int dh) {
  const int keys = kSimtKeys * simt_pitch(dh), weights = kSimtRows * (kSimtKeys + 4);
  return (kSimtRows * simt_pitch(dh) + (keys > weights ? keys : weights) + keys) * 4;
}

// COLS: groups of 64 columns of the head.
template <int COLS>
__global__ void __launch_bounds__(kSimtThreads, 2) extend_simt(const __grid_constant__ ExtArgs A, int vec) {
  extern __shared__ __align__(16) float sm[];
  __shared__ ExtItem sh_it;
  const int dh = A.dh, pitch = simt_pitch(dh), d4 = (dh + 3) / 4;
  float* sq = sm;                                 // [64][pitch], times scale * log2(e)
  float* sk = sm + kSimtRows * pitch;             // [64][pitch], then the weights [64][68]
  float* sv = sm + simt_smem(dh) / 4 - kSimtKeys * pitch;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, x = tid & 15, y = tid >> 4;
  launch_dependents();
  wait_for_previous();
  ExtCursor cur;
  bool more = false;
  if (warp == 0) more = cur.begin(A, blockIdx.x);
  while (true) {
    if (warp == 0) {
      ExtItem next;
      next.tiles = 0;
      if (more) more = cur.next(A, next);
      if (!more) next.tiles = 0;
      if (lane == 0) sh_it = next;
    }
    __syncthreads();
    const ExtItem it = sh_it;
    if (it.tiles == 0) break;
    const int rows = it.ntok * A.hb;
    // a row of 4 elements, of memory whose rows need not be aligned
    auto copy_row4 = [&](const float* src, float* dst, int d, bool on, float mul) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (on) {
        if (vec) {
          v = *reinterpret_cast<const float4*>(src + d);
        } else {
          v.x = src[d];
          if (d + 1 < dh) v.y = src[d + 1];
          if (d + 2 < dh) v.z = src[d + 2];
          if (d + 3 < dh) v.w = src[d + 3];
        }
      }
      *reinterpret_cast<float4*>(dst + d) = make_float4(v.x * mul, v.y * mul, v.z * mul, v.w * mul);
    };
    for (int i = tid; i < kSimtRows * d4; i += kSimtThreads) {
      const int r = i / d4, d = (i - r * d4) * 4, tok = r / A.hb, h = r - tok * A.hb;
      const bool on = r < rows && h < it.heads;
      const int64_t at = static_cast<int64_t>(it.tok0 + tok) * A.hq + it.hk * A.group + it.g0 + h;
      copy_row4(static_cast<const float*>(A.q) + (on ? at * dh : 0), sq + r * pitch, d, on, A.scale_log2);
    }
    int hi[4], lo[4];
    bool valid[4];
    float m[4], l[4], o[4][COLS][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * y + r, tok = row / A.hb;
      valid[r] = row < rows && row - tok * A.hb < it.heads;
      hi[r] = !valid[r] ? 0 : it.shared ? it.end : it.base + tok + 1;
      lo[r] = A.sh.window > 0 ? max(0, hi[r] - A.sh.window) : 0;
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < COLS; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][c][e] = 0.f;
    }
    const bool idle = 8 * warp >= rows;  // a warp without rows helps with the copies only
    for (int j = it.j0; j < it.j0 + it.tiles; ++j) {
      const int k0 = ext_tile(it.walk, j) * kSimtKeys;
      const int sinks = A.sh.window > 0 ? min(A.sh.sinks, it.end) : 0;
      // keys that some row sees; the rest of the tile is 0
      __syncthreads();  // the tile before has been read
      for (int r = warp; r < kSimtKeys; r += kSimtThreads / 32) {
        const int key = k0 + r;
        const bool on = key < sinks || (key >= it.low && key < it.end);
        int64_t at = 0;
        if (on) {
          const int page = key / A.page_size;
          at = ext_page(A, it.seq, page, &g_status_extend) * A.page_stride + static_cast<int64_t>(key - page * A.page_size) * A.slot_stride +
               it.hk * A.head_stride;
        }
        for (int d = lane; d < d4; d += 32) {
          copy_row4(static_cast<const float*>(A.k_pages) + at, sk + r * pitch, 4 * d, on, 1.f);
          copy_row4(static_cast<const float*>(A.v_pages) + at, sv + r * pitch, 4 * d, on, 1.f);
        }
      }
      __syncthreads();
      float s[4][4] = {};
      if (!idle) {
        for (int d = 0; d < d4; ++d) {
          float4 q[4], k[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) q[r] = *reinterpret_cast<const float4*>(sq + (4 * y + r) * pitch + 4 * d);
#pragma unroll
          for (int c = 0; c < 4; ++c) k[c] = *reinterpret_cast<const float4*>(sk + (x + 16 * c) * pitch + 4 * d);
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              s[r][c] += q[r].x * k[c].x;
              s[r][c] += q[r].y * k[c].y;
              s[r][c] += q[r].z * k[c].z;
              s[r][c] += q[r].w * k[c].w;
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float mx = m[r];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = k0 + x + 16 * c;
            if (!(key < hi[r] && (key >= lo[r] || key < A.sh.sinks))) s[r][c] = -INFINITY;
            mx = fmaxf(mx, s[r][c]);
          }
#pragma unroll
          for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          const float ref = mx == -INFINITY ? 0.f : mx, alpha = exp2f(m[r] - ref);
          float sum = 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            s[r][c] = exp2f(s[r][c] - ref);
            sum += s[r][c];
          }
#pragma unroll
          for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
          m[r] = mx;
          l[r] = l[r] * alpha + sum;
#pragma unroll
          for (int c = 0; c < COLS; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][c][e] *= alpha;
        }
      }
      __syncthreads();  // the keys have been read: the weights go there
      if (!idle) {
        float* p = sk;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) p[(4 * y + r) * (kSimtKeys + 4) + x + 16 * c] = s[r][c];
        __syncwarp();  // a row's weights are its own warp's
        for (int k = 0; k < kSimtKeys; k += 4) {
          float4 w[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) w[r] = *reinterpret_cast<const float4*>(p + (4 * y + r) * (kSimtKeys + 4) + k);
#pragma unroll
          for (int c = 0; c < COLS; ++c) {
            const int d = 64 * c + 4 * x;
            if (d >= 4 * d4) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 v = *reinterpret_cast<const float4*>(sv + (k + i) * pitch + d);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float pw = i == 0 ? w[r].x : i == 1 ? w[r].y : i == 2 ? w[r].z : w[r].w;
                o[r][c][0] += pw * v.x;
                o[r][c][1] += pw * v.y;
                o[r][c][2] += pw * v.z;
                o[r][c][3] += pw * v.w;
              }
            }
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (!valid[r]) continue;
      const int row = 4 * y + r, tok = row / A.hb;
      const int64_t at = static_cast<int64_t>(it.tok0 + tok) * A.hq + it.hk * A.group + it.g0 + row - tok * A.hb;
      const int64_t to = it.dest == kExtFinal ? at
                         : it.dest == kExtRows ? static_cast<int64_t>(it.slot) * A.n_tokens * A.hq + at
                                               : static_cast<int64_t>(it.slot) * A.slot_rows + row;
      float* out = (it.dest == kExtFinal ? static_cast<float*>(A.out) : it.dest == kExtRows ? A.row_o : A.part_o) + to * dh;
      const float inv = it.dest != kExtFinal ? 1.f : l[r] > 0.f ? 1.f / l[r] : 0.f;
#pragma unroll
      for (int c = 0; c < COLS; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (64 * c + 4 * x + e < dh) out[64 * c + 4 * x + e] = o[r][c][e] * inv;
      if (x == 0) {
        if (it.dest == kExtFinal) A.lse[at] = l[r] > 0.f ? (m[r] + log2f(l[r])) * 0.69314718055994531f : -INFINITY;
        else (it.dest == kExtRows ? A.row_ml : A.part_ml)[to] = make_float2(m[r], l[r]);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- the join
constexpr int kJoinThreads = 256;

// The parts of a block: CTAs c0 .. c1 (c0 == c1: it is whole, in the row buffers).
struct Cut {
  int c0, c1;
  int tok0;  // token row of its first row
};
__device__ __forceinline__ Cut cut_of(const ExtArgs& A, const ExtSeg& g, int pair, int blk) {
  const int64_t units = A.head->units;
  const int ctas = A.head->ctas;
  const int64_t base = g.unit0 + pair * g.units + ext_units_before(A.sh, g, blk);
  Cut c;
  c.tok0 = g.t0 + blk * A.sh.bt;
  c.c0 = ext_cta_of(units, ctas, base);
  c.c1 = ext_cta_of(units, ctas,
                    base + static_cast<int64_t>(ext_walk(A.sh, g, blk).count - 1) * ext_weight(A.sh, g, blk));
  return c;
}

template <typename T> __device__ __forceinline__ void put(T* p, float v);
template <> __device__ __forceinline__ void put<float>(float* p, float v) { *p = v; }
template <> __device__ __forceinline__ void put<__nv_bfloat16>(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// A block for the rows of a block of one sequence's tokens (x: block and pair): nothing to do where one
// CTA had it whole and no prefix is shared; 0 and -inf where nothing is seen. Threads take a row's
// columns, E at a time, and where the block has few rows a share of the parts each; sums are taken in a
// fixed order.
template <typename T, int E>
__global__ void __launch_bounds__(kJoinThreads) extend_join(const __grid_constant__ ExtArgs A) {
  __shared__ Cut sh_cut[3];  // own, the prefix's block of the first token, the next one
  __shared__ ExtSeg sh_seg;
  __shared__ int sh_blk, sh_pair;
  __shared__ float sums[kJoinThreads * E];
  __shared__ float sh_l[kJoinThreads];
  const int tid = threadIdx.x, dh = A.dh, bt = A.sh.bt;
  wait_for_previous();
  const int pairs = A.hkv * A.blocks_per_kv;
  if (tid < 32) {
    const int lane = tid, block = blockIdx.x / pairs, pair = blockIdx.x - block * pairs;
    const bool some = block < A.head->own_blocks;
    int blk = -1;
    if (some) {
      // the last segment that begins at the block or before: 32 places at a time
      int lo = A.n_groups, n = A.n_seqs;
      while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool before = at < lo + n && A.segs[at].blocks0 <= block;
        const int next = lo + (__popc(__ballot_sync(0xffffffffu, before)) - 1) * step;
        n = min(step, lo + n - next);
        lo = next;
      }
      const ExtSeg g = A.segs[lo];
      blk = block - g.blocks0;
      if (lane < 3) {
        Cut c = {0, -1, 0};
        if (lane == 0 && g.units > 0) c = cut_of(A, g, pair, blk);
        if (lane > 0 && g.prefix >= 0) {
          const ExtSeg p = A.segs[g.prefix];
          const int i = (g.t0 + blk * bt - p.t0) / bt + lane - 1;
          if (i < ext_blocks(A.sh, p.n)) c = cut_of(A, p, pair, i);
        }
        sh_cut[lane] = c;
      }
      if (lane == 0) sh_seg = g;
    }
    if (lane == 0) {
      sh_blk = blk;
      sh_pair = pair;
    }
  }
  __syncthreads();
  if (sh_blk < 0) return;
  const ExtSeg& g = sh_seg;
  const bool empty = g.units == 0, joined = g.prefix >= 0;
  if (!empty && !joined && sh_cut[0].c0 == sh_cut[0].c1) return;
  const int hk = sh_pair / A.blocks_per_kv, g0 = sh_pair % A.blocks_per_kv * A.hb, heads = min(A.hb, A.group - g0);
  const int tok0 = g.t0 + sh_blk * bt, ntok = min(bt, g.n - sh_blk * bt);
  const int cols = dh / E, work = ntok * heads * cols;
  int split = 1;  // shares of the parts
  while (split < 8 && 2 * split * work <= kJoinThreads) split *= 2;
  const int per = kJoinThreads / split, share = tid / per;
  for (int w0 = 0; w0 < work; w0 += per) {
    const int w = w0 + tid - share * per;
    const bool on = w < work;
    float x[E], l = 0.f, mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
    const int r = on ? w / cols : 0, d = on ? (w - r * cols) * E : 0, tok = r / heads, h = r - tok * heads;
    const int64_t at = static_cast<int64_t>(tok0 + tok) * A.hq + hk * A.group + g0 + h;
    if (on && !empty) {
      const Cut own = sh_cut[0];
      Cut pre = {0, -1, 0};
      if (joined) pre = tok0 + tok - sh_cut[1].tok0 < bt ? sh_cut[1] : sh_cut[2];
      const int n0 = own.c1 - own.c0 + 1, n = n0 + pre.c1 - pre.c0 + 1;
      const int own_row = tok * A.hb + h, pre_row = (tok0 + tok - pre.tok0) * A.hb + h;
      // part i: its state and its sums
      auto place = [&](int i, const float2** ml, const float** o) {
        const bool mine = i < n0;
        const Cut& c = mine ? own : pre;
        if (!mine) i -= n0;
        const bool whole = c.c0 == c.c1;
        const int64_t row = whole ? (mine ? static_cast<int64_t>(A.n_tokens) * A.hq : 0) + at
                                  : (static_cast<int64_t>(c.c0 + i) * 2 + (i == 0 ? 1 : 0)) * A.slot_rows +
                                        (mine ? own_row : pre_row);
        *ml = (whole ? A.row_ml : A.part_ml) + row;
        *o = (whole ? A.row_o : A.part_o) + row * dh + d;
      };
      const float2* ml;
      const float* o;
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        place(i, &ml, &o);
        mx = fmaxf(mx, ml->x);
      }
      const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
      for (int i = share; i < n; i += split) {
        place(i, &ml, &o);
        const float2 s = *ml;
        const float f = exp2f(s.x - ref);
        l += f * s.y;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(o);
          x[0] += f * v.x;
          x[1] += f * v.y;
          x[2] += f * v.z;
          x[3] += f * v.w;
        } else {
          x[0] += f * *o;
        }
      }
    }
    if (split > 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) sums[tid * E + e] = x[e];
      sh_l[tid] = l;
      __syncthreads();
      if (share == 0) {
        for (int k = 1; k < split; ++k) {
          l += sh_l[tid + k * per];
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] += sums[(tid + k * per) * E + e];
        }
      }
    }
    if (on && share == 0) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) put<T>(static_cast<T*>(A.out) + at * dh + d + e, x[e] * inv);
      if (d == 0) A.lse[at] = l > 0.f ? (mx + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
    if (split > 1) __syncthreads();
  }
}

// ---------------------------------------------------------------- host
cudaError_t launch_after(const void* kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t st, void** args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t launch_extend_simt(ExtArgs& A, cudaStream_t st) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(A.q) | reinterpret_cast<uintptr_t>(A.k_pages) |
                      reinterpret_cast<uintptr_t>(A.v_pages);
  int vec = p % 16 == 0 && A.dh % 4 == 0 && A.page_stride % 4 == 0 && A.slot_stride % 4 == 0 && A.head_stride % 4 == 0;
  const void* kernel = A.dh > 64 ? reinterpret_cast<const void*>(extend_simt<2>) : reinterpret_cast<const void*>(extend_simt<1>);
  const int smem = simt_smem(A.dh);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  void* args[] = {&A, &vec};
  return launch_after(kernel, A.most_ctas, kSimtThreads, smem, st, args);
}

// Blocks of query heads of one K/V head, as even as can be.
void head_blocks(int group, int most, int* hb, int* blocks) {
  *blocks = (group + most - 1) / most;
  *hb = (group + *blocks - 1) / *blocks;
  *blocks = (group + *hb - 1) / *hb;
}

ExtShape shape_of(int dtype, int hb, int window, int sinks) {
  ExtShape s;
  s.half = (dtype == RA_BF16 ? 128 : kSimtRows) / hb;
  s.bt = dtype == RA_BF16 ? 2 * s.half : s.half;
  s.wide = dtype == RA_BF16 ? 2 : 1;
  s.shift = dtype == RA_BF16 ? 7 : 6;
  s.window = window;
  s.sinks = sinks;
  return s;
}

// The workspace's regions, one after the other.
struct Regions {
  size_t segs, part_o, part_ml, row_o, row_ml, total;
};
Regions regions_of(const ra_paged_cache* c, int n_groups, int n_tokens, int hq) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  int hb, blocks;
  head_blocks(hq / c->hkv, c->dtype == RA_BF16 ? 128 : kSimtRows, &hb, &blocks);
  const ExtShape s = shape_of(c->dtype, hb, 0, 0);
  const size_t ctas = (c->dtype == RA_BF16 ? 1 : 2) * kExtSms;
  const size_t slot_rows = static_cast<size_t>(n_tokens < s.bt ? n_tokens : s.bt) * hb, parts = ctas * 2 * slot_rows;
  const size_t rows = n_groups > 0 ? size_t(2) * n_tokens * hq : 0;
  Regions r;
  r.segs = 256;
  r.part_o = r.segs + up((static_cast<size_t>(n_groups) + c->n_seqs) * sizeof(ExtSeg));
  r.part_ml = r.part_o + up(parts * c->head_dim * 4);
  r.row_o = r.part_ml + up(parts * 8);
  r.row_ml = r.row_o + up(rows * c->head_dim * 4);
  r.total = r.row_ml + up(rows * 8);
  return r;
}

int check_extend(const ra_paged_cache* c, int n_groups, int n_tokens, int hq) {
  if (hq < 1 || hq % c->hkv)
    return record_error(RA_ERR_UNSUPPORTED, "hq (%d) must be a positive multiple of hkv (%d)", hq, c->hkv);
  if (n_tokens < 0 || n_groups < 0) return record_error(RA_ERR_INVALID_ARG, "n_tokens and n_groups must be >= 0");
  if (n_groups > c->n_seqs)
    return record_error(RA_ERR_SHAPE, "more groups (%d) than sequences (%d)", n_groups, c->n_seqs);
  if (static_cast<int64_t>(n_tokens) * hq >= (int64_t(1) << 31))
    return record_error(RA_ERR_UNSUPPORTED, "tokens x query heads must stay below 2^31");
  return RA_OK;
}

}  // namespace

cudaError_t extend_status(unsigned int value[2], bool reset) {
  unsigned int index = 0;
  cudaError_t e = extend_tc_status(value, reset);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&index, g_status_extend, sizeof index);
  if (e == cudaSuccess && reset) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_status_extend, &zero, sizeof zero);
  }
  value[1] |= index;
  return e;
}

}  // namespace ra

using namespace ra;

extern "C" size_t ra_paged_extend_workspace_bytes(const ra_paged_cache* c, int n_groups, int n_tokens, int hq) {
  if (check_cache(c) != RA_OK || check_extend(c, n_groups, n_tokens, hq) != RA_OK) return 0;
  return regions_of(c, n_groups, n_tokens, hq).total;
}

extern "C" int ra_paged_attn_extend(const ra_paged_cache* c, const ra_shared_prefix* shared, int n_tokens, int hq,
                                    float scale, int window, int sinks, const void* q, const int32_t* seq_lens,
                                    const int32_t* cu_new, void* out, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  if (int e = check_cache(c)) return e;
  const int n_groups = shared != nullptr ? shared->n_groups : 0;
  if (int e = check_extend(c, n_groups, n_tokens, hq)) return e;
  const bool some = n_tokens > 0 && c->n_seqs > 0;  // empty tensors may have null pointers
  if (some && (!q || !seq_lens || !out || !lse)) return record_error(RA_ERR_INVALID_ARG, "null tensor pointer");
  if (cu_new == nullptr && n_tokens != c->n_seqs)
    return record_error(RA_ERR_SHAPE, "without cu_new there is one token for each of the %d sequences (got %d)",
                        c->n_seqs, n_tokens);
  if (std::isnan(scale) || std::isinf(scale)) return record_error(RA_ERR_INVALID_ARG, "scale is not finite");
  if (window < 0 || sinks < 0 || sinks > RA_MAX_SINKS)
    return record_error(RA_ERR_INVALID_ARG, "window must be >= 0, sinks 0..%d", RA_MAX_SINKS);
  if (n_groups > 0 && (!shared->cu_groups || !shared->prefix_lens))
    return record_error(RA_ERR_INVALID_ARG, "null pointer in the shared prefixes");
  if (n_groups > 0 && window > 0)
    return record_error(RA_ERR_UNSUPPORTED, "shared prefixes and a window do not go together");
  const Regions at = regions_of(c, n_groups, n_tokens, hq);
  if (workspace_bytes < at.total)
    return record_error(RA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, at.total);
  if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256)
    return record_error(RA_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
  if (!some) return record_error(RA_OK, "%s", "");
  if (c->dtype == RA_BF16) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(c->k_pages) | reinterpret_cast<uintptr_t>(c->v_pages) |
                        reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out);
    if (p % 16 || c->page_stride % 8 || c->slot_stride % 8 || c->head_stride % 8)
      return record_error(RA_ERR_INVALID_ARG,
                          "bf16: q, out and pages must be 16-byte aligned, strides multiples of 8 elements");
  }
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return record_error(RA_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
  ExtArgs A = {};
  A.q = q;
  A.k_pages = c->k_pages;
  A.v_pages = c->v_pages;
  A.block_table = c->block_table;
  A.seq_lens = seq_lens;
  A.cu_new = cu_new;
  A.cu_groups = n_groups > 0 ? shared->cu_groups : nullptr;
  A.prefix_lens = n_groups > 0 ? shared->prefix_lens : nullptr;
  A.table_stride = c->table_stride;
  A.page_stride = c->page_stride;
  A.slot_stride = c->slot_stride;
  A.head_stride = c->head_stride;
  A.n_seqs = c->n_seqs;
  A.n_groups = n_groups;
  A.n_tokens = n_tokens;
  A.max_pages = c->max_pages;
  A.page_size = c->page_size;
  A.n_pages = c->n_pages;
  A.hq = hq;
  A.hkv = c->hkv;
  A.group = hq / c->hkv;
  A.dh = c->head_dim;
  head_blocks(A.group, c->dtype == RA_BF16 ? 128 : kSimtRows, &A.hb, &A.blocks_per_kv);
  A.sh = shape_of(c->dtype, A.hb, window, window > 0 ? sinks : 0);
  A.slot_rows = (n_tokens < A.sh.bt ? n_tokens : A.sh.bt) * A.hb;
  A.most_ctas = (c->dtype == RA_BF16 ? 1 : 2) * (n_sm < kExtSms ? n_sm : kExtSms);
  A.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(c->head_dim))) * 1.4426950408889634f;
  A.timeout_ns = kDefaultTimeoutNs;
  char* ws = static_cast<char*>(workspace);
  A.head = reinterpret_cast<ExtHead*>(ws);
  A.segs = reinterpret_cast<ExtSeg*>(ws + at.segs);
  A.part_o = reinterpret_cast<float*>(ws + at.part_o);
  A.part_ml = reinterpret_cast<float2*>(ws + at.part_ml);
  A.row_o = reinterpret_cast<float*>(ws + at.row_o);
  A.row_ml = reinterpret_cast<float2*>(ws + at.row_ml);
  A.out = out;
  A.lse = lse;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ExtMaps maps;
  if (c->dtype == RA_BF16 && (e = make_extend_maps(&maps, c, &A)) != cudaSuccess)
    return record_error(RA_ERR_UNSUPPORTED, "the pages' strides do not fit a tensor map");
  extend_plan<<<1, kPlanThreads, 0, st>>>(A);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = c->dtype == RA_BF16 ? launch_extend_tc(A, maps, st) : launch_extend_simt(A, st);
  if (e == cudaSuccess) {
    // at most one block of a sequence has fewer tokens than the others
    int64_t blocks = static_cast<int64_t>(n_tokens / A.sh.bt) + c->n_seqs;
    if (blocks > n_tokens) blocks = n_tokens;
    void* args[] = {&A};
    const void* kernel = c->dtype == RA_BF16 ? reinterpret_cast<const void*>(extend_join<__nv_bfloat16, 4>)
                         : A.dh % 4 == 0     ? reinterpret_cast<const void*>(extend_join<float, 4>)
                                             : reinterpret_cast<const void*>(extend_join<float, 1>);
    e = launch_after(kernel, static_cast<unsigned>(blocks * A.hkv * A.blocks_per_kv), kJoinThreads, 0, st, args);
  }
  if (e != cudaSuccess) return record_error(RA_ERR_CUDA, "extend attention launch: %s", cudaGetErrorString(e));
  return record_error(RA_OK, "%s", "");
}
