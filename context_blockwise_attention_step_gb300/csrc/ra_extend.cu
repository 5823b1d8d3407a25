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
// Three or four launches, each while the one before still runs (programmatic dependent launch): the
// planning kernel reads the lengths and lists the segments (ra_extend.h); the main kernels, for many
// rows (ra_extend_tc.cu, float32 here) and for few (ra_extend_few.cu), deal them out evenly to their
// CTAs; the join works on the blocks that need it. The host need not know a length. By themselves the plan takes
// 10-16 us (a chain of reads and of sums over the segments, one block), the join 10-15 us for decoding steps
// and 42 where every CTA leaves two parts of 256 rows (38 MB). The plan grows with the sequences: a call of one
// token each of 64, 512, 2048 and 8192 sequences of 100 keys, 8/1 heads of 64, takes 25, 29, 66 and 219 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "ra_extend.cuh"

namespace ra {

static __device__ unsigned int g_status_extend;  // an index outside the cache
static __device__ unsigned int g_status_plan;    // a plan that did not come

namespace {

// ---------------------------------------------------------------- planning
constexpr int kPlanThreads = 640, kPlanWarps = kPlanThreads / 32;

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

__global__ void __launch_bounds__(kPlanThreads, 1) extend_plan(const __grid_constant__ ExtArgs A) {
  __shared__ int64_t scan_units[2][kPlanWarps];
  __shared__ int scan_blocks[kPlanWarps];
  __shared__ int64_t first_units[2][kPlanThreads];  // of the first segments
  __shared__ int group_keys[kPlanThreads];  // of the first groups: the keys that are shared, 0: none
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const ExtShape& s = A.sh[kExtMany];
  launch_dependents();
  if (tid == 0) A.head->ready = 0;
  auto class_of = [&](int n) { return n * int64_t(A.group) <= A.few_rows ? kExtFew : kExtMany; };
  // groups, a warp each: whether the prefix lies before every new token, and whether sharing it pays.
  // Offsets out of order or range share nothing in the whole call: groups that overlap would give a row
  // two prefixes, whose results go to the same place.
  bool disorder = false;
  for (int g = warp; g < A.n_groups; g += kPlanWarps) {
    const int b0 = bounded(A.cu_groups[g], A.n_seqs), b1 = bounded(A.cu_groups[g + 1], A.n_seqs);
    disorder = disorder || b0 != A.cu_groups[g] || b1 != A.cu_groups[g + 1] || b0 > b1;
    const int64_t cap = static_cast<int64_t>(A.max_pages) * A.page_size;
    int p = A.prefix_lens[g];
    if (p > cap) p = static_cast<int>(cap);
    const int tiles = p > 0 ? p >> s.shift : 0;
    int64_t apart = 0;
    int first = A.n_seqs, ok = 1;
    int balance = 0;  // tokens of sequences of few rows, less the others
    for (int b = b0 + lane; b < b1; b += 32) {
      const Tokens t = tokens_of(A, b);
      if (t.bad) ok = 0;
      if (!t.live) continue;
      if (t.len - t.n < tiles << s.shift) ok = 0;
      apart += ext_block_units(s, t.n);
      balance += ext_few(t.n, A.group) ? t.n : -t.n;
      first = min(first, b);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) apart += __shfl_xor_sync(0xffffffffu, apart, o);
    first = __reduce_min_sync(0xffffffffu, first);
    ok = __reduce_min_sync(0xffffffffu, ok);
    balance = __reduce_add_sync(0xffffffffu, balance);
    if (lane == 0) {
      ExtSeg e = {};
      e.shared = balance >= 0 ? 2 : 1;
      e.prefix = -1;
      if (b0 < b1 && first < A.n_seqs && ok) {
        const Tokens a = tokens_of(A, b0), z = tokens_of(A, b1 - 1);
        const int n = z.t0 + z.n - a.t0;
        const int64_t together = ext_block_units(s, n);
        if (n > 0 && ext_worth_sharing(tiles, apart, together)) {
          e.k1 = tiles << s.shift;
          e.t0 = a.t0;
          e.n = n;
          e.seq = first;
          e.cls = class_of(n);
          e.units = ext_units_before(A.sh[e.cls], e, ext_blocks(A.sh[e.cls], n));
        }
      }
      A.segs[g] = e;
      if (g < kPlanThreads) group_keys[g] = e.k1;
    }
  }
  disorder = __syncthreads_or(disorder);
  if (disorder && tid == 0) atomicOr(&g_status_extend, 1u);
  // all segments in order, a thread each
  const int segs = A.n_groups + A.n_seqs, pairs = A.hkv * A.blocks_per_kv;
  int64_t done[2] = {0, 0};
  int done_blocks = 0;
  for (int i0 = 0; i0 < segs; i0 += kPlanThreads) {
    const int i = i0 + tid;
    ExtSeg e = {};
    int blocks = 0;
    if (i < A.n_groups) {
      e = A.segs[i];
      if (disorder) e.units = 0;
    } else if (i < segs) {
      const int b = i - A.n_groups;
      const Tokens t = tokens_of(A, b);
      if (t.bad) atomicOr(&g_status_extend, 1u);
      e.t0 = t.t0;
      e.n = t.n;
      e.base = t.len - t.n;
      e.k1 = t.len;
      e.seq = b;
      e.prefix = -1;
      e.cls = class_of(t.n);
      if (A.n_groups > 0 && t.live && !disorder) {
        int lo = 0, hi = A.n_groups - 1;  // the last group that begins at b or before
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (A.cu_groups[mid] <= b) lo = mid; else hi = mid - 1;
        }
        if (A.cu_groups[lo] <= b && b < A.cu_groups[lo + 1]) {
          e.k0 = lo < kPlanThreads ? group_keys[lo] : A.segs[lo].k1;
          if (e.k0 > 0) e.prefix = lo;
        }
      }
      blocks = ext_blocks(s, t.n);
      if (t.live) e.units = ext_units_before(A.sh[e.cls], e, ext_blocks(A.sh[e.cls], t.n));
    }
    // units of each class and blocks before this segment
    int64_t x[2];
    int y = blocks;
    x[0] = e.cls == kExtMany ? e.units * pairs : 0;
    x[1] = e.cls == kExtFew ? e.units * pairs : 0;
    const int64_t mine[2] = {x[0], x[1]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, x[0], o), v = __shfl_up_sync(0xffffffffu, x[1], o);
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x[0] += u;
        x[1] += v;
        y += z;
      }
    }
    __syncthreads();  // the round before has read the sums
    if (lane == 31) {
      scan_units[0][warp] = x[0];
      scan_units[1][warp] = x[1];
      scan_blocks[warp] = y;
    }
    __syncthreads();
    // each warp sums the warps before it, a lane a warp
    const bool there = lane < kPlanWarps;
    int64_t p0 = there ? scan_units[0][lane] : 0, p1 = there ? scan_units[1][lane] : 0;
    int pb = there ? scan_blocks[lane] : 0;
    int64_t before[2] = {lane < warp ? p0 : 0, lane < warp ? p1 : 0};
    int before_blocks = lane < warp ? pb : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      p0 += __shfl_xor_sync(0xffffffffu, p0, o);
      p1 += __shfl_xor_sync(0xffffffffu, p1, o);
      pb += __shfl_xor_sync(0xffffffffu, pb, o);
      before[0] += __shfl_xor_sync(0xffffffffu, before[0], o);
      before[1] += __shfl_xor_sync(0xffffffffu, before[1], o);
      before_blocks += __shfl_xor_sync(0xffffffffu, before_blocks, o);
    }
    if (i < segs) {
      e.unit0[0] = done[0] + before[0] + x[0] - mine[0];
      e.unit0[1] = done[1] + before[1] + x[1] - mine[1];
      e.blocks0 = done_blocks + before_blocks + y - blocks;
      A.segs[i] = e;
    }
    if (i0 == 0) {
      first_units[0][tid] = e.unit0[0];
      first_units[1][tid] = e.unit0[1];
    }
    done[0] += p0;
    done[1] += p1;
    done_blocks += pb;
  }
  int ctas[2];
  for (int c = 0; c < 2; ++c) ctas[c] = ext_ctas(A.sh[c], done[c], A.part[c].most_ctas);
  if (tid == 0) {
    ExtHead h;
    for (int c = 0; c < 2; ++c) {
      h.units[c] = done[c];
      h.ctas[c] = ctas[c];
    }
    h.segs = segs;
    h.own_blocks = done_blocks;
    h.ready = 0;
    *A.head = h;
  }
  __syncthreads();
  // where each CTA begins
  const int most = A.part[0].most_ctas;
  for (int k = tid; k < most + A.part[1].most_ctas + 2; k += kPlanThreads) {
    const int c = k <= most ? 0 : 1, cta = c == 0 ? k : k - most - 1, n = c == 0 ? ctas[0] : ctas[1];
    const int64_t all = c == 0 ? done[0] : done[1];
    ExtStart to = {};
    const int64_t u0 = cta < n ? ext_first(all, n, cta) : all;
    to.u0 = u0;
    if (cta >= n) {
      A.starts[c][cta] = to;
      continue;
    }
    int lo = 0, hi = segs - 1;  // the last segment that begins at u0 or before
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((mid < kPlanThreads ? first_units[c][mid] : A.segs[mid].unit0[c]) <= u0) lo = mid; else hi = mid - 1;
    }
    const ExtSeg g = A.segs[lo];
    const int64_t unit0 = ext_unit0(g, c), r = u0 - unit0;
    const int pair = static_cast<int>(ext_div(r, g.units));
    const int blk = ext_block_of(A.sh[c], g, r - pair * g.units);
    to.base = unit0 + pair * g.units + ext_units_before(A.sh[c], g, blk);
    to.seg = lo;
    to.hk = pair / A.blocks_per_kv;
    to.hblk = pair - to.hk * A.blocks_per_kv;
    to.blk = blk;
    A.starts[c][cta] = to;
  }
  __syncthreads();
  if (tid == 0) ext_publish(A.head);
}

// ---------------------------------------------------------------- float32
// 64 rows against tiles of 64 keys on the CUDA cores, 256 threads: thread (y, x) works out the scores
// of rows 4y .. 4y+3 and keys x, x + 16, x + 32, x + 48, sixteen lanes have a row's scores, and of the
// result rows 4y .. and the columns 4x .. 4x+3, and 64 + 4x .. What bounds it: 2 dh FMAs a row and key
// and product; eight FMAs a 16-byte word of shared memory. The next tile's keys come by asynchronous
// copies meanwhile, their places in the table are looked up a tile earlier still; one barrier a tile.
constexpr int kSimtThreads = 256, kSimtRows = 64, kSimtKeys = 64, kSimtPitchP = kSimtKeys + 4;
__host__ __device__ constexpr int simt_pitch(int dh) { return (dh + 3) / 4 * 4 + 4; }
// Q, two stages of K and V, the weights; floats. Two CTAs an SM for heads of up to 64.
__host__ __device__ constexpr int simt_floats(int dh) { return (kSimtRows + 4 * kSimtKeys) * simt_pitch(dh) + kSimtRows * kSimtPitchP; }
constexpr int simt_ctas(int dh) { return dh > 64 ? 1 : 2; }

// COLS: groups of 64 columns of the head.
template <int COLS>
__global__ void __launch_bounds__(kSimtThreads, COLS == 1 ? 2 : 1) extend_simt(const __grid_constant__ ExtArgs A, int vec) {
  extern __shared__ __align__(16) float sm[];
  __shared__ ExtItem sh_it;
  __shared__ int64_t sh_at[2][kSimtKeys];  // of a tile's keys: where they are (-1: not read)
  const int dh = A.dh, pitch = simt_pitch(dh), d4 = (dh + 3) / 4;
  float* sq = sm;                                              // [64][pitch], times scale * log2(e)
  float* stage = sm + kSimtRows * pitch;                       // [2][K, V][64][pitch]
  float* weights = stage + 4 * kSimtKeys * pitch;              // [64][68]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, x = tid & 15, y = tid >> 4;
  wait_for_previous();
  launch_dependents();
  ExtCursor<kExtMany> cur;
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
    const int rows = it.ntok * A.hb, j1 = it.j0 + it.tiles;
    const int sinks = A.sh[kExtMany].window > 0 ? min(A.sh[kExtMany].sinks, it.end) : 0;
    // a row's four elements, of memory whose rows need not be aligned
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
    // where the keys of walk index j are that some row sees, by the first threads; what is not seen is 0
    auto look_up = [&](int j) {
      if (tid >= kSimtKeys || j >= j1) return;
      const int key = ext_tile(it.walk, j) * kSimtKeys + tid;
      int64_t at = -1;
      if (key < sinks || (key >= it.low && key < it.end)) {
        const int page = key / A.page_size;
        at = ext_page(A, it.seq, page, &g_status_extend) * A.page_stride +
             static_cast<int64_t>(key - page * A.page_size) * A.slot_stride + it.hk * A.head_stride;
      }
      sh_at[j & 1][tid] = at;
    };
    auto load = [&](int j) {
      if (j >= j1) return;
      float* k = stage + (j & 1) * 2 * kSimtKeys * pitch;
      float* v = k + kSimtKeys * pitch;
      for (int i = tid; i < kSimtKeys * d4; i += kSimtThreads) {
        const int r = i / d4, d = (i - r * d4) * 4;
        const int64_t at = sh_at[j & 1][r];
        if (vec && at >= 0) {
          cp_async16(smem_u32(k + r * pitch + d), static_cast<const float*>(A.k_pages) + at + d);
          cp_async16(smem_u32(v + r * pitch + d), static_cast<const float*>(A.v_pages) + at + d);
        } else {
          copy_row4(static_cast<const float*>(A.k_pages) + (at < 0 ? 0 : at), k + r * pitch, d, at >= 0, 1.f);
          copy_row4(static_cast<const float*>(A.v_pages) + (at < 0 ? 0 : at), v + r * pitch, d, at >= 0, 1.f);
        }
      }
    };
    look_up(it.j0);
    for (int i = tid; i < kSimtRows * d4; i += kSimtThreads) {
      const int r = i / d4, d = (i - r * d4) * 4, tok = r / A.hb, h = r - tok * A.hb;
      const bool on = r < rows && h < it.heads;
      const int64_t at = static_cast<int64_t>(it.tok0 + tok) * A.hq + it.hk * A.group + it.g0 + h;
      copy_row4(static_cast<const float*>(A.q) + (on ? at * dh : 0), sq + r * pitch, d, on, A.scale_log2);
    }
    __syncthreads();
    load(it.j0);
    cp_async_commit();
    look_up(it.j0 + 1);
    int hi[4], lo[4];
    bool valid[4];
    float m[4], l[4], o[4][COLS][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * y + r, tok = row / A.hb;
      valid[r] = row < rows && row - tok * A.hb < it.heads;
      hi[r] = !valid[r] ? 0 : it.shared ? it.end : it.base + tok + 1;
      lo[r] = A.sh[kExtMany].window > 0 ? max(0, hi[r] - A.sh[kExtMany].window) : 0;
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < COLS; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][c][e] = 0.f;
    }
    for (int j = it.j0; j < j1; ++j) {
      cp_async_wait<0>();
      __syncthreads();  // tile j is there, everyone has done with the one before, and the next one's places are known
      load(j + 1);
      cp_async_commit();
      look_up(j + 2);
      if (8 * warp >= rows) continue;  // (a warp without rows helps with the copies only)
      const int k0 = ext_tile(it.walk, j) * kSimtKeys;
      const float* sk = stage + (j & 1) * 2 * kSimtKeys * pitch;
      const float* sv = sk + kSimtKeys * pitch;
      float s[4][4] = {};
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
          if (!(key < hi[r] && (key >= lo[r] || key < A.sh[kExtMany].sinks))) s[r][c] = -INFINITY;
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
      __syncwarp();  // the weights of the tile before have been read (a row's are its own warp's)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) weights[(4 * y + r) * kSimtPitchP + x + 16 * c] = s[r][c];
      __syncwarp();
      for (int k = 0; k < kSimtKeys; k += 4) {
        float4 w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = *reinterpret_cast<const float4*>(weights + (4 * y + r) * kSimtPitchP + k);
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
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (!valid[r]) continue;
      const int row = 4 * y + r, tok = row / A.hb;
      const int64_t at = static_cast<int64_t>(it.tok0 + tok) * A.hq + it.hk * A.group + it.g0 + row - tok * A.hb;
      const int64_t to = it.dest == kExtFinal ? at
                         : it.dest == kExtRows ? static_cast<int64_t>(it.slot) * A.n_tokens * A.hq + at
                                               : static_cast<int64_t>(it.slot) * A.part[kExtMany].rows + row;
      float* out = (it.dest == kExtFinal ? static_cast<float*>(A.out) : it.dest == kExtRows ? A.row_o : A.part[kExtMany].o) + to * dh;
      const float inv = it.dest != kExtFinal ? 1.f : l[r] > 0.f ? 1.f / l[r] : 0.f;
#pragma unroll
      for (int c = 0; c < COLS; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (64 * c + 4 * x + e < dh) out[64 * c + 4 * x + e] = o[r][c][e] * inv;
      if (x == 0) {
        if (it.dest == kExtFinal) A.lse[at] = l[r] > 0.f ? (m[r] + log2f(l[r])) * 0.69314718055994531f : -INFINITY;
        else (it.dest == kExtRows ? A.row_ml : A.part[kExtMany].ml)[to] = make_float2(m[r], l[r]);
      }
    }
    __syncthreads();  // the item, its rows and its last tile have been read
  }
}

// ---------------------------------------------------------------- the join
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

// The parts of a block: CTA c0 of its class, and c0 + skip + 1 .. c1 (c0 == c1: it is whole, in the row
// buffers).
struct Cut {
  int c0, skip, c1, cls;
  int tok0;  // token row of its first row
  __device__ __forceinline__ int parts() const { return c1 - c0 - skip + 1; }
};
__device__ __forceinline__ Cut cut_of(const ExtArgs& A, const ExtHead& head, const ExtSeg& g, int pair, int blk) {
  const ExtShape& sh = A.sh[g.cls];
  const int64_t units = g.cls == kExtMany ? head.units[0] : head.units[1];
  const int ctas = g.cls == kExtMany ? head.ctas[0] : head.ctas[1];
  const int64_t base = ext_unit0(g, g.cls) + pair * g.units + ext_units_before(sh, g, blk);
  Cut c;
  c.cls = g.cls;
  c.tok0 = g.t0 + blk * sh.bt;
  const ExtCtas of = ext_ctas_of(sh, units, ctas, base, ext_weight(sh, g, blk), ext_walk(sh, g, blk).count);
  c.c0 = of.c0;
  c.skip = of.skip;
  c.c1 = of.c1;
  return c;
}

template <typename T> __device__ __forceinline__ void put4(T* p, const float (&v)[4]);
template <> __device__ __forceinline__ void put4<float>(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <> __device__ __forceinline__ void put4<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// A block for the rows of a block of one sequence's tokens (x: block and pair): nothing to do where one
// CTA had it whole and no prefix is shared; 0 and -inf where nothing is seen. A warp takes a row, or
// where there are few rows a share of its parts: a lane has a part's state, all lanes its sums, four
// columns each (QUADS), or every 32nd. BULK: where there are more than eight rows, which have few parts
// each, a warp takes four rows at once, part by part, and few blocks are shared out (y) (16 questions of 500 tokens behind 16384 shared
// keys, 32/8 heads: 40 us, was 77; its registers leave half the blocks on an SM, which decoding steps
// would pay for: 64 sequences 19 us in place of 13). Sums are taken in a fixed order.
template <typename T, bool QUADS, bool BULK>
__global__ void __launch_bounds__(kJoinThreads, BULK ? 2 : 4) extend_join(const __grid_constant__ ExtArgs A) {
  __shared__ Cut sh_cut[3];  // own, the prefix's block of the first token, the next one
  __shared__ ExtSeg sh_seg;
  __shared__ int sh_blk;
  __shared__ float sums[kJoinWarps][128], sum_l[kJoinWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, dh = A.dh, bt = A.sh[kExtMany].bt;
  const int pairs = A.hkv * A.blocks_per_kv, block = blockIdx.x / pairs, pair = blockIdx.x - block * pairs;
  // the block's parts by the plan, which is there when this kernel may start, then the results
  if (warp == 0) {
    const bool planned = __all_sync(0xffffffffu, ext_acquire(A.head, A.timeout_ns, &g_status_plan));
    const ExtHead head = *A.head;
    int lo = A.n_groups, n = A.n_seqs, blk = -1;
    if (!planned) {
    } else if (A.cu_new == nullptr) {
      lo += block;  // a block is a sequence
      blk = 0;
    } else if (block < head.own_blocks) {
      // the last segment that begins at the block or before: 32 places at a time
      while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool before = at < lo + n && A.segs[at].blocks0 <= block;
        const int next = lo + (__popc(__ballot_sync(0xffffffffu, before)) - 1) * step;
        n = min(step, lo + n - next);
        lo = next;
      }
      blk = block - A.segs[lo].blocks0;
    }
    if (blk >= 0 && lane < 3) {
      const ExtSeg g = A.segs[lo];
      Cut c = {0, 0, -1, 0, 0};
      if (lane == 0 && g.units > 0) c = cut_of(A, head, g, pair, g.cls == kExtFew ? 0 : blk);
      if (lane > 0 && g.prefix >= 0) {
        const ExtSeg p = A.segs[g.prefix];
        const int i = (g.t0 + blk * bt - p.t0) / A.sh[p.cls].bt + lane - 1;
        if (i < ext_blocks(A.sh[p.cls], p.n)) c = cut_of(A, head, p, pair, i);
      }
      sh_cut[lane] = c;
      if (lane == 0) sh_seg = g;
    }
    if (lane == 0) sh_blk = blk;
  }
  wait_for_previous();  // in every block: what follows in the stream waits for this kernel alone
  __syncthreads();
  if (sh_blk < 0) return;
  const ExtSeg& g = sh_seg;
  const bool empty = g.units == 0, joined = g.prefix >= 0;
  const Cut own = sh_cut[0];
  if (!empty && !joined && own.c0 == own.c1) return;
  const int hk = pair / A.blocks_per_kv, g0 = pair % A.blocks_per_kv * A.hb, heads = min(A.hb, A.group - g0);
  const int tok0 = g.t0 + sh_blk * bt, rows = min(bt, g.n - sh_blk * bt) * heads;
  // the parts of a row, and the row of part i: in the row buffers, or among its class's parts
  struct Row {
    int pre;  // which of sh_cut
    int n0, n, tok, h;
    int64_t at;
  };
  auto row_of = [&](int r) {
    Row w;
    w.tok = r / heads;
    w.h = r - w.tok * heads;
    w.at = static_cast<int64_t>(tok0 + w.tok) * A.hq + hk * A.group + g0 + w.h;
    w.pre = tok0 + w.tok - sh_cut[1].tok0 < A.sh[sh_cut[1].cls].bt ? 1 : 2;  // (without a prefix both are empty)
    w.n0 = own.parts();
    w.n = w.n0 + sh_cut[w.pre].parts();
    return w;
  };
  auto place = [&](const Row& w, int i, const float2** ml, const float** o) {
    const bool mine = i < w.n0;
    const Cut& c = sh_cut[mine ? 0 : w.pre];
    if (!mine) i -= w.n0;
    const bool whole = c.c0 == c.c1, few = c.cls == kExtFew;
    const int64_t row = whole ? (mine ? static_cast<int64_t>(A.n_tokens) * A.hq : 0) + w.at
                              : (static_cast<int64_t>(i == 0 ? c.c0 : c.c0 + c.skip + i) * 2 + (i == 0 ? 1 : 0)) * (few ? A.part[1].rows : A.part[0].rows) +
                                    (tok0 + w.tok - c.tok0) * A.hb + w.h;
    *ml = (whole ? A.row_ml : few ? A.part[1].ml : A.part[0].ml) + row;
    *o = (whole ? A.row_o : few ? A.part[1].o : A.part[0].o) + row * dh;
  };
  auto store = [&](int64_t at, float mx, float l, float (&x)[4]) {
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= inv;
    T* out = static_cast<T*>(A.out) + at * dh;
    if constexpr (QUADS) {
      if (4 * lane < dh) put4<T>(out + 4 * lane, x);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (lane + 32 * e < dh) out[lane + 32 * e] = static_cast<T>(x[e]);
    }
    if (lane == 0) A.lse[at] = l > 0.f ? (mx + log2f(l)) * 0.69314718055994531f : -INFINITY;
  };
  auto fetch = [&](const float* o, float (&v)[4]) {
    if constexpr (QUADS) {
      if (4 * lane < dh) {
        const float4 q = *reinterpret_cast<const float4*>(o + 4 * lane);
        v[0] = q.x;
        v[1] = q.y;
        v[2] = q.z;
        v[3] = q.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (lane + 32 * e < dh) v[e] = o[lane + 32 * e];
    }
  };
  if (BULK && rows > kJoinWarps) {
    constexpr int U = 4;
    for (int r0 = (blockIdx.y * kJoinWarps + warp) * U; r0 < rows; r0 += gridDim.y * kJoinWarps * U) {
      float x[U][4] = {}, l[U] = {}, mx[U];
      int64_t at[U];
      int most = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        mx[u] = -INFINITY;
        const Row w = row_of(min(r0 + u, rows - 1));
        at[u] = w.at;
        most = max(most, w.n);
      }
      for (int i = 0; i < most; ++i) {
        float2 s[U];
        float v[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const Row w = row_of(min(r0 + u, rows - 1));
          const float2* ml;
          const float* o;
          s[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[u][e] = 0.f;
          if (i < w.n) {
            place(w, i, &ml, &o);
            s[u] = *ml;
            fetch(o, v[u]);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float top = fmaxf(mx[u], s[u].x), ref = top == -INFINITY ? 0.f : top;
          const float a = exp2f(mx[u] - ref), f = exp2f(s[u].x - ref);
          mx[u] = top;
          l[u] = a * l[u] + f * s[u].y;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[u][e] = a * x[u][e] + f * v[u][e];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r0 + u < rows) store(at[u], mx[u], l[u], x[u]);
    }
    return;
  }
  if (BULK && blockIdx.y > 0) return;
  int split = 1;  // warps of a row
  while (split < kJoinWarps && 2 * split * rows <= kJoinWarps) split *= 2;
  const int share = warp % split, at_once = kJoinWarps / split;
  for (int r = warp / split; r < (rows + at_once - 1) / at_once * at_once; r += at_once) {
    const bool on = r < rows;
    const Row w = row_of(on ? r : 0);
    float x[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f, mx = -INFINITY;
    if (on) {
      const int n = w.n;
      // 32 parts of this warp at a time: their states, then their sums
      for (int i0 = share; i0 < n; i0 += 32 * split) {
        const int i = i0 + lane * split;
        const float2* ml = nullptr;
        const float* o = nullptr;
        float2 s = make_float2(-INFINITY, 0.f);
        if (i < n) {
          place(w, i, &ml, &o);
          s = *ml;
        }
        float top = s.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = fmaxf(top, mx);
        const float ref = top == -INFINITY ? 0.f : top, alpha = exp2f(mx - ref), f = exp2f(s.x - ref);
        mx = top;
        float part_l = f * s.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) part_l += __shfl_xor_sync(0xffffffffu, part_l, d);
        l = l * alpha + part_l;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= alpha;
        const int count = min(32, (n - i0 + split - 1) / split);
#pragma unroll 8
        for (int k = 0; k < count; ++k) {
          const float fk = __shfl_sync(0xffffffffu, f, k);
          const float* ok = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(o), k));
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          fetch(ok, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] += fk * v[e];
        }
      }
    }
    if (split > 1) {  // (one round of the loop: the rows' warps are all here)
      if (lane == 0) sum_l[warp] = mx;
      __syncthreads();
      float top = -INFINITY;
      for (int k = 0; k < split; ++k) top = fmaxf(top, sum_l[warp - share + k]);
      const float f = exp2f(mx - (top == -INFINITY ? 0.f : top));
      mx = top;
      __syncthreads();
      if (lane == 0) sum_l[warp] = l * f;
#pragma unroll
      for (int e = 0; e < 4; ++e) sums[warp][QUADS ? (4 * lane + e) : (lane + 32 * e)] = x[e] * f;
      __syncthreads();
      if (share != 0) continue;
      l = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = 0.f;
      for (int k = 0; k < split; ++k) {
        l += sum_l[warp + k];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += sums[warp + k][QUADS ? (4 * lane + e) : (lane + 32 * e)];
      }
    }
    if (on) store(w.at, mx, l, x);
  }
}

// ---------------------------------------------------------------- host
cudaError_t launch_after(const void* kernel, dim3 grid, unsigned threads, size_t smem, cudaStream_t st, void** args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

template <typename T, bool QUADS>
const void* join_of(bool bulk) {
  return bulk ? reinterpret_cast<const void*>(extend_join<T, QUADS, true>)
              : reinterpret_cast<const void*>(extend_join<T, QUADS, false>);
}

// The SMs of a device, looked up once.
cudaError_t sm_count_of(int dev, int* n_sm) {
  static std::atomic<int> known[kExtDevices];
  if (dev < kExtDevices && (*n_sm = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  const cudaError_t e = cudaDeviceGetAttribute(n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < kExtDevices) known[dev].store(*n_sm, std::memory_order_relaxed);
  return e;
}

cudaError_t launch_extend_simt(ExtArgs& A, cudaStream_t st) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(A.q) | reinterpret_cast<uintptr_t>(A.k_pages) |
                      reinterpret_cast<uintptr_t>(A.v_pages);
  int vec = p % 16 == 0 && A.dh % 4 == 0 && A.page_stride % 4 == 0 && A.slot_stride % 4 == 0 && A.head_stride % 4 == 0;
  const void* kernel = A.dh > 64 ? reinterpret_cast<const void*>(extend_simt<2>) : reinterpret_cast<const void*>(extend_simt<1>);
  const int smem = simt_floats(A.dh) * 4;
  static std::atomic<bool> done[2][kExtDevices];  // (allowed once, for the largest head of each kernel)
  const cudaError_t e = ext_allow_smem(kernel, simt_floats(A.dh > 64 ? 128 : 64) * 4, done[A.dh > 64 ? 1 : 0]);
  if (e != cudaSuccess) return e;
  void* args[] = {&A, &vec};
  return launch_after(kernel, dim3(A.part[kExtMany].most_ctas), kSimtThreads, smem, st, args);
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
  // what a block takes beside its tiles: its rows and first keys come from memory, its sums go there. bf16:
  // about four whole tiles (16 questions of up to 300 tokens behind 16384 shared keys, 32/8 heads of 128,
  // the prefix shared: 1287 us at 1 unit, 761 at 4, 661 at 8; 12 and 16 no faster). float32: little of a
  // tile, which is ten times longer (16 sequences of up to 16 tokens, 16/16 heads of 64: 39 us at 0, 43 at 1,
  // 45 at 2; a prompt of 695 tokens, 32/8 heads of 48: 111, 111 and 119).
  s.lead = dtype == RA_BF16 ? 8 : 0;
  // (8 prompts of up to 30 tokens, 32/8 heads of 128: 31 us at 2, 24 at 3, from 4 the same; one of 200 behind
  // 500: 39, 39, 41 at 4, 45 at 8)
  s.least = dtype == RA_BF16 ? 3 : 1;
  s.shift = dtype == RA_BF16 ? 7 : 6;
  s.window = window;
  s.sinks = sinks;
  return s;
}

// Rows of a K/V head up to which a segment goes to the kernel for few rows, bf16: 16, or 8 where the
// sequences have no more than that on average and the kernel for 8 rows, which is faster, will do.
int few_rows_of(const ra_paged_cache* c, bool decode, int n_tokens, int hq) {
  const int group = hq / c->hkv;
  if (c->dtype != RA_BF16 || group > kExtFewRows || c->n_seqs == 0) return 0;
  const int64_t rows = (decode ? 1 : (static_cast<int64_t>(n_tokens) + c->n_seqs - 1) / c->n_seqs) * group;
  return rows <= 8 ? 8 : kExtFewRows;
}

// One new token of every sequence, and so small a cache that the attention of one token (ra_decode.cu),
// which reads every sequence's keys by itself and has half the launches, is faster, whatever the
// sequences share. It is what the block table has room for that decides, as the lengths are on the
// device: with a table much wider than the sequences are long, steps that would be faster apart are
// not read apart. Measured with tables of the sequences' lengths and one prefix (us apart and shared), 32/8 heads of
// 128, bf16: 16 sequences of 2048 keys, 138 MB, 28 and 39; 16 of 4096, 273 MB, 41 and 36; 32 of 4096,
// 545 MB, 68 and 39. 8/8 heads of 64: 32 of 4096, 273 MB, 43 and 35. float32, 16/4 heads of 64: 32 of 2048, 138 MB,
// 39 and 45; 32 of 4096, 273 MB, 61 and 51.
bool read_apart(const ra_paged_cache* c) {
  const double keys = static_cast<double>(c->n_seqs) * c->max_pages * c->page_size;
  return keys * c->hkv * c->head_dim * (c->dtype == RA_BF16 ? 2 : 4) * 2 <= 256e6;
}

// The workspace's regions, one after the other.
struct Regions {
  size_t segs, starts[2], part_o[2], part_ml[2], row_o, row_ml, total;
  int rows[2], ctas[2];  // of the parts of each class
};
Regions regions_of(const ra_paged_cache* c, int n_groups, int n_tokens, int hq) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  int hb, blocks;
  head_blocks(hq / c->hkv, c->dtype == RA_BF16 ? 128 : kSimtRows, &hb, &blocks);
  const ExtShape s = shape_of(c->dtype, hb, 0, 0);
  Regions r;
  r.ctas[kExtMany] = (c->dtype == RA_BF16 ? 1 : simt_ctas(c->head_dim)) * kExtSms;
  r.rows[kExtMany] = (n_tokens < s.bt ? n_tokens : s.bt) * hb;
  r.ctas[kExtFew] = c->dtype == RA_BF16 ? extend_few_ctas(c->head_dim) : 0;
  r.rows[kExtFew] = r.ctas[kExtFew] > 0 ? 16 : 0;
  const size_t rows = n_groups > 0 ? size_t(2) * n_tokens * hq : 0;
  r.segs = 256;
  size_t at = r.segs + up((static_cast<size_t>(n_groups) + c->n_seqs) * sizeof(ExtSeg));
  for (int k = 0; k < 2; ++k) {
    r.starts[k] = at;
    at += up((r.ctas[k] + 1) * sizeof(ExtStart));
    const size_t parts = static_cast<size_t>(r.ctas[k]) * 2 * r.rows[k];
    r.part_o[k] = at;
    r.part_ml[k] = r.part_o[k] + up(parts * c->head_dim * 4);
    at = r.part_ml[k] + up(parts * 8);
  }
  r.row_o = at;
  r.row_ml = r.row_o + up(rows * c->head_dim * 4);
  r.total = r.row_ml + up(rows * 8);
  const size_t apart = ra_paged_workspace_bytes(c, hq);  // (see read_apart)
  if (r.total < apart) r.total = apart;
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
  unsigned int index = 0, plan = 0, few = 0;
  cudaError_t e = extend_tc_status(value, reset);
  if (e == cudaSuccess) e = extend_few_status(&few, reset);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&index, g_status_extend, sizeof index);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&plan, g_status_plan, sizeof plan);
  if (e == cudaSuccess && reset) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_status_extend, &zero, sizeof zero);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_status_plan, &zero, sizeof zero);
  }
  value[0] |= plan;
  value[1] |= index | few;
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
  if (cu_new == nullptr && (n_groups == 0 || read_apart(c)))
    return ra_paged_attn_decode(c, hq, scale, window, sinks, q, seq_lens, out, lse, workspace, workspace_bytes, stream);
  if (c->dtype == RA_BF16) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(c->k_pages) | reinterpret_cast<uintptr_t>(c->v_pages) |
                        reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out);
    if (p % 16 || c->page_stride % 8 || c->slot_stride % 8 || c->head_stride % 8)
      return record_error(RA_ERR_INVALID_ARG,
                          "bf16: q, out and pages must be 16-byte aligned, strides multiples of 8 elements");
  }
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = sm_count_of(dev, &n_sm);
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
  A.sh[kExtMany] = shape_of(c->dtype, A.hb, window, window > 0 ? sinks : 0);
  A.few_rows = few_rows_of(c, cu_new == nullptr, n_tokens, hq);
  // one block, tiles of 64 keys; its start and end take about three of them (64 sequences of up to 4 new
  // tokens and 8000 keys, 32/8 heads of 128: 250 us at 1, 225 at 2, 213 from 3 on; 100 of 2 and 3000,
  // window 300: 37, 37, 39)
  A.sh[kExtFew] = {16, 16, 1, 3, 2, 6, window, window > 0 ? sinks : 0};
  const int sms = n_sm < kExtSms ? n_sm : kExtSms;
  A.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(c->head_dim))) * 1.4426950408889634f;
  A.timeout_ns = kDefaultTimeoutNs;
  char* ws = static_cast<char*>(workspace);
  A.head = reinterpret_cast<ExtHead*>(ws);
  A.segs = reinterpret_cast<ExtSeg*>(ws + at.segs);
  for (int k = 0; k < 2; ++k) {
    A.starts[k] = reinterpret_cast<ExtStart*>(ws + at.starts[k]);
    A.part[k] = {reinterpret_cast<float*>(ws + at.part_o[k]), reinterpret_cast<float2*>(ws + at.part_ml[k]),
                 k == kExtFew ? A.few_rows : at.rows[k], at.ctas[k] / kExtSms * sms};
  }
  A.row_o = reinterpret_cast<float*>(ws + at.row_o);
  A.row_ml = reinterpret_cast<float2*>(ws + at.row_ml);
  A.out = out;
  A.lse = lse;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ExtMaps maps;
  if (c->dtype == RA_BF16 && (e = make_extend_maps(&maps, c, &A)) != cudaSuccess)
    return record_error(RA_ERR_UNSUPPORTED, "the pages' strides do not fit a tensor map");
  // the kernels that can have work
  const bool many = A.few_rows == 0 || static_cast<int64_t>(n_tokens) * A.group > A.few_rows;
  extend_plan<<<1, kPlanThreads, 0, st>>>(A);
  e = cudaGetLastError();
  if (e == cudaSuccess && A.few_rows > 0) e = launch_extend_few(A, st);
  if (e == cudaSuccess && many) e = c->dtype == RA_BF16 ? launch_extend_tc(A, maps, st) : launch_extend_simt(A, st);
  if (e == cudaSuccess) {
    // at most one block of a sequence has fewer tokens than the others
    int64_t blocks = static_cast<int64_t>(n_tokens / A.sh[kExtMany].bt) + c->n_seqs;
    if (blocks > n_tokens) blocks = n_tokens;
    void* args[] = {&A};
    const bool quads = A.dh % 4 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;  // (bf16 always)
    const bool bulk = static_cast<int64_t>(n_tokens) * A.group > static_cast<int64_t>(kJoinWarps) * c->n_seqs;
    const void* kernel = c->dtype == RA_BF16 ? join_of<__nv_bfloat16, true>(bulk)
                         : quads              ? join_of<float, true>(bulk)
                                              : join_of<float, false>(bulk);
    // (up to eight blocks an SM's share: 16 prompts of up to 300 tokens, 32/8 heads of 128, 82 us at four, 70 at
    // eight, 72 at 14, 84 at 28, as blocks whose rows need no join take their time to start too)
    const int64_t all = blocks * A.hkv * A.blocks_per_kv, most_y = (A.part[kExtMany].rows + 31) / 32;
    const int64_t y = bulk ? std::max<int64_t>(1, std::min<int64_t>(most_y, 8 * sms / all)) : 1;
    e = launch_after(kernel, dim3(static_cast<unsigned>(all), static_cast<unsigned>(y)), kJoinThreads, 0, st, args);
  }
  if (e != cudaSuccess) return record_error(RA_ERR_CUDA, "extend attention launch: %s", cudaGetErrorString(e));
  return record_error(RA_OK, "%s", "");
}
