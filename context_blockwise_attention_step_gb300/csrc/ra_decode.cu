// ra_decode.cu — attention of one new token of every sequence over a paged cache.
//
// The visible keys of all (sequence, K/V head) pairs are cut into units of 64 keys and the
// units, in order, are dealt out evenly to the CTAs: CTA i takes the units [N*i/G, N*(i+1)/G).
// So every SM gets the same share of the cache whatever the lengths, one long sequence as well
// as a ragged batch, and the host need not know the lengths. A CTA whose share covers a pair
// whole writes its result; else it writes its part of the pair (running max m, denominator l,
// unnormalised sum) to the workspace, at most two parts (the first and the last pair of its
// share). A pair is cut only where one CTA's share ends and the next one's begins, so a second
// kernel looks at these places and joins the parts of each cut pair in the order of the CTAs:
//
//   M = max m_i,  l = sum 2^(m_i - M) l_i,  out = sum 2^(m_i - M) o_i / l,
//   lse = (M + log2 l) ln 2
//
// which is the log-sum-exp merge of the ring's blocks (nanotron how-to page, "Numerically-
// Stable Output Fusion") on unnormalised parts. m counts in units of log2: scores are scaled
// by scale * log2(e).
//
// The keys a query sees: with a window, of the n = seq_lens[b] keys the first
// min(sinks, n - window) and the last min(window, n); without one all n. Both runs are read as
// one list of `vis` keys: list index i is key i for i < head, else i + skip.
//
// What bounds it is the cache's bytes: a group's query heads (<= 16) are the 16 rows of one
// m16n8k16 product, so that the tensor cores are 18 % busy with mma.sync and a wider instruction
// would only have more empty rows. The join kernel is launched while the main one runs
// (programmatic dependent launch), works out what it has to join, and then waits for the main
// kernel's end. Measured on GB300 with 32/8 heads of 128, bf16: one sequence of 131072 keys 91 us
// (5.9 TB/s), 64 ragged ones of up to 16384 keys 335 to 345 us (6.2 to 6.4 TB/s), one of 700 keys 7.5
// us, which is two launches and one trip to memory each.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "ra_internal.h"
#include "ra_ptx.cuh"

namespace ra {

static __device__ unsigned int g_status_decode;

namespace {

constexpr int kUnit = 64;       // keys of a unit
constexpr int kSms = 152;
constexpr int kMaxPerSm = 3;
constexpr int kMaxCtas = kMaxPerSm * kSms;
constexpr int kThreads = 128;
constexpr int kJoinThreads = 256;

struct DecodeArgs {
  const void* q;
  const void* k_pages;
  const void* v_pages;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int64_t table_stride, page_stride, slot_stride, head_stride;
  int32_t n_seqs, max_pages, page_size, n_pages;
  int32_t hq, hkv, group, dh;
  int32_t blocks_per_kv;  // blocks of query heads of one K/V head
  int32_t block_heads;    // query heads of a block (the last block may have fewer)
  int32_t window, sinks;
  float scale_log2;
  float* parts;  // [CTA][2] parts of block_heads * (dh + 2) floats
  void* out;
  float* lse;
};

template <typename T> __device__ __forceinline__ void stv(T* p, float v);
template <> __device__ __forceinline__ void stv<float>(float* p, float v) { *p = v; }
template <> __device__ __forceinline__ void stv<__nv_bfloat16>(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}

struct Visible {
  int vis, head, skip;  // keys seen; of these the first `head` are keys 0.. , the rest skip + i
};

__device__ __forceinline__ Visible visible(const DecodeArgs& A, int b, bool flag) {
  int n = A.seq_lens[b];
  const int64_t cap = static_cast<int64_t>(A.max_pages) * A.page_size;
  if (n < 0 || n > cap) {
    if (flag) atomicOr(&g_status_decode, 1u);
    n = n < 0 ? 0 : static_cast<int>(cap);
  }
  Visible v;
  v.vis = n;
  v.head = n;
  v.skip = 0;
  if (A.window > 0 && n > A.window) {
    v.head = min(A.sinks, n - A.window);
    v.skip = n - A.window - v.head;
    v.vis = A.window + v.head;
  }
  return v;
}

__device__ __forceinline__ int units_of(const DecodeArgs& A, int b) {
  return (visible(A, b, false).vis + kUnit - 1) / kUnit;
}

// Row (token) of key list index i of sequence b: element offset of its K/V head 0.
__device__ __forceinline__ int64_t key_row(const DecodeArgs& A, int b, const Visible& v, int i) {
  const int key = i < v.head ? i : i + v.skip;
  const int page = key / A.page_size;
  int at = A.block_table[b * A.table_stride + page];
  if (at < 0 || at >= A.n_pages) {
    atomicOr(&g_status_decode, 1u);
    at = 0;
  }
  return at * A.page_stride + static_cast<int64_t>(key - page * A.page_size) * A.slot_stride;
}

// CTAs that get work, and the first unit of CTA i.
__device__ __forceinline__ int active_ctas(int64_t units, int ctas) {
  return units < ctas ? static_cast<int>(units) : ctas;
}
__device__ __forceinline__ int64_t first_unit(int64_t units, int ctas, int i) { return units * i / ctas; }
// The CTA that has unit u: the largest i with first_unit(i) <= u.
__device__ __forceinline__ int cta_of(int64_t units, int ctas, int64_t u) {
  return static_cast<int>(((u + 1) * ctas - 1) / units);
}

// A walk over the pieces of a CTA's share: (sequence, block of query heads) and a range of its
// units. `u` is the next unit; the sequence is found once and then stepped.
struct Share {
  int64_t u, end;       // units of the share left
  int64_t base;         // first unit of the current pair
  int b, pair, units;   // sequence, pair within it (hk * blocks_per_kv + block), its units
};

// The share of CTA `cta` of `grid`, worked out by the block's THREADS threads; false if it is empty.
// `scan`: 8 values in shared memory.
template <int THREADS>
__device__ __forceinline__ bool share_of(const DecodeArgs& A, int cta, int grid, Share& S, int64_t* scan,
                                         int64_t* total, int* ctas) {
  const int tid = threadIdx.x;
  const int per = A.hkv * A.blocks_per_kv;
  const int chunk = (A.n_seqs + THREADS - 1) / THREADS;
  const int b0 = min(A.n_seqs, tid * chunk), b1 = min(A.n_seqs, b0 + chunk);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += units_of(A, b);
  // inclusive scan over the warp, then over the warps
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if ((tid & 31) >= o) x += y;
  }
  if ((tid & 31) == 31) scan[tid >> 5] = x;
  __syncthreads();
  int64_t before = 0, sum = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < tid >> 5) before += scan[w];
    sum += scan[w];
  }
  before += x - mine;  // units (per pair) before this thread's sequences
  const int64_t units = sum * per;
  *total = units;
  *ctas = active_ctas(units, grid);
  __syncthreads();
  if (cta >= *ctas) return false;
  S.u = first_unit(units, *ctas, cta);
  S.end = first_unit(units, *ctas, cta + 1);
  // the thread whose sequences hold unit S.u finds the pair
  if (S.u >= before * per && S.u < (before + mine) * per) {
    int64_t base = before * per;
    int b = b0, n = units_of(A, b);
    while (S.u >= base + static_cast<int64_t>(n) * per) {
      base += static_cast<int64_t>(n) * per;
      n = units_of(A, ++b);
    }
    const int pair = static_cast<int>((S.u - base) / n);
    scan[0] = base + static_cast<int64_t>(pair) * n;
    scan[1] = b;
    scan[2] = pair;
    scan[3] = n;
  }
  __syncthreads();
  S.base = scan[0];
  S.b = static_cast<int>(scan[1]);
  S.pair = static_cast<int>(scan[2]);
  S.units = static_cast<int>(scan[3]);
  return true;
}

// To the next pair with keys (the caller has checked that units are left).
__device__ __forceinline__ void share_next(const DecodeArgs& A, Share& S) {
  S.base += S.units;
  S.u = S.base;
  if (++S.pair == A.hkv * A.blocks_per_kv) {
    S.pair = 0;
    do {
      S.units = units_of(A, ++S.b);
    } while (S.units == 0);
  }
}

// A main CTA's start: lets the join kernel launch, finds its share of the units.
__device__ __forceinline__ bool share_begin(const DecodeArgs& A, Share& S, int64_t* scan) {
  launch_dependents();
  int64_t total;
  int ctas;
  return share_of<kThreads>(A, blockIdx.x, gridDim.x, S, scan, &total, &ctas);
}

// A main CTA's end: the results of its part of the idle sequences (lengths outside the cache are
// reported here too). 32 sequences a warp at once.
template <typename T>
__device__ __forceinline__ void finish_idle(const DecodeArgs& A) {
  const int lane = threadIdx.x & 31, step = gridDim.x * (kThreads / 32);
  for (int b0 = blockIdx.x + gridDim.x * (threadIdx.x >> 5); b0 < A.n_seqs; b0 += 32 * step) {
    const int b = b0 + lane * step;
    unsigned idle = __ballot_sync(0xffffffffu, b < A.n_seqs && visible(A, b, true).vis == 0);
    for (; idle != 0; idle &= idle - 1) {
      const int64_t row = static_cast<int64_t>(b0 + (__ffs(idle) - 1) * step) * A.hq;
      for (int i = lane; i < A.hq * A.dh; i += 32) stv<T>(static_cast<T*>(A.out) + row * A.dh + i, 0.f);
      for (int h = lane; h < A.hq; h += 32) A.lse[row + h] = -INFINITY;
    }
  }
}

__device__ __forceinline__ float* part_of(const DecodeArgs& A, int cta, int which) {
  return A.parts + (static_cast<int64_t>(cta) * 2 + which) * A.block_heads * (A.dh + 2);
}

// ---------------------------------------------------------------- CUDA cores, any head size
// N sums over the 32 lanes at once: every halving step adds the partner's half and keeps half
// of the values, so N values cost N - 1 shuffles and 5 - log2(N) more. Lane l ends up with
// value l / (32 / N).
template <int N>
__device__ __forceinline__ float lane_sums(float (&x)[N], int lane) {
#pragma unroll
  for (int n = N, o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool hi = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i < n) {
          const float send = hi ? x[i] : x[i + n];
          const float keep = hi ? x[i + n] : x[i];
          x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
    } else {
      x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
    }
  }
  return x[0];
}


// 1 / l; a query whose every score is -inf has l = 0 and gets out = 0, lse = -inf.
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

__device__ __forceinline__ void store_lse(const DecodeArgs& A, int b, int h, float m, float l) {
  A.lse[static_cast<int64_t>(b) * A.hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// The four warps' states of a block of query heads into the result of the pair, or into a part of it
// (units u0 .. u1 - 1).
template <int HB, int W>
__device__ __forceinline__ void store_pair(const DecodeArgs& A, const Share& S, int64_t share0, int u0, int u1, int h0,
                                           int heads, const float (&sm_m)[4][HB], const float (&sm_l)[4][HB],
                                           const float (&sm_o)[4][HB][W]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dh = A.dh;
  const bool whole = u0 == 0 && u1 == S.units;
  float* part = part_of(A, blockIdx.x, S.u == share0 ? 0 : 1);
  for (int h = warp; h < heads; h += 4) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sm_m[w][h]);
    const float ref = M == -INFINITY ? 0.f : M;
    float f[4], L = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      f[w] = exp2f(sm_m[w][h] - ref);
      L += f[w] * sm_l[w][h];
    }
    const float inv = whole ? inverse(L) : 1.f;
    for (int d = lane; d < dh; d += 32) {
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) x += f[w] * sm_o[w][h][d];
      if (whole)
        static_cast<float*>(A.out)[(static_cast<int64_t>(S.b) * A.hq + h0 + h) * dh + d] = x * inv;
      else
        part[h * (dh + 2) + d] = x;
    }
    if (lane == 0) {
      if (whole) {
        store_lse(A, S.b, h0 + h, M, L);
      } else {
        part[h * (dh + 2) + dh] = M;
        part[h * (dh + 2) + dh + 1] = L;
      }
    }
  }
}

// Float32, any size and alignment (decode_f32 takes what it can). Four warps, each 16 keys of a unit, four keys at a time; lane l holds elements l, l + 32, ...
// of q, of the keys and of the sums, for HB query heads.
template <int HB>
__global__ void __launch_bounds__(kThreads, HB == 8 ? 2 : 3) decode_simt(const __grid_constant__ DecodeArgs A) {
  constexpr int NI = 4;  // elements per lane: head_dim <= 128
  __shared__ int64_t scan[8];
  __shared__ float sm_m[4][HB], sm_l[4][HB], sm_o[4][HB][128];
  Share S;
  const bool some = share_begin(A, S, scan);
  const int64_t share0 = S.u;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dh = A.dh;
  const float* kp = static_cast<const float*>(A.k_pages);
  const float* vp = static_cast<const float*>(A.v_pages);
  while (some) {
    const int hk = S.pair / A.blocks_per_kv, blk = S.pair % A.blocks_per_kv;
    const int g0 = blk * HB, heads = min(HB, A.group - g0), h0 = hk * A.group + g0;
    const Visible vis = visible(A, S.b, true);
    const int u0 = static_cast<int>(S.u - S.base);
    const int u1 = static_cast<int>(min(static_cast<int64_t>(S.units), S.end - S.base));
    float qr[HB][NI], o[HB][NI], m[HB], l[HB];
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int d = lane + 32 * i;
        o[h][i] = 0.f;
        qr[h][i] = h < heads && d < dh
                       ? *(static_cast<const float*>(A.q) + (static_cast<int64_t>(S.b) * A.hq + h0 + h) * dh + d)
                       : 0.f;
      }
    }
    // four keys at a time, the next four loaded meanwhile (step i: keys 4i .. 4i+3 of this warp's 16
    // of unit u0 + i/4)
    float kr[4][NI], vr[4][NI];
    auto first_key = [&](int i) { return (u0 + (i >> 2)) * kUnit + warp * 16 + (i & 3) * 4; };
    auto fetch = [&](int i) {
      const int key0 = first_key(i);
      if (i >= 4 * (u1 - u0) || key0 >= vis.vis) return;
      int64_t row = 0;
      if (lane < 4) row = key_row(A, S.b, vis, min(key0 + lane, vis.vis - 1)) + hk * A.head_stride;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = __shfl_sync(0xffffffffu, row, j);
#pragma unroll
        for (int e = 0; e < NI; ++e) {
          const int d = lane + 32 * e;
          kr[j][e] = d < dh ? kp[at + d] : 0.f;
          vr[j][e] = d < dh ? vp[at + d] : 0.f;
        }
      }
    };
    fetch(0);
    for (int i = 0; i < 4 * (u1 - u0); ++i) {
      const int key0 = first_key(i);
      float s[4 * HB], vc[4][NI];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          float x = 0.f;
#pragma unroll
          for (int e = 0; e < NI; ++e) x += qr[h][e] * kr[j][e];
          s[j * HB + h] = x;
        }
#pragma unroll
        for (int e = 0; e < NI; ++e) vc[j][e] = vr[j][e];
      }
      fetch(i + 1);
      if (key0 >= vis.vis) continue;
      const float mine = lane_sums<4 * HB>(s, lane) * A.scale_log2;
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        float x[4], mx = m[h];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = __shfl_sync(0xffffffffu, mine, (j * HB + h) * (32 / (4 * HB)));
          if (key0 + j >= vis.vis) x[j] = -INFINITY;
          mx = fmaxf(mx, x[j]);
        }
        const float ref = mx == -INFINITY ? 0.f : mx;
        const float alpha = exp2f(m[h] - ref);
        m[h] = mx;
        l[h] *= alpha;
#pragma unroll
        for (int e = 0; e < NI; ++e) o[h][e] *= alpha;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(x[j] - ref);
          l[h] += p;
#pragma unroll
          for (int e = 0; e < NI; ++e) o[h][e] += key0 + j < vis.vis ? p * vc[j][e] : 0.f;
        }
      }
    }
    // the four warps' states into one
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      if (lane == 0) {
        sm_m[warp][h] = m[h];
        sm_l[warp][h] = l[h];
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) sm_o[warp][h][lane + 32 * i] = o[h][i];
    }
    __syncthreads();
    store_pair<HB, 128>(A, S, share0, u0, u1, h0, heads, sm_m, sm_l, sm_o);
    __syncthreads();
    if (S.base + S.units >= S.end) break;
    share_next(A, S);
  }
  finish_idle<float>(A);
}

// Float32 in 16-byte loads: LANES lanes take a key, lane c of a key the pieces c, c + LANES, ... of
// four elements (E of them; head_dim <= 4 LANES E). The lanes of a key keep a state of their own, so
// that a weight is worked out once a key and not once a lane, and the states are joined when the
// pair ends. Keys are loaded a step ahead, their places in the table two. What bounds it is the products'
// instructions: 16 sequences of 8192 keys of 128, 32/8 heads 203 us (5.3 TB/s), 8/8 heads 166 us
// (6.5 TB/s), where decode_simt takes 300 and 260.
template <int HB, int E, int LANES>
__global__ void __launch_bounds__(kThreads, HB * E > 8 ? 2 : 3) decode_f32(const __grid_constant__ DecodeArgs A) {
  __shared__ int64_t scan[8];
  __shared__ float sm_m[4][HB], sm_l[4][HB];
  __shared__ __align__(16) float sm_o[4][HB][4 * LANES * E];
  constexpr int KEYS = 32 / LANES, SPLIT = 16 / KEYS;  // a warp's keys at a time, steps of its 16 of a unit
  Share S;
  const bool some = share_begin(A, S, scan);
  const int64_t share0 = S.u;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % LANES, dh = A.dh;
  const float* kp = static_cast<const float*>(A.k_pages);
  const float* vp = static_cast<const float*>(A.v_pages);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  auto has = [&](int e) { return 4 * (c + LANES * e) < dh; };
  while (some) {
    const int hk = S.pair / A.blocks_per_kv, blk = S.pair % A.blocks_per_kv;
    const int g0 = blk * HB, heads = min(HB, A.group - g0), h0 = hk * A.group + g0;
    const Visible vis = visible(A, S.b, true);
    const int u0 = static_cast<int>(S.u - S.base);
    const int u1 = static_cast<int>(min(static_cast<int64_t>(S.units), S.end - S.base));
    float4 q[HB][E], o[HB][E];
    float m[HB], l[HB];
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      const float* row = static_cast<const float*>(A.q) + (static_cast<int64_t>(S.b) * A.hq + h0 + h) * dh;
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o[h][e] = zero;
        q[h][e] = h < heads && has(e) ? *reinterpret_cast<const float4*>(row + 4 * (c + LANES * e)) : zero;
      }
    }
    const int steps = SPLIT * (u1 - u0);
    auto key_of = [&](int i) { return (u0 + i / SPLIT) * kUnit + warp * 16 + i % SPLIT * KEYS + lane / LANES; };
    auto seen = [&](int i) { return i < steps && key_of(i) < vis.vis; };
    auto place = [&](int i) { return seen(i) ? key_row(A, S.b, vis, key_of(i)) + hk * A.head_stride : int64_t(-1); };
    float4 kn[E], vn[E];
    auto load = [&](int64_t at) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool in = at >= 0 && has(e);
        kn[e] = in ? *reinterpret_cast<const float4*>(kp + at + 4 * (c + LANES * e)) : zero;
        vn[e] = in ? *reinterpret_cast<const float4*>(vp + at + 4 * (c + LANES * e)) : zero;
      }
    };
    load(place(0));
    int64_t next = place(1);
    for (int i = 0; i < steps; ++i) {
      float4 v[E];
      float x[HB];
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        x[h] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          x[h] += q[h][e].x * kn[e].x;
          x[h] += q[h][e].y * kn[e].y;
          x[h] += q[h][e].z * kn[e].z;
          x[h] += q[h][e].w * kn[e].w;
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = vn[e];
      load(next);
      next = place(i + 2);
      const bool hidden = !seen(i);
#pragma unroll
      for (int h = 0; h < HB; ++h) {
#pragma unroll
        for (int w = LANES / 2; w > 0; w >>= 1) x[h] += __shfl_xor_sync(0xffffffffu, x[h], w);
        x[h] = hidden ? -INFINITY : x[h] * A.scale_log2;
        const float mx = fmaxf(m[h], x[h]), ref = mx == -INFINITY ? 0.f : mx;
        if (__any_sync(0xffffffffu, mx > m[h])) {
          const float alpha = exp2f(m[h] - ref);
          m[h] = mx;
          l[h] *= alpha;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            o[h][e].x *= alpha;
            o[h][e].y *= alpha;
            o[h][e].z *= alpha;
            o[h][e].w *= alpha;
          }
        }
        const float p = exp2f(x[h] - ref);  // 0 for a hidden key, whose v is 0 too
        l[h] += p;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          o[h][e].x += p * v[e].x;
          o[h][e].y += p * v[e].y;
          o[h][e].z += p * v[e].z;
          o[h][e].w += p * v[e].w;
        }
      }
    }
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      float M = m[h];
#pragma unroll
      for (int w = LANES; w < 32; w <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
      const float f = exp2f(m[h] - (M == -INFINITY ? 0.f : M));
      l[h] *= f;
#pragma unroll
      for (int w = LANES; w < 32; w <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float y[4] = {o[h][e].x * f, o[h][e].y * f, o[h][e].z * f, o[h][e].w * f};
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int w = LANES; w < 32; w <<= 1) y[n] += __shfl_xor_sync(0xffffffffu, y[n], w);
        if (lane < LANES) *reinterpret_cast<float4*>(&sm_o[warp][h][4 * (c + LANES * e)]) = make_float4(y[0], y[1], y[2], y[3]);
      }
      if (lane == 0) {
        sm_m[warp][h] = M;
        sm_l[warp][h] = l[h];
      }
    }
    __syncthreads();
    store_pair<HB, 4 * LANES * E>(A, S, share0, u0, u1, h0, heads, sm_m, sm_l, sm_o);
    __syncthreads();
    if (S.base + S.units >= S.end) break;
    share_next(A, S);
  }
  finish_idle<float>(A);
}

// ---------------------------------------------------------------- bf16: matrix instructions
// Memory-bound: 4 * dh bytes of K and V per key and K/V head, whose 2 * heads * dh products go
// through mma.sync m16n8k16 with the query heads of the K/V head as its 16 rows (the rows
// beyond them are zero; tcgen05's 64 or 128 rows would be emptier still, and its operands would
// have to go through shared memory in whole 128-row tiles). A warp takes 16 keys of each unit
// and is on its own until its share of a pair is done: it copies its keys' rows by cp.async
// into its own ring of stages (rows 16 bytes longer than the data, so that ldmatrix meets every
// bank once), the page of the next tile's keys looked up while the copies of this one fly, and
// keeps running max, sum and O = P V in registers. The ring runs on over the end of a pair.
// S = Q K^T as [heads x keys], so that P is the A operand of P V without any exchange. O is
// rescaled only when a row's max grows by more than 2^8 (the same values in exact arithmetic).
// P is given to the product as two bf16 numbers, its rounding and the rounding of what that leaves
// out: 2^-16 of P, so that the result's own rounding is the only one that shows (one bf16 number
// alone put 0.0012 of `out` beside that rounding's 0.0017, relative L2). Up to 8 query heads the
// second number takes the product's empty rows and costs no instruction. The sums of the second
// numbers are kept apart until a pair ends, for an infinite v takes its sign from P alone: there
// they count for nothing. P's own sum is taken before, in float32.
//
// WIDE: more than 8 query heads per K/V head (rows 8..15 of the products are used).
template <int DH, bool WIDE>
struct MmaCfg {
  static constexpr int PITCH = DH * 2 + 16;                  // bytes of a key's row in a stage
  static constexpr int STAGE = 2 * 16 * PITCH;               // a warp's K and V of 16 keys
  // Measured on GB300 (ragged batch of 64, heads of 128; windowed batch of 33, heads of 64): two
  // stages and two CTAs an SM 343 us, three stages 349, five and one CTA 419; heads of 64 three
  // stages and three CTAs 17 us, two CTAs 20.
  static constexpr int STAGES = DH == 128 ? 2 : 3;
  static constexpr int CTAS = DH == 128 ? 2 : 3;             // on an SM
  static constexpr int RING = 4 * STAGES * STAGE;
  static constexpr int CHUNK = 8192 / (4 * DH * 4);          // rows joined at a time
  static constexpr int SMEM = RING + 8192;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A walk over the tiles of a CTA's share: the pieces (pairs) of the share, and their units.
struct Cursor {
  Share S;
  Visible vis;
  int hk, blk;  // K/V head, block of its query heads
  int u, u1;    // next unit and last + 1 of this piece
  bool more;

  __device__ __forceinline__ void piece(const DecodeArgs& A, bool flag) {
    hk = S.pair / A.blocks_per_kv;
    blk = S.pair - hk * A.blocks_per_kv;
    vis = visible(A, S.b, flag);
    u = static_cast<int>(S.u - S.base);
    u1 = static_cast<int>(min(static_cast<int64_t>(S.units), S.end - S.base));
  }
  __device__ __forceinline__ void begin(const DecodeArgs& A, const Share& share, bool flag) {
    S = share;
    more = true;
    piece(A, flag);
  }
  __device__ __forceinline__ void next_piece(const DecodeArgs& A, bool flag) {
    if (S.base + S.units >= S.end) {
      more = false;
      return;
    }
    share_next(A, S);
    piece(A, flag);
  }
};

template <int DH, bool WIDE>
__global__ void __launch_bounds__(kThreads, (MmaCfg<DH, WIDE>::CTAS)) decode_mma(const __grid_constant__ DecodeArgs A) {
  using C = MmaCfg<DH, WIDE>;
  constexpr int KS = DH / 16;                  // steps of 16 elements
  constexpr int LANES = DH * 2 / 16;           // lanes that copy one row
  constexpr int ROWS = 32 / LANES;             // rows of one copy instruction
  constexpr int NS = C::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scan[8];
  __shared__ float sm_m[4][16], sm_l[4][16];
  Share share;
  if (!share_begin(A, share, scan)) {
    finish_idle<__nv_bfloat16>(A);
    return;
  }
  const int64_t share0 = share.u;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * NS * C::STAGE;
  float* joined = reinterpret_cast<float*>(smem + C::RING);  // [4][CHUNK][DH]
  const char* kp = static_cast<const char*>(A.k_pages);
  const char* vp = static_cast<const char*>(A.v_pages);

  // the load side: rows of the next tile's keys (lane i: key i; -1: no tile), then its copies
  Cursor load;
  load.begin(A, share, true);
  int64_t row = -1;
  auto look_up = [&]() {
    row = -1;
    if (!load.more) return;
    const int key0 = load.u * kUnit + warp * 16;
    if (key0 < load.vis.vis)
      row = (key_row(A, load.S.b, load.vis, min(key0 + (lane & 15), load.vis.vis - 1)) + load.hk * A.head_stride) * 2;
    if (++load.u == load.u1) load.next_piece(A, true);
  };
  auto copy = [&](int stage) {
    if (__shfl_sync(0xffffffffu, row, 0) >= 0) {
      const uint32_t dst = ring + stage * C::STAGE + (lane / LANES) * C::PITCH + (lane % LANES) * 16;
#pragma unroll
      for (int i = 0; i < 16 / ROWS; ++i) {
        const int64_t at = __shfl_sync(0xffffffffu, row, i * ROWS + lane / LANES) + (lane % LANES) * 16;
        cp_async16(dst + i * ROWS * C::PITCH, kp + at);
        cp_async16(dst + i * ROWS * C::PITCH + 16 * C::PITCH, vp + at);
      }
    }
    cp_async_commit();
  };
  look_up();
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) {
    copy(i);
    look_up();
  }

  int stage = 0;
  Cursor at;
  at.begin(A, share, false);
  while (at.more) {
    const int heads = min(A.block_heads, A.group - at.blk * A.block_heads);
    const int h0 = at.hk * A.group + at.blk * A.block_heads;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(A.q) + (static_cast<int64_t>(at.S.b) * A.hq + h0) * DH;
    uint32_t qa[KS][WIDE ? 4 : 2];
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int i = 0; i < (WIDE ? 4 : 2); ++i) {  // i: element half, then row half
        const int r = g + (i >> 1) * 8, d = 16 * k + (i & 1) * 8 + 2 * c;
        qa[k][i] = r < heads ? *reinterpret_cast<const uint32_t*>(q + r * DH + d) : 0u;
      }
    float o[DH / 8][4], small[DH / 8][4];  // P V, and that of P's second numbers (not WIDE: o's rows 8..15)
#pragma unroll
    for (int n = 0; n < DH / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = small[n][i] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    const int u0 = at.u;
    for (; at.u < at.u1; ++at.u) {
      copy(stage == 0 ? NS - 1 : stage - 1);
      look_up();
      cp_async_wait<NS - 1>();
      __syncwarp();
      const int key0 = at.u * kUnit + warp * 16;
      if (key0 < at.vis.vis) {
        const uint32_t ks = ring + stage * C::STAGE, vs = ks + 16 * C::PITCH;
        float s[2][4] = {};
        const uint32_t ka = ks + ((lane & 7) + (lane >> 4) * 8) * C::PITCH + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t b[4];
          ldmatrix4(b, ka + k * 32);
          if constexpr (WIDE) {
            mma_bf16(s[0], qa[k][0], qa[k][2], qa[k][1], qa[k][3], b[0], b[1]);
            mma_bf16(s[1], qa[k][0], qa[k][2], qa[k][1], qa[k][3], b[2], b[3]);
          } else {
            mma_bf16(s[0], qa[k][0], 0u, qa[k][1], 0u, b[0], b[1]);
            mma_bf16(s[1], qa[k][0], 0u, qa[k][1], 0u, b[2], b[3]);
          }
        }
        uint32_t p[2][2], rest[2][2];  // [row half][key half]
        const bool part = key0 + 16 > at.vis.vis;
#pragma unroll
        for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = s[i >> 1][2 * r + (i & 1)] * A.scale_log2;
            if (part && key0 + (i >> 1) * 8 + 2 * c + (i & 1) >= at.vis.vis) x[i] = -INFINITY;
          }
          float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const bool grow = mx > m[r] + 8.f;  // also of the first finite score
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = grow ? (m[r] == -INFINITY ? 0.f : ex2(m[r] - mx)) : 1.f;
            if (grow) m[r] = mx;
            l[r] *= alpha;
#pragma unroll
            for (int n = 0; n < DH / 8; ++n) {
              o[n][2 * r] *= alpha;
              o[n][2 * r + 1] *= alpha;
              (WIDE ? small[n][2 * r] : o[n][2]) *= alpha;
              (WIDE ? small[n][2 * r + 1] : o[n][3]) *= alpha;
            }
          }
          const float ref = m[r] == -INFINITY ? 0.f : m[r];
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = ex2(x[i] - ref);
          l[r] += (e[0] + e[1]) + (e[2] + e[3]);
          p[r][0] = pack_bf16x2(e[0], e[1]);
          p[r][1] = pack_bf16x2(e[2], e[3]);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            rest[r][i] = pack_bf16x2(e[2 * i] - __uint_as_float(p[r][i] << 16),
                                     e[2 * i + 1] - __uint_as_float(p[r][i] & 0xffff0000u));
        }
        const uint32_t va = vs + ((lane & 7) + ((lane >> 3) & 1) * 8) * C::PITCH + (lane >> 4) * 16;
#pragma unroll
        for (int d = 0; d < KS; ++d) {
          uint32_t b[4];
          ldmatrix4_trans(b, va + d * 32);
          if constexpr (WIDE) {
            mma_bf16(o[2 * d], p[0][0], p[1][0], p[0][1], p[1][1], b[0], b[1]);
            mma_bf16(o[2 * d + 1], p[0][0], p[1][0], p[0][1], p[1][1], b[2], b[3]);
            mma_bf16(small[2 * d], rest[0][0], rest[1][0], rest[0][1], rest[1][1], b[0], b[1]);
            mma_bf16(small[2 * d + 1], rest[0][0], rest[1][0], rest[0][1], rest[1][1], b[2], b[3]);
          } else {
            mma_bf16(o[2 * d], p[0][0], rest[0][0], p[0][1], rest[0][1], b[0], b[1]);
            mma_bf16(o[2 * d + 1], p[0][0], rest[0][0], p[0][1], rest[0][1], b[2], b[3]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage: the next copy may go there
      stage = stage + 1 == NS ? 0 : stage + 1;
    }

    auto sum_of = [&](int n, int r, int i) {  // of row half r, with what is finite of the second numbers'
      const float x = WIDE ? small[n][2 * r + i] : o[n][2 + i];
      return o[n][2 * r + i] + (fabsf(x) <= 3.402823466e38f ? x : 0.f);
    };
    // the four warps' states into one, CHUNK heads at a time
#pragma unroll
    for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (c == 0) {
        sm_m[warp][g + 8 * r] = m[r];
        sm_l[warp][g + 8 * r] = l[r];
      }
    }
    const bool whole = u0 == 0 && at.u1 == at.S.units;
    float* part = part_of(A, blockIdx.x, at.S.u == share0 ? 0 : 1);
    for (int r0 = 0; r0 < heads; r0 += C::CHUNK) {
#pragma unroll
      for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
        const int h = g + 8 * r - r0;
        if (h >= 0 && h < C::CHUNK) {
#pragma unroll
          for (int n = 0; n < DH / 8; ++n)
            *reinterpret_cast<float2*>(joined + (warp * C::CHUNK + h) * DH + 8 * n + 2 * c) =
                make_float2(sum_of(n, r, 0), sum_of(n, r, 1));
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < C::CHUNK * (DH / 4); i += kThreads) {
        const int h = i / (DH / 4), d = i % (DH / 4) * 4, hh = r0 + h;
        if (hh >= heads) break;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, sm_m[w][hh]);
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = ex2(sm_m[w][hh] - ref);
          const float4 y = *reinterpret_cast<const float4*>(joined + (w * C::CHUNK + h) * DH + d);
          L += f * sm_l[w][hh];
          x.x += f * y.x;
          x.y += f * y.y;
          x.z += f * y.z;
          x.w += f * y.w;
        }
        if (whole) {
          const float inv = inverse(L);
          uint2 u;
          u.x = pack_bf16x2(x.x * inv, x.y * inv);
          u.y = pack_bf16x2(x.z * inv, x.w * inv);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(A.out) +
                                    (static_cast<int64_t>(at.S.b) * A.hq + h0 + hh) * DH + d) = u;
          if (d == 0) store_lse(A, at.S.b, h0 + hh, M, L);
        } else {
          float* to = part + hh * (DH + 2);
          *reinterpret_cast<float2*>(to + d) = make_float2(x.x, x.y);
          *reinterpret_cast<float2*>(to + d + 2) = make_float2(x.z, x.w);
          if (d == 0) {
            to[DH] = M;
            to[DH + 1] = L;
          }
        }
      }
      __syncthreads();
    }
    at.next_piece(A, false);
  }
  finish_idle<__nv_bfloat16>(A);
}

// ---------------------------------------------------------------- the join
// Units (of one pair each) before sequence b, and of all sequences, by the block's threads.
__device__ __forceinline__ void count_units(const DecodeArgs& A, int b, int64_t* before, int64_t* all,
                                            int64_t* scan) {
  int64_t lo = 0, sum = 0;
  for (int i = threadIdx.x; i < A.n_seqs; i += kJoinThreads) {
    const int u = units_of(A, i);
    sum += u;
    if (i < b) lo += u;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo += __shfl_xor_sync(0xffffffffu, lo, o);
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  if ((threadIdx.x & 31) == 0) {
    scan[threadIdx.x >> 5] = lo;
    scan[8 + (threadIdx.x >> 5)] = sum;
  }
  __syncthreads();
  *before = *all = 0;
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    *before += scan[w];
    *all += scan[8 + w];
  }
}

// The blocks that go by pairs (few pairs, of many parts): x the pair, y the query head of its block
// of heads, the eight warps every eighth part each. The blocks that go by cuts: x the pair that CTA
// x's share ends in, if it goes on in CTA x + 1 and begins in CTA x; two warps a head, four heads
// at a time. The lanes take four elements each; every sum is taken in a fixed order. (Most blocks
// start when the main kernel's end leaves room for them, so few blocks matter more than short
// ones. In all, by pairs and by cuts: one sequence of 700 keys, 8 pairs, 7.7 and 9.1 us; 16
// sequences of 8000, 32/1 heads, 27 and 43 us; 1000 sequences of 100, 32/8 heads, 230 and 112 us.)
template <typename T, bool PAIRS>
__global__ void __launch_bounds__(kJoinThreads) decode_join(const __grid_constant__ DecodeArgs A, int grid) {
  constexpr int ROWS = PAIRS ? 1 : 4, WARPS = kJoinThreads / 32 / ROWS;
  __shared__ int64_t scan[16];
  __shared__ float sums[kJoinThreads / 32][128], sm_l[kJoinThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dh = A.dh;
  Share S;
  int64_t total;
  int ctas;
  bool some;
  if constexpr (PAIRS) {
    const int per = A.hkv * A.blocks_per_kv;
    S.b = blockIdx.x / per;
    S.pair = blockIdx.x - S.b * per;
    S.units = units_of(A, S.b);
    int64_t before;
    count_units(A, S.b, &before, &total, scan);
    total *= per;
    ctas = active_ctas(total, grid);
    S.base = before * per + static_cast<int64_t>(S.pair) * S.units;
    some = S.units > 0;
  } else {  // the pair of the next CTA's first unit
    some = share_of<kJoinThreads>(A, blockIdx.x + 1, grid, S, scan, &total, &ctas) && S.base < S.u;
  }
  int c0 = 0, c1 = 0;
  if (some) {
    c0 = cta_of(total, ctas, S.base);
    c1 = cta_of(total, ctas, S.base + S.units - 1);
  }
  wait_for_previous();  // in every block: what follows in the stream waits for this kernel alone
  if (c0 == c1 || (!PAIRS && c0 != static_cast<int>(blockIdx.x))) return;  // not cut, or cut earlier
  const int hk = S.pair / A.blocks_per_kv, blk = S.pair - hk * A.blocks_per_kv;
  const int heads = min(A.block_heads, A.group - blk * A.block_heads), parts = c1 - c0 + 1;
  for (int row0 = PAIRS ? blockIdx.y : 0; row0 < heads; row0 += PAIRS ? heads : ROWS) {
    const int row = row0 + warp / WARPS, w = warp % WARPS;
    const bool mine = row < heads;
    auto part = [&](int i) {  // the pair is the first of a CTA's share, or its last
      return part_of(A, c0 + i, S.base <= first_unit(total, ctas, c0 + i) ? 0 : 1) + row * (dh + 2);
    };
    float mx = -INFINITY, l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
    if (mine) {  // every warp of a head takes the maximum of all parts
      for (int i = lane; i < parts; i += 32) mx = fmaxf(mx, part(i)[dh]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
      for (int i = w; i < parts; i += WARPS) {
        const float* p = part(i);
        const float f = exp2f(p[dh] - ref);
        l += f * p[dh + 1];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (lane + 32 * e < dh) x[e] += f * p[lane + 32 * e];
      }
    }
    if (lane == 0) sm_l[warp] = l;
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[warp][lane + 32 * e] = x[e];
    __syncthreads();
    if (mine && w == 0) {
      const int h = hk * A.group + blk * A.block_heads + row;
      l = 0.f;
      for (int k = 0; k < WARPS; ++k) l += sm_l[warp + k];
      T* out = static_cast<T*>(A.out) + (static_cast<int64_t>(S.b) * A.hq + h) * dh;
      for (int d = lane; d < dh; d += 32) {
        float s = 0.f;
        for (int k = 0; k < WARPS; ++k) s += sums[warp + k][d];
        stv<T>(out + d, s * inverse(l));
      }
      if (lane == 0) store_lse(A, S.b, h, mx, l);
    }
    __syncthreads();
  }
}

// Query heads that share one read of a K/V head: on the CUDA cores a power of two up to 8 (the
// states of 8 heads fill a thread's registers), for the matrix instructions up to their 16 rows,
// evenly.
int heads_of_block(int dtype, int group) {
  if (dtype == RA_F32) return group >= 8 ? 8 : group >= 4 ? 4 : group >= 2 ? 2 : 1;
  const int blocks = (group + 15) / 16;
  return (group + blocks - 1) / blocks;
}

int ctas_per_sm(int dtype, int dh) { return dtype == RA_F32 ? 3 : dh == 64 ? MmaCfg<64, false>::CTAS : MmaCfg<128, false>::CTAS; }

template <int DH, bool WIDE>
cudaError_t launch_mma(const DecodeArgs& A, int grid, cudaStream_t st) {
  using C = MmaCfg<DH, WIDE>;
  const cudaError_t e =
      cudaFuncSetAttribute(decode_mma<DH, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  decode_mma<DH, WIDE><<<grid, kThreads, C::SMEM, st>>>(A);
  return cudaGetLastError();
}

// Whether every row of a float32 call starts on 16 bytes.
bool wide_f32(const DecodeArgs& A) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(A.q) | reinterpret_cast<uintptr_t>(A.k_pages) |
                      reinterpret_cast<uintptr_t>(A.v_pages);
  return p % 16 == 0 && A.dh % 4 == 0 && A.page_stride % 4 == 0 && A.slot_stride % 4 == 0 && A.head_stride % 4 == 0;
}

// Lanes of a key, and pieces of a lane. Four lanes where their pieces fit the registers: half the
// steps of eight, and with them half the sums over lanes and half the weights (16 sequences of 16384
// keys of 64, 32/8 heads: 205 against 246 us).
int f32_lanes(int dh) { return dh <= 64 ? 4 : 8; }
int f32_pieces(int dh) { return (dh + 4 * f32_lanes(dh) - 1) / (4 * f32_lanes(dh)); }

template <int HB>
void launch_f32(const DecodeArgs& A, int grid, cudaStream_t st) {
  const int e = f32_pieces(A.dh);
  if (f32_lanes(A.dh) == 8) {
    if (e == 3) decode_f32<HB, 3, 8><<<grid, kThreads, 0, st>>>(A);
    else decode_f32<HB, 4, 8><<<grid, kThreads, 0, st>>>(A);
  } else {
    switch (e) {
      case 1: decode_f32<HB, 1, 4><<<grid, kThreads, 0, st>>>(A); break;
      case 2: decode_f32<HB, 2, 4><<<grid, kThreads, 0, st>>>(A); break;
      case 3: decode_f32<HB, 3, 4><<<grid, kThreads, 0, st>>>(A); break;
      default: decode_f32<HB, 4, 4><<<grid, kThreads, 0, st>>>(A); break;
    }
  }
}

template <typename T>
cudaError_t launch_join(cudaLaunchConfig_t& cfg, const DecodeArgs& A, int grid) {
  const int64_t pairs = static_cast<int64_t>(A.n_seqs) * A.hkv * A.blocks_per_kv;
  if (pairs * A.block_heads <= 4 * grid) {
    cfg.gridDim = dim3(static_cast<unsigned>(pairs), A.block_heads);
    return cudaLaunchKernelEx(&cfg, decode_join<T, true>, A, grid);
  }
  cfg.gridDim = dim3(grid - 1);
  return cudaLaunchKernelEx(&cfg, decode_join<T, false>, A, grid);
}

cudaError_t launch(DecodeArgs& A, int dtype, cudaStream_t st) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int per_sm = ctas_per_sm(dtype, A.dh);
  if (dtype == RA_F32 && (wide_f32(A) ? A.block_heads * f32_pieces(A.dh) > 8 : A.block_heads == 8))
    per_sm = 2;  // their registers
  const int grid = per_sm * (n_sm < kSms ? n_sm : kSms);
  if (dtype == RA_F32 && wide_f32(A)) {
    switch (A.block_heads) {
      case 1: launch_f32<1>(A, grid, st); break;
      case 2: launch_f32<2>(A, grid, st); break;
      default: launch_f32<4>(A, grid, st); break;
    }
    e = cudaGetLastError();
  } else if (dtype == RA_F32) {
    switch (A.block_heads) {
      case 1: decode_simt<1><<<grid, kThreads, 0, st>>>(A); break;
      case 2: decode_simt<2><<<grid, kThreads, 0, st>>>(A); break;
      case 4: decode_simt<4><<<grid, kThreads, 0, st>>>(A); break;
      default: decode_simt<8><<<grid, kThreads, 0, st>>>(A); break;
    }
    e = cudaGetLastError();
  } else if (A.dh == 128) {
    e = A.block_heads > 8 ? launch_mma<128, true>(A, grid, st) : launch_mma<128, false>(A, grid, st);
  } else {
    e = A.block_heads > 8 ? launch_mma<64, true>(A, grid, st) : launch_mma<64, false>(A, grid, st);
  }
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return dtype == RA_F32 ? launch_join<float>(cfg, A, grid) : launch_join<__nv_bfloat16>(cfg, A, grid);
}

size_t workspace_of(const ra_paged_cache* c, int hq) {
  const size_t part = heads_of_block(c->dtype, hq / c->hkv) * (c->head_dim + 2) * sizeof(float);
  return (2 * ctas_per_sm(c->dtype, c->head_dim) * kSms * part + 255) & ~size_t(255);
}

int check_heads(const ra_paged_cache* c, int hq) {
  if (hq < 1 || hq % c->hkv)
    return record_error(RA_ERR_UNSUPPORTED, "hq (%d) must be a positive multiple of hkv (%d)", hq, c->hkv);
  if (static_cast<int64_t>(c->n_seqs) * hq >= (int64_t(1) << 31))
    return record_error(RA_ERR_UNSUPPORTED, "sequences x query heads must stay below 2^31");
  return RA_OK;
}

}  // namespace

cudaError_t decode_status(unsigned int* value, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_status_decode, sizeof(unsigned int));
  if (e == cudaSuccess && reset) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_status_decode, &zero, sizeof(unsigned int));
  }
  return e;
}

}  // namespace ra

using namespace ra;

extern "C" size_t ra_paged_workspace_bytes(const ra_paged_cache* c, int hq) {
  if (check_cache(c) != RA_OK || check_heads(c, hq) != RA_OK) return 0;
  return workspace_of(c, hq);
}

extern "C" int ra_paged_attn_decode(const ra_paged_cache* c, int hq, float scale, int window, int sinks,
                                    const void* q, const int32_t* seq_lens, void* out, float* lse,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (int e = check_cache(c)) return e;
  if (int e = check_heads(c, hq)) return e;
  if (c->n_seqs > 0 && (!q || !seq_lens || !out || !lse)) return record_error(RA_ERR_INVALID_ARG, "null tensor pointer");
  if (std::isnan(scale) || std::isinf(scale)) return record_error(RA_ERR_INVALID_ARG, "scale is not finite");
  if (window < 0 || sinks < 0) return record_error(RA_ERR_INVALID_ARG, "window and sinks must be >= 0");
  if (workspace_bytes < workspace_of(c, hq))
    return record_error(RA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes,
                        workspace_of(c, hq));
  if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256)
    return record_error(RA_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
  if (c->n_seqs == 0) return record_error(RA_OK, "%s", "");
  if (c->dtype == RA_BF16) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(c->k_pages) | reinterpret_cast<uintptr_t>(c->v_pages) |
                        reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out);
    if (p % 16 || c->page_stride % 8 || c->slot_stride % 8 || c->head_stride % 8)
      return record_error(RA_ERR_INVALID_ARG,
                          "bf16 decode: q, out and pages must be 16-byte aligned, strides multiples of 8 elements");
  }
  DecodeArgs A;
  A.q = q;
  A.k_pages = c->k_pages;
  A.v_pages = c->v_pages;
  A.block_table = c->block_table;
  A.seq_lens = seq_lens;
  A.table_stride = c->table_stride;
  A.page_stride = c->page_stride;
  A.slot_stride = c->slot_stride;
  A.head_stride = c->head_stride;
  A.n_seqs = c->n_seqs;
  A.max_pages = c->max_pages;
  A.page_size = c->page_size;
  A.n_pages = c->n_pages;
  A.hq = hq;
  A.hkv = c->hkv;
  A.group = hq / c->hkv;
  A.dh = c->head_dim;
  A.block_heads = heads_of_block(c->dtype, A.group);
  // the 16-byte kernel's states of four heads of 128 fill a thread's registers
  if (c->dtype == RA_F32 && A.block_heads > 4 && wide_f32(A)) A.block_heads = 4;
  A.blocks_per_kv = (A.group + A.block_heads - 1) / A.block_heads;
  A.window = window;
  A.sinks = sinks;
  A.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(c->head_dim))) * 1.4426950408889634f;
  A.parts = static_cast<float*>(workspace);
  A.out = out;
  A.lse = lse;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch(A, c->dtype, st);
  if (e != cudaSuccess) return record_error(RA_ERR_CUDA, "decode attention launch: %s", cudaGetErrorString(e));
  return record_error(RA_OK, "%s", "");
}
