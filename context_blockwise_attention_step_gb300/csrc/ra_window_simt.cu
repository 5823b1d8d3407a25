// ra_window_simt.cu — windowed ring attention on the CUDA cores: the float32 path (any head_dim <=
// 128) and a cross-check for bf16 inputs; and the sum of the sinks' gradients of both paths.
//
// A CTA owns 32 rows of one head (queries for out and dq, keys for dk and dv) and walks the runs of
// the other side that some of its rows meets, 64 at a time, through shared memory: for each shard
// the sinks, then the window of the rows (a zigzag shard's two chunks on their own). The runs begin
// where the window does, on any row, so the last tile of a run alone is not full. A thread has 4
// rows x 4 columns of the products, and 4 rows x head_dim / 16 elements of the sums: what bounds
// such kernels is the 128 bytes a cycle that shared memory gives an SM, and 4 x 4 takes two
// multiplications from every word (1 x 4 took less than one, and 10.5 against 5.5 ms for a forward
// and backward of 4096 tokens, 16/4 heads of 128, window 1024). Rows of a tile are 16 bytes longer
// than the data, so that eight threads on eight rows meet every bank once. Weights are exchanged
// between the sixteen threads of a row through shared memory. dq's kernel starts while that of dk and dv, which has
// fewer CTAs, is running, and float32 tiles are loaded by asynchronous copies. CTAs of 16 rows are
// slower, backward and forward, at eight of nine sizes (2048 tokens, 4/2 heads of 64, window 300: forward 63 against 56 us, before
// the copies), for a tile's loads then feed half the products.
// Measured on GB300: that size 45 us forward, 137 us backward (one warp a row, eight keys at a
// time, took 119 and 251); 4096 tokens, 16/4 heads of 128, window 1024: 4.5 ms in all, 23 TFLOP/s.
//
// A sink is seen by the whole sequence: its far queries go, a chunk of a rank at a time, to CTAs
// of their own, which leave float32 sums in the slots that ra_plan.h describes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ra_internal.h"
#include "ra_plan.h"
#include "ra_ptx.cuh"
#include "ra_window.cuh"

namespace ra {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 32;   // rows of a CTA
constexpr int kCols = 64;   // columns (rows of the other side) at a time
constexpr int kPStride = kCols + 4;

__device__ __forceinline__ float ldf(const float* p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void stf(float* p, float v) { *p = v; }
__device__ __forceinline__ void stf(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Four elements into shared memory, zeros if not `in`: float32 by an asynchronous copy, so that all
// the loads of a tile are under way together, without registers.
__device__ __forceinline__ void copy4(float* to, const float* from, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(float* to, const __nv_bfloat16* from, bool in) {
  *reinterpret_cast<float4*>(to) = in ? ld4(from) : make_float4(0.f, 0.f, 0.f, 0.f);
}
// All tiles that the threads have loaded are there.
__device__ __forceinline__ void wait_tiles() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
}

// Rows row0 .. row0 + n - 1 of head h of a [rows, heads, dh] tensor into a tile of ROWS rows, zeros
// behind them and behind dh. vec: dh and the tensor allow loads of four elements.
template <typename T, int DHP, int ROWS>
__device__ __forceinline__ void load_tile(float* to, const T* from, int64_t row0, int n, int heads, int h, int dh,
                                          bool vec) {
  if (vec) {
#pragma unroll 4
    for (int i = threadIdx.x; i < ROWS * (DHP / 4); i += kThreads) {
      const int r = i / (DHP / 4), d = i % (DHP / 4) * 4;
      const bool in = r < n && d < dh;
      const T* at = from + (in ? ((row0 + r) * heads + h) * dh + d : 0);
      copy4(to + r * (DHP + 4) + d, at, in);
    }
  } else {
#pragma unroll 4
    for (int i = threadIdx.x; i < ROWS * DHP; i += kThreads) {
      const int r = i / DHP, d = i % DHP;
      to[r * (DHP + 4) + d] = r < n && d < dh ? ldf(from + ((row0 + r) * heads + h) * dh + d) : 0.f;
    }
  }
}

// x[i][j] = row 4 ty + i of A times row tx + 16 j of B, j < J.
template <int DHP, int J>
__device__ __forceinline__ void products_of(const float* A, const float* B, int ty, int tx, float (&x)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < DHP; d += 4) {
    float4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * (DHP + 4) + d);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * (DHP + 4) + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i][j] += u[i].x * v.x;
        x[i][j] += u[i].y * v.y;
        x[i][j] += u[i].z * v.z;
        x[i][j] += u[i].w * v.w;
      }
    }
  }
}

// The first n of the 64 columns: a tile of a few first tokens takes a quarter of the products.
template <int DHP>
__device__ __forceinline__ void products(const float* A, const float* B, int ty, int tx, int n, float (&x)[4][4]) {
  if (n <= 16) products_of<DHP, 1>(A, B, ty, tx, x);
  else products_of<DHP, 4>(A, B, ty, tx, x);
}

// acc[i][4 j + e] (row 4 ty + i, element 4 tx + 64 j + e) += sum over the first n columns c of W[row][c] B[c]
// (W is 0 from n on).
template <int DHP>
struct Acc {
  static constexpr int J = DHP >= 64 ? DHP / 64 : 1;  // DHP 32: the upper eight threads of a row idle
  float v[4][4 * J];
};
template <int DHP>
__device__ __forceinline__ void accumulate(const float* W, const float* B, int ty, int tx, int n, Acc<DHP>& acc) {
  if (4 * tx >= DHP) return;
#pragma unroll 2
  for (int c0 = 0; c0 < n; c0 += 4) {
    float w[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = *reinterpret_cast<const float4*>(W + (4 * ty + i) * kPStride + c0);
      w[i][0] = t.x;
      w[i][1] = t.y;
      w[i][2] = t.z;
      w[i][3] = t.w;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < Acc<DHP>::J; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(B + (c0 + c) * (DHP + 4) + 4 * tx + 64 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc.v[i][4 * j] += w[i][c] * v.x;
          acc.v[i][4 * j + 1] += w[i][c] * v.y;
          acc.v[i][4 * j + 2] += w[i][c] * v.z;
          acc.v[i][4 * j + 3] += w[i][c] * v.w;
        }
      }
  }
}
template <typename T, int DHP>
__device__ __forceinline__ void store_row(T* to, int tx, int dh, const float (&acc)[4 * Acc<DHP>::J], float mul) {
#pragma unroll
  for (int j = 0; j < Acc<DHP>::J; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 4 * tx + 64 * j + e;
      if (d < dh) stf(to + d, acc[4 * j + e] * mul);
    }
}
// Over the sixteen threads of a row.
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The query block of a CTA: kRows rows of rank r, head h.
struct QBlock {
  int h, r, a0, n;      // first row, rows
  int64_t row, lse;     // of a0
};
__device__ __forceinline__ QBlock query_block(const Plan& P, const SeqDesc& sd, int x) {
  QBlock q;
  const int blocks = ceil_div(sd.L, kRows);
  q.h = x % P.hq;
  x /= P.hq;
  q.r = x / blocks;
  q.a0 = (blocks - 1 - x % blocks) * kRows;
  q.n = min(kRows, sd.L - q.a0);
  q.row = sd.row_off + static_cast<int64_t>(q.r) * P.shard_stride + q.a0;
  q.lse = sd.lse_off + static_cast<int64_t>(q.h) * P.lse_hstride + static_cast<int64_t>(q.r) * P.shard_stride + q.a0;
  return q;
}

// Which keys of the current shard the block's rows see: lo .. lim of each, and those before sk.
struct RowKeys {
  int lim[kRows], lo[kRows];
};

// Calls tile(j, sk, first key, keys) for the keys of shard j that some of the block's rows sees, for
// every shard, after the rows' limits in the shard have been put into `keys` (shared memory; tile()
// begins with a barrier).
template <typename TileF>
__device__ __forceinline__ void for_each_key_tile(const Plan& P, int L, const QBlock& q, RowKeys& keys, TileF&& tile) {
  auto pos = [&](int a) { return static_cast<int>(layout_pos(P.layout, P.D, L, q.r, a)); };
  const int a1 = q.a0 + q.n - 1;
  const bool two = straddles(P, L, q.a0, a1);
  const int mid = two ? L >> 1 : q.a0;
  const KeyLimit before0 = key_limit_of(P, pos(q.a0) - P.window), upto0 = key_limit_of(P, pos(two ? mid - 1 : a1)),
                 before1 = key_limit_of(P, pos(mid) - P.window), upto1 = key_limit_of(P, pos(a1));
  KeyLimit before, upto;  // of row threadIdx.x
  const bool valid = threadIdx.x < q.n;
  if (threadIdx.x < kRows) {
    const int p = valid ? pos(q.a0 + threadIdx.x) : 0;
    upto = key_limit_of(P, p);
    before = key_limit_of(P, p - P.window);
  }
  for (int s = 0; s < P.D; ++s) {
    const int j = shard_at_step(P.D, q.r, s);
    const int lim = limit_in(P, L, j, upto1);
    if (lim < 0) continue;
    const int sk = sink_rows(P, L, j);
    __syncthreads();  // the last tile's weights are done
    if (threadIdx.x < kRows) {
      keys.lim[threadIdx.x] = valid ? limit_in(P, L, j, upto) : -1;
      keys.lo[threadIdx.x] = limit_in(P, L, j, before) + 1;
    }
    // run 0: the sinks; 1, 2: the window of the rows before and after the chunks' border
    int next = 0;
    for (int run = 0; run < 3; ++run) {
      int from, to;
      if (run == 0) {
        from = 0;
        to = min(sk - 1, lim);
      } else {
        if (run == 1 && !two) continue;
        from = max(next, limit_in(P, L, j, run == 1 ? before0 : before1) + 1);
        to = run == 1 ? limit_in(P, L, j, upto0) : lim;
      }
      next = max(next, to + 1);
      for (int b = from; b <= to; b += kCols) tile(j, sk, b, min(kCols, to + 1 - b));
    }
  }
}

template <int DHP, int ROWS>
constexpr int tile_floats() { return ROWS * (DHP + 4); }

template <typename T, int DHP>
__global__ void __launch_bounds__(kThreads)
    window_fwd_simt(const __grid_constant__ Plan P, const T* __restrict__ q, const T* __restrict__ k,
                    const T* __restrict__ v, T* __restrict__ out, float* __restrict__ lse, bool vec) {
  extern __shared__ float4 smem4[];
  float* sq = reinterpret_cast<float*>(smem4);
  float *sk_ = sq + tile_floats<DHP, kRows>(), *sv = sk_ + tile_floats<DHP, kCols>(), *sp = sv + tile_floats<DHP, kCols>();
  __shared__ RowKeys keys;
  const SeqDesc& sd = P.seq[blockIdx.y];
  const int L = sd.L, dh = P.head_dim, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  if (static_cast<int64_t>(blockIdx.x) >= static_cast<int64_t>(ceil_div(L, kRows)) * P.D * P.hq) return;
  const QBlock b = query_block(P, sd, blockIdx.x);
  const int hk = b.h / P.group;
  load_tile<T, DHP, kRows>(sq, q, b.row, b.n, P.hq, b.h, dh, vec);
  float m[4], l[4];
  Acc<DHP> acc = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  for_each_key_tile(P, L, b, keys, [&](int j, int sk, int k0, int n) {
    const int64_t krow = sd.row_off + static_cast<int64_t>(j) * P.shard_stride + k0;
    __syncthreads();
    load_tile<T, DHP, kCols>(sk_, k, krow, n, P.hkv, hk, dh, vec);
    load_tile<T, DHP, kCols>(sv, v, krow, n, P.hkv, hk, dh, vec);
    wait_tiles();
    float x[4][4];
    products<DHP>(sq, sk_, ty, tx, n, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lim = keys.lim[4 * ty + i], lo = keys.lo[4 * ty + i];
      float mx = m[i];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = tx + 16 * c, key = k0 + col;
        const bool see = col < n && key <= lim && (key >= lo || key < sk);
        x[i][c] = see ? x[i][c] * P.scale : -INFINITY;
        mx = fmaxf(mx, x[i][c]);
      }
      mx = row_max(mx);
      const float ref = mx == -INFINITY ? 0.f : mx, alpha = expf(m[i] - ref);
      m[i] = mx;
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float e = expf(x[i][c] - ref);
        sum += e;
        sp[(4 * ty + i) * kPStride + tx + 16 * c] = e;
      }
      l[i] = l[i] * alpha + row_sum(sum);
#pragma unroll
      for (int d = 0; d < 4 * Acc<DHP>::J; ++d) acc.v[i][d] *= alpha;
    }
    __syncwarp();  // a row's sixteen threads are in one warp
    accumulate<DHP>(sp, sv, ty, tx, n, acc);
  });
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * ty + i;
    if (row >= b.n) break;
    store_row<T, DHP>(out + ((b.row + row) * P.hq + b.h) * dh, tx, dh, acc.v[i], l[i] > 0.f ? 1.f / l[i] : 0.f);
    if (tx == 0) lse[b.lse + row] = l[i] > 0.f ? m[i] + logf(l[i]) : -INFINITY;
  }
}

template <typename T, int DHP>
__global__ void __launch_bounds__(kThreads)
    window_dq_simt(const __grid_constant__ Plan P, const T* __restrict__ q, const T* __restrict__ k,
                   const T* __restrict__ v, const T* __restrict__ dout, const float* __restrict__ lse,
                   const float* __restrict__ delta, T* __restrict__ dq, bool vec) {
  extern __shared__ float4 smem4[];
  float* sq = reinterpret_cast<float*>(smem4);
  float *sdo = sq + tile_floats<DHP, kRows>(), *sk_ = sdo + tile_floats<DHP, kRows>(),
        *sv = sk_ + tile_floats<DHP, kCols>(), *sp = sv + tile_floats<DHP, kCols>();
  __shared__ RowKeys keys;
  const SeqDesc& sd = P.seq[blockIdx.y];
  const int L = sd.L, dh = P.head_dim, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  if (static_cast<int64_t>(blockIdx.x) >= static_cast<int64_t>(ceil_div(L, kRows)) * P.D * P.hq) return;
  const QBlock b = query_block(P, sd, blockIdx.x);
  const int hk = b.h / P.group;
  load_tile<T, DHP, kRows>(sq, q, b.row, b.n, P.hq, b.h, dh, vec);
  load_tile<T, DHP, kRows>(sdo, dout, b.row, b.n, P.hq, b.h, dh, vec);
  float la[4], da[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    la[i] = 4 * ty + i < b.n ? lse[b.lse + 4 * ty + i] : 0.f;
    da[i] = 4 * ty + i < b.n ? delta[b.lse + 4 * ty + i] : 0.f;
  }
  Acc<DHP> acc = {};
  for_each_key_tile(P, L, b, keys, [&](int j, int sk, int k0, int n) {
    const int64_t krow = sd.row_off + static_cast<int64_t>(j) * P.shard_stride + k0;
    __syncthreads();
    load_tile<T, DHP, kCols>(sk_, k, krow, n, P.hkv, hk, dh, vec);
    load_tile<T, DHP, kCols>(sv, v, krow, n, P.hkv, hk, dh, vec);
    wait_tiles();
    float x[4][4], y[4][4];
    products<DHP>(sq, sk_, ty, tx, n, x);
    products<DHP>(sdo, sv, ty, tx, n, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lim = keys.lim[4 * ty + i], lo = keys.lo[4 * ty + i];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = tx + 16 * c, key = k0 + col;
        const bool see = col < n && key <= lim && (key >= lo || key < sk);
        sp[(4 * ty + i) * kPStride + col] = see ? expf(x[i][c] * P.scale - la[i]) * (y[i][c] - da[i]) : 0.f;
      }
    }
    __syncwarp();
    accumulate<DHP>(sp, sk_, ty, tx, n, acc);
  });
  wait_for_previous();  // so that the end of this kernel is that of window_dkv_simt too
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (4 * ty + i < b.n)
      store_row<T, DHP>(dq + ((b.row + 4 * ty + i) * P.hq + b.h) * dh, tx, dh, acc.v[i], P.scale);
}

// Blocks: the sinks' far queries (sink shard, 32 sink rows, rank, chunk, K/V head), then the key
// blocks with the queries of their windows.
template <typename T, int DHP>
__global__ void __launch_bounds__(kThreads)
    window_dkv_simt(const __grid_constant__ Plan P, const T* __restrict__ q, const T* __restrict__ k,
                    const T* __restrict__ v, const T* __restrict__ dout, const float* __restrict__ lse,
                    const float* __restrict__ delta, T* __restrict__ dk, T* __restrict__ dv, bool vec) {
  extern __shared__ float4 smem4[];
  float* sk_ = reinterpret_cast<float*>(smem4);
  float *sv = sk_ + tile_floats<DHP, kRows>(), *sq = sv + tile_floats<DHP, kRows>(),
        *sdo = sq + tile_floats<DHP, kCols>(), *sp = sdo + tile_floats<DHP, kCols>();
  launch_dependents();
  __shared__ float s_lse[kCols], s_delta[kCols];
  __shared__ int s_lo[kRows], s_hi[kRows];
  const SeqDesc& sd = P.seq[blockIdx.y];
  const int L = sd.L, dh = P.head_dim, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int chunks = sink_chunks(P, L), sink_blocks = ceil_div(P.sink_stride, kRows);
  const int64_t far_blocks = static_cast<int64_t>(sink_items_of(P, L)) * sink_blocks;
  int j, b0, hk, far_r = -1, chunk = 0, n_rows;
  if (static_cast<int64_t>(blockIdx.x) < far_blocks) {
    unsigned x = blockIdx.x;
    hk = x % P.hkv;
    x /= P.hkv;
    chunk = x % chunks;
    x /= chunks;
    far_r = x % P.D;
    x /= P.D;
    b0 = (x % sink_blocks) * kRows;
    j = x / sink_blocks;
    n_rows = min(kRows, sink_rows(P, L, j) - b0);
  } else {
    const int64_t y = static_cast<int64_t>(blockIdx.x) - far_blocks;
    const int blocks = ceil_div(L, kRows);
    if (y >= static_cast<int64_t>(blocks) * P.D * P.hkv) return;
    unsigned x = static_cast<unsigned>(y);
    hk = x % P.hkv;
    x /= P.hkv;
    j = x / blocks;
    b0 = (x % blocks) * kRows;
    n_rows = min(kRows, L - b0);
  }
  if (n_rows <= 0) return;
  const int64_t krow = sd.row_off + static_cast<int64_t>(j) * P.shard_stride + b0;
  load_tile<T, DHP, kRows>(sk_, k, krow, n_rows, P.hkv, hk, dh, vec);
  load_tile<T, DHP, kRows>(sv, v, krow, n_rows, P.hkv, hk, dh, vec);
  auto pos = [&](int b) { return static_cast<int>(layout_pos(P.layout, P.D, L, j, b)); };
  auto end_of = [&](int p) {  // the last position that sees position p through the window
    return key_limit_of(P, static_cast<int>(min(static_cast<int64_t>(p) + P.window - 1, int64_t(0x7fffffff))));
  };
  const int b1 = b0 + n_rows - 1;
  const bool valid = threadIdx.x < n_rows;
  KeyLimit last, first;  // of row threadIdx.x
  if (threadIdx.x < kRows) {
    const int p = valid ? pos(b0 + threadIdx.x) : 0;
    last = end_of(p);
    first = key_limit_of(P, p - 1);
  }
  const bool two = straddles(P, L, b0, b1);
  const int mid = two ? L >> 1 : b0;
  const KeyLimit first0 = key_limit_of(P, pos(b0) - 1), last0 = end_of(pos(two ? mid - 1 : b1)),
                 first1 = key_limit_of(P, pos(mid) - 1), last1 = end_of(pos(b1)), far0 = end_of(pos(b0));
  Acc<DHP> dka = {}, dva = {};
  for (int s = far_r >= 0 ? far_r : 0; s < (far_r >= 0 ? far_r + 1 : P.D); ++s) {
    const int r = far_r >= 0 ? far_r : rank_at_step(P.D, j, s);
    __syncthreads();
    if (threadIdx.x < kRows) {  // the rows' queries in rank r
      s_lo[threadIdx.x] = limit_in(P, L, r, far_r >= 0 ? last : first) + 1;
      s_hi[threadIdx.x] = !valid ? -1 : far_r >= 0 ? L - 1 : limit_in(P, L, r, last);
    }
    const int64_t row0 = sd.row_off + static_cast<int64_t>(r) * P.shard_stride;
    for (int g = 0; g < P.group; ++g) {
      const int h = hk * P.group + g;
      const int64_t li0 = sd.lse_off + static_cast<int64_t>(h) * P.lse_hstride + static_cast<int64_t>(r) * P.shard_stride;
      int next = 0;
      for (int run = two && far_r < 0 ? 0 : 1; run < 2; ++run) {
        int from, to;
        if (far_r >= 0) {
          from = max(limit_in(P, L, r, far0) + 1, chunk * P.sink_chunk * kQTileRows);
          to = min(L, (chunk + 1) * P.sink_chunk * kQTileRows) - 1;
        } else {
          from = max(next, limit_in(P, L, r, run ? first1 : first0) + 1);
          to = limit_in(P, L, r, run ? last1 : last0);
        }
        next = max(next, to + 1);
        for (int a = from; a <= to; a += kCols) {
          const int n = min(kCols, to + 1 - a);
          __syncthreads();
          load_tile<T, DHP, kCols>(sq, q, row0 + a, n, P.hq, h, dh, vec);
          load_tile<T, DHP, kCols>(sdo, dout, row0 + a, n, P.hq, h, dh, vec);
          if (threadIdx.x < n) {
            s_lse[threadIdx.x] = lse[li0 + a + threadIdx.x];
            s_delta[threadIdx.x] = delta[li0 + a + threadIdx.x];
          }
          wait_tiles();
          float x[4][4], y[4][4];
          products<DHP>(sk_, sq, ty, tx, n, x);
          products<DHP>(sv, sdo, ty, tx, n, y);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int lo = s_lo[4 * ty + i], hi = s_hi[4 * ty + i];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int col = tx + 16 * c;
              const bool see = col < n && a + col >= lo && a + col <= hi;
              const float p = see ? expf(x[i][c] * P.scale - s_lse[col]) : 0.f;
              sp[(4 * ty + i) * kPStride + col] = p;
              y[i][c] = see ? p * (y[i][c] - s_delta[col]) : 0.f;
            }
          }
          __syncwarp();
          accumulate<DHP>(sp, sdo, ty, tx, n, dva);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) sp[(4 * ty + i) * kPStride + tx + 16 * c] = y[i][c];
          __syncwarp();
          accumulate<DHP>(sp, sq, ty, tx, n, dka);
        }
      }
    }
  }
  wait_tiles();  // (a block without queries)
  const int sinks = sink_rows(P, L, j);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * ty + i, b = b0 + row;
    if (row >= n_rows) break;
    if (b < sinks) {
      const int64_t slot = sink_slot(P, sd, j, hk, far_r < 0 ? 0 : 1 + far_r * chunks + chunk);
      float* to = P.sink_sums + (slot * 2 * P.sink_stride + b) * dh;
      store_row<float, DHP>(to, tx, dh, dka.v[i], P.scale);
      store_row<float, DHP>(to + static_cast<int64_t>(P.sink_stride) * dh, tx, dh, dva.v[i], 1.f);
    } else {
      store_row<T, DHP>(dk + ((krow + row) * P.hkv + hk) * dh, tx, dh, dka.v[i], P.scale);
      store_row<T, DHP>(dv + ((krow + row) * P.hkv + hk) * dh, tx, dh, dva.v[i], 1.f);
    }
  }
}

// dk and dv of the sink rows: the sum of their slots. Block x: a sink row of a sink shard and K/V head
// (all in x: y ends at 65535, which 128 sink shards of 512 heads reach); y: sequence. Threads: dk's
// head_dim elements, then dv's.
template <typename T>
__global__ void __launch_bounds__(256)
    sink_sum_kernel(const __grid_constant__ Plan P, T* __restrict__ dk, T* __restrict__ dv) {
  const SeqDesc& s = P.seq[blockIdx.y];
  const int dh = P.head_dim, row = blockIdx.x % P.sink_stride, head = blockIdx.x / P.sink_stride;
  const int j = head / P.hkv, hk = head % P.hkv;
  if (j >= sink_shards(P, s.L) || row >= sink_rows(P, s.L, j) || threadIdx.x >= 2 * dh) return;
  const int which = threadIdx.x / dh, d = threadIdx.x % dh, n = sink_slots(P, s.L);
  const int64_t slot = sink_slot(P, s, j, hk, 0);
  const float* src = P.sink_sums + ((slot * 2 + which) * P.sink_stride + row) * dh + d;
  float sum = 0.f;
#pragma unroll 8
  for (int i = 0; i < n; ++i) sum += src[static_cast<int64_t>(i) * 2 * P.sink_stride * dh];
  const int64_t krow = s.row_off + static_cast<int64_t>(j) * P.shard_stride + row;
  stf((which ? dv : dk) + (krow * P.hkv + hk) * dh + d, sum);
}

// Most blocks of a sequence; < 0 if they are too many for a launch.
template <typename F>
int64_t most_blocks(const Plan& P, F&& of) {
  int64_t m = 1;
  for (int i = 0; i < P.n_seqs; ++i) m = of(P.seq[i].L) > m ? of(P.seq[i].L) : m;
  return m < (int64_t(1) << 31) ? m : -1;
}

// Whether rows can be read four elements at a time.
bool can_vec(const Plan& P, const void* a, const void* b, const void* c, const void* d) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
                      reinterpret_cast<uintptr_t>(c) | reinterpret_cast<uintptr_t>(d);
  return P.head_dim % 4 == 0 && p % 16 == 0;
}

template <typename K>
cudaError_t allow_smem(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int DHP>
cudaError_t fwd(const Plan& P, const void* q, const void* k, const void* v, void* out, float* lse, cudaStream_t st) {
  constexpr int smem = (tile_floats<DHP, kRows>() + 2 * tile_floats<DHP, kCols>() + kRows * kPStride) * sizeof(float);
  const int64_t blocks = most_blocks(P, [&](int L) { return static_cast<int64_t>(ceil_div(L, kRows)) * P.D * P.hq; });
  cudaError_t e = blocks < 0 ? cudaErrorInvalidConfiguration : allow_smem(window_fwd_simt<T, DHP>, smem);
  if (e != cudaSuccess) return e;
  window_fwd_simt<T, DHP><<<dim3(static_cast<unsigned>(blocks), P.n_seqs), kThreads, smem, st>>>(
      P, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), static_cast<T*>(out), lse,
      can_vec(P, q, k, v, nullptr));
  return cudaGetLastError();
}

template <typename T, int DHP>
cudaError_t bwd(const Plan& P, const void* q, const void* k, const void* v, const void* dout, const float* lse,
                const float* delta, void* dq, void* dk, void* dv, cudaStream_t st) {
  const T *q_ = static_cast<const T*>(q), *k_ = static_cast<const T*>(k), *v_ = static_cast<const T*>(v),
          *do_ = static_cast<const T*>(dout);
  constexpr int tiles = 2 * tile_floats<DHP, kRows>() + 2 * tile_floats<DHP, kCols>();
  constexpr int smem = (tiles + kRows * kPStride) * sizeof(float);
  const int64_t kv_blocks = most_blocks(P, [&](int L) {
    return static_cast<int64_t>(ceil_div(L, kRows)) * P.D * P.hkv +
           static_cast<int64_t>(sink_items_of(P, L)) * ceil_div(P.sink_stride, kRows);
  });
  const int64_t q_blocks = most_blocks(P, [&](int L) { return static_cast<int64_t>(ceil_div(L, kRows)) * P.D * P.hq; });
  cudaError_t e = kv_blocks < 0 || q_blocks < 0 ? cudaErrorInvalidConfiguration : allow_smem(window_dkv_simt<T, DHP>, smem);
  if (e == cudaSuccess) e = allow_smem(window_dq_simt<T, DHP>, smem);
  if (e != cudaSuccess) return e;
  window_dkv_simt<T, DHP><<<dim3(static_cast<unsigned>(kv_blocks), P.n_seqs), kThreads, smem, st>>>(
      P, q_, k_, v_, do_, lse, delta, static_cast<T*>(dk), static_cast<T*>(dv), can_vec(P, q, k, v, dout));
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // dq needs nothing of dk and dv: its CTAs start as soon as theirs have all begun.
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(q_blocks), P.n_seqs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, window_dq_simt<T, DHP>, P, q_, k_, v_, do_, lse, delta, static_cast<T*>(dq),
                            can_vec(P, q, k, v, dout));
}

}  // namespace

cudaError_t launch_window_fwd_simt(const Plan& P, int dtype, const void* q, const void* k, const void* v, void* out,
                                   float* lse, cudaStream_t st) {
  if (P.n_seqs == 0) return cudaSuccess;
  if (dtype == RA_BF16)  // head_dim 64 or 128
    return P.head_dim == 128 ? fwd<__nv_bfloat16, 128>(P, q, k, v, out, lse, st)
                             : fwd<__nv_bfloat16, 64>(P, q, k, v, out, lse, st);
  if (P.head_dim <= 32) return fwd<float, 32>(P, q, k, v, out, lse, st);
  return P.head_dim <= 64 ? fwd<float, 64>(P, q, k, v, out, lse, st) : fwd<float, 128>(P, q, k, v, out, lse, st);
}

cudaError_t launch_window_bwd_simt(const Plan& P, int dtype, const void* q, const void* k, const void* v,
                                   const void* dout, const float* lse, const float* delta, void* dq, void* dk,
                                   void* dv, cudaStream_t st) {
  if (P.n_seqs == 0) return cudaSuccess;
  cudaError_t e;
  if (dtype == RA_BF16)
    e = P.head_dim == 128 ? bwd<__nv_bfloat16, 128>(P, q, k, v, dout, lse, delta, dq, dk, dv, st)
                          : bwd<__nv_bfloat16, 64>(P, q, k, v, dout, lse, delta, dq, dk, dv, st);
  else if (P.head_dim <= 32) e = bwd<float, 32>(P, q, k, v, dout, lse, delta, dq, dk, dv, st);
  else if (P.head_dim <= 64) e = bwd<float, 64>(P, q, k, v, dout, lse, delta, dq, dk, dv, st);
  else e = bwd<float, 128>(P, q, k, v, dout, lse, delta, dq, dk, dv, st);
  return e == cudaSuccess ? launch_sink_sum(P, dtype, dk, dv, st) : e;
}

cudaError_t launch_sink_sum(const Plan& P, int dtype, void* dk, void* dv, cudaStream_t st) {
  if (P.sinks == 0 || P.n_seqs == 0) return cudaSuccess;
  int shards = 0;
  for (int i = 0; i < P.n_seqs; ++i) {
    const int n = sink_shards(P, P.seq[i].L);
    shards = n > shards ? n : shards;
  }
  const int64_t blocks = static_cast<int64_t>(P.sink_stride) * shards * P.hkv;
  if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks), P.n_seqs);
  if (dtype == RA_F32)
    sink_sum_kernel<float><<<grid, 256, 0, st>>>(P, static_cast<float*>(dk), static_cast<float*>(dv));
  else
    sink_sum_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(P, static_cast<__nv_bfloat16*>(dk),
                                                              static_cast<__nv_bfloat16*>(dv));
  return cudaGetLastError();
}

}  // namespace ra
