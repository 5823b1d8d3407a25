// ra_window_simt.cu — windowed ring attention on the CUDA cores: the float32 path (any head_dim <=
// 128) and a cross-check for bf16 inputs; and the sum of the sinks' gradients of both paths.
//
// One warp per query row and head (per key row and K/V head for dk, dv), the lanes over the head
// dimension as in the ring's CUDA-core kernels. What bounds such kernels is the exchange between
// lanes, five shuffles for every dot product: eight dot products are reduced together instead
// (halving the values with every step: nine shuffles for eight), which leaves each value on four
// lanes, where its exponential is taken once and from where it is broadcast. Measured on GB300
// (2048 tokens, 4/2 heads of 64, window 300): one key at a time 310 us forward and 2.66 ms
// backward, eight at a time 123 us and 253 us.
//
// A sink is seen by the whole sequence: its far queries go, a chunk of a rank at a time, to warps
// of their own, which leave float32 sums in the slots that ra_plan.h describes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ra_internal.h"
#include "ra_plan.h"
#include "ra_window.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 8;  // keys (queries) at a time

__device__ __forceinline__ float ldf(const float* p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void stf(float* p, float v) { *p = v; }
__device__ __forceinline__ void stf(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Eight sums over the lanes: value i ends up on lanes 4i .. 4i+3.
__device__ __forceinline__ float sums8(float (&x)[kBatch], int lane) {
#pragma unroll
  for (int n = 4, o = 16; n >= 1; n >>= 1, o >>= 1) {
    const bool hi = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < n) {
        const float send = hi ? x[i] : x[i + n];
        const float keep = hi ? x[i + n] : x[i];
        x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
  }
  x[0] += __shfl_xor_sync(0xffffffffu, x[0], 2);
  return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 1);
}
// Over the eight values.
__device__ __forceinline__ float max8(float x) {
#pragma unroll
  for (int o = 16; o >= 4; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float sum8(float x) {
#pragma unroll
  for (int o = 16; o >= 4; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Rows base .. base + 7 (those past the last are the last again) of a [rows, heads, dh] tensor.
template <typename T, int NI>
__device__ __forceinline__ void load8(const T* p, int64_t stride, int n, int dh, int lane, float (&r)[kBatch][NI]) {
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const T* row = p + min(b, n - 1) * stride;
#pragma unroll
    for (int i = 0; i < NI; ++i) r[b][i] = lane + 32 * i < dh ? ldf(row + lane + 32 * i) : 0.f;
  }
}
template <typename T, int NI>
__device__ __forceinline__ void load1(const T* row, int dh, int lane, float (&r)[NI]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) r[i] = lane + 32 * i < dh ? ldf(row + lane + 32 * i) : 0.f;
}
template <int NI>
__device__ __forceinline__ float dot8(const float (&x)[NI], const float (&r)[kBatch][NI], int lane) {
  float s[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    s[b] = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) s[b] += x[i] * r[b][i];
  }
  return sums8(s, lane);
}

// One query row: rank, row, head; and its rows in the tensors.
struct QRow {
  int r, a, h;
  int64_t row, li;
};
__device__ __forceinline__ QRow query_row(const Plan& P, const SeqDesc& sd, uint32_t u) {
  QRow q;
  const uint32_t x = u / P.hq;
  q.h = static_cast<int>(u - x * P.hq);
  q.r = static_cast<int>(x / sd.L);
  q.a = static_cast<int>(x - q.r * sd.L);
  q.row = sd.row_off + static_cast<int64_t>(q.r) * P.shard_stride + q.a;
  q.li = sd.lse_off + static_cast<int64_t>(q.h) * P.lse_hstride + static_cast<int64_t>(q.r) * P.shard_stride + q.a;
  return q;
}

// Calls f(row of the first key, keys) for the keys that the query sees, eight at a time.
template <typename F>
__device__ __forceinline__ void for_each_keys(const Plan& P, const SeqDesc& sd, const QRow& q, F&& f) {
  const int L = sd.L, pq = static_cast<int>(layout_pos(P.layout, P.D, L, q.r, q.a));
  const KeyLimit upto = key_limit_of(P, pq), before = key_limit_of(P, pq - P.window);
  for (int s = 0; s < P.D; ++s) {
    const int j = shard_at_step(P.D, q.r, s);
    const int lim = limit_in(P, L, j, upto);
    if (lim < 0) continue;
    const int64_t row0 = sd.row_off + static_cast<int64_t>(j) * P.shard_stride;
    const int sk = min(sink_rows(P, L, j), lim + 1);
    const int lo = max(limit_in(P, L, j, before) + 1, sk);
    for (int b = 0; b < sk; b += kBatch) f(row0 + b, min(kBatch, sk - b));
    for (int b = lo; b <= lim; b += kBatch) f(row0 + b, min(kBatch, lim + 1 - b));
  }
}

template <typename T, int NI>
__global__ void __launch_bounds__(kThreads)
    window_fwd_simt(const __grid_constant__ Plan P, const T* __restrict__ q, const T* __restrict__ k,
                    const T* __restrict__ v, T* __restrict__ out, float* __restrict__ lse) {
  const SeqDesc& sd = P.seq[blockIdx.y];
  const int dh = P.head_dim, lane = threadIdx.x & 31;
  const uint32_t units = static_cast<uint32_t>(P.D) * sd.L * P.hq;
  for (uint32_t u = blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kWarps) {
    const QRow x = query_row(P, sd, u);
    const int hk = x.h / P.group;
    const int64_t stride = static_cast<int64_t>(P.hkv) * dh;
    float qr[NI], acc[NI] = {}, m = -INFINITY, l = 0.f;
    load1(q + (x.row * P.hq + x.h) * dh, dh, lane, qr);
    for_each_keys(P, sd, x, [&](int64_t row, int n) {
      float r[kBatch][NI];
      load8(k + row * stride + hk * dh, stride, n, dh, lane, r);
      float s = dot8(qr, r, lane) * P.scale;
      if ((lane >> 2) >= n) s = -INFINITY;
      load8(v + row * stride + hk * dh, stride, n, dh, lane, r);
      const float m_new = fmaxf(m, max8(s));
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = expf(m - ref), p = expf(s - ref);
      m = m_new;
      l = l * alpha + sum8(p);
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[i] *= alpha;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float pb = __shfl_sync(0xffffffffu, p, 4 * b);
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] += pb * r[b][i];
      }
    });
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (lane + 32 * i < dh) stf(out + (x.row * P.hq + x.h) * dh + lane + 32 * i, acc[i] * inv);
    if (lane == 0) lse[x.li] = l > 0.f ? m + logf(l) : -INFINITY;
  }
}

template <typename T, int NI>
__global__ void __launch_bounds__(kThreads)
    window_dq_simt(const __grid_constant__ Plan P, const T* __restrict__ q, const T* __restrict__ k,
                   const T* __restrict__ v, const T* __restrict__ dout, const float* __restrict__ lse,
                   const float* __restrict__ delta, T* __restrict__ dq) {
  const SeqDesc& sd = P.seq[blockIdx.y];
  const int dh = P.head_dim, lane = threadIdx.x & 31;
  const uint32_t units = static_cast<uint32_t>(P.D) * sd.L * P.hq;
  for (uint32_t u = blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kWarps) {
    const QRow x = query_row(P, sd, u);
    const int hk = x.h / P.group;
    const int64_t stride = static_cast<int64_t>(P.hkv) * dh, at = (x.row * P.hq + x.h) * dh;
    const float la = lse[x.li], da = delta[x.li];
    float qr[NI], dr[NI], acc[NI] = {};
    load1(q + at, dh, lane, qr);
    load1(dout + at, dh, lane, dr);
    for_each_keys(P, sd, x, [&](int64_t row, int n) {
      float kr[kBatch][NI], vr[kBatch][NI];
      load8(k + row * stride + hk * dh, stride, n, dh, lane, kr);
      load8(v + row * stride + hk * dh, stride, n, dh, lane, vr);
      const float x = dot8(qr, kr, lane), y = dot8(dr, vr, lane);
      const float ds = (lane >> 2) < n ? expf(x * P.scale - la) * (y - da) : 0.f;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float d = __shfl_sync(0xffffffffu, ds, 4 * b);
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] += d * kr[b][i];
      }
    });
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (lane + 32 * i < dh) stf(dq + at + lane + 32 * i, acc[i] * P.scale);
  }
}

// Units: the sinks' far queries (sink shard, sink row, K/V head, rank, chunk), then the key rows
// with the queries of their window.
template <typename T, int NI>
__global__ void __launch_bounds__(kThreads)
    window_dkv_simt(const __grid_constant__ Plan P, const T* __restrict__ q, const T* __restrict__ k,
                    const T* __restrict__ v, const T* __restrict__ dout, const float* __restrict__ lse,
                    const float* __restrict__ delta, T* __restrict__ dk, T* __restrict__ dv) {
  const SeqDesc& sd = P.seq[blockIdx.y];
  const int L = sd.L, dh = P.head_dim, lane = threadIdx.x & 31;
  const int chunks = sink_chunks(P, L);
  const uint32_t far_units = static_cast<uint32_t>(sink_items_of(P, L)) * P.sink_stride;
  const uint32_t units = far_units + static_cast<uint32_t>(P.D) * L * P.hkv;
  for (uint32_t u = blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kWarps) {
    int j, b, hk, far_r = -1, chunk = 0;
    if (u < far_units) {
      uint32_t x = u;
      hk = x % P.hkv;
      x /= P.hkv;
      chunk = x % chunks;
      x /= chunks;
      far_r = x % P.D;
      x /= P.D;
      b = x % P.sink_stride;
      j = x / P.sink_stride;
      if (b >= sink_rows(P, L, j)) continue;
    } else {
      uint32_t x = u - far_units;
      hk = x % P.hkv;
      x /= P.hkv;
      j = x / L;
      b = x - j * L;
    }
    const bool sink = b < sink_rows(P, L, j);
    const int64_t krow = sd.row_off + static_cast<int64_t>(j) * P.shard_stride + b;
    const int64_t at = (krow * P.hkv + hk) * dh, stride = static_cast<int64_t>(P.hq) * dh;
    float kr[NI], vr[NI], dka[NI] = {}, dva[NI] = {};
    load1(k + at, dh, lane, kr);
    load1(v + at, dh, lane, vr);
    const int64_t pk = layout_pos(P.layout, P.D, L, j, b);
    const KeyLimit last = key_limit_of(P, static_cast<int>(min(pk + P.window - 1, int64_t(0x7fffffff))));
    const KeyLimit before = key_limit_of(P, static_cast<int>(pk) - 1);
    for (int s = far_r >= 0 ? far_r : 0; s < (far_r >= 0 ? far_r + 1 : P.D); ++s) {
      const int r = far_r >= 0 ? far_r : rank_at_step(P.D, j, s);
      int lo = limit_in(P, L, r, far_r >= 0 ? last : before) + 1;
      int hi = far_r >= 0 ? L - 1 : limit_in(P, L, r, last);
      if (far_r >= 0) {
        lo = max(lo, chunk * P.sink_chunk * kQTileRows);
        hi = min(hi, (chunk + 1) * P.sink_chunk * kQTileRows - 1);
      }
      const int64_t row0 = sd.row_off + static_cast<int64_t>(r) * P.shard_stride;
      for (int g = 0; g < P.group; ++g) {
        const int h = hk * P.group + g;
        const int64_t li0 = sd.lse_off + static_cast<int64_t>(h) * P.lse_hstride + static_cast<int64_t>(r) * P.shard_stride;
        for (int a = lo; a <= hi; a += kBatch) {
          const int n = min(kBatch, hi + 1 - a);
          const int64_t from = (row0 + a) * stride + h * dh;
          const int mine = min(lane >> 2, n - 1);
          const float la = lse[li0 + a + mine], da = delta[li0 + a + mine];
          float qr[kBatch][NI], dr[kBatch][NI];
          load8(q + from, stride, n, dh, lane, qr);
          load8(dout + from, stride, n, dh, lane, dr);
          const float x = dot8(kr, qr, lane), y = dot8(vr, dr, lane);
          const float p = (lane >> 2) < n ? expf(x * P.scale - la) : 0.f;
          const float ds = p * (y - da);
#pragma unroll
          for (int c = 0; c < kBatch; ++c) {
            const float pc = __shfl_sync(0xffffffffu, p, 4 * c), dc = __shfl_sync(0xffffffffu, ds, 4 * c);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              dva[i] += pc * dr[c][i];
              dka[i] += dc * qr[c][i];
            }
          }
        }
      }
    }
    const int64_t slot = sink ? sink_slot(P, sd, j, hk, far_r < 0 ? 0 : 1 + far_r * chunks + chunk) : 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int d = lane + 32 * i;
      if (d < dh) {
        if (sink) {
          P.sink_sums[((slot * 2 + 0) * P.sink_stride + b) * dh + d] = dka[i] * P.scale;
          P.sink_sums[((slot * 2 + 1) * P.sink_stride + b) * dh + d] = dva[i];
        } else {
          stf(dk + at + d, dka[i] * P.scale);
          stf(dv + at + d, dva[i]);
        }
      }
    }
  }
}

// dk and dv of the sink rows: the sum of their slots. Block x: a sink row; y: sink shard and K/V
// head; z: sequence. Threads: dk's head_dim elements, then dv's.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    sink_sum_kernel(const __grid_constant__ Plan P, T* __restrict__ dk, T* __restrict__ dv) {
  const SeqDesc& s = P.seq[blockIdx.z];
  const int dh = P.head_dim, j = blockIdx.y / P.hkv, hk = blockIdx.y % P.hkv, row = blockIdx.x;
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

int max_len(const Plan& P) {
  int m = 0;
  for (int i = 0; i < P.n_seqs; ++i) m = P.seq[i].L > m ? P.seq[i].L : m;
  return m;
}

dim3 grid_of(const Plan& P, int64_t units) {
  int64_t blocks = (units + kWarps - 1) / kWarps;
  blocks = blocks > 16384 ? 16384 : blocks < 1 ? 1 : blocks;
  return dim3(static_cast<unsigned>(blocks), P.n_seqs);
}

template <typename T, int NI>
cudaError_t fwd(const Plan& P, const void* q, const void* k, const void* v, void* out, float* lse, cudaStream_t st) {
  window_fwd_simt<T, NI><<<grid_of(P, static_cast<int64_t>(P.D) * max_len(P) * P.hq), kThreads, 0, st>>>(
      P, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), static_cast<T*>(out), lse);
  return cudaGetLastError();
}

template <typename T, int NI>
cudaError_t bwd(const Plan& P, const void* q, const void* k, const void* v, const void* dout, const float* lse,
                const float* delta, void* dq, void* dk, void* dv, cudaStream_t st) {
  const T *q_ = static_cast<const T*>(q), *k_ = static_cast<const T*>(k), *v_ = static_cast<const T*>(v),
          *do_ = static_cast<const T*>(dout);
  int64_t far = 0;
  for (int i = 0; i < P.n_seqs; ++i) {
    const int64_t f = static_cast<int64_t>(sink_items_of(P, P.seq[i].L)) * P.sink_stride;
    far = f > far ? f : far;
  }
  window_dkv_simt<T, NI><<<grid_of(P, far + static_cast<int64_t>(P.D) * max_len(P) * P.hkv), kThreads, 0, st>>>(
      P, q_, k_, v_, do_, lse, delta, static_cast<T*>(dk), static_cast<T*>(dv));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  window_dq_simt<T, NI><<<grid_of(P, static_cast<int64_t>(P.D) * max_len(P) * P.hq), kThreads, 0, st>>>(
      P, q_, k_, v_, do_, lse, delta, static_cast<T*>(dq));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_fwd_simt(const Plan& P, int dtype, const void* q, const void* k, const void* v, void* out,
                                   float* lse, cudaStream_t st) {
  if (P.n_seqs == 0) return cudaSuccess;
  if (dtype == RA_BF16)  // head_dim 64 or 128
    return P.head_dim == 128 ? fwd<__nv_bfloat16, 4>(P, q, k, v, out, lse, st)
                             : fwd<__nv_bfloat16, 2>(P, q, k, v, out, lse, st);
  if (P.head_dim <= 32) return fwd<float, 1>(P, q, k, v, out, lse, st);
  return P.head_dim <= 64 ? fwd<float, 2>(P, q, k, v, out, lse, st) : fwd<float, 4>(P, q, k, v, out, lse, st);
}

cudaError_t launch_window_bwd_simt(const Plan& P, int dtype, const void* q, const void* k, const void* v,
                                   const void* dout, const float* lse, const float* delta, void* dq, void* dk,
                                   void* dv, cudaStream_t st) {
  if (P.n_seqs == 0) return cudaSuccess;
  cudaError_t e;
  if (dtype == RA_BF16)
    e = P.head_dim == 128 ? bwd<__nv_bfloat16, 4>(P, q, k, v, dout, lse, delta, dq, dk, dv, st)
                          : bwd<__nv_bfloat16, 2>(P, q, k, v, dout, lse, delta, dq, dk, dv, st);
  else if (P.head_dim <= 32) e = bwd<float, 1>(P, q, k, v, dout, lse, delta, dq, dk, dv, st);
  else if (P.head_dim <= 64) e = bwd<float, 2>(P, q, k, v, dout, lse, delta, dq, dk, dv, st);
  else e = bwd<float, 4>(P, q, k, v, dout, lse, delta, dq, dk, dv, st);
  return e == cudaSuccess ? launch_sink_sum(P, dtype, dk, dv, st) : e;
}

cudaError_t launch_sink_sum(const Plan& P, int dtype, void* dk, void* dv, cudaStream_t st) {
  if (P.sinks == 0 || P.n_seqs == 0) return cudaSuccess;
  int shards = 0;
  for (int i = 0; i < P.n_seqs; ++i) {
    const int n = sink_shards(P, P.seq[i].L);
    shards = n > shards ? n : shards;
  }
  const dim3 grid(P.sink_stride, shards * P.hkv, P.n_seqs);
  if (dtype == RA_F32)
    sink_sum_kernel<float><<<grid, kThreads, 0, st>>>(P, static_cast<float*>(dk), static_cast<float*>(dv));
  else
    sink_sum_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(P, static_cast<__nv_bfloat16*>(dk),
                                                              static_cast<__nv_bfloat16*>(dv));
  return cudaGetLastError();
}

}  // namespace ra
