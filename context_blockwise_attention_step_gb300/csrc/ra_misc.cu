// ra_misc.cu — the HBM-bound kernels of the path: the standalone update_out_and_lse merge,
// the backward preprocess (delta = rowsum(dO * O)) and postprocess (f32 dq -> dq), and the
// natural <-> shard-major permutations.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ra_internal.h"
#include "ra_plan.h"

namespace ra {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float ldf(const float* p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ size_t lse_index(const Plan& P, const SeqDesc& sd, int h, int r, int a) {
  return sd.lse_off + static_cast<size_t>(h) * P.lse_hstride + static_cast<size_t>(r) * P.shard_stride + a;
}

unsigned grid_for(long work, long per_block) {
  long b = (work + per_block - 1) / per_block;
  if (b > 8192) b = 8192;
  return static_cast<unsigned>(b < 1 ? 1 : b);
}

long max_len(const Plan& P) {
  long m = 0;
  for (int i = 0; i < P.n_seqs; ++i) m = P.seq[i].L > m ? P.seq[i].L : m;
  return m;
}

// ------------------------------------------------------------------ update_out_and_lse
// lse' = log(e^lse + e^blse); out' = e^(lse-lse') out + e^(blse-lse') bout; -inf identity.
// One warp per (row, head): lane 0 reads both lse values and broadcasts them, the lanes
// walk the row in VEC-element pieces (VEC = 4 when head_dim % 4 == 0; head_dim <= 128, so
// one piece per lane), and lane 0 writes the merged lse only after the broadcast, so no
// lane can read an already-merged lse. The row's out / block loads are issued before the
// broadcast so that their latency overlaps the lse loads'.
// At most 32 registers (8 blocks of 256 threads per SM), so that 64 warps per SM have their
// loads in flight: measured on GB300 at 131072 tokens, 32 heads, 5.2 against 4.7 TB/s with
// the 33 registers the compiler picks unbounded (48 warps).
template <typename BT, int VEC>
__global__ void __launch_bounds__(kThreads, 8)
    merge_kernel(const __grid_constant__ Plan P, float* __restrict__ out, float* __restrict__ lse,
                 const BT* __restrict__ bout, const float* __restrict__ blse) {
  const SeqDesc& sd = P.seq[blockIdx.y];
  const int L = sd.L, dh = P.head_dim, nv = dh / VEC, lane = threadIdx.x & 31;
  const long units = static_cast<long>(plan_ranks(P)) * L * P.hq;
  constexpr int kWarps = kThreads / 32;
  for (long u = static_cast<long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<long>(gridDim.x) * kWarps) {
    const int h = static_cast<int>(u % P.hq);
    const long x = u / P.hq;
    const int a = static_cast<int>(x % L);
    const int r = P.rank_only >= 0 ? P.rank_only : static_cast<int>(x / L);
    const size_t li = lse_index(P, sd, h, r, a);
    const size_t row = static_cast<size_t>(sd.row_off + r * P.shard_stride + a);
    const size_t rb = (row * P.hq + h) * dh;
    float l1 = 0.f, l2 = 0.f;
    if (lane == 0) {
      l1 = lse[li];
      l2 = blse[li];
    }
    if constexpr (VEC == 4) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float b[4] = {0.f, 0.f, 0.f, 0.f};
      const bool mine = lane < nv;
      if (mine) {
        o = *reinterpret_cast<const float4*>(out + rb + 4 * lane);
        if constexpr (sizeof(BT) == 4) {
          const float4 t = *reinterpret_cast<const float4*>(bout + rb + 4 * lane);
          b[0] = t.x; b[1] = t.y; b[2] = t.z; b[3] = t.w;
        } else {
          const uint2 t = *reinterpret_cast<const uint2*>(bout + rb + 4 * lane);
          const __nv_bfloat162 p0 = *reinterpret_cast<const __nv_bfloat162*>(&t.x);
          const __nv_bfloat162 p1 = *reinterpret_cast<const __nv_bfloat162*>(&t.y);
          b[0] = __low2float(p0); b[1] = __high2float(p0);
          b[2] = __low2float(p1); b[3] = __high2float(p1);
        }
      }
      l1 = __shfl_sync(0xffffffffu, l1, 0);
      l2 = __shfl_sync(0xffffffffu, l2, 0);
      const float mx = fmaxf(l1, l2);
      float w1 = 0.f, w2 = 0.f, lnew = -INFINITY;
      if (mx != -INFINITY) {
        const float e1 = expf(l1 - mx), e2 = expf(l2 - mx);
        const float sum = e1 + e2;
        lnew = mx + logf(sum);
        w1 = e1 / sum;
        w2 = e2 / sum;
      }
      if (lane == 0) lse[li] = lnew;
      if (mine && mx != -INFINITY) {
        o.x = w1 * o.x + w2 * b[0];
        o.y = w1 * o.y + w2 * b[1];
        o.z = w1 * o.z + w2 * b[2];
        o.w = w1 * o.w + w2 * b[3];
        *reinterpret_cast<float4*>(out + rb + 4 * lane) = o;
      }
    } else {
      l1 = __shfl_sync(0xffffffffu, l1, 0);
      l2 = __shfl_sync(0xffffffffu, l2, 0);
      const float mx = fmaxf(l1, l2);
      float w1 = 0.f, w2 = 0.f, lnew = -INFINITY;
      if (mx != -INFINITY) {
        const float e1 = expf(l1 - mx), e2 = expf(l2 - mx);
        const float sum = e1 + e2;
        lnew = mx + logf(sum);
        w1 = e1 / sum;
        w2 = e2 / sum;
      }
      if (lane == 0) lse[li] = lnew;
      if (mx == -INFINITY) continue;
      for (int c = lane; c < nv; c += 32) out[rb + c] = w1 * out[rb + c] + w2 * ldf(bout + rb + c);
    }
  }
}

// ------------------------------------------------------------------ backward preprocess
// delta[row, h] = sum_d dO[row, h, d] * O[row, h, d]  (f32), one warp per (row, head). A warp has
// the loads of kDeltaRows of them in flight, and 32-bit divisions (measured on GB300, 65536 tokens,
// 32 heads of 128: 0.1 ms less than one row at a time with 64-bit ones); every row is summed in the
// same order whatever the count.
constexpr int kDeltaRows = 4;
template <typename T>
__global__ void __launch_bounds__(kThreads)
    delta_kernel(const __grid_constant__ Plan P, const T* __restrict__ o, const T* __restrict__ dout,
                 float* __restrict__ delta) {
  const SeqDesc& sd = P.seq[blockIdx.y];
  const int L = sd.L, dh = P.head_dim, lane = threadIdx.x & 31;
  // tokens x query heads stay below 2^31: 32-bit divisions
  const uint32_t units = static_cast<uint32_t>(plan_ranks(P)) * L * P.hq;
  constexpr uint32_t kWarps = kThreads / 32;
  for (uint32_t u0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kDeltaRows; u0 < units;
       u0 += gridDim.x * kWarps * kDeltaRows) {
    float s[kDeltaRows];
    size_t out[kDeltaRows];
#pragma unroll
    for (int k = 0; k < kDeltaRows; ++k) {
      const uint32_t u = u0 + k;
      s[k] = 0.f;
      out[k] = 0;
      if (u < units) {
        const uint32_t x = u / P.hq;
        const int h = static_cast<int>(u - x * P.hq);
        const int ri = static_cast<int>(x / L), a = static_cast<int>(x - ri * L);
        const int r = P.rank_only >= 0 ? P.rank_only : ri;
        const size_t base = (static_cast<size_t>(sd.row_off + r * P.shard_stride + a) * P.hq + h) * dh;
        out[k] = lse_index(P, sd, h, r, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // head_dim <= 128
          const int d = lane + 32 * i;
          if (d < dh) s[k] += ldf(o + base + d) * ldf(dout + base + d);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kDeltaRows; ++k) {
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], w);
      if (lane == 0 && u0 + k < units) delta[out[k]] = s[k];
    }
  }
}

// ------------------------------------------------------------------ backward postprocess
// dq = bf16(dq sums); the tensor-core kernel already applied the softmax scale.
__global__ void __launch_bounds__(kThreads)
    dq_convert_kernel(const float4* __restrict__ acc, uint2* __restrict__ dq, long n4, float scale) {
  for (long i = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x; i < n4;
       i += static_cast<long>(gridDim.x) * kThreads) {
    const float4 a = acc[i];
    const __nv_bfloat162 p0 = __floats2bfloat162_rn(a.x * scale, a.y * scale);
    const __nv_bfloat162 p1 = __floats2bfloat162_rn(a.z * scale, a.w * scale);
    uint2 o;
    o.x = *reinterpret_cast<const uint32_t*>(&p0);
    o.y = *reinterpret_cast<const uint32_t*>(&p1);
    dq[i] = o;
  }
}

// ------------------------------------------------------------------ permutations
// direction 0: natural -> shard-major; 1: shard-major -> natural. One warp per token row.
template <typename V>
__global__ void __launch_bounds__(kThreads)
    shard_tokens_kernel(const __grid_constant__ Plan P, int direction, const V* __restrict__ src,
                        V* __restrict__ dst, int nvec) {
  const SeqDesc& sd = P.seq[blockIdx.y];
  const int L = sd.L, lane = threadIdx.x & 31;
  const long units = static_cast<long>(P.D) * L;
  constexpr int kWarps = kThreads / 32;
  for (long u = static_cast<long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<long>(gridDim.x) * kWarps) {
    const int a = static_cast<int>(u % L);
    const int r = static_cast<int>(u / L);
    const size_t sm = static_cast<size_t>(sd.row_off) + static_cast<size_t>(r) * P.shard_stride + a;
    const size_t nat = static_cast<size_t>(sd.nat_off) + static_cast<size_t>(layout_pos(P.layout, P.D, L, r, a));
    const size_t from = direction == 0 ? nat : sm, to = direction == 0 ? sm : nat;
    for (int c = lane; c < nvec; c += 32) dst[to * nvec + c] = src[from * nvec + c];
  }
}

__global__ void __launch_bounds__(kThreads)
    shard_lse_kernel(const __grid_constant__ Plan P, int direction, const float* __restrict__ src,
                     float* __restrict__ dst) {
  const SeqDesc& sd = P.seq[blockIdx.y];
  const int L = sd.L;
  const long units = static_cast<long>(P.hq) * P.D * L;
  for (long u = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x; u < units;
       u += static_cast<long>(gridDim.x) * kThreads) {
    const int a = static_cast<int>(u % L);
    const int r = static_cast<int>((u / L) % P.D);
    const int h = static_cast<int>(u / (static_cast<long>(L) * P.D));
    const size_t sm = lse_index(P, sd, h, r, a);
    const size_t nat = static_cast<size_t>(sd.lse_nat_off) + static_cast<size_t>(h) * P.lse_hstride +
                       static_cast<size_t>(layout_pos(P.layout, P.D, L, r, a));
    if (direction == 0) dst[sm] = src[nat]; else dst[nat] = src[sm];
  }
}

}  // namespace

cudaError_t launch_merge(const Plan& P, float* out, float* lse, const void* block_out,
                         int block_f32, const float* block_lse, cudaStream_t st) {
  const bool aligned = (reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(block_out)) % 16 == 0;
  const int vec = P.head_dim % 4 == 0 && aligned ? 4 : 1;
  const long work = plan_ranks(P) * max_len(P) * P.hq;  // one warp per (row, head)
  const dim3 grid(grid_for(work, kThreads / 32), P.n_seqs);
  if (block_f32) {
    if (vec == 4) merge_kernel<float, 4><<<grid, kThreads, 0, st>>>(P, out, lse, (const float*)block_out, block_lse);
    else merge_kernel<float, 1><<<grid, kThreads, 0, st>>>(P, out, lse, (const float*)block_out, block_lse);
  } else {
    if (vec == 4) merge_kernel<__nv_bfloat16, 4><<<grid, kThreads, 0, st>>>(P, out, lse, (const __nv_bfloat16*)block_out, block_lse);
    else merge_kernel<__nv_bfloat16, 1><<<grid, kThreads, 0, st>>>(P, out, lse, (const __nv_bfloat16*)block_out, block_lse);
  }
  return cudaGetLastError();
}

cudaError_t launch_bwd_delta(const Plan& P, int dtype, const void* out, const void* dout,
                             float* delta, cudaStream_t st) {
  const long work = plan_ranks(P) * max_len(P) * P.hq;
  const dim3 grid(grid_for(work, kThreads / 32 * kDeltaRows), P.n_seqs);
  if (dtype == RA_F32)
    delta_kernel<float><<<grid, kThreads, 0, st>>>(P, (const float*)out, (const float*)dout, delta);
  else
    delta_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(P, (const __nv_bfloat16*)out, (const __nv_bfloat16*)dout, delta);
  return cudaGetLastError();
}

cudaError_t launch_dq_convert(const Plan& P, const float* dq_acc, void* dq, cudaStream_t st) {
  const long n4 = static_cast<long>(P.n_rows) * P.hq * P.head_dim / 4;
  dq_convert_kernel<<<grid_for(n4, kThreads), kThreads, 0, st>>>(
      reinterpret_cast<const float4*>(dq_acc), reinterpret_cast<uint2*>(dq), n4, 1.f);
  return cudaGetLastError();
}

cudaError_t launch_shard_tokens(const Plan& P, int direction, const void* src, void* dst,
                                int64_t row_bytes, cudaStream_t st) {
  const long work = P.D * max_len(P);
  const dim3 grid(grid_for(work, kThreads / 32), P.n_seqs);
  const uintptr_t al = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst);
  if (row_bytes % 16 == 0 && al % 16 == 0)
    shard_tokens_kernel<uint4><<<grid, kThreads, 0, st>>>(P, direction, (const uint4*)src, (uint4*)dst, (int)(row_bytes / 16));
  else if (row_bytes % 4 == 0 && al % 4 == 0)
    shard_tokens_kernel<uint32_t><<<grid, kThreads, 0, st>>>(P, direction, (const uint32_t*)src, (uint32_t*)dst, (int)(row_bytes / 4));
  else
    shard_tokens_kernel<uint8_t><<<grid, kThreads, 0, st>>>(P, direction, (const uint8_t*)src, (uint8_t*)dst, (int)row_bytes);
  return cudaGetLastError();
}

cudaError_t launch_shard_lse(const Plan& P, int direction, const float* src, float* dst,
                             cudaStream_t st) {
  const long work = static_cast<long>(P.hq) * P.D * max_len(P);
  const dim3 grid(grid_for(work, kThreads), P.n_seqs);
  shard_lse_kernel<<<grid, kThreads, 0, st>>>(P, direction, src, dst);
  return cudaGetLastError();
}

}  // namespace ra
