// ra_extend_few.cu — the part of the attention of new tokens over a paged cache (ra_extend.cu) that has
// at most 8 or 16 rows a K/V head: one token or a few of a sequence behind a shared prefix, drafted tokens
// to be checked, a short prefix of a small group. bf16.
//
// Memory-bound like the decode attention, and made like it: the rows, (token, query head), are the 16
// rows of m16n8k16 products; a warp takes 16 of a tile's 64 keys, copies them by cp.async into its own
// ring of stages and keeps running max, sum and O = P V in registers; the four warps' states are
// joined when a piece ends, and the ring runs on over its end. P goes into the product as two bf16
// numbers (2^-16). What is added are masks by row: a row at position p sees the keys up to p, and
// with a window those from p - window + 1 on and the first few. Keys that no row sees are not read.
//
// What bounds it: the start, about 6 us from the plan over the block table to the first keys, then memory: 33
// sequences of up to 4 drafted tokens, window 1024 + 4, 8 heads of 64, 70 MB in 23 us; 64 sequences' own keys
// behind a shared prefix, 32/8 heads of 128, 63 MB in 27 us.
//
// WIDE: more than 8 rows in some segment (else the second numbers of P take the product's empty rows).
#include <cuda_bf16.h>

#include "ra_extend.cuh"

namespace ra {

static __device__ unsigned int g_status_few;  // an index outside the cache

namespace {

constexpr int kThreads = 128;
constexpr int kKeys = 64;  // of a tile

template <int DH>
struct Cfg {
  static constexpr int PITCH = DH * 2 + 16;     // bytes of a key's row in a stage: ldmatrix meets every bank once
  static constexpr int STAGE = 2 * 16 * PITCH;  // a warp's K and V of 16 keys
  static constexpr int STAGES = DH == 128 ? 2 : 3;  // as in the decode attention, where it is measured
  static constexpr int CTAS = DH == 128 ? 2 : 3;    // on an SM
  static constexpr int RING = 4 * STAGES * STAGE;
  static constexpr int CHUNK = 8192 / (4 * DH * 4);  // rows joined at a time
  static constexpr int SMEM = RING + 8192;
};

// A walk over the tiles of a CTA's share.
struct Tiles {
  ExtCursor<kExtFew> cur;
  ExtItem it;
  int j;
  bool more;

  __device__ __forceinline__ void begin(const ExtArgs& A) {
    more = cur.begin(A, blockIdx.x) && cur.next(A, it);
    j = it.j0;
  }
  __device__ __forceinline__ bool last() const { return j + 1 == it.j0 + it.tiles; }
  __device__ __forceinline__ void next_item(const ExtArgs& A) {
    more = cur.next(A, it);
    j = it.j0;
  }
};

// Of the 16 keys from key0 on, of walk index j: whether a row sees some of them.
__device__ __forceinline__ bool some_seen(const ExtItem& it, int j, int key0, int sinks) {
  return key0 < sinks || (j >= it.walk.ns && key0 < it.end && key0 + 16 > it.low);
}

template <int DH, bool WIDE>
__global__ void __launch_bounds__(kThreads, Cfg<DH>::CTAS) extend_few(const __grid_constant__ ExtArgs A) {
  using C = Cfg<DH>;
  constexpr int KS = DH / 16;                  // steps of 16 elements
  constexpr int LANES = DH * 2 / 16;           // lanes that copy one row
  constexpr int ROWS = 32 / LANES;             // rows of one copy instruction
  constexpr int NS = C::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sm_m[4][16], sm_l[4][16];
  wait_for_previous();
  launch_dependents();  // (after it: the kernel for many rows relies on that)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * NS * C::STAGE;
  float* joined = reinterpret_cast<float*>(smem + C::RING);  // [4][CHUNK][DH]
  const char* kp = static_cast<const char*>(A.k_pages);
  const char* vp = static_cast<const char*>(A.v_pages);
  const int window = A.sh[kExtFew].window;

  // the load side: rows of the next tile's keys (lane i: key i; -1: no tile), then its copies
  Tiles load;
  load.begin(A);
  Tiles at = load;  // the side that computes
  int64_t row = -1;
  auto look_up = [&]() {
    row = -1;
    if (!load.more) return;
    const ExtItem& it = load.it;
    const int key0 = ext_tile(it.walk, load.j) * kKeys + warp * 16;
    const int sinks = window > 0 ? min(A.sh[kExtFew].sinks, it.end) : 0;
    if (some_seen(it, load.j, key0, sinks)) {
      int key = key0 + (lane & 15);  // a key that is not seen: one that is, in its place
      if (key >= sinks) key = load.j < it.walk.ns ? sinks - 1 : min(max(key, it.low), it.end - 1);
      const int page = key / A.page_size;
      row = (ext_page(A, it.seq, page, &g_status_few) * A.page_stride +
             static_cast<int64_t>(key - page * A.page_size) * A.slot_stride + it.hk * A.head_stride) * 2;
    }
    if (load.last()) load.next_item(A); else ++load.j;
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
  while (at.more) {
    const ExtItem& it = at.it;
    const int rows = it.ntok * it.heads, heads = it.heads;
    const int64_t q0 = static_cast<int64_t>(it.tok0) * A.hq + it.hk * A.group;  // (token, head) of row 0
    uint32_t qa[KS][WIDE ? 4 : 2];
    int hi[2], lo[2];  // of this lane's rows: keys lo .. hi - 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i, tok = r / heads;
      const bool on = r < rows;
      hi[i] = !on || it.shared ? it.end : it.base + tok + 1;
      lo[i] = window > 0 ? max(0, hi[i] - window) : 0;
      if (i == 1 && !WIDE) continue;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(A.q) +
                               (q0 + static_cast<int64_t>(tok) * A.hq + r - tok * heads) * DH;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)  // element half
          qa[k][2 * i + e] = on ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 * e + 2 * c) : 0u;
    }
    // keys that every row sees: from..to-1
    const int from = window > 0 ? max(0, it.end - window) : 0, to = it.shared ? it.end : it.base + 1;
    const int sinks = window > 0 ? min(A.sh[kExtFew].sinks, it.end) : 0;
    float o[DH / 8][4], small[DH / 8][4];  // P V, and that of P's second numbers (not WIDE: o's rows 8..15)
#pragma unroll
    for (int n = 0; n < DH / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = small[n][i] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (const int j1 = it.j0 + it.tiles; at.j < j1; ++at.j) {
      copy(stage == 0 ? NS - 1 : stage - 1);
      look_up();
      cp_async_wait<NS - 1>();
      __syncwarp();
      const int key0 = ext_tile(it.walk, at.j) * kKeys + warp * 16;
      if (some_seen(it, at.j, key0, sinks)) {
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
        const bool part = key0 < from || key0 + 16 > to;
#pragma unroll
        for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = s[i >> 1][2 * r + (i & 1)] * A.scale_log2;
            if (part) {
              const int key = key0 + (i >> 1) * 8 + 2 * c + (i & 1);
              if (!(key < hi[r] && (key >= lo[r] || key < sinks))) x[i] = -INFINITY;
            }
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

    auto sum_of = [&](int n, int r, int i) {
      const float x = WIDE ? small[n][2 * r + i] : o[n][2 + i];
      return o[n][2 * r + i] + (fabsf(x) <= 3.402823466e38f ? x : 0.f);  // (of an infinite v P's own sign counts)
    };
    // the four warps' states into one, CHUNK rows at a time
#pragma unroll
    for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (c == 0) {
        sm_m[warp][g + 8 * r] = m[r];
        sm_l[warp][g + 8 * r] = l[r];
      }
    }
    const int dest = it.dest;
    for (int r0 = 0; r0 < rows; r0 += C::CHUNK) {
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
        const int h = i / (DH / 4), d = i % (DH / 4) * 4, r = r0 + h;
        if (r >= rows) break;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, sm_m[w][r]);
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = ex2(sm_m[w][r] - ref);
          const float4 y = *reinterpret_cast<const float4*>(joined + (w * C::CHUNK + h) * DH + d);
          L += f * sm_l[w][r];
          x.x += f * y.x;
          x.y += f * y.y;
          x.z += f * y.z;
          x.w += f * y.w;
        }
        const int tok = r / heads;
        const int64_t where = q0 + static_cast<int64_t>(tok) * A.hq + r - tok * heads;
        if (dest == kExtFinal) {
          const float inv = L > 0.f ? 1.f / L : 0.f;
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(A.out) + where * DH + d) =
              make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
          if (d == 0) A.lse[where] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
        } else {
          const int64_t to = dest == kExtRows ? static_cast<int64_t>(it.slot) * A.n_tokens * A.hq + where
                                              : static_cast<int64_t>(it.slot) * A.part[kExtFew].rows + r;
          *reinterpret_cast<float4*>((dest == kExtRows ? A.row_o : A.part[kExtFew].o) + to * DH + d) = x;
          if (d == 0) (dest == kExtRows ? A.row_ml : A.part[kExtFew].ml)[to] = make_float2(M, L);
        }
      }
      __syncthreads();
    }
    at.next_item(A);
  }
}

template <int DH, bool WIDE>
cudaError_t launch(const ExtArgs& A, cudaStream_t st) {
  auto kernel = extend_few<DH, WIDE>;
  static std::atomic<bool> done[kExtDevices];
  const cudaError_t e = ext_allow_smem(kernel, Cfg<DH>::SMEM, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(A.part[kExtFew].most_ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<DH>::SMEM;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, A);
}

}  // namespace

int extend_few_ctas(int head_dim) { return (head_dim == 128 ? Cfg<128>::CTAS : Cfg<64>::CTAS) * kExtSms; }

cudaError_t extend_few_status(unsigned int* value, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_status_few, sizeof g_status_few);
  if (e == cudaSuccess && reset) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_status_few, &zero, sizeof zero);
  }
  return e;
}

cudaError_t launch_extend_few(const ExtArgs& A, cudaStream_t st) {
  const bool wide = A.part[kExtFew].rows > 8;
  if (A.dh == 128) return wide ? launch<128, true>(A, st) : launch<128, false>(A, st);
  return wide ? launch<64, true>(A, st) : launch<64, false>(A, st);
}

}  // namespace ra
