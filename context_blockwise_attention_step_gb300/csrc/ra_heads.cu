// ra_heads.cu — per-head norm of queries and keys with the rotation by position in the same
// pass (forward and backward over a ring problem's rows), and the append of new tokens to a
// paged cache, which does the same on its way there.
//
//   n = x * r,  r = rsqrt(mean(x^2) + eps);   y = R(pos) (n * w)
//   backward: g = R(pos)^T dy;  dw = sum g * n;  h = g * w;  dx = r * (h - n * mean(h * n))
//
// A token's position is its place in its sequence, or it has positions on several axes (time, height,
// width), given with the tokens, and every pair of the rotation turns by one of them.
//
// Angles: pair i turns by pos * inv_freq[i]. A float product would lose the angle at far
// positions (at 2^17 the spacing of floats near pos * 1 rad is 2^-7 rad), so inv_freq / 2pi is
// kept as a 64-bit fraction of a turn: its product with the position, modulo 2^64, is the
// angle within the turn, and the top 32 bits, rounded to a float, go to sincospif: 2^-26 of a turn at
// any position.
//
// What bounds these kernels is the bytes: every element is read once and written once, statistics
// and angles stay in registers. 131072 tokens, 32/8 heads of 128, bf16, on GB300: forward 440 us
// (6.10 TB/s), backward 669 us (6.02 TB/s); 16 prompts of up to 8192 tokens into a cache 260 us
// (6.2 TB/s); 2 x 4096 tokens, 8 heads of 64: 11 and 16 us, four new tokens 4 us, which is latency.
// Positions on three axes cost 12 bytes a token and a load beside each angle, of a line that is in L1: 1112
// us forward and backward of the first (1109 by place), 267 us the second.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "ra_internal.h"
#include "ra_layout.h"
#include "ra_ptx.cuh"

namespace ra {

static __device__ unsigned int g_status_append;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Rows of a ring problem, in natural order of the sequences (unlike the launch plans' table,
// which is sorted by length).
struct RingRows {
  int32_t layout, D, n_seqs;
  int32_t seqlen;                     // batch mode: S; varlen mode: 0
  int32_t shard_rows;                 // varlen mode: rows of one rank's buffer (T / D)
  int32_t cu_local[RA_MAX_SEQS + 1];  // varlen mode: cu_seqlens / D
};

// Rows of new tokens of the sequences of a paged cache.
struct CacheRows {
  const int32_t* seq_lens;
  const int32_t* cu_new;  // null: row b is the one new token of sequence b
  const int32_t* block_table;
  int64_t table_stride, page_stride, slot_stride, head_stride;
  int32_t n_seqs, max_pages, page_size, n_pages;
};

// Positions on several axes: `stride` elements from one row's to the next.
struct AxisPos {
  const int32_t* pos;
  int64_t stride;
  uint8_t axis[RA_MAX_ROTARY_DIM / 2];  // of every pair
};
// The rows of a ring problem, whose order does not matter then, and of a cache.
struct RingAxisRows {
  AxisPos at;
};
struct CacheAxisRows {
  CacheRows rows;
  AxisPos at;
};

// One token: its position, and where its k and v go.
struct Token {
  int64_t pos;
  int64_t kv;        // element offset of head 0 in k_out / v_out
  bool absent;       // a row that belongs to no sequence: nothing is written
  bool idle;         // q_out = 0, no k and v
};

__device__ __forceinline__ Token locate(const RingRows& R, int row, int64_t kv_row) {
  Token t;
  t.absent = t.idle = false;
  t.kv = static_cast<int64_t>(row) * kv_row;
  if (R.seqlen > 0) {
    const int x = row % R.seqlen, L = R.seqlen / R.D;
    t.pos = layout_pos(R.layout, R.D, L, x / L, x % L);
  } else {
    const int r = row / R.shard_rows, x = row % R.shard_rows;
    int lo = 0, hi = R.n_seqs - 1;  // the last sequence that starts at or before x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (R.cu_local[mid] <= x) lo = mid; else hi = mid - 1;
    }
    const int a0 = R.cu_local[lo];
    t.pos = layout_pos(R.layout, R.D, R.cu_local[lo + 1] - a0, r, x - a0);
  }
  return t;
}

__device__ __forceinline__ Token locate(const CacheRows& R, int row, int64_t) {
  Token t;
  t.kv = 0;
  t.pos = 0;
  t.absent = t.idle = false;
  int b = row;
  int64_t behind = 0;  // tokens of the sequence after this one
  if (R.cu_new != nullptr) {
    if (row < R.cu_new[0] || row >= R.cu_new[R.n_seqs]) {
      t.absent = true;
      return t;
    }
    int lo = 0, hi = R.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (R.cu_new[mid] <= row) lo = mid; else hi = mid - 1;
    }
    b = lo;
    behind = static_cast<int64_t>(R.cu_new[b + 1]) - 1 - row;
  }
  const int len = R.seq_lens[b];
  t.pos = static_cast<int64_t>(len) - 1 - behind;
  if (len == 0 && R.cu_new == nullptr) {
    t.idle = true;
    return t;
  }
  const int64_t page = t.pos / R.page_size;
  int64_t at = -1;
  if (t.pos >= 0 && page < R.max_pages) at = R.block_table[b * R.table_stride + page];
  if (at < 0 || at >= R.n_pages) {
    t.idle = true;
    atomicOr(&g_status_append, 1u);
    return t;
  }
  t.kv = at * R.page_stride + (t.pos - page * R.page_size) * R.slot_stride;
  return t;
}

__device__ __forceinline__ Token locate(const RingAxisRows&, int row, int64_t kv_row) {
  Token t;
  t.absent = t.idle = false;
  t.kv = static_cast<int64_t>(row) * kv_row;
  t.pos = 0;
  return t;
}
__device__ __forceinline__ Token locate(const CacheAxisRows& R, int row, int64_t kv_row) {
  return locate(R.rows, row, kv_row);
}

// The position that pair `pair` of row `row` turns by; `place` is the row's place in its sequence.
template <typename Rows>
__device__ __forceinline__ int64_t turn_by(const Rows&, int64_t, int64_t place, int) {
  return place;
}
__device__ __forceinline__ int64_t turn_by(const AxisPos& P, int64_t row, int pair) {
  return P.pos[row * P.stride + P.axis[pair]];
}
__device__ __forceinline__ int64_t turn_by(const RingAxisRows& R, int64_t row, int64_t, int pair) {
  return turn_by(R.at, row, pair);
}
__device__ __forceinline__ int64_t turn_by(const CacheAxisRows& R, int64_t row, int64_t, int pair) {
  return turn_by(R.at, row, pair);
}

__device__ __forceinline__ float ldf(const float* p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void stf(float* p, float v) { *p = v; }
__device__ __forceinline__ void stf(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float2 cos_sin(uint64_t turns, int64_t pos) {
  const int32_t t = static_cast<int32_t>((turns * static_cast<uint64_t>(pos)) >> 32);
  float s, c;
  sincospif(static_cast<float>(t) * 4.656612873077393e-10f, &s, &c);  // half turns: t * 2^-31
  return make_float2(c, s);
}

// What every kernel here gets by value.
struct HeadArgs {
  ra_rope rope;  // rotary_dim 0: none
  float eps;
  int hq, hkv, dh, n_rows;
  int64_t q_stride, k_stride, v_stride;  // elements between the rows of the inputs
  int64_t kv_head;                       // elements between the heads of k_out and v_out
};

// ---------------------------------------------------------------- any head size and alignment
// Lane l holds elements l, l + 32, ... of a head; a head's row goes through shared memory to reach
// the lanes' rotation partners: y[d] = cs[d] x[d] + sn[d] x[other[d]]. A warp takes a token (or a
// share of its heads), so that a token's position and angles are worked out once.
constexpr int kPerLane = 4;  // head_dim <= 128
struct LaneTurn {
  float cs[kPerLane], sn[kPerLane];
  int other[kPerLane];
};
template <typename Rows>
__device__ __forceinline__ LaneTurn lane_turn(const HeadArgs& A, const Rows& R, int64_t token, int64_t place, int lane,
                                              float sign) {
  LaneTurn t;
  const int rd = A.rope.rotary_dim;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int d = lane + 32 * i;
    t.cs[i] = 1.f;
    t.sn[i] = 0.f;
    t.other[i] = d;
    if (d < rd) {
      const bool second = A.rope.interleaved ? d & 1 : d >= rd / 2;
      const int pair = A.rope.interleaved ? d >> 1 : second ? d - rd / 2 : d;
      t.other[i] = A.rope.interleaved ? d ^ 1 : second ? d - rd / 2 : d + rd / 2;
      const float2 c = cos_sin(A.rope.turns[pair], turn_by(R, token, place, pair));
      t.cs[i] = c.x;
      t.sn[i] = second ? sign * c.y : -sign * c.y;
    }
  }
  return t;
}
__device__ __forceinline__ void apply(const LaneTurn& t, float* row, int dh, int lane, float (&x)[kPerLane]) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPerLane; ++i)
    if (lane + 32 * i < dh) row[lane + 32 * i] = x[i];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPerLane; ++i)  // (what is not rotated stays as it is, infinities too)
    if (lane + 32 * i < dh && t.other[i] != lane + 32 * i) x[i] = t.cs[i] * x[i] + t.sn[i] * row[t.other[i]];
}
template <typename T>
__device__ __forceinline__ void load_lane(const T* p, int dh, int lane, float (&x)[kPerLane]) {
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) x[i] = lane + 32 * i < dh ? ldf(p + lane + 32 * i) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store_lane(T* p, int dh, int lane, const float (&x)[kPerLane]) {
#pragma unroll
  for (int i = 0; i < kPerLane; ++i)
    if (lane + 32 * i < dh) stf(p + lane + 32 * i, x[i]);
}

// Heads first, first + step, ... of a token's q, k or v, U of them loaded ahead.
template <typename T>
__device__ __forceinline__ void any_run(const HeadArgs& A, const T* w, bool turned, const LaneTurn& turn,
                                        const T* src, T* dst, int64_t dst_head, int heads, int first, int step,
                                        float* row, int lane) {
  constexpr int U = 2;
  const int dh = A.dh;
  float wl[kPerLane];
  if (w != nullptr) load_lane(w, dh, lane, wl);
  for (int h0 = first; h0 < heads; h0 += U * step) {
    float x[U][kPerLane];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h0 + u * step < heads) load_lane(src + static_cast<int64_t>(h0 + u * step) * dh, dh, lane, x[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
      if (h >= heads) break;
      if (w != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) ss += x[u][i] * x[u][i];
        const float r = rsqrtf(warp_sum(ss) / dh + A.eps);
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) x[u][i] = lane + 32 * i < dh ? x[u][i] * r * wl[i] : 0.f;
      }
      if (turned) apply(turn, row, dh, lane, x[u]);
      store_lane(dst + h * dst_head, dh, lane, x[u]);
    }
  }
}

template <typename T, typename Rows, bool CACHE>
__global__ void __launch_bounds__(kThreads)
    heads_fwd_any(const __grid_constant__ HeadArgs A, const __grid_constant__ Rows R, int parts,
                  const T* __restrict__ qw, const T* __restrict__ kw, const T* q, const T* k, const T* v,
                  T* q_out, T* k_out, T* v_out) {
  __shared__ float rows[kWarps][128];
  const int lane = threadIdx.x & 31, dh = A.dh;
  float* row = rows[threadIdx.x >> 5];
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t t = unit / parts;
  const int part = static_cast<int>(unit - t * parts);
  if (t >= A.n_rows) return;
  const Token tok = locate(R, static_cast<int>(t), A.hkv * static_cast<int64_t>(dh));
  if (tok.absent) return;
  T* qo = q_out + t * A.hq * dh;
  if (tok.idle) {
    const float zero[kPerLane] = {};
    for (int h = part; h < A.hq; h += parts) store_lane(qo + static_cast<int64_t>(h) * dh, dh, lane, zero);
    return;
  }
  const bool turned = A.rope.rotary_dim > 0;
  const LaneTurn turn = lane_turn(A, R, t, tok.pos, lane, 1.f);
  any_run(A, qw, turned, turn, q + t * A.q_stride, qo, dh, A.hq, part, parts, row, lane);
  // the next run of heads goes on with the part after the last one's
  const int pk = ((part - A.hq) % parts + parts) % parts;
  any_run(A, kw, turned, turn, k + t * A.k_stride, k_out + tok.kv, A.kv_head, A.hkv, pk, parts, row, lane);
  if constexpr (CACHE) {
    const int pv = ((pk - A.hkv) % parts + parts) % parts;
    any_run<T>(A, nullptr, false, turn, v + t * A.v_stride, v_out + tok.kv, A.kv_head, A.hkv, pv, parts, row, lane);
  }
}

// The weight gradients of the lanes' elements are summed in registers over a warp's tokens, over
// the block's warps in shared memory, and written per block. `parts` as above (a part's heads stay
// the same, so that the sums do not depend on the order).
template <typename T>
__device__ __forceinline__ void any_run_bwd(const HeadArgs& A, const T* w, bool turned, const LaneTurn& turn,
                                            const T* x, const T* dy, T* dx, int heads, int first, int step,
                                            float* row, int lane, float (&acc)[kPerLane]) {
  const int dh = A.dh;
  float wl[kPerLane];
  if (w != nullptr) load_lane(w, dh, lane, wl);
  constexpr int U = 2;
  for (int h0 = first; h0 < heads; h0 += U * step) {
    float gu[U][kPerLane], nu[U][kPerLane];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t h = h0 + u * step;
      if (h < heads) {
        load_lane(dy + h * dh, dh, lane, gu[u]);
        if (w != nullptr) load_lane(x + h * dh, dh, lane, nu[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
      if (h >= heads) break;
      float (&g)[kPerLane] = gu[u], (&n)[kPerLane] = nu[u];
      if (turned) apply(turn, row, dh, lane, g);
      if (w != nullptr) {
        float ss = 0.f, hn = 0.f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) ss += n[i] * n[i];
        const float r = rsqrtf(warp_sum(ss) / dh + A.eps);
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
          n[i] *= r;
          acc[i] += g[i] * n[i];
          g[i] = lane + 32 * i < dh ? g[i] * wl[i] : 0.f;
          hn += g[i] * n[i];
        }
        const float mean = warp_sum(hn) / dh;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) g[i] = r * (g[i] - n[i] * mean);
      }
      store_lane(dx + static_cast<int64_t>(h) * dh, dh, lane, g);
    }
  }
}

template <typename T, typename Rows>
__global__ void __launch_bounds__(kThreads)
    heads_bwd_any(const __grid_constant__ HeadArgs A, const __grid_constant__ Rows R, int parts,
                  const T* __restrict__ qw, const T* __restrict__ kw, const T* __restrict__ q,
                  const T* __restrict__ k, const T* dq_out, const T* dk_out, T* dq, T* dk,
                  float* __restrict__ partial) {
  __shared__ float rows[kWarps][128];
  __shared__ float sums[kWarps][2][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dh = A.dh;
  float* row = rows[warp];
  float acc[2][kPerLane] = {};
  const bool turned = A.rope.rotary_dim > 0;
  const int64_t units = static_cast<int64_t>(A.n_rows) * parts;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < units;
       u += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t t = u / parts;
    const int part = static_cast<int>(u - t * parts);
    const LaneTurn turn = lane_turn(A, R, t, locate(R, static_cast<int>(t), 0).pos, lane, -1.f);
    const int64_t oq = t * A.hq * dh, ok = t * A.hkv * dh;
    any_run_bwd(A, qw, turned, turn, q + t * A.q_stride, dq_out + oq, dq + oq, A.hq, part, parts, row, lane, acc[0]);
    const int pk = ((part - A.hq) % parts + parts) % parts;
    any_run_bwd(A, kw, turned, turn, k + t * A.k_stride, dk_out + ok, dk + ok, A.hkv, pk, parts, row, lane, acc[1]);
  }
  if (qw == nullptr) return;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    sums[warp][0][lane + 32 * i] = acc[0][i];
    sums[warp][1][lane + 32 * i] = acc[1][i];
  }
  __syncthreads();
  {
    const int which = threadIdx.x >> 7, d = threadIdx.x & 127;  // kThreads = 2 * 128
    float s = 0.f;
    for (int w = 0; w < kWarps; ++w) s += sums[w][which][d];
    if (d < dh) partial[(static_cast<int64_t>(blockIdx.x) * 2 + which) * dh + d] = s;
  }
}

// ---------------------------------------------------------------- 16-byte loads
// A head is held by LANES lanes, each with two 16-byte pieces: the c-th of the first half and the
// c-th of the second half of the rotated elements, so that both members of a rotated pair are in
// one thread (interleaved pairs are anyway), or two neighbouring pieces of what is not rotated.
// The HEADS heads of a warp are loaded together.
// DH is the head size (64 or 128), or -32, -64, -128 for a multiple of 8 up to that: the last lanes
// of a head then have nothing, and HeadArgs has the size.
template <typename T, int DH>
struct Vec {
  static constexpr int SPAN = DH < 0 ? -DH : DH;
  static constexpr int N = 16 / sizeof(T);          // elements of a piece
  static constexpr int LANES = SPAN / 2 / N;        // lanes of a head
  static constexpr int HEADS = 32 / LANES;          // heads of a warp at a time
  static constexpr int PER = N / HEADS > 0 ? N / HEADS : 1;  // angles a lane works out
};

template <int DH>
__device__ __forceinline__ int size_of(const HeadArgs& A) {
  return DH < 0 ? A.dh : DH;
}
// Whether lane c of a head has pieces.
template <typename T, int DH>
__device__ __forceinline__ bool has_piece(const HeadArgs& A, int c) {
  return DH > 0 || c * 2 * Vec<T, DH>::N < A.dh;
}

template <typename T, int DH>
struct Piece {  // a lane's two pieces, as loaded
  uint4 a, b;
};
struct Place {
  int a, b;  // first elements of a lane's two pieces
};
template <typename T, int DH, bool INTER>
__device__ __forceinline__ Place place_of(const HeadArgs& A, int c) {
  constexpr int N = Vec<T, DH>::N;
  const int rd = A.rope.rotary_dim, turned = rd / 2 / N;  // lanes with pairs (not interleaved)
  if (INTER || rd == 0) return {c * N, size_of<DH>(A) / 2 + c * N};
  if (c < turned) return {c * N, rd / 2 + c * N};
  return {rd + (c - turned) * 2 * N, rd + (c - turned) * 2 * N + N};
}
template <typename T, int DH>
__device__ __forceinline__ Piece<T, DH> load_piece(const T* head, Place at) {
  Piece<T, DH> p;
  p.a = *reinterpret_cast<const uint4*>(head + at.a);
  p.b = *reinterpret_cast<const uint4*>(head + at.b);
  return p;
}
template <typename T, int DH>
__device__ __forceinline__ void store_piece(T* head, Place at, const Piece<T, DH>& p) {
  *reinterpret_cast<uint4*>(head + at.a) = p.a;
  *reinterpret_cast<uint4*>(head + at.b) = p.b;
}

__device__ __forceinline__ void widen(const uint4& v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x);
  x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z);
  x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void widen(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 narrow(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Cosines and sines of the pairs of this lane's pieces. The HEADS lanes that hold the same
// pieces of different heads need the same angles: each works out its share, and they exchange.
template <typename T, int DH, bool INTER, typename Rows>
__device__ __forceinline__ void piece_angles(const HeadArgs& A, const Rows& R, int64_t token, int64_t place, int lane,
                                             float (&cs)[Vec<T, DH>::N], float (&sn)[Vec<T, DH>::N]) {
  using V = Vec<T, DH>;
  const int c = lane % V::LANES, sub = lane / V::LANES;
  float2 mine[V::PER];
#pragma unroll
  for (int k = 0; k < V::PER; ++k) {
    const int j = (sub * V::PER + k) % V::N;
    const int pair = !INTER ? c * V::N + j : j < V::N / 2 ? c * V::N / 2 + j : size_of<DH>(A) / 4 + c * V::N / 2 + j - V::N / 2;
    mine[k] = pair < A.rope.rotary_dim / 2 ? cos_sin(A.rope.turns[pair], turn_by(R, token, place, pair)) : make_float2(1.f, 0.f);
  }
#pragma unroll
  for (int j = 0; j < V::N; ++j) {
    const int from = j / V::PER * V::LANES + c;
    cs[j] = __shfl_sync(0xffffffffu, mine[j % V::PER].x, from);
    sn[j] = __shfl_sync(0xffffffffu, mine[j % V::PER].y, from);
  }
}

// The rotated pairs of a lane's pieces: if interleaved, the first `a` of the first piece's and the
// first `b` of the second's; else all pairs that the two pieces make if a > 0, or none. What is not
// rotated stays as it is: turned by nothing, an infinity would make its neighbour and itself NaN. (1 %
// of the time where the whole head is rotated; a branch of its own for that case costs 1 % more.)
struct Turned {
  int a, b;
};
template <typename T, int DH, bool INTER>
__device__ __forceinline__ Turned turned_of(const HeadArgs& A, int c) {
  constexpr int N = Vec<T, DH>::N;
  const int pairs = A.rope.rotary_dim / 2;
  if (INTER) return {pairs - c * N / 2, pairs - size_of<DH>(A) / 4 - c * N / 2};
  return {pairs - c * N, 0};
}
// Turns a lane's pieces by +angle (sign 1) or -angle (sign -1).
template <int N, bool INTER>
__device__ __forceinline__ void turn(float (&a)[N], float (&b)[N], const float (&cs)[N], const float (&sn)[N],
                                     float sign, Turned n) {
  if constexpr (INTER) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const float x = a[2 * j], y = a[2 * j + 1], s = sign * sn[j];
      if (j < n.a) {
        a[2 * j] = x * cs[j] - y * s;
        a[2 * j + 1] = y * cs[j] + x * s;
      }
      const float u = b[2 * j], v = b[2 * j + 1], t = sign * sn[N / 2 + j];
      if (j < n.b) {
        b[2 * j] = u * cs[N / 2 + j] - v * t;
        b[2 * j + 1] = v * cs[N / 2 + j] + u * t;
      }
    }
  } else if (n.a > 0) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float x = a[j], y = b[j], s = sign * sn[j];
      a[j] = x * cs[j] - y * s;
      b[j] = y * cs[j] + x * s;
    }
  }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The heads `first`, `first + step`, ... (in warps' loads of HEADS heads) of one token's q, k or
// v: U loads in flight, then norm, rotation and store of each. The token's cosines and sines are in
// registers; prepare() is called once, with the first loads under way.
template <typename T, int DH, bool INTER, int U, typename F>
__device__ __forceinline__ void head_run(const HeadArgs& A, const T* __restrict__ w, bool turned, const T* src,
                                         T* dst, int64_t dst_head, int heads, int first, int step, int lane,
                                         const float (&cs)[Vec<T, DH>::N], const float (&sn)[Vec<T, DH>::N],
                                         F&& prepare) {
  using V = Vec<T, DH>;
  const Place at = place_of<T, DH, INTER>(A, lane % V::LANES);
  const int sub = lane / V::LANES, runs = (heads + V::HEADS - 1) / V::HEADS, dh = size_of<DH>(A);
  const bool on = has_piece<T, DH>(A, lane % V::LANES);
  const float per_dh = 1.f / dh;
  const Turned rotated = turned_of<T, DH, INTER>(A, lane % V::LANES);
  Piece<T, DH> wp = {};
  if (w != nullptr && on) wp = load_piece<T, DH>(w, at);
  for (int i0 = first; i0 < runs; i0 += step * U) {
    Piece<T, DH> p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (i0 + u * step) * V::HEADS + sub;
      if (DH < 0 && !on) p[u] = {};
      if (h < heads && on) p[u] = load_piece<T, DH>(src + h * dh, at);
    }
    if (i0 == first) prepare();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (i0 + u * step) * V::HEADS + sub;
      if (i0 + u * step >= runs) break;  // (the same for the whole warp)
      if (w != nullptr || turned) {
        float a[V::N], b[V::N];
        widen(p[u].a, a);
        widen(p[u].b, b);
        if (w != nullptr) {
          float ss = 0.f, wa[V::N], wb[V::N];
#pragma unroll
          for (int j = 0; j < V::N; ++j) ss += a[j] * a[j] + b[j] * b[j];
          const float r = rsqrtf(group_sum<V::LANES>(ss) * per_dh + A.eps);
          widen(wp.a, wa);
          widen(wp.b, wb);
#pragma unroll
          for (int j = 0; j < V::N; ++j) {
            a[j] *= r * wa[j];
            b[j] *= r * wb[j];
          }
        }
        if (turned) turn<V::N, INTER>(a, b, cs, sn, 1.f, rotated);
        p[u].a = narrow(a);
        p[u].b = narrow(b);
      }
      if (h < heads && on) store_piece<T, DH>(dst + h * dst_head, at, p[u]);
    }
  }
}

// A warp takes a token, or one of `parts` shares of its heads. Three blocks an SM with two loads of a
// lane in flight, measured at 131072 tokens, 32/8 heads of 128, bf16 (when it took 436 us): two blocks
// with four loads 450, three with four 485, four with two 475, three with one 487.
template <typename T, int DH, bool INTER, typename Rows, bool CACHE>
__global__ void __launch_bounds__(kThreads, 3)
    heads_fwd_vec(const __grid_constant__ HeadArgs A, const __grid_constant__ Rows R, int parts,
                  const T* __restrict__ qw, const T* __restrict__ kw, const T* q, const T* k, const T* v,
                  T* q_out, T* k_out, T* v_out) {
  using V = Vec<T, DH>;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t t = unit / parts;
  const int part = static_cast<int>(unit - t * parts), dh = size_of<DH>(A);
  if (t >= A.n_rows) return;
  const Token tok = locate(R, static_cast<int>(t), A.hkv * static_cast<int64_t>(dh));
  if (tok.absent) return;
  T* qo = q_out + t * A.hq * dh;
  if (tok.idle) {
    for (int h = part * V::HEADS + lane / V::LANES; h < A.hq; h += parts * V::HEADS) {
      Piece<T, DH> zero = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      if (has_piece<T, DH>(A, lane % V::LANES)) store_piece<T, DH>(qo + h * dh, place_of<T, DH, INTER>(A, lane % V::LANES), zero);
    }
    return;
  }
  float cs[V::N], sn[V::N];
  const bool turned = A.rope.rotary_dim > 0;
  auto angles = [&]() {
    if (turned) piece_angles<T, DH, INTER>(A, R, t, tok.pos, lane, cs, sn);
  };
  auto none = []() {};
  const int runs_q = (A.hq + V::HEADS - 1) / V::HEADS, runs_k = (A.hkv + V::HEADS - 1) / V::HEADS;
  if (part >= runs_q) angles();
  head_run<T, DH, INTER, 2>(A, qw, turned, q + t * A.q_stride, qo, dh, A.hq, part, parts, lane, cs, sn, angles);
  // the next run of heads goes on with the part after the last one's
  const int pk = ((part - runs_q) % parts + parts) % parts;
  head_run<T, DH, INTER, 2>(A, kw, turned, k + t * A.k_stride, k_out + tok.kv, A.kv_head, A.hkv, pk, parts, lane,
                            cs, sn, none);
  if constexpr (CACHE) {
    const int pv = ((pk - runs_k) % parts + parts) % parts;
    head_run<T, DH, INTER, 2>(A, nullptr, false, v + t * A.v_stride, v_out + tok.kv, A.kv_head, A.hkv, pv, parts,
                              lane, cs, sn, none);
  }
}

constexpr int kBwdThreads = 128;

// Backward of one token's q or k heads; `acc` gathers g * n of the lane's elements.
template <typename T, int DH, bool INTER, int U, typename F>
__device__ __forceinline__ void head_run_bwd(const HeadArgs& A, const T* __restrict__ w, bool turned, const T* x,
                                             const T* dy, T* dx, int heads, int lane,
                                             const float (&cs)[Vec<T, DH>::N], const float (&sn)[Vec<T, DH>::N],
                                             float (&acc_a)[Vec<T, DH>::N], float (&acc_b)[Vec<T, DH>::N],
                                             F&& prepare) {
  using V = Vec<T, DH>;
  const Place at = place_of<T, DH, INTER>(A, lane % V::LANES);
  const int sub = lane / V::LANES, dh = size_of<DH>(A);
  const bool on = has_piece<T, DH>(A, lane % V::LANES);
  const float per_dh = 1.f / dh;
  const Turned rotated = turned_of<T, DH, INTER>(A, lane % V::LANES);
  Piece<T, DH> wp = {};
  if (w != nullptr && on) wp = load_piece<T, DH>(w, at);
  for (int h0 = sub; h0 - sub < heads; h0 += V::HEADS * U) {
    Piece<T, DH> g[U], p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * V::HEADS;
      g[u].a = g[u].b = p[u].a = p[u].b = make_uint4(0u, 0u, 0u, 0u);
      if (h < heads && on) {
        g[u] = load_piece<T, DH>(dy + h * dh, at);
        if (w != nullptr) p[u] = load_piece<T, DH>(x + h * dh, at);
      }
    }
    if (h0 == sub) prepare();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * V::HEADS;
      if (h - sub >= heads) break;  // (the same for the whole warp)
      float a[V::N], b[V::N];
      widen(g[u].a, a);
      widen(g[u].b, b);
      if (turned) turn<V::N, INTER>(a, b, cs, sn, -1.f, rotated);
      if (w != nullptr) {
        float xa[V::N], xb[V::N], wv[V::N], ss = 0.f, hn = 0.f;
        widen(p[u].a, xa);
        widen(p[u].b, xb);
#pragma unroll
        for (int j = 0; j < V::N; ++j) ss += xa[j] * xa[j] + xb[j] * xb[j];
        const float r = rsqrtf(group_sum<V::LANES>(ss) * per_dh + A.eps);
        widen(wp.a, wv);
#pragma unroll
        for (int j = 0; j < V::N; ++j) {
          xa[j] *= r;
          acc_a[j] += a[j] * xa[j];
          a[j] *= wv[j];
          hn += a[j] * xa[j];
        }
        widen(wp.b, wv);
#pragma unroll
        for (int j = 0; j < V::N; ++j) {
          xb[j] *= r;
          acc_b[j] += b[j] * xb[j];
          b[j] *= wv[j];
          hn += b[j] * xb[j];
        }
        const float mean = group_sum<V::LANES>(hn) * per_dh;
#pragma unroll
        for (int j = 0; j < V::N; ++j) {
          a[j] = r * (a[j] - xa[j] * mean);
          b[j] = r * (b[j] - xb[j] * mean);
        }
      }
      g[u].a = narrow(a);
      g[u].b = narrow(b);
      if (h < heads && on) store_piece<T, DH>(dx + h * dh, at, g[u]);
    }
  }
}

// Four blocks an SM with two heads' loads of a lane in flight, at the same size (659 us then):
// four with one 777, five with one 933, three with two 946.
template <typename T, int DH, bool INTER, typename Rows>
__global__ void __launch_bounds__(kBwdThreads, 4)
    heads_bwd_vec(const __grid_constant__ HeadArgs A, const __grid_constant__ Rows R,
                  const T* __restrict__ qw, const T* __restrict__ kw, const T* __restrict__ q,
                  const T* __restrict__ k, const T* dq_out, const T* dk_out, T* dq, T* dk,
                  float* __restrict__ partial) {
  using V = Vec<T, DH>;
  constexpr int WARPS = kBwdThreads / 32;
  __shared__ float sums[WARPS][2][V::SPAN];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dh = size_of<DH>(A);
  const bool turned = A.rope.rotary_dim > 0;
  float acc[2][2][V::N] = {};
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * WARPS + warp; t < A.n_rows;
       t += static_cast<int64_t>(gridDim.x) * WARPS) {
    float cs[V::N], sn[V::N];
    const int64_t oq = t * A.hq * dh, ok = t * A.hkv * dh;
    head_run_bwd<T, DH, INTER, 2>(
        A, qw, turned, q + t * A.q_stride, dq_out + oq, dq + oq, A.hq, lane, cs, sn, acc[0][0], acc[0][1], [&]() {
          if (turned) piece_angles<T, DH, INTER>(A, R, t, locate(R, static_cast<int>(t), 0).pos, lane, cs, sn);
        });
    head_run_bwd<T, DH, INTER, 2>(A, kw, turned, k + t * A.k_stride, dk_out + ok, dk + ok, A.hkv, lane, cs, sn,
                                  acc[1][0], acc[1][1], []() {});
  }
  if (qw == nullptr) return;
  const Place at = place_of<T, DH, INTER>(A, lane % V::LANES);
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int j = 0; j < V::N; ++j) {
        float x = acc[which][half][j];  // over the heads of the warp: lanes with the same pieces
#pragma unroll
        for (int o = V::LANES; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane < V::LANES && has_piece<T, DH>(A, lane)) sums[warp][which][(half ? at.b : at.a) + j] = x;
      }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * dh; i += kBwdThreads) {
    float s = 0.f;
    for (int w = 0; w < WARPS; ++w) s += sums[w][i / dh][i % dh];
    partial[static_cast<int64_t>(blockIdx.x) * 2 * dh + i] = s;
  }
}

// Sums the blocks' weight gradients: a block for 32 of the 2*dh columns, a warp-row for every
// 32nd partial.
__global__ void __launch_bounds__(1024)
    weight_grad_sum(const float* __restrict__ partial, int n, int dh, float* __restrict__ dqw,
                    float* __restrict__ dkw) {
  __shared__ float s[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + x;
  float sum = 0.f;
  if (col < 2 * dh)
    for (int i = y; i < n; i += 32) sum += partial[static_cast<int64_t>(i) * 2 * dh + col];
  s[y][x] = sum;
  __syncthreads();
  sum = warp_sum(s[x][y]);  // column y of this block, summed over the rows
  const int out = blockIdx.x * 32 + y;
  if (x == 0 && out < 2 * dh) (out < dh ? dqw[out] : dkw[out - dh]) = sum;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
  return n < 1 ? 1 : n;
}

unsigned blocks_for(int64_t units, int per_block, int most) {
  int64_t b = (units + per_block - 1) / per_block;
  return static_cast<unsigned>(b < 1 ? 1 : b > most ? most : b);
}

int check_rope(const ra_rope* rope, int head_dim) {
  if (rope == nullptr) return RA_OK;
  if (rope->rotary_dim < 2 || rope->rotary_dim > RA_MAX_ROTARY_DIM || rope->rotary_dim % 2)
    return record_error(RA_ERR_INVALID_ARG, "rope: rotary_dim must be even, 2..%d (use ra_rope_init)",
                        RA_MAX_ROTARY_DIM);
  if (rope->rotary_dim > head_dim)
    return record_error(RA_ERR_SHAPE, "rotary_dim %d > head_dim %d", rope->rotary_dim, head_dim);
  return RA_OK;
}

int check_norm(const void* qw, const void* kw, float eps) {
  if ((qw == nullptr) != (kw == nullptr))
    return record_error(RA_ERR_INVALID_ARG, "pass both weights or neither");
  if (qw != nullptr && !(eps >= 0.f && std::isfinite(eps)))
    return record_error(RA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return RA_OK;
}

// The rows of a (validated) problem.
int rows_of(const ra_problem* p) { return p->batch > 0 ? p->batch * p->seqlen : p->cu_seqlens[p->n_seqs]; }

void fill_rows(const ra_problem* p, RingRows* R) {
  R->layout = p->layout;
  R->D = p->D;
  R->cu_local[0] = 0;
  if (p->batch > 0) {
    R->seqlen = p->seqlen;
    R->shard_rows = 0;
    R->n_seqs = p->batch;
  } else {
    R->seqlen = 0;
    R->n_seqs = p->n_seqs;
    for (int i = 0; i <= p->n_seqs; ++i) R->cu_local[i] = p->cu_seqlens[i] / p->D;
    R->shard_rows = rows_of(p) / p->D;
  }
}

void fill_args(HeadArgs* A, const ra_rope* rope, float eps, int hq, int hkv, int dh, int n_rows) {
  if (rope != nullptr) A->rope = *rope; else A->rope.rotary_dim = A->rope.interleaved = 0;
  A->eps = eps;
  A->hq = hq;
  A->hkv = hkv;
  A->dh = dh;
  A->n_rows = n_rows;
  A->kv_head = dh;
  A->q_stride = A->k_stride = A->v_stride = 0;
}

// Few tokens: the `runs` of their heads are shared between warps until there are 16 warps for every
// SM.
int parts_of(int n_rows, int runs) {
  const int want = (16 * sm_count() + n_rows - 1) / n_rows;
  return want < 1 ? 1 : want > runs ? runs : want;
}

// Whether the 16-byte kernels can take a call: heads of 64 or 128, in float32 any multiple of 8, a
// rotation that falls into whole pieces, and rows that all start on 16 bytes. (Measured, forward
// and backward: 131072 tokens, 32/8 heads of 128, bf16, 1.15 ms against the others' 3.9 ms; 32768
// tokens, float32 heads of 80, 0.40 against 0.69 ms.)
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool can_vec(const HeadArgs& A, int elem) {
  auto rows16 = [&](int64_t stride) { return stride * elem % 16 == 0; };
  return (A.dh == 64 || A.dh == 128 || (elem == 4 && A.dh % 8 == 0)) && (A.rope.interleaved || A.rope.rotary_dim % (32 / elem) == 0) &&
         rows16(A.q_stride) && rows16(A.k_stride) && rows16(A.v_stride) && rows16(A.kv_head);
}

// Calls f with the 16-byte kernels' DH for the call's head size.
template <typename T, typename F>
auto with_span(const HeadArgs& A, F&& f) {
  if (A.dh == 128) return f(std::integral_constant<int, 128>());
  if constexpr (sizeof(T) == 4) {
    if (A.dh <= 32) return f(std::integral_constant<int, -32>());
    if (A.dh < 64) return f(std::integral_constant<int, -64>());
    if (A.dh > 64) return f(std::integral_constant<int, -128>());
  }
  return f(std::integral_constant<int, 64>());
}

template <typename T, int DH, bool INTER, typename Rows, bool CACHE>
cudaError_t fwd_vec(const HeadArgs& A, const Rows& R, const void* qw, const void* kw, const void* q,
                    const void* k, const void* v, void* q_out, void* k_out, void* v_out, cudaStream_t st) {
  using V = Vec<T, DH>;
  const int runs = (A.hq + V::HEADS - 1) / V::HEADS + (A.hkv + V::HEADS - 1) / V::HEADS * (CACHE ? 2 : 1);
  const int parts = parts_of(A.n_rows, runs);
  const int64_t units = static_cast<int64_t>(A.n_rows) * parts;
  heads_fwd_vec<T, DH, INTER, Rows, CACHE><<<static_cast<unsigned>((units + kWarps - 1) / kWarps), kThreads, 0, st>>>(
      A, R, parts, static_cast<const T*>(qw), static_cast<const T*>(kw), static_cast<const T*>(q),
      static_cast<const T*>(k), static_cast<const T*>(v), static_cast<T*>(q_out), static_cast<T*>(k_out),
      static_cast<T*>(v_out));
  return cudaGetLastError();
}

template <typename T, typename Rows, bool CACHE>
cudaError_t launch_fwd(const HeadArgs& A, const Rows& R, const void* qw, const void* kw,
                       const void* q, const void* k, const void* v, void* q_out, void* k_out,
                       void* v_out, bool aligned, cudaStream_t st) {
  if (aligned && can_vec(A, sizeof(T)) && aligned16(qw) && aligned16(kw) && aligned16(q) && aligned16(k) &&
      aligned16(v) && aligned16(q_out) && aligned16(k_out) && aligned16(v_out)) {
    return with_span<T>(A, [&](auto span) {
      constexpr int DH = decltype(span)::value;
      return A.rope.interleaved
                 ? fwd_vec<T, DH, true, Rows, CACHE>(A, R, qw, kw, q, k, v, q_out, k_out, v_out, st)
                 : fwd_vec<T, DH, false, Rows, CACHE>(A, R, qw, kw, q, k, v, q_out, k_out, v_out, st);
    });
  }
  const int parts = parts_of(A.n_rows, A.hq + A.hkv * (CACHE ? 2 : 1));
  const int64_t units = static_cast<int64_t>(A.n_rows) * parts;
  heads_fwd_any<T, Rows, CACHE><<<static_cast<unsigned>((units + kWarps - 1) / kWarps), kThreads, 0, st>>>(
      A, R, parts, static_cast<const T*>(qw), static_cast<const T*>(kw), static_cast<const T*>(q),
      static_cast<const T*>(k), static_cast<const T*>(v), static_cast<T*>(q_out),
      static_cast<T*>(k_out), static_cast<T*>(v_out));
  return cudaGetLastError();
}

template <typename T, int DH, bool INTER, typename Rows>
void bwd_vec(unsigned blocks, const HeadArgs& A, const Rows& R, const void* qw, const void* kw, const void* q,
             const void* k, const void* dq_out, const void* dk_out, void* dq, void* dk, float* partial,
             cudaStream_t st) {
  heads_bwd_vec<T, DH, INTER, Rows><<<blocks, kBwdThreads, 0, st>>>(
      A, R, static_cast<const T*>(qw), static_cast<const T*>(kw), static_cast<const T*>(q),
      static_cast<const T*>(k), static_cast<const T*>(dq_out), static_cast<const T*>(dk_out),
      static_cast<T*>(dq), static_cast<T*>(dk), partial);
}

template <typename T, typename Rows>
cudaError_t launch_bwd(const HeadArgs& A, const Rows& R, const void* qw, const void* kw,
                       const void* q, const void* k, const void* dq_out, const void* dk_out,
                       void* dq, void* dk, float* partial, float* dqw, float* dkw, cudaStream_t st) {
  unsigned blocks;
  if (can_vec(A, sizeof(T)) && aligned16(qw) && aligned16(kw) && aligned16(q) && aligned16(k) &&
      aligned16(dq_out) && aligned16(dk_out) && aligned16(dq) && aligned16(dk)) {
    blocks = blocks_for(A.n_rows, kBwdThreads / 32, kHeadBwdBlocks);
    with_span<T>(A, [&](auto span) {
      constexpr int DH = decltype(span)::value;
      if (A.rope.interleaved) bwd_vec<T, DH, true>(blocks, A, R, qw, kw, q, k, dq_out, dk_out, dq, dk, partial, st);
      else bwd_vec<T, DH, false>(blocks, A, R, qw, kw, q, k, dq_out, dk_out, dq, dk, partial, st);
    });
  } else {
    const int parts = parts_of(A.n_rows, A.hq + A.hkv);
    blocks = blocks_for(static_cast<int64_t>(A.n_rows) * parts, kWarps, kHeadBwdBlocks);
    heads_bwd_any<T, Rows><<<blocks, kThreads, 0, st>>>(
        A, R, parts, static_cast<const T*>(qw), static_cast<const T*>(kw), static_cast<const T*>(q),
        static_cast<const T*>(k), static_cast<const T*>(dq_out), static_cast<const T*>(dk_out),
        static_cast<T*>(dq), static_cast<T*>(dk), partial);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || qw == nullptr) return e;
  weight_grad_sum<<<(2 * A.dh + 31) / 32, 1024, 0, st>>>(partial, blocks, A.dh, dqw, dkw);
  return cudaGetLastError();
}

}  // namespace

cudaError_t append_status(unsigned int* value, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_status_append, sizeof(unsigned int));
  if (e == cudaSuccess && reset) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_status_append, &zero, sizeof(unsigned int));
  }
  return e;
}

// Shared with the decode attention. Leaves dtype-specific demands (alignment) to the caller.
int check_cache(const ra_paged_cache* c) {
  if (c == nullptr) return record_error(RA_ERR_INVALID_ARG, "cache is NULL");
  if (c->dtype != RA_F32 && c->dtype != RA_BF16)
    return record_error(RA_ERR_INVALID_ARG, "bad dtype %d", c->dtype);
  if (c->hkv < 1 || c->head_dim < 1 || c->page_size < 1 || c->n_pages < 1 || c->n_seqs < 0 ||
      c->max_pages < 0)
    return record_error(RA_ERR_INVALID_ARG, "cache: heads, head_dim, page_size and n_pages must be >= 1, "
                                            "n_seqs and max_pages >= 0");
  if (c->dtype == RA_BF16 && c->head_dim != 64 && c->head_dim != 128)
    return record_error(RA_ERR_UNSUPPORTED, "bf16 supports head_dim 64 or 128 (got %d)", c->head_dim);
  if (c->head_dim > 128)
    return record_error(RA_ERR_UNSUPPORTED, "f32 supports head_dim <= 128 (got %d)", c->head_dim);
  if (c->n_seqs > RA_MAX_CACHE_SEQS)
    return record_error(RA_ERR_UNSUPPORTED, "n_seqs > %d", RA_MAX_CACHE_SEQS);
  // (the decode kernels round a length up to units of 64 keys in 32 bits)
  if (static_cast<int64_t>(c->max_pages) * c->page_size > (int64_t(1) << 31) - 64)
    return record_error(RA_ERR_UNSUPPORTED, "max_pages * page_size must be 2^31 - 64 at most");
  if (c->page_stride < 1 || c->slot_stride < 1 || c->head_stride < 1 || c->table_stride < c->max_pages)
    return record_error(RA_ERR_INVALID_ARG, "cache: strides must be positive, table_stride >= max_pages");
  if (c->k_pages == nullptr || c->v_pages == nullptr ||
      (c->block_table == nullptr && c->n_seqs > 0 && c->max_pages > 0))
    return record_error(RA_ERR_INVALID_ARG, "null cache pointer");
  return RA_OK;
}

// |x| / 2pi modulo 1 in units of 2^-64, to a unit, and its negative for x < 0. 1 / 2pi is two doubles
// (hi + lo, from the decimal expansion of pi), and what the product with hi is rounded by comes back
// from an fma: one double product would be off by up to 2^10 units for x = 1, which a position of 2^30
// makes 2^-24 of a turn. (volatile: the product has to be the rounded one everywhere.)
uint64_t turns_of(double x) {
  constexpr double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
  const double f = std::fabs(x);
  volatile double product = f * hi;
  const double p = product;
  double rest = std::fma(f, hi, -p) + f * lo;  // f / 2pi = p + rest
  rest -= std::rint(rest);
  const double a = (p - std::floor(p)) * 18446744073709551616.0, whole = std::floor(a);  // exact
  double b = std::rint(rest * 18446744073709551616.0 + (a - whole));
  if (b >= 9223372036854775808.0) b = -9223372036854775808.0;  // half a turn either way
  const uint64_t t = static_cast<uint64_t>(whole) + static_cast<uint64_t>(static_cast<int64_t>(b));
  return x < 0 ? uint64_t(0) - t : t;
}

size_t heads_bwd_workspace(int head_dim) {
  return static_cast<size_t>(kHeadBwdBlocks) * 2 * head_dim * sizeof(float);
}

}  // namespace ra

using namespace ra;

extern "C" int ra_rope_init(ra_rope* rope, int rotary_dim, int interleaved, const double* inv_freq) {
  if (rope == nullptr || inv_freq == nullptr) return record_error(RA_ERR_INVALID_ARG, "null pointer");
  if (rotary_dim < 2 || rotary_dim > RA_MAX_ROTARY_DIM || rotary_dim % 2)
    return record_error(RA_ERR_INVALID_ARG, "rotary_dim must be even, 2..%d (got %d)", RA_MAX_ROTARY_DIM,
                        rotary_dim);
  rope->rotary_dim = rotary_dim;
  rope->interleaved = interleaved ? 1 : 0;
  for (int i = 0; i < RA_MAX_ROTARY_DIM / 2; ++i) rope->turns[i] = 0;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    if (!std::isfinite(inv_freq[i])) return record_error(RA_ERR_INVALID_ARG, "inv_freq[%d] is not finite", i);
    rope->turns[i] = turns_of(inv_freq[i]);
  }
  record_error(RA_OK, "%s", "");
  return RA_OK;
}

namespace {

// Positions on several axes of a call: none for a rotation by place.
struct Axes {
  const ra_axis_rope* rope;
  const int32_t* pos;
  int64_t stride;
};
constexpr Axes kNoAxes = {nullptr, nullptr, 0};

int check_axes(const ra_axis_rope* rope, const int32_t* pos, int64_t stride, bool some) {
  if (rope == nullptr) return record_error(RA_ERR_INVALID_ARG, "rope is NULL");
  if (rope->n_axes < 1 || rope->n_axes > RA_MAX_AXES)
    return record_error(RA_ERR_INVALID_ARG, "rope: n_axes must be 1..%d (use ra_axis_rope_init)", RA_MAX_AXES);
  for (int i = 0; i < rope->rope.rotary_dim / 2 && i < RA_MAX_ROTARY_DIM / 2; ++i)
    if (rope->axis[i] >= rope->n_axes)
      return record_error(RA_ERR_INVALID_ARG, "rope: axis[%d] is %d of %d axes", i, rope->axis[i], rope->n_axes);
  if (some && pos == nullptr) return record_error(RA_ERR_INVALID_ARG, "positions is NULL");
  if (stride < rope->n_axes)
    return record_error(RA_ERR_SHAPE, "pos_row_stride must be >= n_axes (%d)", rope->n_axes);
  return RA_OK;
}

AxisPos axis_pos(const Axes& x) {
  AxisPos a;
  a.pos = x.pos;
  a.stride = x.stride;
  for (int i = 0; i < RA_MAX_ROTARY_DIM / 2; ++i) a.axis[i] = x.rope->axis[i];
  return a;
}

// Calls f with the rows of a ring problem.
template <typename F>
cudaError_t with_rows(const ra_problem* p, const Axes& x, F&& f) {
  if (x.rope != nullptr) return f(RingAxisRows{axis_pos(x)});
  RingRows R;
  fill_rows(p, &R);
  return f(R);
}

int norm_rope_fwd(const ra_problem* p, const ra_rope* rope, const Axes& axes, float eps, const void* q,
                  int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* q_weight,
                  const void* k_weight, void* q_out, void* k_out, void* stream) {
  const bool some = rows_of(p) > 0;  // empty tensors may have null pointers
  if (some && (!q || !k || !q_out || !k_out)) return record_error(RA_ERR_INVALID_ARG, "null tensor pointer");
  if (int e = check_rope(rope, p->head_dim)) return e;
  if (int e = check_norm(q_weight, k_weight, eps)) return e;
  if (rope == nullptr && q_weight == nullptr)
    return record_error(RA_ERR_INVALID_ARG, "neither weights nor a rotation: nothing to do");
  const int64_t nq = static_cast<int64_t>(p->hq) * p->head_dim, nk = static_cast<int64_t>(p->hkv) * p->head_dim;
  if (q_row_stride < nq || k_row_stride < nk)
    return record_error(RA_ERR_SHAPE, "row strides must be >= heads * head_dim");
  if (some && ((q == q_out && q_row_stride != nq) || (k == k_out && k_row_stride != nk)))
    return record_error(RA_ERR_INVALID_ARG, "in place wants contiguous rows");
  if (!some) return record_error(RA_OK, "%s", "");
  HeadArgs A;
  fill_args(&A, rope, eps, p->hq, p->hkv, p->head_dim, rows_of(p));
  A.q_stride = q_row_stride;
  A.k_stride = k_row_stride;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = with_rows(p, axes, [&](const auto& R) {
    using Rows = std::decay_t<decltype(R)>;
    return p->dtype == RA_F32
               ? launch_fwd<float, Rows, false>(A, R, q_weight, k_weight, q, k, nullptr, q_out, k_out, nullptr, true, st)
               : launch_fwd<__nv_bfloat16, Rows, false>(A, R, q_weight, k_weight, q, k, nullptr, q_out, k_out,
                                                        nullptr, true, st);
  });
  if (e != cudaSuccess) return record_error(RA_ERR_CUDA, "norm and rotation launch: %s", cudaGetErrorString(e));
  return record_error(RA_OK, "%s", "");
}

int norm_rope_bwd(const ra_problem* p, const ra_rope* rope, const Axes& axes, float eps, const void* dq_out,
                  const void* dk_out, const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                  const void* q_weight, const void* k_weight, void* dq, void* dk, float* dq_weight,
                  float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
  const bool some = rows_of(p) > 0;  // empty tensors may have null pointers
  if (some && (!dq_out || !dk_out || !dq || !dk)) return record_error(RA_ERR_INVALID_ARG, "null tensor pointer");
  if (int e = check_rope(rope, p->head_dim)) return e;
  if (int e = check_norm(q_weight, k_weight, eps)) return e;
  if (rope == nullptr && q_weight == nullptr)
    return record_error(RA_ERR_INVALID_ARG, "neither weights nor a rotation: nothing to do");
  if (q_weight != nullptr) {
    if ((some && (!q || !k)) || !dq_weight || !dk_weight) return record_error(RA_ERR_INVALID_ARG, "null tensor pointer");
    if (q_row_stride < static_cast<int64_t>(p->hq) * p->head_dim ||
        k_row_stride < static_cast<int64_t>(p->hkv) * p->head_dim)
      return record_error(RA_ERR_SHAPE, "row strides must be >= heads * head_dim");
    if (workspace_bytes < heads_bwd_workspace(p->head_dim))
      return record_error(RA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes,
                          heads_bwd_workspace(p->head_dim));
    if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256)
      return record_error(RA_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
  }
  const int n_rows = rows_of(p);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (!some) {
    if (q_weight != nullptr) {
      e = cudaMemsetAsync(dq_weight, 0, p->head_dim * sizeof(float), st);
      if (e == cudaSuccess) e = cudaMemsetAsync(dk_weight, 0, p->head_dim * sizeof(float), st);
    }
  } else {
    HeadArgs A;
    fill_args(&A, rope, eps, p->hq, p->hkv, p->head_dim, n_rows);
    A.q_stride = q_row_stride;
    A.k_stride = k_row_stride;
    float* partial = static_cast<float*>(workspace);
    e = with_rows(p, axes, [&](const auto& R) {
      return p->dtype == RA_F32 ? launch_bwd<float>(A, R, q_weight, k_weight, q, k, dq_out, dk_out, dq, dk, partial,
                                                    dq_weight, dk_weight, st)
                                : launch_bwd<__nv_bfloat16>(A, R, q_weight, k_weight, q, k, dq_out, dk_out, dq, dk,
                                                            partial, dq_weight, dk_weight, st);
    });
  }
  if (e != cudaSuccess)
    return record_error(RA_ERR_CUDA, "norm and rotation backward launch: %s", cudaGetErrorString(e));
  return record_error(RA_OK, "%s", "");
}

int cache_append(const ra_paged_cache* c, const ra_rope* rope, const Axes& axes, float eps, int n_tokens, int hq,
                 const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                 int64_t v_row_stride, const void* q_weight, const void* k_weight, const int32_t* seq_lens,
                 const int32_t* cu_new, void* q_out, void* stream) {
  if ((q == nullptr) != (q_out == nullptr)) return record_error(RA_ERR_INVALID_ARG, "pass both q and q_out or neither");
  const bool some = n_tokens > 0 && c->n_seqs > 0;  // empty tensors may have null pointers
  if (some && (!k || !v || !seq_lens)) return record_error(RA_ERR_INVALID_ARG, "null tensor pointer");
  if (n_tokens < 0) return record_error(RA_ERR_INVALID_ARG, "n_tokens must be >= 0");
  if (q != nullptr && (hq < 1 || hq % c->hkv))
    return record_error(RA_ERR_UNSUPPORTED, "hq (%d) must be a multiple of hkv (%d)", hq, c->hkv);
  if (cu_new == nullptr && n_tokens != c->n_seqs)
    return record_error(RA_ERR_SHAPE, "without cu_new there is one token for each of the %d sequences (got %d)",
                        c->n_seqs, n_tokens);
  if (int e = check_rope(rope, c->head_dim)) return e;
  if (int e = check_norm(q_weight, k_weight, eps)) return e;
  const int heads_q = q != nullptr ? hq : 0;
  const int64_t nq = static_cast<int64_t>(heads_q) * c->head_dim, nk = static_cast<int64_t>(c->hkv) * c->head_dim;
  if ((q != nullptr && q_row_stride < nq) || k_row_stride < nk || v_row_stride < nk)
    return record_error(RA_ERR_SHAPE, "row strides must be >= heads * head_dim");
  if (q != nullptr && q == q_out && q_row_stride != nq)
    return record_error(RA_ERR_INVALID_ARG, "in place wants contiguous rows");
  if (!some) return record_error(RA_OK, "%s", "");
  CacheRows R;
  R.seq_lens = seq_lens;
  R.cu_new = cu_new;
  R.block_table = c->block_table;
  R.table_stride = c->table_stride;
  R.page_stride = c->page_stride;
  R.slot_stride = c->slot_stride;
  R.head_stride = c->head_stride;
  R.n_seqs = c->n_seqs;
  R.max_pages = c->max_pages;
  R.page_size = c->page_size;
  R.n_pages = c->n_pages;
  HeadArgs A;
  fill_args(&A, rope, eps, heads_q, c->hkv, c->head_dim, n_tokens);
  A.q_stride = q_row_stride;
  A.k_stride = k_row_stride;
  A.v_stride = v_row_stride;
  A.kv_head = c->head_stride;
  const int elem = c->dtype == RA_F32 ? 4 : 2;  // of the pages, kv_head is looked at with the rows
  const bool pages16 = c->page_stride * elem % 16 == 0 && c->slot_stride * elem % 16 == 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto put = [&](const auto& rows) {
    using Rows = std::decay_t<decltype(rows)>;
    return c->dtype == RA_F32
               ? launch_fwd<float, Rows, true>(A, rows, q_weight, k_weight, q, k, v, q_out, c->k_pages, c->v_pages, pages16, st)
               : launch_fwd<__nv_bfloat16, Rows, true>(A, rows, q_weight, k_weight, q, k, v, q_out, c->k_pages,
                                                       c->v_pages, pages16, st);
  };
  const cudaError_t e = axes.rope != nullptr ? put(CacheAxisRows{R, axis_pos(axes)}) : put(R);
  if (e != cudaSuccess) return record_error(RA_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
  return record_error(RA_OK, "%s", "");
}

}  // namespace

extern "C" int ra_qk_norm_rope_fwd(const ra_problem* p, const ra_rope* rope, float eps, const void* q,
                                   int64_t q_row_stride, const void* k, int64_t k_row_stride,
                                   const void* q_weight, const void* k_weight, void* q_out, void* k_out,
                                   void* stream) {
  if (int e = ra_validate(p)) return e;
  return norm_rope_fwd(p, rope, kNoAxes, eps, q, q_row_stride, k, k_row_stride, q_weight, k_weight, q_out, k_out,
                       stream);
}

extern "C" int ra_qk_norm_rope_bwd(const ra_problem* p, const ra_rope* rope, float eps, const void* dq_out,
                                   const void* dk_out, const void* q, int64_t q_row_stride, const void* k,
                                   int64_t k_row_stride, const void* q_weight, const void* k_weight, void* dq,
                                   void* dk, float* dq_weight, float* dk_weight, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (int e = ra_validate(p)) return e;
  return norm_rope_bwd(p, rope, kNoAxes, eps, dq_out, dk_out, q, q_row_stride, k, k_row_stride, q_weight, k_weight, dq,
                       dk, dq_weight, dk_weight, workspace, workspace_bytes, stream);
}

extern "C" int ra_kv_cache_append(const ra_paged_cache* c, const ra_rope* rope, float eps, int n_tokens, int hq,
                                  const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                                  const void* v, int64_t v_row_stride, const void* q_weight,
                                  const void* k_weight, const int32_t* seq_lens, const int32_t* cu_new,
                                  void* q_out, void* stream) {
  if (int e = check_cache(c)) return e;
  return cache_append(c, rope, kNoAxes, eps, n_tokens, hq, q, q_row_stride, k, k_row_stride, v, v_row_stride, q_weight,
                      k_weight, seq_lens, cu_new, q_out, stream);
}

extern "C" int ra_axis_rope_init(ra_axis_rope* rope, int rotary_dim, int interleaved, const double* inv_freq,
                                 int n_axes, const int32_t* axis) {
  if (rope == nullptr || axis == nullptr) return record_error(RA_ERR_INVALID_ARG, "null pointer");
  if (n_axes < 1 || n_axes > RA_MAX_AXES)
    return record_error(RA_ERR_INVALID_ARG, "n_axes must be 1..%d (got %d)", RA_MAX_AXES, n_axes);
  if (int e = ra_rope_init(&rope->rope, rotary_dim, interleaved, inv_freq)) return e;
  rope->n_axes = n_axes;
  for (int i = 0; i < RA_MAX_ROTARY_DIM / 2; ++i) {
    const int a = i < rotary_dim / 2 ? axis[i] : 0;
    if (a < 0 || a >= n_axes) return record_error(RA_ERR_INVALID_ARG, "axis[%d] is %d of %d axes", i, a, n_axes);
    rope->axis[i] = static_cast<uint8_t>(a);
  }
  return record_error(RA_OK, "%s", "");
}

extern "C" int ra_qk_norm_axis_rope_fwd(const ra_problem* p, const ra_axis_rope* rope, const int32_t* positions,
                                        int64_t pos_row_stride, float eps, const void* q, int64_t q_row_stride,
                                        const void* k, int64_t k_row_stride, const void* q_weight,
                                        const void* k_weight, void* q_out, void* k_out, void* stream) {
  if (int e = ra_validate(p)) return e;
  if (int e = check_axes(rope, positions, pos_row_stride, rows_of(p) > 0)) return e;
  return norm_rope_fwd(p, &rope->rope, {rope, positions, pos_row_stride}, eps, q, q_row_stride, k, k_row_stride,
                       q_weight, k_weight, q_out, k_out, stream);
}

extern "C" int ra_qk_norm_axis_rope_bwd(const ra_problem* p, const ra_axis_rope* rope, const int32_t* positions,
                                        int64_t pos_row_stride, float eps, const void* dq_out, const void* dk_out,
                                        const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                                        const void* q_weight, const void* k_weight, void* dq, void* dk,
                                        float* dq_weight, float* dk_weight, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  if (int e = ra_validate(p)) return e;
  if (int e = check_axes(rope, positions, pos_row_stride, rows_of(p) > 0)) return e;
  return norm_rope_bwd(p, &rope->rope, {rope, positions, pos_row_stride}, eps, dq_out, dk_out, q, q_row_stride, k,
                       k_row_stride, q_weight, k_weight, dq, dk, dq_weight, dk_weight, workspace, workspace_bytes,
                       stream);
}

extern "C" int ra_kv_cache_append_axes(const ra_paged_cache* c, const ra_axis_rope* rope, const int32_t* positions,
                                       int64_t pos_row_stride, float eps, int n_tokens, int hq, const void* q,
                                       int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                                       int64_t v_row_stride, const void* q_weight, const void* k_weight,
                                       const int32_t* seq_lens, const int32_t* cu_new, void* q_out, void* stream) {
  if (int e = check_cache(c)) return e;
  if (int e = check_axes(rope, positions, pos_row_stride, n_tokens > 0 && c->n_seqs > 0)) return e;
  return cache_append(c, &rope->rope, {rope, positions, pos_row_stride}, eps, n_tokens, hq, q, q_row_stride, k,
                      k_row_stride, v, v_row_stride, q_weight, k_weight, seq_lens, cu_new, q_out, stream);
}
