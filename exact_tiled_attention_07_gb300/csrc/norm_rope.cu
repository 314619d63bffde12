// Queries and keys normed head by head (root mean square, learned weight) and rotated by their position, in one pass,
// and its gradients.
//
// A row x of d channels of one head, at position p:
//     r = 1 / sqrt(mean(x^2) + eps),  y = x r w,  (a, b) -> (a c - b s, b c + a s) for each rotated pair of channels,
// with c, s = cos, sin of the pair's angle at p from the caller's table.  The rotation R is orthogonal, so with
// u = R^T dy:
//     g = u w,  xh = x r,   dx = r (g - xh mean(g xh)),   dw = sum over rows of u xh.
// The backward recomputes r from x (it reads x anyway) instead of keeping it.
//
// Bound: HBM.  Every row is read and written once and a channel takes about ten instructions, so the layout is made for
// wide loads and few of them: a lane holds eight channels of a row, the two halves of four rotated pairs (two 8-byte
// pieces rotary / 2 channels apart, or 16 bytes in a row where pairs are adjacent), so that a pair never crosses lanes and
// only the sum of a row does.  d / 8 lanes make a row, two or four rows a warp.  A group of lanes takes kUnit heads of
// one token: their loads are all in flight before the first is used, and cos and sin are read once for all of them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

// Four consecutive channels of a row as they lie in memory.
template <typename T>
struct Four {
  using Raw = uint2;
  static __device__ __forceinline__ void open(const Raw& r, float* v) {
    const float2 a = unpack2<std::is_same<T, __nv_bfloat16>::value>(r.x);
    const float2 b = unpack2<std::is_same<T, __nv_bfloat16>::value>(r.y);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  }
  static __device__ __forceinline__ Raw close(const float* v) {
    return make_uint2(pack2<std::is_same<T, __nv_bfloat16>::value>(v[0], v[1]),
                      pack2<std::is_same<T, __nv_bfloat16>::value>(v[2], v[3]));
  }
};
template <>
struct Four<float> {
  using Raw = float4;
  static __device__ __forceinline__ void open(const Raw& r, float* v) { v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w; }
  static __device__ __forceinline__ Raw close(const float* v) { return make_float4(v[0], v[1], v[2], v[3]); }
};

__device__ __forceinline__ float weight_at(const void* w, int kind, int c) {
  if (!w) return 1.f;
  if (kind == DT_FP32) return static_cast<const float*>(w)[c];
  if (kind == DT_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]);
  return __half2float(static_cast<const __half*>(w)[c]);
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Where a lane's channels are: pieces of four channels at `a` and `b`; pair t of its four is (v[t], v[4 + t]), or
// (v[2 t], v[2 t + 1]) where pairs are adjacent.
struct Pieces {
  int a, b;
  int pair;  // its first pair's place in the table, -1: not rotated
};
__device__ __forceinline__ Pieces pieces_of(int lane, int rotary, bool adjacent) {
  Pieces p;
  const int at = 8 * lane;
  if (at < rotary) {
    p.pair = 4 * lane;
    p.a = adjacent ? at : 4 * lane;
    p.b = adjacent ? at + 4 : 4 * lane + rotary / 2;
  } else {
    p.pair = -1;
    p.a = at;
    p.b = at + 4;
  }
  return p;
}

// cos and sin of a lane's four pairs at a token (1 and 0 where it is not rotated).  A position outside the table is
// clamped to it and recorded.
__device__ __forceinline__ void angles(const NormRopeArgs& p, int64_t t, int n, const Pieces& at, float (&c)[4],
                                       float (&s)[4]) {
  c[0] = c[1] = c[2] = c[3] = 1.f;
  s[0] = s[1] = s[2] = s[3] = 0.f;
  if (p.rotary == 0) return;
  int pos = p.positions ? p.positions[t] : n;
  if (pos < 0 || pos >= p.table_len) {
    report_error(p.err, DERR_BAD_ARG, 300);
    pos = pos < 0 ? 0 : p.table_len - 1;
  }
  if (at.pair < 0) return;
  const float* row = p.table + (int64_t)pos * p.rotary + at.pair;
  const float4 c4 = *reinterpret_cast<const float4*>(row);
  const float4 s4 = *reinterpret_cast<const float4*>(row + p.rotary / 2);
  c[0] = c4.x, c[1] = c4.y, c[2] = c4.z, c[3] = c4.w;
  s[0] = s4.x, s[1] = s4.y, s[2] = s4.z, s[3] = s4.w;
}

template <bool ADJ>
__device__ __forceinline__ void rotate(float (&v)[8], const float (&c)[4], const float (&s)[4], float sign) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    float& a = v[ADJ ? 2 * t : t];
    float& b = v[ADJ ? 2 * t + 1 : 4 + t];
    const float x = a, y = b, si = sign * s[t];
    a = x * c[t] - y * si;
    b = y * c[t] + x * si;
  }
}

// A unit: up to UNIT heads of one token, all queries or all keys.
struct Unit {
  int64_t t;  // token b N + n
  int b, n;
  int h0, heads;
  bool key;
};
template <int UNIT>
__device__ __forceinline__ Unit unit_of(const NormRopeArgs& p, int u) {
  const int uq = (p.h + UNIT - 1) / UNIT, uk = (p.hkv + UNIT - 1) / UNIT;
  Unit w;
  const int t = u / (uq + uk);
  int i = u - t * (uq + uk);
  w.key = i >= uq;
  if (w.key) i -= uq;
  w.t = t;
  w.b = t / p.n;
  w.n = t - w.b * p.n;
  w.h0 = i * UNIT;
  w.heads = min(UNIT, (w.key ? p.hkv : p.h) - w.h0);
  return w;
}

// The row of head h0 of a unit in a tensor.
template <typename T, typename P>
__device__ __forceinline__ T* rows_of(P* base, const NormRopeStrides& st, const Unit& w) {
  return const_cast<T*>(reinterpret_cast<const T*>(base)) + w.b * st.batch + w.n * st.token + w.h0 * st.head;
}

template <typename T, int LANES, bool ADJ, int UNIT>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs p, int units) {
  using F = Four<T>;
  const int lane = threadIdx.x % LANES;
  const int u = (int)(((int64_t)blockIdx.x * kThreads + threadIdx.x) / LANES);
  const bool active = u < units && 8 * lane < p.d;
  const Unit w = unit_of<UNIT>(p, min(u, units - 1));
  const Pieces at = pieces_of(8 * lane < p.d ? lane : 0, p.rotary, ADJ);
  const NormRopeStrides& si = w.key ? p.k_st : p.q_st;
  const T* x = rows_of<T>(w.key ? p.k : p.q, si, w);
  typename F::Raw ra[UNIT], rb[UNIT];
#pragma unroll
  for (int i = 0; i < UNIT; ++i) {
    if (active && i < w.heads) {
      ra[i] = *reinterpret_cast<const typename F::Raw*>(x + i * si.head + at.a);
      rb[i] = *reinterpret_cast<const typename F::Raw*>(x + i * si.head + at.b);
    }
  }
  float c[4], s[4], wt[8];
  angles(p, w.t, w.n, at, c, s);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    wt[t] = weight_at(w.key ? p.wk : p.wq, p.wdtype, at.a + t);
    wt[4 + t] = weight_at(w.key ? p.wk : p.wq, p.wdtype, at.b + t);
  }
  const NormRopeStrides& so = w.key ? p.ko_st : p.qo_st;
  T* y = rows_of<T>(w.key ? p.ko : p.qo, so, w);
  const float inv_d = 1.f / (float)p.d;
#pragma unroll
  for (int i = 0; i < UNIT; ++i) {
    float v[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = 0.f;
    const bool mine = active && i < w.heads;
    if (mine) {
      F::open(ra[i], v);
      F::open(rb[i], v + 4);
    }
    float sq = 0.f;
#pragma unroll
    for (int t = 0; t < 8; ++t) sq = fmaf(v[t], v[t], sq);
    const float r = __frsqrt_rn(fmaf(row_sum<LANES>(sq), inv_d, p.eps));
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] *= r * wt[t];
    rotate<ADJ>(v, c, s, 1.f);
    if (mine) {
      *reinterpret_cast<typename F::Raw*>(y + i * so.head + at.a) = F::close(v);
      *reinterpret_cast<typename F::Raw*>(y + i * so.head + at.b) = F::close(v + 4);
    }
  }
}

// Backward.  A group of lanes walks units of one kind (blocks below q_blocks take queries, the others keys), so that its
// eight sums of dw stay in registers; the block adds its groups' sums in shared memory, in a fixed order, into one row
// of partials for the finishing kernel.  Sums are in 32 bits, in three levels (a group's rows, a block's groups, blocks).
template <typename T, int LANES, bool ADJ, int UNIT>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs p, int q_blocks) {
  using F = Four<T>;
  constexpr int GROUPS = kThreads / LANES;
  __shared__ float part[GROUPS][8 * LANES];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const bool key = (int)blockIdx.x >= q_blocks;
  const int heads = key ? p.hkv : p.h;
  const int per_token = (heads + UNIT - 1) / UNIT;
  const int units = (int)((int64_t)p.b * p.n) * per_token;
  const int first = ((int)blockIdx.x - (key ? q_blocks : 0)) * GROUPS + group;
  const int step = (key ? (int)gridDim.x - q_blocks : q_blocks) * GROUPS;
  const bool in_row = 8 * lane < p.d;
  const Pieces at = pieces_of(in_row ? lane : 0, p.rotary, ADJ);
  const NormRopeStrides &sx = key ? p.k_st : p.q_st, &sy = key ? p.ko_st : p.qo_st, &sd = key ? p.dk_st : p.dq_st;
  float wt[8], dw[8];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    wt[t] = weight_at(key ? p.wk : p.wq, p.wdtype, at.a + t);
    wt[4 + t] = weight_at(key ? p.wk : p.wq, p.wdtype, at.b + t);
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) dw[t] = 0.f;
  const float inv_d = 1.f / (float)p.d;
  // (all groups of a warp go round together: the sums of rows are taken by the whole warp)
  for (int u0 = first - group % (32 / LANES); u0 < units; u0 += step) {
    const int u = u0 + group % (32 / LANES);
    Unit w;
    const int t = min(u, units - 1) / per_token;
    w.t = t;
    w.b = t / p.n;
    w.n = t - w.b * p.n;
    w.h0 = (min(u, units - 1) - t * per_token) * UNIT;
    w.heads = min(UNIT, heads - w.h0);
    const bool active = u < units && in_row;
    const T* x = rows_of<T>(key ? p.k : p.q, sx, w);
    const T* dy = rows_of<T>(key ? p.ko : p.qo, sy, w);
    T* dx = rows_of<T>(key ? p.dk : p.dq, sd, w);
    typename F::Raw xa[UNIT], xb[UNIT], ya[UNIT], yb[UNIT];
#pragma unroll
    for (int i = 0; i < UNIT; ++i) {
      if (active && i < w.heads) {
        xa[i] = *reinterpret_cast<const typename F::Raw*>(x + i * sx.head + at.a);
        xb[i] = *reinterpret_cast<const typename F::Raw*>(x + i * sx.head + at.b);
        ya[i] = *reinterpret_cast<const typename F::Raw*>(dy + i * sy.head + at.a);
        yb[i] = *reinterpret_cast<const typename F::Raw*>(dy + i * sy.head + at.b);
      }
    }
    float c[4], s[4];
    angles(p, w.t, w.n, at, c, s);
#pragma unroll
    for (int i = 0; i < UNIT; ++i) {
      float v[8], g[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) v[t] = g[t] = 0.f;
      const bool mine = active && i < w.heads;
      if (mine) {
        F::open(xa[i], v);
        F::open(xb[i], v + 4);
        F::open(ya[i], g);
        F::open(yb[i], g + 4);
      }
      float sq = 0.f;
#pragma unroll
      for (int t = 0; t < 8; ++t) sq = fmaf(v[t], v[t], sq);
      const float r = __frsqrt_rn(fmaf(row_sum<LANES>(sq), inv_d, p.eps));
      rotate<ADJ>(g, c, s, -1.f);
      float dot = 0.f;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        v[t] *= r;
        if (mine) dw[t] = fmaf(g[t], v[t], dw[t]);
        g[t] *= wt[t];
        dot = fmaf(g[t], v[t], dot);
      }
      dot = row_sum<LANES>(dot) * inv_d;
#pragma unroll
      for (int t = 0; t < 8; ++t) g[t] = r * fmaf(-v[t], dot, g[t]);
      if (mine) {
        *reinterpret_cast<typename F::Raw*>(dx + i * sd.head + at.a) = F::close(g);
        *reinterpret_cast<typename F::Raw*>(dx + i * sd.head + at.b) = F::close(g + 4);
      }
    }
  }
  if (in_row) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      part[group][at.a + t] = dw[t];
      part[group][at.b + t] = dw[4 + t];
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < p.d) {
    float sum = 0.f;
#pragma unroll 4
    for (int g = 0; g < GROUPS; ++g) sum += part[g][threadIdx.x];
    p.partials[(int64_t)blockIdx.x * p.d + threadIdx.x] = sum;
  }
}

// dw of the queries (block 0) and of the keys (block 1): the blocks' partial sums, every channel by kFinish / 32 warps.
constexpr int kFinish = 1024;
__global__ void __launch_bounds__(kFinish) norm_rope_finish(const __grid_constant__ NormRopeArgs p, int q_blocks, int blocks) {
  __shared__ float part[kFinish];
  const bool key = blockIdx.y == 1;
  void* out = key ? p.dwk : p.dwq;
  if (!out) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  const int from = key ? q_blocks : 0, to = key ? blocks : q_blocks;
  float sum = 0.f;
  if (c < p.d) {
#pragma unroll 4
    for (int i = from + slice; i < to; i += kFinish / 32) sum += p.partials[(int64_t)i * p.d + c];
  }
  part[threadIdx.x] = sum;
  __syncthreads();
  if (slice != 0 || c >= p.d) return;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < kFinish / 32; ++i) sum += part[i * 32 + threadIdx.x];
  if (p.wdtype == DT_FP32) static_cast<float*>(out)[c] = sum;
  else if (p.wdtype == DT_BF16) static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(sum);
  else static_cast<__half*>(out)[c] = __float2half_rn(sum);
}

constexpr int kUnit = 4;

template <typename T, int LANES, bool ADJ>
cudaError_t forward_l(const NormRopeArgs& a) {
  const int64_t per_token = (a.h + kUnit - 1) / kUnit + (a.hkv + kUnit - 1) / kUnit;
  const int64_t units = (int64_t)a.b * a.n * per_token;
  const int64_t blocks = (units * LANES + kThreads - 1) / kThreads;
  norm_rope_kernel<T, LANES, ADJ, kUnit><<<(unsigned)blocks, kThreads, 0, a.stream>>>(a, (int)units);
  return cudaGetLastError();
}

template <typename T, int LANES, bool ADJ>
cudaError_t backward_l(const NormRopeArgs& a) {
  constexpr int UNIT = kUnit / 2, GROUPS = kThreads / LANES;
  const int64_t tokens = (int64_t)a.b * a.n;
  const int64_t uq = tokens * ((a.h + UNIT - 1) / UNIT), uk = tokens * ((a.hkv + UNIT - 1) / UNIT);
  // blocks that fill the GPU, shared out by the units of each kind, at most one unit too many a group
  int64_t qb = 0, kb = 0;
  if (uq + uk > 0) {
    const int64_t all = norm_rope_bwd_blocks();
    qb = uq ? std::max<int64_t>(1, (all - 2) * uq / (uq + uk)) : 0;
    kb = uk ? std::max<int64_t>(1, (all - 2) * uk / (uq + uk)) : 0;
    qb = std::min(qb, (uq + GROUPS - 1) / GROUPS);
    kb = std::min(kb, (uk + GROUPS - 1) / GROUPS);
    norm_rope_bwd_kernel<T, LANES, ADJ, UNIT><<<(unsigned)(qb + kb), kThreads, 0, a.stream>>>(a, (int)qb);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.dwq || a.dwk)
    norm_rope_finish<<<dim3((a.d + 31) / 32, 2), kFinish, 0, a.stream>>>(a, (int)qb, (int)(qb + kb));
  return cudaGetLastError();
}

template <typename T, bool ADJ>
cudaError_t pick_lanes(const NormRopeArgs& a) {
  if (a.d <= 64) return a.backward ? backward_l<T, 8, ADJ>(a) : forward_l<T, 8, ADJ>(a);
  if (a.d <= 128) return a.backward ? backward_l<T, 16, ADJ>(a) : forward_l<T, 16, ADJ>(a);
  return a.backward ? backward_l<T, 32, ADJ>(a) : forward_l<T, 32, ADJ>(a);
}

template <typename T>
cudaError_t pick_pairs(const NormRopeArgs& a) {
  return a.adjacent ? pick_lanes<T, true>(a) : pick_lanes<T, false>(a);
}

}  // namespace

int norm_rope_bwd_blocks() { return 4 * device_sm_count(); }

cudaError_t launch_norm_rope(const NormRopeArgs& a) {
  switch (a.dtype) {
    case DT_BF16: return pick_pairs<__nv_bfloat16>(a);
    case DT_FP16: return pick_pairs<__half>(a);
    default: return pick_pairs<float>(a);
  }
}

}  // namespace fa
