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
// Bound: HBM (each row read and written once; backward x and dy read).  A channel costs 5 to 10 instructions, which is enough to
// matter at 6 TB/s, so the layout saves them: a lane holds 16 channels of a row (8 in fp32, and where the row or its rotated
// part is no multiple of 16), as two pieces of 8 that are the two halves of its rotated pairs (rotary / 2 channels apart, or
// one behind the other where pairs are adjacent): a pair never crosses lanes, only a row's sums do, and arithmetic runs on
// paired fp32 instructions.  Measured on one GB300: 34,001 tokens of 32 + 8 heads of 128 (bf16) 111 us, 6.4 TB/s of 6.8; 8 x 4096
// tokens, 16 + 16 heads, into the layout of attention 87 us (6.2 TB/s), gradients 130 us (6.2 TB/s).  Steps there (gradients of the
// second, TB/s): 8 channels a lane, loads in registers 3.3; loads one row ahead 4.1; a ring in shared memory 4.9; no
// divisions, rsqrtf, no zero fills 5.3; units of four heads 5.8 (figures of the steps with L2 full of data to be written back).
// Groups side by side on tokens instead of heads: 90 and 132 us there, 128 us for the packed tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxOcc = 3;

// P consecutive channels of a row as they lie in memory, and as P / 2 pairs of floats.
template <typename T, int P>
struct Piece {
  static constexpr int kWords = P * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kWords == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void open(float2* v) const {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      else v[i] = unpack2<std::is_same<T, __nv_bfloat16>::value>(w[i]);
    }
  }
  __device__ __forceinline__ void close(const float2* v) {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      if constexpr (sizeof(T) == 4) w[2 * i] = __float_as_uint(v[i].x), w[2 * i + 1] = __float_as_uint(v[i].y);
      else w[i] = pack2<std::is_same<T, __nv_bfloat16>::value>(v[i].x, v[i].y);
    }
  }
};

// Four channels of a weight (1 where there is none).
__device__ __forceinline__ float4 weight4(const void* w, int kind, int c) {
  if (!w) return make_float4(1.f, 1.f, 1.f, 1.f);
  if (kind == DT_FP32) return *reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
  const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + c);
  const float2 lo = kind == DT_BF16 ? unpack2<true>(v.x) : unpack2<false>(v.x);
  const float2 hi = kind == DT_BF16 ? unpack2<true>(v.y) : unpack2<false>(v.y);
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}
template <int P>
__device__ __forceinline__ void load_weights(float2 (&wt)[P], const void* w, int kind, int a, int b) {
#pragma unroll
  for (int i = 0; i < P / 4; ++i) {
    const float4 x = weight4(w, kind, a + 4 * i), y = weight4(w, kind, b + 4 * i);
    wt[2 * i] = make_float2(x.x, x.y), wt[2 * i + 1] = make_float2(x.z, x.w);
    wt[P / 2 + 2 * i] = make_float2(y.x, y.y), wt[P / 2 + 2 * i + 1] = make_float2(y.z, y.w);
  }
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Where a lane's 2 P channels are: pieces of P at `a` and `b`; pair t of its P is (a + t, b + t), or where pairs are
// adjacent (a + 2 t, a + 2 t + 1), b then being a + P.
struct Pieces {
  int a, b;
  int pair;  // its first pair's place in the table, -1: not rotated
};
template <int P, bool ADJ>
__device__ __forceinline__ Pieces pieces_of(int lane, int rotary) {
  Pieces p;
  const int at = 2 * P * lane;
  const bool turned = at < rotary;
  p.pair = turned ? P * lane : -1;
  p.a = turned && !ADJ ? P * lane : at;
  p.b = turned && !ADJ ? P * lane + rotary / 2 : at + P;
  return p;
}

// cos and sin of a lane's P pairs at a token (not set where it is not rotated), two pairs to a float2.  A position outside the
// table is clamped to it and recorded.
template <int P>
struct Angles {
  float2 c[P / 2], s[P / 2];
  __device__ __forceinline__ void load(const NormRopeArgs& p, int64_t t, int n, const Pieces& at) {
    if (p.rotary == 0) return;
    int pos = p.positions ? p.positions[t] : n;
    if (pos < 0 || pos >= p.table_len) {
      report_error(p.err, DERR_BAD_ARG, 300);
      pos = pos < 0 ? 0 : p.table_len - 1;
    }
    if (at.pair < 0) return;
    const float* row = p.table + (int64_t)pos * p.rotary + at.pair;
#pragma unroll
    for (int i = 0; i < P / 4; ++i) {
      const float4 c4 = *reinterpret_cast<const float4*>(row + 4 * i);
      const float4 s4 = *reinterpret_cast<const float4*>(row + p.rotary / 2 + 4 * i);
      c[2 * i] = make_float2(c4.x, c4.y), c[2 * i + 1] = make_float2(c4.z, c4.w);
      s[2 * i] = make_float2(s4.x, s4.y), s[2 * i + 1] = make_float2(s4.z, s4.w);
    }
  }
  // v turned by the angles (BACK: by their opposites)
  template <bool ADJ, bool BACK>
  __device__ __forceinline__ void turn(float2 (&v)[P]) const {
    if constexpr (ADJ) {
#pragma unroll
      for (int t = 0; t < P; ++t) {
        const float ct = t & 1 ? c[t / 2].y : c[t / 2].x, st = t & 1 ? s[t / 2].y : s[t / 2].x;
        const float2 x = fmul2(make_float2(v[t].y, v[t].x), BACK ? make_float2(st, -st) : make_float2(-st, st));
        v[t] = ffma2(v[t], ct, x);
      }
    } else {
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        const float2 a = v[i], b = v[P / 2 + i];
        const float2 ms = make_float2(-s[i].x, -s[i].y);
        v[i] = ffma2v(b, BACK ? s[i] : ms, fmul2(a, c[i]));
        v[P / 2 + i] = ffma2v(a, BACK ? ms : s[i], fmul2(b, c[i]));
      }
    }
  }
};

// The row of head h0 of token (b, n) in a tensor.
template <typename T>
__device__ __forceinline__ const T* rows_of(const void* base, const NormRopeStrides& st, int b, int n, int h0) {
  return static_cast<const T*>(base) + b * st.batch + n * st.token + h0 * st.head;
}

template <int P>
__device__ __forceinline__ float squares(const float2 (&v)[P]) {
  float2 sq = fmul2(v[0], v[0]);
#pragma unroll
  for (int t = 1; t < P; ++t) sq = ffma2v(v[t], v[t], sq);
  return sq.x + sq.y;
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_async(void* smem, const void* g) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
}

__host__ __device__ constexpr int unit_of(int heads) { return heads % 4 == 0 ? 4 : (heads % 2 == 0 ? 2 : 1); }

// The row that a group of lanes is at: head h of token t = b n_tokens + n.  A group takes units of up to four heads of a
// token, one row after the other, so that it reads cos and sin once for them, and goes on by the same number of units each
// time, which is added digit by digit (a division costs as much as a fifth of the work on a row).
struct Row {
  int t, b, n, h, sub;
  __device__ __forceinline__ void set(int u, int unit, int heads, int tokens) {
    const int per_token = heads / unit;
    t = u / per_token;
    h = (u - t * per_token) * unit;
    b = t / tokens;
    n = t - b * tokens;
    sub = 0;
  }
  __device__ __forceinline__ void add(const Row& step, int unit, int heads, int tokens) {
    ++h;
    if (++sub < unit) return;
    sub = 0;
    h += step.h - unit;
    const int carry = h >= heads;
    h -= carry ? heads : 0;
    t += step.t + carry;
    n += step.n + carry;
    b += step.b;
    if (n >= tokens) {
      n -= tokens;
      ++b;
    }
  }
};

// A group of LANES lanes walks the rows of one kind (blocks below q_blocks take queries, the others keys): weights, and
// backward the sums of dw, stay in its registers.  A lane copies its own pieces of the rows to come into a ring of STAGES
// places in shared memory (asynchronously, and nobody else reads them, so that no barrier is needed): the bytes in flight
// that HBM's latency asks for do not fit into registers beside 2 P weights, sums, channels and gradients.
// Backward: a block adds its groups' sums in shared memory, in a fixed order, into one row of partials for the finishing
// kernel.  Sums are in 32 bits, in three levels (a group's rows, a block's groups, blocks).
template <typename T, int P, bool BWD>
struct RopeCfg {
  static constexpr int PIECE = P * (int)sizeof(T);  // bytes: 8 or 16
  static constexpr int PIECES = BWD ? 4 : 2;        // of x (and dy) for every lane
  static constexpr int STAGE = kThreads * PIECES * PIECE;
  // Blocks an SM and rows in flight.  Two blocks with 128 registers a thread where a lane has 16 channels (three spill, 102 us
  // against 93 for norm and rotation of 8 x 4096 tokens, 16 + 16 heads of 128 in bf16), three where it has 8; deeper rings
  // measured the same.
  static constexpr int OCC = P == 8 ? 2 : 3;
  static constexpr int STAGES = (BWD ? 3 : 4) * 16 / PIECE;
  static constexpr int SMEM = STAGES * STAGE;
  static_assert(OCC <= kMaxOcc && OCC * (SMEM + 1024) <= 228 * 1024, "shared memory, partials");
};
template <typename T, int P, int LANES, bool ADJ, bool BWD>
__global__ void __launch_bounds__(kThreads, RopeCfg<T, P, BWD>::OCC)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs p, int q_blocks) {
  using C = RopeCfg<T, P, BWD>;
  constexpr int GROUPS = kThreads / LANES;
  extern __shared__ __align__(16) uint8_t ring[];
  static_assert(!BWD || C::SMEM >= GROUPS * 2 * P * LANES * 4, "the sums of dw go where the ring was");
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const bool key = (int)blockIdx.x >= q_blocks;
  const int heads = key ? p.hkv : p.h;
  const int unit = unit_of(heads), units = p.b * p.n * (heads / unit);
  const int step = (key ? (int)gridDim.x - q_blocks : q_blocks) * GROUPS;
  const bool in_row = 2 * P * lane < p.d;
  const Pieces at = pieces_of<P, ADJ>(in_row ? lane : 0, p.rotary);
  const NormRopeStrides &xs = key ? p.k_st : p.q_st, &ys = key ? p.ko_st : p.qo_st, &ds = key ? p.dk_st : p.dq_st;
  const void *xbase = key ? p.k : p.q, *ybase = key ? p.ko : p.qo, *dbase = key ? p.dk : p.dq;
  float2 wt[P], dw[P];
  load_weights(wt, key ? p.wk : p.wq, p.wdtype, at.a, at.b);
#pragma unroll
  for (int c = 0; c < P; ++c) dw[c] = make_float2(0.f, 0.f);
  const float inv_d = 1.f / (float)p.d;
  auto place = [&](int stage, int piece) { return ring + stage * C::STAGE + (piece * kThreads + threadIdx.x) * C::PIECE; };
  auto fetch = [&](const Row& w, int stage) {
    const T* x = rows_of<T>(xbase, xs, w.b, w.n, w.h);
    copy_async<C::PIECE>(place(stage, 0), x + at.a);
    copy_async<C::PIECE>(place(stage, 1), x + at.b);
    if constexpr (BWD) {
      const T* dy = rows_of<T>(ybase, ys, w.b, w.n, w.h);
      copy_async<C::PIECE>(place(stage, 2), dy + at.a);
      copy_async<C::PIECE>(place(stage, 3), dy + at.b);
    }
  };
  // (all groups of a warp go round together: the sums of rows are taken by the whole warp.  A group that is behind the last
  // row works on what lies in its places and stores nothing.)
  const int u0 = ((int)blockIdx.x - (key ? q_blocks : 0)) * GROUPS + group;
  const int ahead = group % (32 / LANES);  // units between the warp's first group and this one
  const int count = (u0 < units ? (units - 1 - u0) / step + 1 : 0) * unit;  // rows of this group
  const int rounds = (u0 - ahead < units ? (units - 1 - (u0 - ahead)) / step + 1 : 0) * unit;  // of the warp's first: the most
  Row now, next, by;
  by.set(step, unit, heads, p.n);
  now.set(min(u0, units - 1), unit, heads, p.n);
  next = now;
  Angles<P> turn;
#pragma unroll
  for (int k = 0; k < C::STAGES - 1; ++k) {
    if (k < count) fetch(next, k);
    copies_commit();
    next.add(by, unit, heads, p.n);
  }
  int stage = 0;
  for (int i = 0; i < rounds; ++i) {
    const bool mine = i < count && in_row;
    if (now.sub == 0 && i < count) turn.load(p, now.t, now.n, at);
    if (i + C::STAGES - 1 < count) fetch(next, stage == 0 ? C::STAGES - 1 : stage - 1);
    copies_commit();
    next.add(by, unit, heads, p.n);
    copies_wait<C::STAGES - 1>();
    float2 v[P];
    Piece<T, P> piece;
    piece.load(reinterpret_cast<const T*>(place(stage, 0)));
    piece.open(v);
    piece.load(reinterpret_cast<const T*>(place(stage, 1)));
    piece.open(v + P / 2);
    // (lanes behind a row's end hold a copy of its first pieces)
    const float sq = row_sum<LANES>(in_row ? squares(v) : 0.f);
    const float r = rsqrtf(fmaf(sq, inv_d, p.eps));
    const float2 r2 = make_float2(r, r);
    if constexpr (!BWD) {
#pragma unroll
      for (int c = 0; c < P; ++c) v[c] = fmul2(fmul2(v[c], r2), wt[c]);
      if (at.pair >= 0) turn.template turn<ADJ, false>(v);
      if (mine) {
        T* y = const_cast<T*>(rows_of<T>(ybase, ys, now.b, now.n, now.h));
        piece.close(v);
        piece.store(y + at.a);
        piece.close(v + P / 2);
        piece.store(y + at.b);
      }
    } else {
      float2 g[P];
      piece.load(reinterpret_cast<const T*>(place(stage, 2)));
      piece.open(g);
      piece.load(reinterpret_cast<const T*>(place(stage, 3)));
      piece.open(g + P / 2);
      if (at.pair >= 0) turn.template turn<ADJ, true>(g);
      float2 dot = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < P; ++c) {
        v[c] = fmul2(v[c], r2);
        if (mine) dw[c] = ffma2v(g[c], v[c], dw[c]);
        g[c] = fmul2(g[c], wt[c]);
        dot = ffma2v(g[c], v[c], dot);
      }
      const float m = -row_sum<LANES>(in_row ? dot.x + dot.y : 0.f) * inv_d;
#pragma unroll
      for (int c = 0; c < P; ++c) g[c] = fmul2(ffma2(v[c], m, g[c]), r2);
      if (mine) {
        T* dx = const_cast<T*>(rows_of<T>(dbase, ds, now.b, now.n, now.h));
        piece.close(g);
        piece.store(dx + at.a);
        piece.close(g + P / 2);
        piece.store(dx + at.b);
      }
    }
    stage = stage + 1 == C::STAGES ? 0 : stage + 1;
    now.add(by, unit, heads, p.n);
  }
  copies_wait<0>();
  if constexpr (BWD) {
    __syncthreads();  // every lane has read what it copied
    float* part = reinterpret_cast<float*>(ring);  // [GROUPS][d]
    if (in_row) {
#pragma unroll
      for (int c = 0; c < P / 2; ++c) {
        *reinterpret_cast<float2*>(part + group * p.d + at.a + 2 * c) = dw[c];
        *reinterpret_cast<float2*>(part + group * p.d + at.b + 2 * c) = dw[P / 2 + c];
      }
    }
    __syncthreads();
    if ((int)threadIdx.x < p.d) {
      float sum = 0.f;
#pragma unroll 4
      for (int g = 0; g < GROUPS; ++g) sum += part[g * p.d + threadIdx.x];
      p.partials[(int64_t)blockIdx.x * p.d + threadIdx.x] = sum;
    }
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

template <typename T, int P, int LANES, bool ADJ, bool BWD>
cudaError_t launch_l(const NormRopeArgs& a) {
  using C = RopeCfg<T, P, BWD>;
  constexpr int GROUPS = kThreads / LANES;
  const int64_t rq = (int64_t)a.b * a.n * a.h, rk = (int64_t)a.b * a.n * a.hkv;
  // blocks that fill the GPU, shared out by the rows of each kind, no more than there are units
  int64_t qb = 0, kb = 0;
  if (rq + rk > 0) {
    const int64_t all = C::OCC * device_sm_count();
    qb = rq ? std::max<int64_t>(1, std::min<int64_t>(all - (rk ? 1 : 0), (all * rq + (rq + rk) / 2) / (rq + rk))) : 0;
    kb = rk ? std::max<int64_t>(1, all - qb) : 0;
    qb = std::min(qb, (rq / unit_of(a.h) + GROUPS - 1) / GROUPS);
    kb = std::min(kb, (rk / unit_of(a.hkv) + GROUPS - 1) / GROUPS);
    auto kern = norm_rope_kernel<T, P, LANES, ADJ, BWD>;
    static std::atomic<unsigned long long> allowed;
    cudaError_t e = allow_smem(kern, C::SMEM, &allowed);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(qb + kb), kThreads, C::SMEM, a.stream>>>(a, (int)qb);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (BWD && (a.dwq || a.dwk))
    norm_rope_finish<<<dim3((a.d + 31) / 32, 2), kFinish, 0, a.stream>>>(a, (int)qb, (int)(qb + kb));
  return cudaGetLastError();
}

template <typename T, bool ADJ, bool BWD>
cudaError_t pick_lanes(const NormRopeArgs& a) {
  if constexpr (sizeof(T) == 2) {
    // sixteen channels a lane where the row and its rotated part are whole numbers of them
    if (a.d % 16 == 0 && a.rotary % 16 == 0) {
      if (a.d <= 64) return launch_l<T, 8, 4, ADJ, BWD>(a);
      if (a.d <= 128) return launch_l<T, 8, 8, ADJ, BWD>(a);
      return launch_l<T, 8, 16, ADJ, BWD>(a);
    }
  }
  if (a.d <= 64) return launch_l<T, 4, 8, ADJ, BWD>(a);
  if (a.d <= 128) return launch_l<T, 4, 16, ADJ, BWD>(a);
  return launch_l<T, 4, 32, ADJ, BWD>(a);
}

template <typename T>
cudaError_t pick_pairs(const NormRopeArgs& a) {
  if (a.backward) return a.adjacent ? pick_lanes<T, true, true>(a) : pick_lanes<T, false, true>(a);
  return a.adjacent ? pick_lanes<T, true, false>(a) : pick_lanes<T, false, false>(a);
}

}  // namespace

int norm_rope_bwd_blocks() { return kMaxOcc * device_sm_count(); }

cudaError_t launch_norm_rope(const NormRopeArgs& a) {
  switch (a.dtype) {
    case DT_BF16: return pick_pairs<__nv_bfloat16>(a);
    case DT_FP16: return pick_pairs<__half>(a);
    default: return pick_pairs<float>(a);
  }
}

}  // namespace fa
