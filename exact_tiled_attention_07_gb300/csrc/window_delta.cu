// D of the backward where queries see few keys (bf16/fp16, head dims 64/128/256): D_i = sum_j P_ij (dO_i . V_j), P and the products in
// 32 bits, instead of dO_i . O_i from the O that was rounded to 16 bits.
//
// Why: dS_ij = P_ij (dP_ij - D_i).  With few keys in sight dP and D are of one size and nearly cancel (with one key they are
// equal and dQ is 0), so that half a step of O is no longer small in dS.
//
// Which rows: all where window + sinks <= 32, else the 64 (a block) that each sequence begins with, as query i sees i + 1 keys at most.
// What dQ is off, relative to its norm, by the number of keys that a query sees (bf16, d = 128; fp16 the same in its steps; its own rounding
// is 0.0017 of it and that of dS as much again; dK the same within 0.0001):
//                     2       3       4       6       8       12      16      24      32      48      64      128
//   D from O          0.0038  0.0032  0.0030  0.0028  0.0027  0.0026  0.0025  0.0025  0.0025  0.0024  0.0024  0.0024
//   D from the keys   0.0024 (0.00235) at any number
// 32 keys: up to there the rounded O adds 5 % and more to what the result is off anyway (8 % at 16, 14 % at 8, 60 % at 2), behind it less.
//
// Work: a block takes 64 queries of a head, a warp 16 of them, whose Q and dO stay in registers as operands of m16n8k16; tiles
// of 64 keys and values come to shared memory, and of those a warp multiplies the 16 keys at a time that some of its queries see: 16 +
// window keys a query and no maximum, as L is known.  (The 128-row tiles of tcgen05 would multiply 128 + window keys a query, and
// wait for one another; here nothing waits but the block for its own copies.)  No mask but the window's: keys outside it reach nothing.
// The preprocess, which clears the workspace and writes D of the other rows, is launched to run beside it.
//
// Bound: HBM, Q, K, V and dO once.  8 x 16 heads of 4,096 rows, d = 128 (537 MB), all rows: 103 us (5.2 TB/s) for a window of 16.  The
// whole backward there with D from the keys and with D from O: windows of 2 to 16 438, 361 us, of 32 449, 361 (d = 64 327, 269; d = 256,
// 4 x 16 heads, 533, 456).  With the first blocks alone: window 1,024 722, 717; 2 x 16 heads of 1,000, d = 64, window 256 39, 37.
#include <cuda.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int ROWS = 64;      // queries of a block, keys of a tile
constexpr int THREADS = 128;  // a warp 16 queries

template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void matrices4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 64 rows of 16-bit elements in shared memory: 16-byte chunk c of row r at place c ^ (r & 7), so that eight rows of a matrix
// lie in eight different bank groups
template <int D>
__device__ __forceinline__ uint32_t chunk_at(uint32_t base, int r, int c) {
  return base + (uint32_t)(r * (D / 8) + (c ^ (r & 7))) * 16;
}

// rows [row0, row0 + 64) of a head of n rows on their way to shared memory; rows behind the last are zeros
template <int D>
__device__ __forceinline__ void copy_rows(uint32_t dst, const uint16_t* head, int row0, int n) {
#pragma unroll 4
  for (int x = threadIdx.x; x < ROWS * (D / 8); x += THREADS) {
    const int r = x / (D / 8), c = x % (D / 8);
    const bool there = row0 + r < n;
    const uint16_t* from = head + (int64_t)(there ? row0 + r : 0) * D + c * 8;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(chunk_at<D>(dst, r, c)), "l"(from), "r"(there ? 16 : 0)
                 : "memory");
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS)
    window_delta_kernel(const uint16_t* __restrict__ q, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                        const uint16_t* __restrict__ dout, const float* __restrict__ lse, float* __restrict__ delta, int n,
                        int npad, int tiles, int group, float scale_log2, int window, int sinks) {
  extern __shared__ __align__(1024) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;");
  const uint32_t first = smem_u32(smem), second = first + ROWS * D * 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x / tiles, q0 = (blockIdx.x - head * tiles) * ROWS;
  const int64_t at = (int64_t)head * n * D, kv_at = (int64_t)(head / group) * n * D;

  copy_rows<D>(first, q + at, q0, n);
  copy_rows<D>(second, dout + at, q0, n);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  uint32_t qa[D / 16][4], oa[D / 16][4];
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const int r = warp * 16 + lane % 16, c = kk * 2 + lane / 16;
    matrices4(qa[kk], chunk_at<D>(first, r, c));
    matrices4(oa[kk], chunk_at<D>(second, r, c));
  }
  // this thread's two queries of the warp's 16
  const int w0 = q0 + warp * 16, w1 = min(w0 + 15, n - 1);
  const int i[2] = {w0 + lane / 4, w0 + lane / 4 + 8};
  float minus_l[2], sum[2] = {0.f, 0.f};
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float l = i[r] < n ? lse[(int64_t)head * n + i[r]] : -INFINITY;  // (as the preprocess: P = 0 on rows without a finite score)
    minus_l[r] = l > -INFINITY ? -l * 1.4426950408889634f : -INFINITY;
  }

  const int begin = max(0, q0 - window + 1) / ROWS, end = min(q0 + ROWS - 1, n - 1) / ROWS;  // tiles of the window
  const int sink_tiles = min(begin, min(sinks, n) / ROWS + (min(sinks, n) % ROWS != 0));
  for (int t = 0; t < sink_tiles + end + 1 - begin; ++t) {
    const int j0 = (t < sink_tiles ? t : t - sink_tiles + begin) * ROWS;
    __syncthreads();  // what was in shared memory has been read
    copy_rows<D>(first, k + kv_at, j0, n);
    copy_rows<D>(second, v + kv_at, j0, n);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll 1
    for (int p = 0; p < ROWS / 16; ++p) {
      const int jp = j0 + p * 16;
      // none of the warp's queries sees a key of these 16
      if (jp > w1 || (w0 - (jp + 15) >= window && jp >= sinks)) continue;
      float s[2][4] = {}, dp[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int r = p * 16 + lane / 16 * 8 + lane % 8, c = kk * 2 + lane / 8 % 2;
        uint32_t kb[4], vb[4];
        matrices4(kb, chunk_at<D>(first, r, c));
        matrices4(vb, chunk_at<D>(second, r, c));
        mma16<BF16>(s[0], qa[kk], kb[0], kb[1]);
        mma16<BF16>(dp[0], oa[kk], vb[0], vb[1]);
        mma16<BF16>(s[1], qa[kk], kb[2], kb[3]);
        mma16<BF16>(dp[1], oa[kk], vb[2], vb[3]);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int r = x / 2 % 2, j = jp + x / 4 * 8 + lane % 4 * 2 + x % 2;
        const bool see = j <= i[r] && (i[r] - j < window || j < sinks);
        const float pr = ex2(fmaf(s[x / 4][x % 4], scale_log2, minus_l[r]));
        if (see) sum[r] = fmaf(pr, dp[x / 4][x % 4], sum[r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
    sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
    if (lane % 4 == 0 && i[r] < n) delta[(int64_t)head * npad + i[r]] = sum[r];
  }
}

template <int D, bool BF16>
cudaError_t launch_d(const BwdArgs& a) {
  const int tiles = (a.delta_rows + ROWS - 1) / ROWS, smem = 2 * ROWS * D * 2;
  auto kern = window_delta_kernel<D, BF16>;
  static std::atomic<unsigned long long> allowed;
  cudaError_t e = allow_smem(kern, smem, &allowed);
  if (e != cudaSuccess) return e;
  auto p = [](const void* x) { return static_cast<const uint16_t*>(x); };
  kern<<<(unsigned)((int64_t)a.bh * tiles), THREADS, smem, a.stream>>>(p(a.q), p(a.k), p(a.v), p(a.dout), a.lse, a.delta, a.n,
                                                                       (int)padded_rows(a.n), tiles, a.group,
                                                                       a.scale * 1.4426950408889634f, a.window, a.sinks);
  return cudaGetLastError();
}

}  // namespace

// All rows where none sees more than 32 keys, else a block of each sequence's first ones: see above.
int window_delta_rows(int n, int window, int sinks) { return (int64_t)window + sinks <= 32 ? n : n < ROWS ? n : ROWS; }

cudaError_t launch_window_delta(const BwdArgs& a) {
  const bool bf = a.dtype == DT_BF16;
  switch (a.d) {
    case 64: return bf ? launch_d<64, true>(a) : launch_d<64, false>(a);
    case 128: return bf ? launch_d<128, true>(a) : launch_d<128, false>(a);
    case 256: return bf ? launch_d<256, true>(a) : launch_d<256, false>(a);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace fa
