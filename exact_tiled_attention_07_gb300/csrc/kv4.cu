// The 4-bit key/value cache (layout: kv4.cuh): rows written (append), read back (read) and the
// cache thinned out by accumulated attention weight (evict).
//
// Quantisation of a group x of 64 channels of a row, every step an fp32 operation rounded to
// nearest unless said otherwise:
//   lo = min x, hi = max x
//   step   = fp16((hi - lo) / 15), rounded up, so that 15 steps cover [lo, hi]
//   middle = fp16(lo + 8 step), rounded to nearest
//   code   = clamp(rint((x - middle) / step), -8, 7) + 8     (8 when step is 0)
// so |middle + step (code - 8) - x| <= max(step / 2, 2^-11 |middle|) up to fp32 rounding.  The
// quotient and the two sums are IEEE operations: the codes are the same wherever they are taken.
#include <cuda_runtime.h>
#include <cstdint>

#include "kernels.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr uint32_t kSiteAppend = 920, kSiteRead = 921, kSiteEvict = 922;

template <typename T>
struct Elem;  // eight consecutive elements of a row as fp32, and back (rounded to nearest)
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<true>(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<true>(x[0], x[1]), pack2<true>(x[2], x[3]), pack2<true>(x[4], x[5]),
                                              pack2<true>(x[6], x[7]));
  }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<false>(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void store8(__half* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<false>(x[0], x[1]), pack2<false>(x[2], x[3]),
                                              pack2<false>(x[4], x[5]), pack2<false>(x[6], x[7]));
  }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// Slot that packed row r of sequence b takes: the sequence's rows are the last ones of its
// lens[b] cached slots.  False (with the device error recorded) when that is not inside the cache.
__device__ __forceinline__ bool row_slot(const Kv4RowArgs& a, int r, int b, int64_t* slot, uint32_t site) {
  *slot = (int64_t)a.lens[b] - a.cu[b + 1] + r;
  if (*slot >= 0 && *slot < a.capacity) return true;
  report_error(a.err, DERR_BAD_ARG, site);
  return false;
}

// One thread per 8 channels of a row (one 32-bit word of codes); the 8 threads of a group find its
// minimum and maximum with three shuffles.  Bound by HBM: 8 elements in, 4.5 bytes out a thread.
template <typename T>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4RowArgs a, int words_per_row) {
  const int64_t per_row = (int64_t)a.hkv * words_per_row;
  const int64_t total = (int64_t)a.t * per_row;
  // words_per_row is a multiple of 8 and a group's words are 8 consecutive threads of a warp: all
  // 8 have the same row, head and fate, so the shuffles stay inside them
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= total) return;
  const int r = (int)(i / per_row);
  const int rest = (int)(i - (int64_t)r * per_row);
  const int h = rest / words_per_row, word = rest - h * words_per_row;
  const int b = packed_sequence(a.cu, a.b, r);
  if (b < 0) return;
  int64_t slot;
  if (!row_slot(a, r, b, &slot, kSiteAppend)) return;
  const int d = a.d;
  uint8_t* block = a.cache + (((int64_t)b * a.hkv + h) * (a.capacity / kKv4Block) + slot / kKv4Block) * kv4_block_bytes(d);
  const int in = (int)(slot % kKv4Block);
  const unsigned lanes = 0xFFu << (threadIdx.x & 24);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const T* src = which ? static_cast<const T*>(a.v) + r * a.v_ts + h * a.v_hs
                         : static_cast<const T*>(a.k) + r * a.k_ts + h * a.k_hs;
    float x[8];
    Elem<T>::load8(src + word * 8, x);
    float lo = x[0], hi = x[0];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      bad |= !(fabsf(x[j]) <= kKv4Limit);
      lo = fminf(lo, x[j]);
      hi = fmaxf(hi, x[j]);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(lanes, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(lanes, hi, o));
    }
    bad = __any_sync(lanes, bad);
    const __half step = __float2half_ru(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const float s = __half2float(step);
    const __half middle = __float2half_rn(__fadd_rn(lo, 8.f * s));
    const float m = __half2float(middle);
    uint32_t codes = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float c = 0.f;
      if (!bad && s > 0.f) c = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[j], m), s)), -8.f), 7.f);
      codes |= (uint32_t)((int)c + 8) << (4 * j);
    }
    *reinterpret_cast<uint32_t*>(block + kv4_codes_at(d, which) + in * kv4_code_bytes(d) + word * 4) = codes;
    if ((word & 7) == 0) {
      const uint32_t par = bad ? kKv4NanParam
                               : (uint32_t)__half_as_ushort(step) | ((uint32_t)__half_as_ushort(middle) << 16);
      *reinterpret_cast<uint32_t*>(block + kv4_params_at(d, which) + (in * kv4_param_words(d) + (word >> 3)) * 4) = par;
    }
  }
  if (a.weights && word == 0) a.weights[((int64_t)b * a.hkv + h) * a.capacity + slot] = 0.f;
}

// The inverse: one thread per 8 channels of a row, middle + step (code - 8) in fp32, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4RowArgs a, int words_per_row) {
  const int64_t per_row = (int64_t)a.hkv * words_per_row;
  const int64_t total = (int64_t)a.t * per_row;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= total) return;
  const int r = (int)(i / per_row);
  const int rest = (int)(i - (int64_t)r * per_row);
  const int h = rest / words_per_row, word = rest - h * words_per_row;
  const int b = packed_sequence(a.cu, a.b, r);
  if (b < 0) return;
  int64_t slot;
  if (!row_slot(a, r, b, &slot, kSiteRead)) return;
  const int d = a.d;
  const uint8_t* block =
      a.cache + (((int64_t)b * a.hkv + h) * (a.capacity / kKv4Block) + slot / kKv4Block) * kv4_block_bytes(d);
  const int in = (int)(slot % kKv4Block);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const uint32_t codes =
        *reinterpret_cast<const uint32_t*>(block + kv4_codes_at(d, which) + in * kv4_code_bytes(d) + word * 4);
    const uint32_t par = *reinterpret_cast<const uint32_t*>(block + kv4_params_at(d, which) +
                                                            (in * kv4_param_words(d) + (word >> 3)) * 4);
    const float s = __half2float(__ushort_as_half((unsigned short)(par & 0xFFFF)));
    const float m = __half2float(__ushort_as_half((unsigned short)(par >> 16)));
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = fmaf(s, (float)((int)((codes >> (4 * j)) & 15u) - 8), m);
    T* dst = which ? static_cast<T*>(const_cast<void*>(a.v)) + r * a.v_ts + h * a.v_hs
                   : static_cast<T*>(const_cast<void*>(a.k)) + r * a.k_ts + h * a.k_hs;
    Elem<T>::store8(dst + word * 8, x);
  }
}

template <bool READ>
cudaError_t launch_rows(const Kv4RowArgs& a) {
  const int words = a.d / 8;
  const int64_t threads = (int64_t)a.t * a.hkv * words;
  const unsigned grid = (unsigned)((threads + 255) / 256);
  switch (a.dtype) {
    case DT_BF16:
      if (READ) kv4_read_kernel<__nv_bfloat16><<<grid, 256, 0, a.stream>>>(a, words);
      else kv4_append_kernel<__nv_bfloat16><<<grid, 256, 0, a.stream>>>(a, words);
      break;
    case DT_FP16:
      if (READ) kv4_read_kernel<__half><<<grid, 256, 0, a.stream>>>(a, words);
      else kv4_append_kernel<__half><<<grid, 256, 0, a.stream>>>(a, words);
      break;
    default:
      if (READ) kv4_read_kernel<float><<<grid, 256, 0, a.stream>>>(a, words);
      else kv4_append_kernel<float><<<grid, 256, 0, a.stream>>>(a, words);
  }
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------- eviction
//
// Of a sequence's len slots of one key/value head, `keep` stay: the `recent` newest ones (the last
// slots) and, of the others, those of the largest weight, ties going to the lowest slot.  Kept
// slots keep their order, so the last slots stay the newest.
//
// kv4_select_kernel (one block per head): weights as 32-bit keys that order like the numbers
// (NaN above everything, -0 as 0); the k-th largest key is found digit by digit (8 bits, four
// histogram passes over the keys); then one ordered pass writes the kept slots: those above the
// threshold key, the first ones equal to it, and the newest.
// kv4_gather_kernel: moves rows, 16 bytes a thread.

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int evict_len(const Kv4EvictArgs& a, int b) {
  const int n = a.lens[b];
  if (n < 0 || n > a.capacity) {
    if (threadIdx.x == 0) report_error(a.err, DERR_BAD_ARG, kSiteEvict);
    return n < 0 ? 0 : a.capacity;
  }
  return n;
}

constexpr int kSelThreads = 1024;

__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const Kv4EvictArgs a) {
  const int bh = blockIdx.x, b = bh / a.hkv;
  const int n = evict_len(a, b);
  const int kept_n = min(n, a.keep);
  int32_t* kept = a.kept + (int64_t)bh * a.keep;
  const int tid = threadIdx.x;
  for (int i = kept_n + tid; i < a.keep; i += kSelThreads) kept[i] = -1;
  if (n <= a.keep) {
    for (int i = tid; i < n; i += kSelThreads) kept[i] = i;
    return;
  }
  const float* w = a.weights + (int64_t)bh * a.capacity;
  const int m = n - a.recent;  // candidates: slots [0, m)
  const int k = a.keep - a.recent;  // of which k stay, 0 <= k < m
  __shared__ unsigned hist[256];
  __shared__ unsigned warp_sum[2][32];
  __shared__ unsigned sel_digit, sel_left;
  uint32_t prefix = 0, mask = 0;
  unsigned left = (unsigned)k;  // still to take among the keys that match prefix
  if (k > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = tid; i < m; i += kSelThreads) {
        const uint32_t key = weight_key(w[i]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        unsigned rest = left;
        int digit = 255;
        for (; digit > 0; --digit) {
          if (hist[digit] >= rest) break;
          rest -= hist[digit];
        }
        sel_digit = (unsigned)digit;
        sel_left = rest;
      }
      __syncthreads();
      prefix |= sel_digit << shift;
      mask |= 0xFFu << shift;
      left = sel_left;
      __syncthreads();
    }
  }
  // keys above `prefix` stay, and the first `left` of those equal to it
  unsigned out = 0, eq = 0;  // kept so far, equal ones seen so far (slots before this round)
  for (int base = 0; base < n; base += kSelThreads) {
    const int i = base + tid;
    bool above = false, equal = false;
    if (i < n) {
      if (i >= m) {
        above = true;
      } else if (k > 0) {
        const uint32_t key = weight_key(w[i]);
        above = key > prefix;
        equal = key == prefix;
      }
    }
    const unsigned be = __ballot_sync(0xffffffffu, equal);
    const int warp = tid >> 5, lane = tid & 31;
    if (lane == 0) warp_sum[0][warp] = __popc(be);
    __syncthreads();
    unsigned eq_before = eq, eq_total = 0;
    for (int j = 0; j < 32; ++j) {
      const unsigned v = warp_sum[0][j];
      if (j < warp) eq_before += v;
      eq_total += v;
    }
    const bool take = above || (equal && eq_before + __popc(be & ((1u << lane) - 1u)) < left);
    const unsigned bt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) warp_sum[1][warp] = __popc(bt);
    __syncthreads();
    unsigned at = out, total = 0;
    for (int j = 0; j < 32; ++j) {
      const unsigned v = warp_sum[1][j];
      if (j < warp) at += v;
      total += v;
    }
    if (take) {
      const unsigned pos = at + __popc(bt & ((1u << lane) - 1u));
      if (pos < (unsigned)a.keep) kept[pos] = i;
    }
    out += total;
    eq += eq_total;
    __syncthreads();
  }
}

// One thread per 16 bytes of codes of a kept row (K and V), the first threads of a row also its
// parameters and weight.
__global__ void __launch_bounds__(256) kv4_gather_kernel(const Kv4EvictArgs a) {
  const int d = a.d, per = d / 32;  // 16-byte pieces of a row's codes
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.b; b += blockDim.x) a.out_lens[b] = min(min(max(a.lens[b], 0), a.capacity), a.keep);
  const int64_t row = i / (2 * per);
  if (row >= (int64_t)a.b * a.hkv * a.keep) return;
  const int piece = (int)(i - row * (2 * per));
  const int64_t bh = row / a.keep;
  const int to = (int)(row - bh * a.keep);
  const int from = a.kept[row];
  if (from < 0) return;
  const uint8_t* sb =
      a.cache + (bh * (a.capacity / kKv4Block) + from / kKv4Block) * kv4_block_bytes(d);
  uint8_t* db = a.out_cache + (bh * (a.out_capacity / kKv4Block) + to / kKv4Block) * kv4_block_bytes(d);
  const int si = from % kKv4Block, di = to % kKv4Block;
  const int which = piece / per, part = piece - which * per;
  const int at = kv4_codes_at(d, which) + part * 16;
  *reinterpret_cast<uint4*>(db + at + di * kv4_code_bytes(d)) =
      *reinterpret_cast<const uint4*>(sb + at + si * kv4_code_bytes(d));
  const int pw = kv4_param_words(d);
  if (part < pw)
    *reinterpret_cast<uint32_t*>(db + kv4_params_at(d, which) + (di * pw + part) * 4) =
        *reinterpret_cast<const uint32_t*>(sb + kv4_params_at(d, which) + (si * pw + part) * 4);
  if (piece == 0) a.out_weights[bh * a.out_capacity + to] = a.weights[bh * a.capacity + from];
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowArgs& a) { return launch_rows<false>(a); }
cudaError_t launch_kv4_read(const Kv4RowArgs& a) { return launch_rows<true>(a); }

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a) {
  kv4_select_kernel<<<a.b * a.hkv, kSelThreads, 0, a.stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t threads = (int64_t)a.b * a.hkv * a.keep * 2 * (a.d / 32);
  kv4_gather_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
