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

// Sequence of packed row r for a whole warp (every lane gets it): the number of sequences that end at
// or before r, 32 ends at a time; -1 when r belongs to none.  Any contents of cu give a b in range.
__device__ __forceinline__ int warp_sequence(const int32_t* __restrict__ cu, int B, int r) {
  const int lane = threadIdx.x & 31;
  int b = 0;
  for (int base = 0; base < B; base += 32) {
    const bool past = base + lane < B && cu[base + lane + 1] <= r;
    const int n = __popc(__ballot_sync(0xffffffffu, past));
    b += n;
    if (n < 32) break;
  }
  return b < B && r >= cu[0] ? b : -1;
}

constexpr int kRowWarps = 8;  // rows of a block: one warp each

// A warp takes CH x 32 words (8 channels each) of a row's key/value heads: a lane loads 16 bytes of
// 16-bit elements, keys and values, before anything else is known; the 8 lanes of a group find its minimum and
// maximum with three shuffles and a lane's codes are one 32-bit word.  Bound by HBM: 16 bytes in, 4.5 out
// for 8 channels.  The quotient is taken as a product with 1 / step, whose distance from the IEEE quotient
// is below 2^-20 for |quotient| <= 8.5; only where it lies within 2^-18 of a half (where that could change the
// rounding) is the division done.
template <typename T, int CH>
__global__ void __launch_bounds__(kRowWarps * 32) kv4_append_kernel(const Kv4RowArgs a, int word_shift) {
  const int r = blockIdx.x * kRowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= a.t) return;
  const int words = a.hkv << word_shift;  // of a row
  const int w0 = blockIdx.y * (CH * 32) + lane;
  float x[CH][2][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int w = w0 + c * 32;
    if (w >= words) continue;
    const int h = w >> word_shift, word = w - (h << word_shift);
    Elem<T>::load8(static_cast<const T*>(a.k) + r * a.k_ts + h * a.k_hs + word * 8, x[c][0]);
    Elem<T>::load8(static_cast<const T*>(a.v) + r * a.v_ts + h * a.v_hs + word * 8, x[c][1]);
  }
  const int b = warp_sequence(a.cu, a.b, r);
  if (b < 0) return;
  int64_t slot;
  if (!row_slot(a, r, b, &slot, kSiteAppend)) return;
  const int d = a.d, in = (int)(slot % kKv4Block);
  const unsigned lanes = 0xFFu << (lane & 24);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int w = w0 + c * 32;
    if (w >= words) continue;  // (words is a multiple of 8: a group's lanes go together)
    const int h = w >> word_shift, word = w - (h << word_shift);
    uint8_t* block = a.cache + (((int64_t)b * a.hkv + h) * (a.capacity / kKv4Block) + slot / kKv4Block) * kv4_block_bytes(d);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float(&y)[8] = x[c][which];
      float lo = y[0], hi = y[0];
      bool bad = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        bad |= !(fabsf(y[j]) <= kKv4Limit);
        lo = fminf(lo, y[j]);
        hi = fmaxf(hi, y[j]);
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
      uint32_t codes = 0x88888888u;
      if (!bad && s > 0.f) {
        const float inv = __frcp_rn(s);
        codes = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float diff = __fsub_rn(y[j], m);
          float q = diff * inv;
          if (fabsf(q - rintf(q)) > 0.5f - 0x1p-18f) q = __fdiv_rn(diff, s);
          codes |= (uint32_t)((int)fminf(fmaxf(rintf(q), -8.f), 7.f) + 8) << (4 * j);
        }
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
}

// The inverse, with the same split: middle + step (code - 8) in fp32, rounded once.
template <typename T, int CH>
__global__ void __launch_bounds__(kRowWarps * 32) kv4_read_kernel(const Kv4RowArgs a, int word_shift) {
  const int r = blockIdx.x * kRowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= a.t) return;
  const int words = a.hkv << word_shift;
  const int w0 = blockIdx.y * (CH * 32) + lane;
  const int b = warp_sequence(a.cu, a.b, r);
  if (b < 0) return;
  int64_t slot;
  if (!row_slot(a, r, b, &slot, kSiteRead)) return;
  const int d = a.d, in = (int)(slot % kKv4Block);
  uint32_t codes[CH][2], par[CH][2];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int w = w0 + c * 32;
    if (w >= words) continue;
    const int h = w >> word_shift, word = w - (h << word_shift);
    const uint8_t* block =
        a.cache + (((int64_t)b * a.hkv + h) * (a.capacity / kKv4Block) + slot / kKv4Block) * kv4_block_bytes(d);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      codes[c][which] =
          *reinterpret_cast<const uint32_t*>(block + kv4_codes_at(d, which) + in * kv4_code_bytes(d) + word * 4);
      par[c][which] = *reinterpret_cast<const uint32_t*>(block + kv4_params_at(d, which) +
                                                         (in * kv4_param_words(d) + (word >> 3)) * 4);
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int w = w0 + c * 32;
    if (w >= words) continue;
    const int h = w >> word_shift, word = w - (h << word_shift);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float2 p = unpack2<false>(par[c][which]);
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = fmaf(p.x, (float)((int)((codes[c][which] >> (4 * j)) & 15u) - 8), p.y);
      T* dst = which ? static_cast<T*>(const_cast<void*>(a.v)) + r * a.v_ts + h * a.v_hs
                     : static_cast<T*>(const_cast<void*>(a.k)) + r * a.k_ts + h * a.k_hs;
      Elem<T>::store8(dst + word * 8, x);
    }
  }
}

// Two chunks of 32 words a warp (one where a row has no more) keep 64 bytes a lane in flight.
template <bool READ, typename T>
cudaError_t launch_rows_t(const Kv4RowArgs& a) {
  const int shift = a.d == 64 ? 3 : (a.d == 128 ? 4 : 5);
  const int words = a.hkv << shift;
  const int ch = words > 32 ? 2 : 1;
  const dim3 grid((unsigned)((a.t + kRowWarps - 1) / kRowWarps), (unsigned)((words + 32 * ch - 1) / (32 * ch)));
  auto kern = READ ? (ch == 2 ? kv4_read_kernel<T, 2> : kv4_read_kernel<T, 1>)
                   : (ch == 2 ? kv4_append_kernel<T, 2> : kv4_append_kernel<T, 1>);
  kern<<<grid, kRowWarps * 32, 0, a.stream>>>(a, shift);
  return cudaGetLastError();
}

template <bool READ>
cudaError_t launch_rows(const Kv4RowArgs& a) {
  switch (a.dtype) {
    case DT_BF16: return launch_rows_t<READ, __nv_bfloat16>(a);
    case DT_FP16: return launch_rows_t<READ, __half>(a);
    default: return launch_rows_t<READ, float>(a);
  }
}

// ---------------------------------------------------------------------------- eviction
//
// Of a sequence's len slots of one key/value head, `keep` stay: the `recent` newest ones (the last
// slots) and, of the others, those of the largest weight, ties going to the lowest slot.  Kept
// slots keep their order, so the last slots stay the newest.
//
// kv4_select_kernel (one block per head): weights as 32-bit keys that order like the numbers
// (NaN above everything, -0 as 0); the k-th largest key is found digit by digit (11, 11 and 10 bits:
// three histogram passes over the keys, which stay in L2 or L1); then each warp walks its share of the slots
// twice, counting and writing those above the threshold key, the first ones equal to it, and the newest.
// kv4_gather_kernel: one block per 64 kept slots of a head, a block of the new cache, 16 bytes a thread.

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

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32, kSelBins = 2048;

// Adds this warp's digits to the histogram; lanes that agree throughout (equal weights) add once.
__device__ __forceinline__ void count_digit(unsigned* hist, bool there, uint32_t digit) {
  const unsigned all = __ballot_sync(0xffffffffu, there);
  if (!all) return;
  int same;
  __match_all_sync(0xffffffffu, there ? digit : 0xFFFFFFFFu, &same);
  if (same) {
    if ((threadIdx.x & 31) == 0) atomicAdd(&hist[digit], 32u);
  } else if (there) {
    atomicAdd(&hist[digit], 1u);
  }
}

__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const Kv4EvictArgs a) {
  const int bh = blockIdx.x, b = bh / a.hkv;
  const int n = evict_len(a, b);
  int32_t* kept = a.kept + (int64_t)bh * a.keep;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = min(n, a.keep) + tid; i < a.keep; i += kSelThreads) kept[i] = -1;
  if (n <= a.keep) {
    for (int i = tid; i < n; i += kSelThreads) kept[i] = i;
    return;
  }
  const float* __restrict__ w = a.weights + (int64_t)bh * a.capacity;
  const int m = n - a.recent;       // candidates: slots [0, m)
  const int k = a.keep - a.recent;  // of which k stay, 0 <= k < m
  __shared__ unsigned hist[kSelBins];
  __shared__ unsigned warp_sum[kSelWarps], warp_eq[kSelWarps];
  __shared__ unsigned sel_digit, sel_left;
  uint32_t prefix = 0, mask = 0;
  unsigned left = (unsigned)k;  // still to take among the keys that match prefix
  if (k > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t digits = pass == 2 ? 1023u : 2047u;
      for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      constexpr int U = 8;  // loads in flight
      for (int base = warp * 32; base < m; base += kSelThreads * U) {
        uint32_t key[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = base + u * kSelThreads + lane;
          key[u] = i < m ? weight_key(w[i]) : 0u;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = base + u * kSelThreads + lane;
          count_digit(hist, i < m && (key[u] & mask) == prefix, (key[u] >> shift) & digits);
        }
      }
      __syncthreads();
      // the digit at which the counts from the top reach `left`: thread t holds bins 2047 - 2t and 2046 - 2t
      const int top = kSelBins - 1 - 2 * tid;
      const unsigned c0 = hist[top], c1 = hist[top - 1];
      unsigned incl = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      unsigned before = incl - c0 - c1;
      for (int j = 0; j < warp; ++j) before += warp_sum[j];
      if (before < left && before + c0 + c1 >= left) {
        const bool first = before + c0 >= left;
        sel_digit = (unsigned)(first ? top : top - 1);
        sel_left = left - before - (first ? 0u : c0);
      }
      __syncthreads();
      prefix |= sel_digit << shift;
      mask |= digits << shift;
      left = sel_left;
    }
  }
  // slots of key > prefix stay, the first `left` of those equal to it, and the newest; warp j walks the
  // slots [j * share, (j + 1) * share)
  const int share = ((n + kSelThreads - 1) / kSelThreads) * 32;
  const int from = min(n, warp * share), to = min(n, from + share);
  auto kind = [&](int i, bool* above, bool* equal) {
    *above = *equal = false;
    if (i >= to) return;
    if (i >= m) {
      *above = true;
    } else if (k > 0) {
      const uint32_t key = weight_key(w[i]);
      *above = key > prefix;
      *equal = key == prefix;
    }
  };
  unsigned na = 0, ne = 0;
#pragma unroll 4
  for (int i = from + lane; i - lane < to; i += 32) {
    bool above, equal;
    kind(i, &above, &equal);
    na += above;
    ne += equal;
  }
  na = __reduce_add_sync(0xffffffffu, na);
  ne = __reduce_add_sync(0xffffffffu, ne);
  if (lane == 0) {
    warp_sum[warp] = na;
    warp_eq[warp] = ne;
  }
  __syncthreads();
  unsigned above_before = 0, eq_before = 0;
  for (int j = 0; j < warp; ++j) {
    above_before += warp_sum[j];
    eq_before += warp_eq[j];
  }
  const unsigned under = (1u << lane) - 1u;
#pragma unroll 4
  for (int i = from + lane; i - lane < to; i += 32) {
    bool above, equal;
    kind(i, &above, &equal);
    const unsigned ba = __ballot_sync(0xffffffffu, above), be = __ballot_sync(0xffffffffu, equal);
    const unsigned my_eq = eq_before + __popc(be & under);  // equal ones in front of this slot
    const unsigned pos = above_before + __popc(ba & under) + min(my_eq, left);
    if ((above || (equal && my_eq < left)) && pos < (unsigned)a.keep) kept[pos] = i;
    above_before += __popc(ba);
    eq_before += __popc(be);
  }
}

__global__ void __launch_bounds__(256) kv4_gather_kernel(const Kv4EvictArgs a, int blocks_per_head) {
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.b; b += blockDim.x) a.out_lens[b] = min(min(max(a.lens[b], 0), a.capacity), a.keep);
  const int bh = blockIdx.x / blocks_per_head, blk = blockIdx.x - bh * blocks_per_head;
  const int to0 = blk * kKv4Block;
  __shared__ int from[kKv4Block];
  if (threadIdx.x < kKv4Block)
    from[threadIdx.x] = to0 + (int)threadIdx.x < a.keep ? a.kept[(int64_t)bh * a.keep + to0 + threadIdx.x] : -1;
  __syncthreads();
  const int d = a.d, pw = kv4_param_words(d);
  const int shift = d == 64 ? 1 : (d == 128 ? 2 : 3);  // log2 of the 16-byte pieces of a row's codes
  const uint8_t* src = a.cache + (int64_t)bh * (a.capacity / kKv4Block) * kv4_block_bytes(d);
  uint8_t* dst = a.out_cache + ((int64_t)bh * (a.out_capacity / kKv4Block) + blk) * kv4_block_bytes(d);
  // codes of K, then of V: in the order of the new block
#pragma unroll 2
  for (int i = threadIdx.x; i < 2 * (kKv4Block << shift); i += blockDim.x) {
    const int which = i >> (6 + shift), row = (i >> shift) & (kKv4Block - 1), part = i & ((1 << shift) - 1);
    const int f = from[row];
    if (f < 0) continue;
    const uint8_t* sb = src + (int64_t)(f / kKv4Block) * kv4_block_bytes(d) + kv4_codes_at(d, which) +
                        (f % kKv4Block) * kv4_code_bytes(d);
    *reinterpret_cast<uint4*>(dst + i * 16) = *reinterpret_cast<const uint4*>(sb + part * 16);
  }
  for (int i = threadIdx.x; i < 2 * kKv4Block * pw; i += blockDim.x) {
    const int which = i / (kKv4Block * pw), rest = i - which * (kKv4Block * pw), row = rest / pw;
    const int f = from[row];
    if (f < 0) continue;
    const uint8_t* sb = src + (int64_t)(f / kKv4Block) * kv4_block_bytes(d) + kv4_params_at(d, which) +
                        ((f % kKv4Block) * pw + rest % pw) * 4;
    *reinterpret_cast<uint32_t*>(dst + kv4_params_at(d, 0) + i * 4) = *reinterpret_cast<const uint32_t*>(sb);
  }
  if (threadIdx.x < kKv4Block && from[threadIdx.x] >= 0)
    a.out_weights[(int64_t)bh * a.out_capacity + to0 + threadIdx.x] =
        a.weights[(int64_t)bh * a.capacity + from[threadIdx.x]];
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowArgs& a) { return launch_rows<false>(a); }
cudaError_t launch_kv4_read(const Kv4RowArgs& a) { return launch_rows<true>(a); }

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a) {
  kv4_select_kernel<<<a.b * a.hkv, kSelThreads, 0, a.stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int per_head = (a.keep + kKv4Block - 1) / kKv4Block;
  kv4_gather_kernel<<<(unsigned)per_head * a.b * a.hkv, 256, 0, a.stream>>>(a, per_head);
  return cudaGetLastError();
}

}  // namespace fa
