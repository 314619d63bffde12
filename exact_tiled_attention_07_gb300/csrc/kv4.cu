// The 4-bit key/value cache (layout: kv4.cuh): rows written (append), read back (read) and the
// cache thinned out by accumulated attention weight (evict).
//
// Quantisation of a group x of 64 channels of a row, every step an fp32 operation rounded to
// nearest unless said otherwise:
//   lo = min x, hi = max x
//   step   = fp16((hi - lo) / 15), rounded up, so that 15 steps cover [lo, hi]
//   middle = fp16(lo + 8 step), rounded to nearest
//   code   = clamp(rint((x - middle) / step), -8, 7) + 8     (8 when step is 0)
// so |middle + step (code - 8) - x| <= max(step / 2, 2^-11 |middle| + 2^-25) up to fp32 rounding
// (2^-25: half of fp16's smallest number, which middles below 2^-14 are rounded by).  The
// quotient and the two sums are IEEE operations: the codes are the same wherever they are taken.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "kernels.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr uint32_t kSiteAppend = 920, kSiteRead = 921, kSiteEvict = 922;

template <typename T>
struct Elem;  // eight consecutive elements of a row from fp32 (rounded to nearest)
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<true>(x[0], x[1]), pack2<true>(x[2], x[3]), pack2<true>(x[4], x[5]),
                                              pack2<true>(x[6], x[7]));
  }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ void store8(__half* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<false>(x[0], x[1]), pack2<false>(x[2], x[3]),
                                              pack2<false>(x[4], x[5]), pack2<false>(x[6], x[7]));
  }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// Smallest and largest of a group's 64 elements, eight in this lane (raw: as loaded) and the rest in the
// other seven lanes of the group; NaN when one of them is.  16-bit elements stay packed: the minimum and
// the negated maximum share a register through the shuffles.
template <typename T2>
__device__ __forceinline__ float2 packed_range(const uint32_t (&w)[4]) {
  const T2* v = reinterpret_cast<const T2*>(w);
  const T2 mn = __hmin2_nan(__hmin2_nan(v[0], v[1]), __hmin2_nan(v[2], v[3]));
  const T2 mx = __hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3]));
  T2 r;
  r.x = __hmin_nan(mn.x, mn.y);
  r.y = __hneg(__hmax_nan(mx.x, mx.y));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    const uint32_t u = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&r), o);
    r = __hmin2_nan(r, *reinterpret_cast<const T2*>(&u));
  }
  return make_float2((float)r.x, -(float)r.y);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T>
struct Raw;  // eight elements as loaded
template <>
struct Raw<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ float2 range() const { return packed_range<__nv_bfloat162>(w); }
  __device__ __forceinline__ float2 pair(int i) const { return unpack2<true>(w[i]); }
};
template <>
struct Raw<__half> {
  uint32_t w[4];
  __device__ __forceinline__ float2 range() const { return packed_range<__half2>(w); }
  __device__ __forceinline__ float2 pair(int i) const { return unpack2<false>(w[i]); }
};
template <>
struct Raw<float> {
  uint32_t w[8];
  __device__ __forceinline__ float2 pair(int i) const {
    return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  __device__ __forceinline__ float2 range() const {
    float lo = __uint_as_float(w[0]), nhi = -lo;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      lo = min_nan(lo, __uint_as_float(w[i]));
      nhi = min_nan(nhi, -__uint_as_float(w[i]));
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      nhi = min_nan(nhi, __shfl_xor_sync(0xffffffffu, nhi, o));
    }
    return make_float2(lo, -nhi);
  }
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(r.w) / 16; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    r.w[4 * i] = u.x, r.w[4 * i + 1] = u.y, r.w[4 * i + 2] = u.z, r.w[4 * i + 3] = u.w;
  }
  return r;
}

// x / 15 correctly rounded: a quotient from the rounded reciprocal is within an ulp, and its exact
// remainder times that reciprocal corrects it (Markstein's theorem)
__device__ __forceinline__ float fifteenth(float x) {
  constexpr float r = 1.f / 15.f;
  const float q = x * r;
  return fmaf(fmaf(-15.f, q, x), r, q);
}

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
// 16-bit elements, keys and values, before the row's sequence and slot are known; the 8 lanes of a group find its minimum
// and maximum together and a lane's codes are one 32-bit word.  The quotient is taken as a product with an
// approximate 1 / step (2^-23), which is within 2^-19 of the IEEE quotient for |quotient| <= 8.5;
// where one lies within 2^-17 of a half (exact halves are one in 1,200 of bf16 data) or beyond the codes, the
// division is done for it.  Rounding to an integer is an addition of 1.5 2^23 and its subtraction,
// and four codes are put together by multiply-adds.
// Bound: instructions (160 for 32 words; HBM wants 26 us for 34,001 rows of 8 heads of 128 bf16
// channels, 139 MB in and 39 MB out).  Measured there: 52 us (3.4 TB/s); 109 with conversions to int (16 a clock
// on an SM) and a division each, 58 with shifts and masks for the packing.  One chunk a warp instead of two 96
// against 85 us with the read behind it, four 87.
template <typename T, int D, int CH>
__global__ void __launch_bounds__(kRowWarps * 32) kv4_append_kernel(const Kv4RowArgs a) {
  constexpr int kWords = D / 8;  // of a row of one head
  const int r = blockIdx.x * kRowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= a.t) return;
  // (rows of no sequence need not be there: nothing of them is read)
  if (r < a.cu[0] || r >= a.cu[a.b]) return;
  const int words = a.hkv * kWords;
  const int w0 = blockIdx.y * (CH * 32) + lane;
  int no_abort = 0;
  if (!debug_check(r >= a.cu[0] && r < a.cu[a.b], ErrCtx{a.err, &no_abort}, kSiteAppend)) return;
  Raw<T> x[CH][2];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int w = min(w0 + c * 32, words - 1);  // (lanes behind the row go along, so that the shuffles are whole)
    const int h = w / kWords, word = w % kWords;
    x[c][0] = load_raw(static_cast<const T*>(a.k) + r * a.k_ts + h * a.k_hs + word * 8);
    x[c][1] = load_raw(static_cast<const T*>(a.v) + r * a.v_ts + h * a.v_hs + word * 8);
  }
  const int b = warp_sequence(a.cu, a.b, r);
  if (b < 0) return;
  int64_t slot;
  if (!row_slot(a, r, b, &slot, kSiteAppend)) return;
  const int in = (int)(slot % kKv4Block);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const bool there = w0 + c * 32 < words;  // (words is a multiple of 8: a group's lanes go together)
    const int w = min(w0 + c * 32, words - 1);
    const int h = w / kWords, word = w % kWords;
    uint8_t* block = a.cache + (((int64_t)b * a.hkv + h) * (a.capacity / kKv4Block) + slot / kKv4Block) * kv4_block_bytes(D);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float2 range = x[c][which].range();  // (lo, hi), both NaN when an element is
      const bool bad = !(range.x >= -kKv4Limit && range.y <= kKv4Limit);
      const __half step = __float2half_ru(fifteenth(__fsub_rn(range.y, range.x)));
      const float s = __half2float(step);
      const __half middle = __float2half_rn(__fadd_rn(range.x, 8.f * s));
      const float m = __half2float(middle);
      uint32_t codes = 0x88888888u;
      if (!bad && s > 0.f) {
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
        constexpr float kRound = 12582912.f;  // 1.5 2^23
        float2 n[4];
        float worst = 0.f;  // largest distance from the nearest integer
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 q = fmul2(fsub2(x[c][which].pair(j), make_float2(m, m)), make_float2(inv, inv));
          n[j] = fsub2(fadd2(q, make_float2(kRound, kRound)), make_float2(kRound, kRound));
          const float2 e = fsub2(q, n[j]);
          worst = max3(worst, fabsf(e.x), fabsf(e.y));
        }
        // (the quotients lie between those of lo and hi: where these round to -8 and 7 at the most, none is clamped)
        const bool clamped = !((range.x - m) * inv > -8.49f && (range.y - m) * inv < 7.49f);
        if (worst > 0.5f - 0x1p-17f || clamped) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 y = x[c][which].pair(j / 2);
            const float diff = __fsub_rn(j & 1 ? y.y : y.x, m);
            float& r = j & 1 ? n[j / 2].y : n[j / 2].x;
            if (clamped || fabsf(diff * inv - r) > 0.5f - 0x1p-17f) r = fminf(fmaxf(rintf(__fdiv_rn(diff, s)), -8.f), 7.f);
          }
        }
        // four codes to a sum of codes times powers of 16, exact, which the offset brings to the low 16 bits
        const float a0 = fmaf(fmaf(n[1].y, 16.f, n[1].x), 256.f, fmaf(n[0].y, 16.f, n[0].x)) + (kRound + 34952.f);
        const float a1 = fmaf(fmaf(n[3].y, 16.f, n[3].x), 256.f, fmaf(n[2].y, 16.f, n[2].x)) + (kRound + 34952.f);
        codes = __byte_perm(__float_as_uint(a0), __float_as_uint(a1), 0x5410);
      }
      if (!there) continue;
      *reinterpret_cast<uint32_t*>(block + kv4_codes_at(D, which) + in * kv4_code_bytes(D) + word * 4) = codes;
      if ((word & 7) == 0) {
        const uint32_t par = bad ? kKv4NanParam
                                 : (uint32_t)__half_as_ushort(step) | ((uint32_t)__half_as_ushort(middle) << 16);
        *reinterpret_cast<uint32_t*>(block + kv4_params_at(D, which) + (in * kv4_param_words(D) + (word >> 3)) * 4) = par;
      }
    }
    if (a.weights && there && word == 0) a.weights[((int64_t)b * a.hkv + h) * a.capacity + slot] = 0.f;
  }
}

// The inverse, with the same split: middle + step (code - 8) in fp32, rounded once.  Bound: HBM; 32 us for the rows
// above (5.6 TB/s, 0.83 of the measured copy rate).
template <typename T, int D, int CH>
__global__ void __launch_bounds__(kRowWarps * 32) kv4_read_kernel(const Kv4RowArgs a) {
  constexpr int kWords = D / 8;
  const int r = blockIdx.x * kRowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= a.t) return;
  const int words = a.hkv * kWords;
  const int w0 = blockIdx.y * (CH * 32) + lane;
  const int b = warp_sequence(a.cu, a.b, r);
  if (b < 0) return;
  int64_t slot;
  if (!row_slot(a, r, b, &slot, kSiteRead)) return;
  const int in = (int)(slot % kKv4Block);
  uint32_t codes[CH][2], par[CH][2];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int w = w0 + c * 32;
    if (w >= words) continue;
    const int h = w / kWords, word = w % kWords;
    const uint8_t* block =
        a.cache + (((int64_t)b * a.hkv + h) * (a.capacity / kKv4Block) + slot / kKv4Block) * kv4_block_bytes(D);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      codes[c][which] =
          *reinterpret_cast<const uint32_t*>(block + kv4_codes_at(D, which) + in * kv4_code_bytes(D) + word * 4);
      par[c][which] = *reinterpret_cast<const uint32_t*>(block + kv4_params_at(D, which) +
                                                         (in * kv4_param_words(D) + (word >> 3)) * 4);
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int w = w0 + c * 32;
    if (w >= words) continue;
    const int h = w / kWords, word = w % kWords;
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
template <bool READ, typename T, int D>
cudaError_t launch_rows_d(const Kv4RowArgs& a) {
  const int words = a.hkv * (D / 8);
  const int ch = words > 32 ? 2 : 1;
  const dim3 grid((unsigned)((a.t + kRowWarps - 1) / kRowWarps), (unsigned)((words + 32 * ch - 1) / (32 * ch)));
  auto kern = READ ? (ch == 2 ? kv4_read_kernel<T, D, 2> : kv4_read_kernel<T, D, 1>)
                   : (ch == 2 ? kv4_append_kernel<T, D, 2> : kv4_append_kernel<T, D, 1>);
  kern<<<grid, kRowWarps * 32, 0, a.stream>>>(a);
  return cudaGetLastError();
}

template <bool READ, typename T>
cudaError_t launch_rows_t(const Kv4RowArgs& a) {
  return a.d == 64 ? launch_rows_d<READ, T, 64>(a)
                   : (a.d == 128 ? launch_rows_d<READ, T, 128>(a) : launch_rows_d<READ, T, 256>(a));
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
// kv4_select_kernel (one block per head, or a cluster of 2 to 8 with a run of the slots each): weights
// as 32-bit keys that order like the numbers (NaN above everything, -0 as 0); the k-th largest key is found
// digit by digit (10, 11 and 11 bits: three histogram passes over the keys, which stay in L2 or L1;
// the blocks of a cluster add up each other's histograms through distributed shared memory, so all find the
// same digit); then each lane decides over its slots, and each warp writes those above the threshold key, the
// first ones equal to it, and the newest, behind what the warps and blocks before it keep.  Bound by latency:
// 5,000 cycles until the weights are there, 7,000 for the first pass (its digit, sign, exponent and one bit, takes
// few values: 16 copies of that histogram, one per pair of lanes), 5,000 for each of the others, 8,000 for
// deciding and writing.
// Measured for 8 x 8 heads of up to 32,768 slots, 8,192 to stay: 17 us (two blocks a head).  28 with a branch around
// each weight's load, which made the loads wait for one another, sums over warps one by one, and blocks that stay
// until their stores are done; in that form 44 with one block a head and the keys read again in every pass, 47 with
// four blocks, of which only half are resident.
// kv4_gather_kernel: one block per 64 kept slots of a head, a block of the new cache, all of a thread's loads
// before its stores.  Bound: HBM: 151 MB moved for those heads, and more read beside it, as a kept row of codes is 64
// bytes and its parameters 8: 25 us; 28 with plain loads of codes, for which L2 fetches 128 bytes (140 MB read instead
// of 101 for sequences of 8,000 to 32,768).

__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 -> +0
  return isnan(w) ? 0xFFFFFFFFu : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
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
constexpr int kSelKeys = 16;  // keys of a thread in registers
constexpr int kSelCopies = 16, kSelFirstBins = 1024;
constexpr int kSelSmem = (kSelCopies * kSelFirstBins + 2 * kSelBins) * 4;

template <bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const Kv4EvictArgs a) {
  namespace cg = cooperative_groups;
  asm volatile("griddepcontrol.launch_dependents;");
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
  auto sync_all = [&]() {
    if constexpr (CLUSTER) cluster.sync();
    else __syncthreads();
  };
  auto remote = [&](unsigned* p, int j) -> const unsigned* {
    if constexpr (CLUSTER) return cluster.map_shared_rank(p, j);
    else return p;
  };
  const int bh = blockIdx.x / ctas, b = bh / a.hkv;
  const int n = evict_len(a, b);
  int32_t* kept = a.kept + (int64_t)bh * a.keep;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = min(n, a.keep) + rank * kSelThreads + tid; i < a.keep; i += ctas * kSelThreads) kept[i] = -1;
  if (n <= a.keep) {  // (the whole cluster)
    for (int i = rank * kSelThreads + tid; i < n; i += ctas * kSelThreads) kept[i] = i;
    return;
  }
  const float* __restrict__ w = a.weights + (int64_t)bh * a.capacity;
  const int m = n - a.recent;       // candidates: slots [0, m)
  const int k = a.keep - a.recent;  // of which k stay, 0 <= k < m
  // this block's slots [lo, hi), whole warps' worth of them
  const int share = (n + ctas * 32 - 1) / (ctas * 32) * 32;
  const int lo = min(n, rank * share), hi = min(n, lo + share);
  // warp j has slots [lo + j * part, lo + (j + 1) * part), lane by lane: key[u] is slot from + u * 32 + lane of the
  // panel that is loaded.  One panel, as for up to 16384 slots a block, stays in registers throughout.
  const int part = ((share + kSelThreads - 1) / kSelThreads) * 32;
  const int from = min(hi, lo + warp * part), to = min(hi, from + part);
  const int panels = (part + kSelKeys * 32 - 1) / (kSelKeys * 32);
  uint32_t key[kSelKeys];  // 0, which no number has, behind the candidates
  auto load_panel = [&](int p) {
    // (all the loads, then the keys: a branch for each would make them wait for one another)
#pragma unroll
    for (int u = 0; u < kSelKeys; ++u) {
      const int i = from + (p * kSelKeys + u) * 32 + lane;
      key[u] = __float_as_uint(w[max(min(i, min(to, m) - 1), 0)]);
    }
#pragma unroll
    for (int u = 0; u < kSelKeys; ++u)
      key[u] = from + (p * kSelKeys + u) * 32 + lane < min(to, m) ? weight_key(__uint_as_float(key[u])) : 0u;
  };
  if (panels == 1 && k > 0) load_panel(0);
  // two histograms in turn: the other blocks may still read the last pass's while this one's is filled
  extern __shared__ unsigned copies[];  // [kSelFirstBins][kSelCopies], then the two histograms
  unsigned* hist = copies + kSelCopies * kSelFirstBins;
  __shared__ unsigned warp_sum[kSelWarps], warp_eq[kSelWarps], totals[2];
  __shared__ unsigned sel_digit, sel_left;
  uint32_t prefix = 0, mask = 0;
  unsigned left = (unsigned)k;  // still to take among the keys that match prefix
  if (k > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 22 : (pass == 1 ? 11 : 0);
      const uint32_t digits = pass == 0 ? 1023u : 2047u;
      unsigned* mine = hist + (pass & 1) * kSelBins;
      for (int i = tid; i < kSelBins; i += kSelThreads) mine[i] = 0;
      if (pass == 0)
        for (int i = tid; i < kSelCopies * kSelFirstBins; i += kSelThreads) copies[i] = 0;
      __syncthreads();
      for (int p = 0; p < panels; ++p) {
        if (panels > 1) load_panel(p);
#pragma unroll
        for (int u = 0; u < kSelKeys; ++u) {
          if (from + (p * kSelKeys + u) * 32 >= min(to, m)) break;
          if (pass == 0)  // (bin 0 is no number's)
            atomicAdd(&copies[(key[u] >> shift) * kSelCopies + (lane & (kSelCopies - 1))], 1u);
          else if ((key[u] & mask) == prefix)
            atomicAdd(&mine[(key[u] >> shift) & digits], 1u);
        }
      }
      __syncthreads();
      if (pass == 0) {
        unsigned c = 0;
#pragma unroll
        for (int j = 0; j < kSelCopies; ++j) c += copies[tid * kSelCopies + ((j + tid) & (kSelCopies - 1))];
        mine[tid] = c;  // (the bins above kSelFirstBins stay empty)
      }
      sync_all();
      // the digit at which the counts from the top reach `left`: thread t holds bins 2047 - 2t and 2046 - 2t
      const int top = kSelBins - 1 - 2 * tid;
      unsigned c0 = 0, c1 = 0;
      for (int j = 0; j < ctas; ++j) {
        const uint2 v = *reinterpret_cast<const uint2*>(remote(mine, j) + top - 1);
        c1 += v.x;
        c0 += v.y;
      }
      unsigned incl = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      const unsigned before = incl - c0 - c1 + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u);
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
  // slots of key > prefix stay, the first `left` of those equal to it, and the newest: of a panel's slots, bit u
  // for this lane's u-th one
  auto decide = [&](int p, unsigned* above, unsigned* equal) {
    unsigned gt = 0, eq = 0;
#pragma unroll
    for (int u = 0; u < kSelKeys; ++u) {
      gt |= key[u] > prefix ? 1u << u : 0u;
      eq |= key[u] == prefix ? 1u << u : 0u;
    }
    auto below = [&](int end) {  // bits of the slots in front of `end`
      const int c = (end - (from + p * kSelKeys * 32 + lane) + 31) >> 5;
      return (1u << min(max(c, 0), kSelKeys)) - 1u;
    };
    const unsigned old = below(min(to, m)), any = below(to);
    *above = (any & ~old) | (k > 0 ? gt & old : 0u);
    *equal = k > 0 ? eq & old : 0u;
  };
  unsigned na = 0, ne = 0, above = 0, equal = 0;
  for (int p = 0; p < panels; ++p) {
    if (panels > 1 && k > 0) load_panel(p);
    decide(p, &above, &equal);
    na += __popc(above);
    ne += __popc(equal);
  }
  na = __reduce_add_sync(0xffffffffu, na);
  ne = __reduce_add_sync(0xffffffffu, ne);
  __syncthreads();  // (warp_sum is read above)
  if (lane == 0) {
    warp_sum[warp] = na;
    warp_eq[warp] = ne;
  }
  __syncthreads();
  unsigned above_before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u);
  unsigned eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_eq[lane] : 0u);
  if (tid == kSelThreads - 1) totals[0] = above_before + na, totals[1] = eq_before + ne;
  sync_all();
  for (int j = 0; j < rank; ++j) {
    const unsigned* t = remote(totals, j);
    above_before += t[0];
    eq_before += t[1];
  }
  // no block leaves while another may read its shared memory
  if constexpr (CLUSTER) cluster.barrier_arrive();
  const unsigned under = (1u << lane) - 1u;
  for (int p = 0; p < panels; ++p) {
    if (panels > 1) {
      if (k > 0) load_panel(p);
      decide(p, &above, &equal);
    }
    int i = from + p * kSelKeys * 32 + lane;
    if (ne == 0) {  // (none in the warp's share) four at a time
      unsigned at = above_before + min(eq_before, left);
#pragma unroll 1
      for (int u = 0; u < kSelKeys && i - lane < to; u += 4, i += 128, above >>= 4) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const unsigned ba = __ballot_sync(0xffffffffu, above >> v & 1u), pos = at + __popc(ba & under);
          if ((above >> v & 1u) && pos < (unsigned)a.keep) kept[pos] = i + v * 32;
          at += __popc(ba);
        }
      }
      above_before = at - min(eq_before, left);
      continue;
    }
#pragma unroll 1
    for (int u = 0; u < kSelKeys && i - lane < to; ++u, i += 32, above >>= 1, equal >>= 1) {
      const unsigned ba = __ballot_sync(0xffffffffu, above & 1u), be = __ballot_sync(0xffffffffu, equal & 1u);
      const unsigned my_eq = eq_before + __popc(be & under);  // equal ones in front of this slot
      const unsigned pos = above_before + __popc(ba & under) + min(my_eq, left);
      if (((above & 1u) || ((equal & 1u) && my_eq < left)) && pos < (unsigned)a.keep) kept[pos] = i;
      above_before += __popc(ba);
      eq_before += __popc(be);
    }
  }
  if constexpr (CLUSTER) cluster.barrier_wait();
}

// 16 bytes whose neighbours beyond 64 are not wanted: L2 fetches 64 bytes instead of 128
__device__ __forceinline__ uint4 load_alone(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int D>
__global__ void __launch_bounds__(256) kv4_gather_kernel(const Kv4EvictArgs a, int blocks_per_head) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (launched while the selection is still going)
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.b; b += blockDim.x) a.out_lens[b] = min(min(max(a.lens[b], 0), a.capacity), a.keep);
  const int bh = blockIdx.x / blocks_per_head, blk = blockIdx.x - bh * blocks_per_head;
  const int to0 = blk * kKv4Block;
  __shared__ int from[kKv4Block];
  if (threadIdx.x < kKv4Block)
    from[threadIdx.x] = to0 + (int)threadIdx.x < a.keep ? a.kept[(int64_t)bh * a.keep + to0 + threadIdx.x] : -1;
  __syncthreads();
  constexpr int BYTES = kv4_block_bytes(D), PW = kv4_param_words(D);
  constexpr int PER = D / 32;                   // 16-byte pieces of a row's codes
  constexpr int N = 2 * kKv4Block * PER / 256;  // pieces of a thread: K codes, then V codes, in the new block's order
  constexpr int NP = (2 * kKv4Block * PW + 255) / 256;
  const uint8_t* src = a.cache + (int64_t)bh * (a.capacity / kKv4Block) * BYTES;
  uint8_t* dst = a.out_cache + ((int64_t)bh * (a.out_capacity / kKv4Block) + blk) * BYTES;
  auto row_of = [&](int f, int at, int row_bytes) {
    return src + (int64_t)(f / kKv4Block) * BYTES + at + (f % kKv4Block) * row_bytes;
  };
  uint4 codes[N];
  uint32_t par[NP];
  float w = 0.f;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int i = u * 256 + threadIdx.x, which = i / (kKv4Block * PER), row = (i / PER) % kKv4Block;
    if (from[row] >= 0)
      codes[u] = load_alone(row_of(from[row], kv4_codes_at(D, which), kv4_code_bytes(D)) + i % PER * 16);
  }
#pragma unroll
  for (int u = 0; u < NP; ++u) {
    const int i = u * 256 + threadIdx.x, which = i / (kKv4Block * PW), row = (i / PW) % kKv4Block;
    if (i < 2 * kKv4Block * PW && from[row] >= 0)
      par[u] = *reinterpret_cast<const uint32_t*>(row_of(from[row], kv4_params_at(D, which), PW * 4) + i % PW * 4);
  }
  const bool weighted = threadIdx.x < kKv4Block && from[threadIdx.x % kKv4Block] >= 0;
  if (weighted) w = a.weights[(int64_t)bh * a.capacity + from[threadIdx.x]];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int i = u * 256 + threadIdx.x;
    if (from[(i / PER) % kKv4Block] >= 0) *reinterpret_cast<uint4*>(dst + i * 16) = codes[u];
  }
#pragma unroll
  for (int u = 0; u < NP; ++u) {
    const int i = u * 256 + threadIdx.x;
    if (i < 2 * kKv4Block * PW && from[(i / PW) % kKv4Block] >= 0)
      *reinterpret_cast<uint32_t*>(dst + kv4_params_at(D, 0) + i * 4) = par[u];
  }
  if (weighted) a.out_weights[(int64_t)bh * a.out_capacity + to0 + threadIdx.x] = w;
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowArgs& a) { return launch_rows<false>(a); }
cudaError_t launch_kv4_read(const Kv4RowArgs& a) { return launch_rows<true>(a); }

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a) {
  // blocks per head: as many as there are SMs for (a block's registers fill one), while each has some
  // thousand slots
  int ctas = 1;
  while (ctas < 8 && (int64_t)a.b * a.hkv * ctas * 2 <= device_sm_count() && a.capacity / (ctas * 2) >= 2048) ctas *= 2;
  static std::atomic<unsigned long long> allowed[2];
  cudaError_t e = ctas > 1 ? allow_smem(kv4_select_kernel<true>, kSelSmem, &allowed[1])
                           : allow_smem(kv4_select_kernel<false>, kSelSmem, &allowed[0]);
  if (e != cudaSuccess) return e;
  if (ctas == 1) {
    kv4_select_kernel<false><<<a.b * a.hkv, kSelThreads, kSelSmem, a.stream>>>(a);
    e = cudaGetLastError();
  } else {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.b * a.hkv * ctas));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = kSelSmem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kv4_select_kernel<true>, a);
  }
  if (e != cudaSuccess) return e;
  const int per_head = (a.keep + kKv4Block - 1) / kKv4Block;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)per_head * a.b * a.hkv);
  cfg.blockDim = dim3(256);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, a.d == 64 ? kv4_gather_kernel<64> : (a.d == 128 ? kv4_gather_kernel<128> : kv4_gather_kernel<256>),
                            a, per_head);
}

}  // namespace fa
