// Decode attention over the 4-bit key/value cache (layout: kv4.cuh).
//
// For the R = (H / Hkv) Nq query rows that read one key/value head, with x_hat the value that a
// cached code stands for (x_hat = middle + step (code - 8), one step and middle per 64 channels):
//   S_rj = tau log2e sum_g [ step_K(j, g) (q_r . (code_K(j) - 8))_g + middle_K(j, g) sum_g q_r ]
//   O_r  = sum_j 2^(S_rj - m_r) v_hat_j / l_r,   L_r = (m_r + log2 l_r) ln 2,
//   weights_j += sum_r 2^(S_rj - m_r) / l_r      (when asked for)
// The step and middle of a key enter behind the dot product, in fp32, so keys are never rounded.
//
// Bound: HBM (72 d / 64 bytes for d keys and d values, 9 bits per channel pair), then the
// instructions that turn codes into numbers.  So codes go from shared memory straight into the
// registers of mma.sync operands (m16n8k16): tcgen05 would want them as 16-bit tiles in shared
// or tensor memory, four times the bytes written and read again, for query tiles of 8 rows of
// which it would use 8 in 128.
//
//   S^T = K Q^T: K is the A operand (16 tokens x 16 channels), Q^T the B operand (8 query rows).
//     A 32-bit word of codes holds channels 8w .. 8w + 7; (w >> 4n) & 0x000F000F is channels
//     8w + n and 8w + n + 4 in the two halves of a register: an operand register, once the bits
//     of 128 (bf16) or 1024 (fp16) are or-ed in and that plus 8 is subtracted (exact).  Channels
//     may come in any order in a dot product, so Q is laid out in registers to match.
//   O^T = V^T P^T: V^T is the A operand (16 channels x 16 tokens): a register holds one channel of
//     two tokens, so the words of two tokens are interleaved by halves first.  v_hat is computed in
//     fp16 (one fused multiply-add, rounded once, 2^-11); P is rounded to fp16 (2^-11) scaled by
//     2^8, so that probabilities down to 2^-22 of the row's largest keep their full precision.
//     P^T comes out of the S^T accumulators by movmatrix.
//
// Work split: the 64-slot blocks of all (sequence, key/value head, group of 8 NT query rows) form one list;
// each CTA takes an equal run of it, whatever the lengths of the sequences, found on the device
// from lens.  A head that lies inside one CTA's run is finished there; one that is cut leaves a
// partial (unnormalised O, m, l) per CTA in the workspace, at most two per CTA, and
// decode_kv4_merge joins them in the CTAs' order.  Inside a CTA each warp takes every NW-th block
// through a ring of its own, filled by one bulk copy per block.
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "kernels.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPShift = 8.f;  // P is kept as 2^(S - m + 8)
constexpr uint32_t kSiteKv4Full = 930, kSiteKv4Drain = 931, kSiteKv4Empty = 932, kSiteKv4Len = 933;

template <int D, int NT>
struct Kv4Cfg {
  static constexpr int ROWS = 8 * NT;     // query rows of a CTA
  static constexpr int GROUPS = D / 64;   // parameter groups of a row
  static constexpr int BLOCK = kv4_block_bytes(D);
  static constexpr int NW = 8;            // warps
  static constexpr int TEAM = D == 256 ? 2 : 1;  // warps that share a block
  static constexpr int TEAMS = NW / TEAM;
  static constexpr int TOK = 64 / TEAM;   // tokens of a block for one warp
  static constexpr int STAGES = D == 64 ? 4 : 2;
  static constexpr int THREADS = NW * 32;
  static constexpr int OSTRIDE = 64 + 4;  // floats of a row in the exchange buffer
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_O = TEAMS * STAGES * BLOCK;                // [NW][ROWS][OSTRIDE] fp32
  static constexpr int OFF_ML = OFF_O + NW * ROWS * OSTRIDE * 4;      // [NW][ROWS][2] fp32
  static constexpr int OFF_BAR = OFF_ML + NW * ROWS * 2 * 4;
  static constexpr int NBAR = 2 * TEAMS * STAGES;  // full, then empty
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
  static_assert(SMEM <= 232448, "shared memory");
  static_assert(BLOCK % 16 == 0 && OFF_O % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
};

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8x8 matrix of 16-bit elements transposed across the warp
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// code - 8 of nibbles n and n + 4 of w (n = 0..3), as a pair of 16-bit numbers
template <bool BF16>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int n) {
  const uint32_t bits = (w >> (4 * n)) & 0x000F000Fu;
  if constexpr (BF16) {
    const uint32_t u = bits | 0x43004300u;  // 128 + code
    const uint32_t bias = 0x43084308u;      // 136
    const __nv_bfloat162 r =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), *reinterpret_cast<const __nv_bfloat162*>(&bias));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const uint32_t u = bits | 0x64006400u;  // 1024 + code
    const uint32_t bias = 0x64086408u;      // 1032
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&bias));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// the two tokens' channel n + 4 * hi of words a, b as v_hat pairs: x holds the 16-bit halves of
// both words side by side
__device__ __forceinline__ uint32_t value_pair(uint32_t x, int n, uint32_t step2, uint32_t mid2) {
  const uint32_t c = code_pair<false>(x, n);
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&c), *reinterpret_cast<const __half2*>(&step2),
                            *reinterpret_cast<const __half2*>(&mid2));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ int clamp_len(int n, int capacity) { return min(max(n, 0), capacity); }
__device__ __forceinline__ int blocks_of(int n) { return (n + kKv4Block - 1) / kKv4Block; }

// Position in the list of blocks, which runs over sequences, then heads x row groups, then blocks.
struct Cursor {
  int64_t first;  // list position of sequence b's first block
  int b, nb, len;
};
struct Place {
  int b, hr, blk, nb, len;  // hr: key/value head * row groups + row group
  int64_t seg;              // list position of the segment's (b, hr) first block
};

struct WorkList {
  const int32_t* lens;
  int B, HR, capacity;
  __device__ __forceinline__ void enter(Cursor& c, int b) const {
    c.b = b;
    c.len = b < B ? clamp_len(lens[b], capacity) : 0;
    c.nb = blocks_of(c.len);
  }
  // total number of blocks; the whole warp takes part
  __device__ __forceinline__ int64_t total() const {
    int64_t t = 0;
    for (int b = threadIdx.x & 31; b < B; b += 32) t += blocks_of(clamp_len(lens[b], capacity));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t * HR;
  }
  // cursor at the sequence that list position u (inside the list) belongs to; the whole warp
  __device__ __forceinline__ Cursor find(int64_t u) const {
    const int lane = threadIdx.x & 31;
    int64_t first = 0;
    for (int base = 0; base < B; base += 32) {
      const int n = base + lane < B ? blocks_of(clamp_len(lens[base + lane], capacity)) : 0;
      int64_t incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, first + incl * HR > u);
      if (past) {
        const int at = __ffs(past) - 1;
        Cursor c;
        c.first = first + __shfl_sync(0xffffffffu, (incl - n) * HR, at);
        enter(c, base + at);
        return c;
      }
      first += __shfl_sync(0xffffffffu, incl, 31) * HR;
    }
    Cursor c;
    c.first = first;
    enter(c, B);
    return c;
  }
  // place of list position u >= c.first (inside the list), moving the cursor along
  __device__ __forceinline__ Place at(Cursor& c, int64_t u) const {
    while (u >= c.first + (int64_t)c.nb * HR && c.b < B) {
      c.first += (int64_t)c.nb * HR;
      enter(c, c.b + 1);
    }
    Place p;
    p.b = c.b;
    p.nb = c.nb;
    p.len = c.len;
    const int rel = (int)(u - c.first);
    p.hr = rel / max(c.nb, 1);
    p.blk = rel - p.hr * c.nb;
    p.seg = u - p.blk;
    return p;
  }
};

// The list is cut into one run per CTA, none of them empty (CTAs beyond the list's length have none).
__device__ __forceinline__ int runs_of(int64_t total, int ctas) { return total < ctas ? (int)total : ctas; }
__device__ __forceinline__ int64_t run_start(int64_t total, int g, int G) { return total * g / G; }

// Partials of the merge: per CTA two slots (0: a segment that began in an earlier CTA's run, 1: one that began
// in this CTA's run and goes on), [ROWS][D] unnormalised O and [ROWS][2] (m, l).
__host__ __device__ __forceinline__ size_t partial_floats(int rows, int d) { return (size_t)rows * (d + 2); }

template <int D, bool BF16, int NT, bool SCORES>
__global__ void __launch_bounds__(Kv4Cfg<D, NT>::THREADS, 1)
    decode_kv4_kernel(const DecodeKv4Args a, float* __restrict__ part, float* __restrict__ scores, int row_groups) {
  using C = Kv4Cfg<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;  // mma fragment coordinates
  const int team = warp / C::TEAM, half = warp % C::TEAM;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + team * C::STAGES;
  uint64_t* empty = full + C::TEAMS * C::STAGES;  // (teams of several warps) every warp has read the slot
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + C::NBAR * 8);
  const ErrCtx ctx{a.err, abort_flag};
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    for (int s = 0; s < C::NBAR; ++s) mbar_init(bars + s, s < C::TEAMS * C::STAGES ? 1 : C::TEAM);
    fence_barrier_init();
  }
  __syncthreads();

  const WorkList wl{a.lens, a.b, a.hkv * row_groups, a.capacity};
  const int64_t total = wl.total();
  const int G = runs_of(total, gridDim.x);
  if ((int)blockIdx.x >= G) return;
  const int64_t u0 = run_start(total, blockIdx.x, G), u1 = run_start(total, blockIdx.x + 1, G);
  const int R = (a.h / a.hkv) * a.nq;  // query rows of a key/value head
  const float scale_log2 = a.scale * kLog2e;

  // ring of this warp's team: its i-th block is list position u0 + team + i * TEAMS, in slot i % STAGES
  uint8_t* ring = smem + C::OFF_RING + team * C::STAGES * C::BLOCK;
  Cursor ahead = wl.find(u0);
  Cursor here = ahead;
  int64_t next_load = u0 + team;  // list position of the next block to load
  int loads = 0, uses = 0;
  const bool loader = half == 0 && lane == 0;
  bool ok = true;
  auto load_next = [&]() {
    if (next_load < u1 && ok) {
      if (C::TEAM > 1 && loader && loads >= C::STAGES)
        ok = mbar_wait(empty + loads % C::STAGES, (uint32_t)(loads / C::STAGES - 1) & 1, ctx, kSiteKv4Empty);
      if (loader && ok) {
        const Place p = wl.at(ahead, next_load);
        const int hk = p.hr / row_groups;
        const uint8_t* src =
            a.cache + (((int64_t)p.b * a.hkv + hk) * (a.capacity / kKv4Block) + p.blk) * C::BLOCK;
        const int s = loads % C::STAGES;
        mbar_arrive_expect_tx(full + s, C::BLOCK);
        bulk_load(ring + s * C::BLOCK, src, C::BLOCK, full + s);
      }
      loads += ok;
    }
    next_load += C::TEAMS;
  };
  for (int s = 0; s < C::STAGES; ++s) load_next();

  float o_acc[D / 16][NT][4];
  float m_run[NT][2], l_run[NT][2];
  uint32_t qf[D / 16][NT][2];
  float qsum[C::GROUPS][NT][2];
  float* ml = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* obuf = reinterpret_cast<float*>(smem + C::OFF_O);

  for (int64_t seg_u = u0; seg_u < u1;) {
    // the segment (sequence, head, row group) at seg_u, as far as this CTA's run goes
    const Place sp = wl.at(here, seg_u);
    const int64_t seg_end = sp.seg + sp.nb;
    const int64_t mine_end = seg_end < u1 ? seg_end : u1;
    const int hk = sp.hr / row_groups, rg = sp.hr - hk * row_groups;
    const int row0 = rg * C::ROWS;  // first query row of the group among the R
    // Q rows of this group: rows row0 .. row0 + ROWS of the key/value head, zero past R
    const int64_t q_row0 = ((int64_t)sp.b * a.hkv + hk) * R + row0;  // rows of Q, O, L in [B][H][Nq] order
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + g;
      const bool there = row0 + row < R;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (q_row0 + row) * D);
#pragma unroll
      for (int gr = 0; gr < C::GROUPS; ++gr) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // channels gr * 64 + t * 16 + j * 8 .. + 8
          const uint4 u = there ? src[gr * 8 + t * 2 + j] : make_uint4(0u, 0u, 0u, 0u);
          qf[gr * 4 + j * 2][nt][0] = __byte_perm(u.x, u.z, 0x5410);      // channels 0, 4
          qf[gr * 4 + j * 2][nt][1] = __byte_perm(u.x, u.z, 0x7632);      // 1, 5
          qf[gr * 4 + j * 2 + 1][nt][0] = __byte_perm(u.y, u.w, 0x5410);  // 2, 6
          qf[gr * 4 + j * 2 + 1][nt][1] = __byte_perm(u.y, u.w, 0x7632);  // 3, 7
          const float2 f0 = unpack2<BF16>(u.x), f1 = unpack2<BF16>(u.y), f2 = unpack2<BF16>(u.z), f3 = unpack2<BF16>(u.w);
          sum += ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
        }
        // sum over the group's channels (the four t) of row g, then for this lane's rows 2t, 2t + 1
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        qsum[gr][nt][0] = __shfl_sync(0xffffffffu, sum, (2 * t) * 4);
        qsum[gr][nt][1] = __shfl_sync(0xffffffffu, sum, (2 * t + 1) * 4);
      }
    }
    int last[NT][2];  // one past the newest slot that rows 2t, 2t + 1 see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = row0 + nt * 8 + 2 * t + e;
        last[nt][e] = a.causal ? sp.len - a.nq + row % a.nq + 1 : sp.len;
        m_run[nt][e] = -INFINITY;
        l_run[nt][e] = 0.f;
      }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o_acc[i][nt][e] = 0.f;

    // this team's blocks of the segment: list positions u0 + team + uses * TEAMS while < mine_end
    for (int64_t u = u0 + team + (int64_t)uses * C::TEAMS; ok && u < mine_end; u += C::TEAMS) {
      const int blk = (int)(u - sp.seg);
      const int s = uses % C::STAGES;
      ok = __all_sync(0xffffffffu, mbar_wait(full + s, (uint32_t)(uses / C::STAGES) & 1, ctx, kSiteKv4Full));
      if (!ok) break;
      ++uses;
      uint8_t* blkp = ring + s * C::BLOCK;
      const int slot0 = blk * kKv4Block + half * C::TOK;
      // not every slot of this block is inside every row's range
      const bool edge = blk * kKv4Block + kKv4Block > sp.len - (a.causal ? a.nq - 1 : 0);
      if (edge) {
        // V parameters of slots behind the sequence to zero: v_hat = 0 whatever lies there
        for (int i = lane; i < C::TOK * C::GROUPS; i += 32) {
          const int tok = half * C::TOK + i / C::GROUPS;
          if (blk * kKv4Block + tok >= sp.len)
            reinterpret_cast<uint32_t*>(blkp + kv4_params_at(D, 1))[half * C::TOK * C::GROUPS + i] = 0u;
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int step = 0; step < C::TOK / 32; ++step) {
        const int tok0 = half * C::TOK + step * 32;  // first of this step's 32 tokens in the block
        // ---- S^T of 2 x 16 tokens
        float sc[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const int ta = tok0 + mt * 16 + g;  // this lane's tokens: ta and ta + 8
          const uint8_t* ka = blkp + kv4_codes_at(D, 0) + ta * (D / 2) + t * 8;
          const uint32_t* pa = reinterpret_cast<const uint32_t*>(blkp + kv4_params_at(D, 0)) + ta * C::GROUPS;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
#pragma unroll
          for (int gr = 0; gr < C::GROUPS; ++gr) {
            const uint2 wa = *reinterpret_cast<const uint2*>(ka + gr * 32);
            const uint2 wb = *reinterpret_cast<const uint2*>(ka + gr * 32 + 8 * (D / 2));
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t xa = j ? wa.y : wa.x, xb = j ? wb.y : wb.x;
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t af[4] = {code_pair<BF16>(xa, 2 * k), code_pair<BF16>(xb, 2 * k),
                                        code_pair<BF16>(xa, 2 * k + 1), code_pair<BF16>(xb, 2 * k + 1)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16816<BF16>(acc[nt], af, qf[gr * 4 + j * 2 + k][nt][0], qf[gr * 4 + j * 2 + k][nt][1]);
              }
            }
            const float2 p0 = unpack2<false>(pa[gr]), p1 = unpack2<false>(pa[8 * C::GROUPS + gr]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              sc[mt][nt][0] += fmaf(p0.x, acc[nt][0], p0.y * qsum[gr][nt][0]);
              sc[mt][nt][1] += fmaf(p0.x, acc[nt][1], p0.y * qsum[gr][nt][1]);
              sc[mt][nt][2] += fmaf(p1.x, acc[nt][2], p1.y * qsum[gr][nt][0]);
              sc[mt][nt][3] += fmaf(p1.x, acc[nt][3], p1.y * qsum[gr][nt][1]);
            }
          }
        }
        // ---- log2 units, mask, running maximum
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x = sc[mt][nt][e] * scale_log2;
              if (edge) {
                const int slot = blk * kKv4Block + tok0 + mt * 16 + g + (e >> 1) * 8;
                if (slot >= last[nt][e & 1]) x = -INFINITY;
              }
              sc[mt][nt][e] = x;
              mx[e & 1] = fmaxf(mx[e & 1], x);
            }
          if constexpr (SCORES) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int row = nt * 8 + 2 * t + (e & 1);
                const int slot = blk * kKv4Block + tok0 + mt * 16 + g + (e >> 1) * 8;
                if (row0 + row < R) scores[(q_row0 + row) * a.capacity + slot] = sc[mt][nt][e];
              }
          }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
          }
          float off[2];
          bool grow = false;
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mn = fmaxf(m_run[nt][e], mx[e]);
            alpha[e] = mn == -INFINITY ? 1.f : ex2(m_run[nt][e] - mn);
            grow |= mn > m_run[nt][e];
            m_run[nt][e] = mn;
            off[e] = mn == -INFINITY ? 0.f : kPShift - mn;
          }
          if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) l_run[nt][e] *= alpha[e];
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) o_acc[i][nt][e] *= alpha[e & 1];
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[e] = ex2(sc[mt][nt][e] + off[e & 1]);
              l_run[nt][e & 1] += p[e];
            }
            pf[mt][nt][0] = movmatrix(pack2<false>(p[0], p[1]));
            pf[mt][nt][1] = movmatrix(pack2<false>(p[2], p[3]));
          }
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const int ta = tok0 + mt * 16 + 2 * t;  // tokens ta, ta + 1, ta + 8, ta + 9
          constexpr int VW = D / 64;              // code words of a lane's D / 8 channels
          const uint8_t* vb = blkp + kv4_codes_at(D, 1) + ta * (D / 2) + g * (D / 16);
          const uint32_t* pv = reinterpret_cast<const uint32_t*>(blkp + kv4_params_at(D, 1)) + ta * C::GROUPS +
                               (g * C::GROUPS) / 8;
          const uint32_t w0 = pv[0], w1 = pv[C::GROUPS], w2 = pv[8 * C::GROUPS], w3 = pv[9 * C::GROUPS];
          const uint32_t s_lo = __byte_perm(w0, w1, 0x5410), m_lo = __byte_perm(w0, w1, 0x7632);
          const uint32_t s_hi = __byte_perm(w2, w3, 0x5410), m_hi = __byte_perm(w2, w3, 0x7632);
          uint32_t c[4][VW];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint8_t* src = vb + ((q & 1) + (q >> 1) * 8) * (D / 2);
            if constexpr (VW == 1) {
              c[q][0] = *reinterpret_cast<const uint32_t*>(src);
            } else if constexpr (VW == 2) {
              const uint2 v = *reinterpret_cast<const uint2*>(src);
              c[q][0] = v.x;
              c[q][1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(src);
              c[q][0] = v.x;
              c[q][1] = v.y;
              c[q][2] = v.z;
              c[q][3] = v.w;
            }
          }
#pragma unroll
          for (int w = 0; w < VW; ++w)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              const uint32_t sel = hi ? 0x7632u : 0x5410u;
              const uint32_t x_lo = __byte_perm(c[0][w], c[1][w], sel), x_hi = __byte_perm(c[2][w], c[3][w], sel);
#pragma unroll
              for (int n = 0; n < 4; n += 2) {
                // operand rows g, g + 8: this lane's channels 8 w + 4 hi + n and + 1
                const uint32_t af[4] = {value_pair(x_lo, n, s_lo, m_lo), value_pair(x_lo, n + 1, s_lo, m_lo),
                                        value_pair(x_hi, n, s_hi, m_hi), value_pair(x_hi, n + 1, s_hi, m_hi)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16816<false>(o_acc[w * 4 + hi * 2 + n / 2][nt], af, pf[mt][nt][0], pf[mt][nt][1]);
              }
            }
        }
      }
      // the block is read: its slot takes the team's next one
      if (edge) fence_proxy_async_smem();  // the zeroed parameters come before the next copy into the slot
      __syncwarp();
      if (C::TEAM > 1 && lane == 0) mbar_arrive(empty + s);
      load_next();
    }

    // ---- join the warps: rows' maxima and sums, then O 64 channels at a time
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = l_run[nt][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (g == 0) {
          ml[(warp * C::ROWS + nt * 8 + 2 * t + e) * 2] = m_run[nt][e];
          ml[(warp * C::ROWS + nt * 8 + 2 * t + e) * 2 + 1] = l;
        }
      }
    __syncthreads();
    float f[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float M = -INFINITY;
        for (int w = 0; w < C::NW; ++w) M = fmaxf(M, ml[(w * C::ROWS + nt * 8 + 2 * t + e) * 2]);
        f[nt][e] = m_run[nt][e] == -INFINITY ? 1.f : ex2(m_run[nt][e] - M);
      }
    const bool whole = sp.seg >= u0 && seg_end <= u1;
    float* slot = part + ((size_t)blockIdx.x * 2 + (sp.seg >= u0 ? 1 : 0)) * partial_floats(C::ROWS, D);
#pragma unroll 1
    for (int cc = 0; cc < D / 64; ++cc) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        if (i / 4 != cc) continue;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2*>(obuf + (warp * C::ROWS + nt * 8 + 2 * t + e) * C::OSTRIDE + g * 8 + (i % 4) * 2) =
                make_float2(o_acc[i][nt][e] * f[nt][e], o_acc[i][nt][2 + e] * f[nt][e]);
      }
      __syncthreads();
      // columns: lane group g of the mma holds channels g * D / 8 + cc * 8 .. + 8
      for (int i = threadIdx.x; i < C::ROWS * 32; i += C::THREADS) {
        const int row = i / 32, c2 = i % 32;  // channel pair
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::NW; ++w)
          v = fadd2(v, *reinterpret_cast<const float2*>(obuf + (w * C::ROWS + row) * C::OSTRIDE + c2 * 2));
        const int ch = (c2 / 4) * (D / 8) + cc * 8 + (c2 % 4) * 2;
        if (row0 + row < R) {
          float M = -INFINITY, l = 0.f;
          for (int w = 0; w < C::NW; ++w) M = fmaxf(M, ml[(w * C::ROWS + row) * 2]);
          for (int w = 0; w < C::NW; ++w) {
            const float mw = ml[(w * C::ROWS + row) * 2];
            // (a row whose scores were all NaN has no maximum, but its sum is NaN)
            l += ml[(w * C::ROWS + row) * 2 + 1] * (mw == -INFINITY ? 1.f : ex2(mw - M));
          }
          if (whole) {
            const float inv = l > 0.f ? 1.f / l : 0.f;
            reinterpret_cast<uint32_t*>(a.o)[((q_row0 + row) * D + ch) / 2] = pack2<BF16>(v.x * inv, v.y * inv);
            if (cc == 0 && c2 == 0)
              a.lse[q_row0 + row] = l > 0.f ? (M - kPShift + log2f(l)) * kLn2 : (isnan(l) ? l : -INFINITY);
          } else {
            *reinterpret_cast<float2*>(slot + row * D + ch) = v;
            if (cc == 0 && c2 == 0)
              *reinterpret_cast<float2*>(slot + C::ROWS * D + row * 2) = make_float2(M, l);
          }
        }
      }
      __syncthreads();
    }
    if (*abort_flag) break;
    seg_u = mine_end;
  }
  // every copy must land before the CTA may exit
  if (loader) {
    int no_abort = 0;
    ErrCtx nctx = ctx;
    nctx.abort = &no_abort;
    for (int i = max(0, loads - C::STAGES); i < loads; ++i)
      mbar_wait(full + i % C::STAGES, (uint32_t)(i / C::STAGES) & 1, nctx, kSiteKv4Drain);
  }
}

// Joins the partials of the segments that the runs of several CTAs cut, in the order of the CTAs, and
// writes the rows of empty sequences.  One block per (sequence, key/value head, row group).
template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(128) decode_kv4_merge(const DecodeKv4Args a, const float* __restrict__ part,
                                                       int row_groups, int ctas) {
  constexpr int ROWS = 8 * NT;
  const int hr_count = a.hkv * row_groups;
  const int b = blockIdx.x / hr_count, hr = blockIdx.x - b * hr_count;
  const int hk = hr / row_groups, rg = hr - hk * row_groups;
  const int R = (a.h / a.hkv) * a.nq;
  const int rows = min(ROWS, R - rg * ROWS);
  const int64_t row0 = ((int64_t)b * a.hkv + hk) * R + rg * ROWS;
  if (hr == 0 && threadIdx.x == 0 && clamp_len(a.lens[b], a.capacity) != a.lens[b])
    report_error(a.err, DERR_BAD_ARG, kSiteKv4Len);
  const int nb = blocks_of(clamp_len(a.lens[b], a.capacity));
  if (nb == 0) {
    for (int i = threadIdx.x; i < rows * D / 2; i += blockDim.x) reinterpret_cast<uint32_t*>(a.o)[row0 * D / 2 + i] = 0u;
    for (int i = threadIdx.x; i < rows; i += blockDim.x) a.lse[row0 + i] = -INFINITY;
    return;
  }
  const WorkList wl{a.lens, a.b, hr_count, a.capacity};
  const int64_t total = wl.total();
  const int G = runs_of(total, ctas);
  int64_t before = 0;
  for (int i = threadIdx.x & 31; i < b; i += 32) before += blocks_of(clamp_len(a.lens[i], a.capacity));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  const int64_t s0 = before * hr_count + (int64_t)hr * nb, s1 = s0 + nb;
  // CTA whose run holds list position u: the largest g with total * g / G <= u
  const int g0 = (int)(((s0 + 1) * G - 1) / total), g1 = (int)((s1 * G - 1) / total);
  if (g0 == g1) return;  // finished by that CTA
  const size_t stride = 2 * partial_floats(ROWS, D);
  const float* first = part + g0 * stride + partial_floats(ROWS, D);
  const float* rest = part + (size_t)(g0 + 1) * stride;
  const int n = g1 - g0;
  for (int i = threadIdx.x; i < rows * (D / 4); i += blockDim.x) {
    const int row = i / (D / 4), c = i - row * (D / 4);
    auto mlp = [&](int j) {
      return *reinterpret_cast<const float2*>((j ? rest + (j - 1) * stride : first) + ROWS * D + row * 2);
    };
    float M = -INFINITY;
    for (int j = 0; j <= n; ++j) M = fmaxf(M, mlp(j).x);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j <= n; ++j) {
      const float2 v = mlp(j);
      const float f = v.x == -INFINITY ? 1.f : ex2(v.x - M);  // (no maximum: nothing seen, or only NaN)
      l += v.y * f;
      const float4 x = *reinterpret_cast<const float4*>((j ? rest + (j - 1) * stride : first) + row * D + c * 4);
      o.x += x.x * f, o.y += x.y * f, o.z += x.z * f, o.w += x.w * f;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    reinterpret_cast<uint2*>(a.o)[((row0 + row) * D + c * 4) / 4] =
        make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
    if (c == 0) a.lse[row0 + row] = l > 0.f ? (M - kPShift + log2f(l)) * kLn2 : (isnan(l) ? l : -INFINITY);
  }
}

// weights_out = weights_in + sum over the head's rows of 2^(S - L log2e), for the sequence's slots
__global__ void __launch_bounds__(256) decode_kv4_weights(const DecodeKv4Args a, const float* __restrict__ scores) {
  const int tiles = (a.capacity + 255) / 256;
  const int bh = blockIdx.x / tiles, b = bh / a.hkv;
  const int slot = (blockIdx.x - bh * tiles) * 256 + threadIdx.x;
  if (slot >= clamp_len(a.lens[b], a.capacity)) return;
  const int R = (a.h / a.hkv) * a.nq;
  const float* s = scores + (int64_t)bh * R * a.capacity + slot;
  float w = 0.f;
  for (int r = 0; r < R; ++r) {
    const float L = a.lse[(int64_t)bh * R + r];
    if (L != -INFINITY) w += ex2(s[(int64_t)r * a.capacity] - L * kLog2e);
  }
  const int64_t i = (int64_t)bh * a.capacity + slot;
  a.w_out[i] = (a.w_in ? a.w_in[i] : 0.f) + w;
}

int row_tiles(int h, int hkv, int nq) { return ((h / hkv) * nq > 8) ? 2 : 1; }

// CTAs of the decode kernel: one per SM, no more than there can be blocks
int grid_size(int b, int hkv, int row_groups, int capacity) {
  const int64_t most = (int64_t)b * hkv * row_groups * (capacity / kKv4Block);
  return (int)std::min<int64_t>(most, device_sm_count());
}

template <int D, bool BF16, int NT>
cudaError_t launch_nt(const DecodeKv4Args& a) {
  using C = Kv4Cfg<D, NT>;
  const int R = (a.h / a.hkv) * a.nq;
  const int row_groups = (R + C::ROWS - 1) / C::ROWS;
  const int G = grid_size(a.b, a.hkv, row_groups, a.capacity);
  float* part = static_cast<float*>(a.ws);
  float* scores = part + (size_t)G * 2 * partial_floats(C::ROWS, D);
  auto kern = a.w_out ? decode_kv4_kernel<D, BF16, NT, true> : decode_kv4_kernel<D, BF16, NT, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<G, C::THREADS, C::SMEM, a.stream>>>(a, part, scores, row_groups);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  decode_kv4_merge<D, BF16, NT><<<a.b * a.hkv * row_groups, 128, 0, a.stream>>>(a, part, row_groups, G);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.w_out) {
    decode_kv4_weights<<<(unsigned)((a.capacity + 255) / 256) * a.b * a.hkv, 256, 0, a.stream>>>(a, scores);
    e = cudaGetLastError();
  }
  return e;
}

template <int D>
cudaError_t launch_d(const DecodeKv4Args& a) {
  const bool bf = a.dtype == DT_BF16;
  if (row_tiles(a.h, a.hkv, a.nq) == 1) return bf ? launch_nt<D, true, 1>(a) : launch_nt<D, false, 1>(a);
  return bf ? launch_nt<D, true, 2>(a) : launch_nt<D, false, 2>(a);
}

}  // namespace

size_t decode_kv4_workspace_bytes(int b, int h, int hkv, int nq, int capacity, int d, bool weights) {
  const int rows = 8 * row_tiles(h, hkv, nq);
  const int R = (h / hkv) * nq;
  const int row_groups = (R + rows - 1) / rows;
  size_t n = (size_t)grid_size(b, hkv, row_groups, capacity) * 2 * partial_floats(rows, d);
  if (weights) n += (size_t)b * hkv * R * capacity;
  return n * sizeof(float);
}

cudaError_t launch_decode_kv4(const DecodeKv4Args& a) {
  switch (a.d) {
    case 64: return launch_d<64>(a);
    case 128: return launch_d<128>(a);
    case 256: return launch_d<256>(a);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace fa
