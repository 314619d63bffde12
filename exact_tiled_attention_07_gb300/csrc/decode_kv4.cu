// Decode attention over the 4-bit key/value cache (layout: kv4.cuh).
//
// For the R = (H / Hkv) Nq query rows that read one key/value head, with x_hat the value that a
// cached code stands for (x_hat = middle + step (code - 8), one step and middle per 64 channels):
//   S_rj = tau log2e sum_g [ step_K(j, g) (q_r . code_K(j))_g + (middle_K - 8 step_K)(j, g) sum_g q_r ]
//   O_r  = sum_g [ sum_j P_rj step_V(j, g) code_V(j) + sum_j P_rj (middle_V - 8 step_V)(j, g) ] / l_r
//   P_rj = 2^(S_rj - m_r), l_r = sum_j P_rj, L_r = (m_r + log2 l_r) ln 2
//   weights_j += sum_r P_rj / l_r      (when asked for)
// Steps and middles never touch the codes: those of a key enter behind the dot product, those of a
// value in front of it, in fp32, so keys and values are not rounded.
//
// Bound: HBM (9/16 byte a channel of a key or value), then the instructions that turn codes into
// numbers (282 for 16 tokens of 128 channels in all, 130 of them on the integer pipe, which has half the rate of
// the others).  So codes go from shared memory straight into the registers of mma.sync (m16n8k16,
// fp16, fp32 sums) operands.  Masked out of its word, a nibble is an fp16 subnormal, c 2^-24 where it stands
// lowest and c 2^-20 next to that: 4 masks and a shift for 8 codes, nothing to convert; what the codes are
// multiplied with and the sums carry the powers of two, and the offset of 8 is taken off in fp32.
// Measured, 32 x 8 heads of 32,768 slots, d = 128, four rows a head (1.21 GB): 206 us, 5.9 TB/s, 0.86 of the
// measured copy rate; with the arithmetic left out 194.  Other forms of it (beside 211):
//   * codes to fp16 numbers by or-ing them into 1024 and taking that and 8 off (9 instructions for 8 codes): 236 us,
//     313 with the or's constant as an immediate (each mask-and-or two instructions);
//   * one CTA of 8, 12 or 16 warps an SM instead of four of 4, in that form: 248 to 256 us;
//   * keys as E4M3 bytes 0000cccc, which hold c 2^-9 exactly, by mma.sync: 351 us (it runs as conversions
//     and fp16 products, 523 instructions);
//   * the same bytes by tcgen05, codes unpacked into shared memory, probabilities in three E4M3 pieces: right to
//     the same tolerances, 398 us; a tile's unpacking, product, softmax and product wait for one another,
//     and the bytes written and read again (110 KB for 128 tokens) come near what shared memory moves in that time.
//
//   S^T = K Q^T: K is the A operand (16 tokens x 16 channels).  Channels may come in any order in a
//     dot product, so Q is laid out to match; it is scaled by a power of two that puts the row's
//     largest element in [2^14, 2^15), so a bf16 q is exact in fp16 down to 2^-31 of that (of an odd channel,
//     which is multiplied by 2^-4 as odd codes count 16 times, down to 2^-27).
//   O^T = V^T P^T: V^T is the A operand (16 channels x 16 tokens): a register holds one channel of two
//     tokens, so the words of two tokens are interleaved by halves first.  P step_V is rounded to
//     fp16 (2^-11), and what the offset of 8 takes off is counted with the rounded one, so the error is that of
//     code - 8; for fp16 queries the rounding error is a second operand, so that little more than
//     O's own rounding is left.  P^T comes out of the S^T accumulators by movmatrix.
//     The codes' offset of 8 (with the middles, in fp32: corr) comes off the sums every kFold tokens of a warp, not only
//     at the end: sums of codes 0 to 15 grow to hundreds of times what is left of them, and mma.sync truncates its
//     fp32 sums at every step.  Relative to O's rms over 65,536 slots at 400 blocks a CTA (d = 64, fp16 queries) the
//     error is 2.2e-4, of which 2e-4 are O's own rounding; 4.8e-3 with the offset taken off at the end.
//     1.4 % of the time of the 1.21 GB case, every 256 tokens the same within 2 us.
//     Range: P = 2^(S - m + 8) with a reference m of each row that keeps the products P step_V, which are rounded,
//     inside fp16's range, and not P alone: m is raised where a product might pass 2^15.5 and does pass 2^9, so that the
//     step's largest comes to 2^8.  Whether one might is seen from the largest score and the block's largest step.  So
//     each product keeps fp16's precision down to 2^-22 of the row's largest product (what is smaller, and the rounding
//     error of fp16 queries, an absolute 2^-33 of it), whatever steps other rows' slots or slots of no weight
//     have.  With m the largest score and the steps' largest exponent: 1 to 2.5 % off where a slot of step 4,096 and
//     no weight stands among every 32 of step 0.002; a scale of each row's 64 channels on top of m: 5 to 8 % more time at
//     d = 128 and 256.  A block whose largest step does not allow for P is looked over
//     step by step: where every 32nd slot is of that kind, 244 us instead of 212 for the 1.21 GB case.
//
// Work split: the 64-slot blocks of all (sequence, key/value head, group of 8 NT query rows) form one list;
// each CTA takes an equal run of it, whatever the lengths of the sequences, found on the device
// from lens.  A head that lies inside one CTA's run is finished there; one that is cut leaves a
// partial (unnormalised O, m, l) per CTA in the workspace, at most two per CTA, and
// decode_kv4_finish joins them in the CTAs' order.  Inside a CTA each team of warps takes every TEAMS-th
// block through a ring of its own, filled by one bulk copy per block.  (Equal pieces of every sequence instead,
// sized by the longest: 76 us against 42 for a batch of lengths 1 to 32,768.)
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
constexpr float kMostProduct = 15.5f;  // log2 of P step, at most (fp16 ends below 2^16)
constexpr float kMostP = 28.f;         // log2 of P where no step bounds it (fp16's smallest is 2^-24)
constexpr int kFold = 128;      // tokens of a warp after which the codes' offset comes off its sums
constexpr float kNoScore = 1e30f;  // off before the first score: 2^(-inf + 1e30) is still 0
constexpr uint32_t kSiteKv4Full = 930, kSiteKv4Drain = 931, kSiteKv4Empty = 932, kSiteKv4Len = 933;

template <int D, int NT>
struct Kv4Cfg {
  static constexpr int ROWS = 8 * NT;     // query rows of a CTA
  static constexpr int GROUPS = D / 64;   // parameter groups of a row
  static constexpr int BLOCK = kv4_block_bytes(D);
  // CTAs of 4 warps, four an SM where 128 registers a thread hold a row tile's accumulators, else two: one's start
  // and end of a segment run under the others' loops.  128 x 8 heads of 100 slots, d = 128: 21 us; two CTAs of
  // 8 warps 26, one of 16 warps 38; heads of 32,768 slots measure the same with four and two, 4 % more with one.
  static constexpr int CTAS = NT == 1 && D <= 128 ? 4 : 2;
  static constexpr int NW = 4;  // warps
  static constexpr int TEAM = D == 256 || (D == 128 && NT == 1) ? 2 : 1;  // warps that share a block
  static constexpr int TEAMS = NW / TEAM;
  static constexpr int TOK = 64 / TEAM;   // tokens of a block for one warp
  static constexpr int STAGES = 2;
  static constexpr int THREADS = NW * 32;
  // channels that the warps exchange at a time (a whole row where two CTAs have the shared memory for it)
  static constexpr int OCH = NT == 1 && D <= 128 ? D : 64;
  static constexpr int OSTRIDE = OCH + 4;  // floats of a row in the exchange buffer
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_O = TEAMS * STAGES * BLOCK;                // [NW][ROWS][OSTRIDE] fp32
  static constexpr int OFF_ML = OFF_O + (NW * ROWS * OSTRIDE + NW * ROWS + ROWS * 2) * 4;  // [NW][ROWS][2] fp32
  static constexpr int OFF_BAR = OFF_ML + NW * ROWS * 2 * 4;
  static constexpr int NBAR = 2 * TEAMS * STAGES;  // full, then empty
  static constexpr int OFF_LIST = OFF_BAR + NBAR * 8 + 16;  // [TEAMS] ListPlace
  static constexpr int SMEM = OFF_LIST + TEAMS * 40;
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024 && SMEM <= 232448, "shared memory");
  static_assert(BLOCK % 16 == 0 && OFF_O % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the first product of a sum
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
      "%10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// (a.x b.x + c.x, a.y b.y + c.y)
__device__ __forceinline__ float2 ffma2v(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 8x8 matrix of 16-bit elements transposed across the warp
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// The offset (P = 2^(S + off)) that brings a step's largest product, prod + off, to 2^8 where it is above 2^9, and its
// largest P, top + off, to 2^kMostP where it is more than the smallest step's bound lets by
__device__ __forceinline__ float lowered(float off, float prod, float top) {
  const float next = prod + off > 9.f ? 8.f - prod : off;
  return top + next > kMostProduct + 14.f ? kMostP - top : next;
}

// The four nibbles of each half of x as four pairs of fp16: codes times 2^-24 (even) and 2^-20 (odd), as
// the subnormal numbers that their bits are where they stand
__device__ __forceinline__ void code_pairs(uint32_t x, uint32_t (&out)[4]) {
  const uint32_t y = x >> 8;
  out[0] = x & 0x000F000Fu;
  out[1] = x & 0x00F000F0u;
  out[2] = y & 0x000F000Fu;
  out[3] = y & 0x00F000F0u;
}

__device__ __forceinline__ int clamp_len(int n, int capacity) { return min(max(n, 0), capacity); }
__device__ __forceinline__ int blocks_of(int n) { return (n + kKv4Block - 1) / kKv4Block; }

// The list: sequences, then their heads x row groups (segments), then the segment's nb blocks, each a
// position, behind kSegCost positions that stand for what a segment costs whatever its length (its queries, joining
// the warps, its output: about the time of that many blocks).  With 2, 4, 6, 9 and 12 in turn: 8 sequences of 1 to 32,768
// slots, d = 64: 40, 34, 30, 30, 30 us; d = 128: 50, 40, 40, 40, 40; d = 256: 79, 69, 60, 58, 58; 64 of 300 and 64 of 3,000,
// d = 128: 79, 69, 71, 71, 71.
constexpr int kSegCost = 6;

struct Cursor {
  int64_t first;  // list position of sequence b's first segment
  int b, nb, len;
};
struct Place {
  int b, hr, nb, len;  // hr: key/value head * row groups + row group
  int64_t seg;         // list position of the segment
};

struct WorkList {
  const int32_t* lens;
  int B, HR, capacity;
  __device__ __forceinline__ static int positions(int nb) { return nb > 0 ? nb + kSegCost : 0; }
  __device__ __forceinline__ int blocks(int b) const { return blocks_of(clamp_len(lens[b], capacity)); }
  __device__ __forceinline__ void enter(Cursor& c, int b) const {
    c.b = b;
    c.len = b < B ? clamp_len(lens[b], capacity) : 0;
    c.nb = blocks_of(c.len);
  }
  // positions of sequences [0, end); the whole warp takes part
  __device__ __forceinline__ int64_t total(int end) const {
    int64_t t = 0;
    for (int b = threadIdx.x & 31; b < end; b += 32) t += positions(blocks(b));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t * HR;
  }
  // cursor at the sequence that list position u (inside the list) belongs to; the whole warp
  __device__ __forceinline__ Cursor find(int64_t u) const {
    const int lane = threadIdx.x & 31;
    int64_t first = 0;
    for (int base = 0; base < B; base += 32) {
      const int n = base + lane < B ? positions(blocks(base + lane)) : 0;
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
  // segment of list position u >= c.first (inside the list), moving the cursor along
  __device__ __forceinline__ Place at(Cursor& c, int64_t u) const {
    int64_t span = (int64_t)positions(c.nb) * HR;
    while (u >= c.first + span && c.b < B) {
      c.first += span;
      enter(c, c.b + 1);
      span = (int64_t)positions(c.nb) * HR;
    }
    Place p;
    p.b = c.b;
    p.nb = c.nb;
    p.len = c.len;
    const int per = max(positions(c.nb), 1);
    p.hr = (int)(u - c.first) / per;
    p.seg = c.first + (int64_t)p.hr * per;
    return p;
  }
};

// The list is cut into one run per CTA, none of them empty (CTAs beyond the list's length have none).
__device__ __forceinline__ int runs_of(int64_t total, int ctas) { return total < ctas ? (int)total : ctas; }
__device__ __forceinline__ int64_t run_start(int64_t total, int g, int G) { return total * g / G; }
// CTA whose run holds list position u: the largest g with total * g / G <= u
__device__ __forceinline__ int run_of(int64_t total, int64_t u, int G) { return (int)(((u + 1) * G - 1) / total); }
// blocks [first, end) of a segment that lie in the run [u0, u1)
__device__ __forceinline__ void run_blocks(int64_t seg, int nb, int64_t u0, int64_t u1, int* first, int* end) {
  const int64_t at = seg + kSegCost;
  *first = (int)max((int64_t)0, min((int64_t)nb, u0 - at));
  *end = (int)max((int64_t)*first, min((int64_t)nb, u1 - at));
}

// Where a loading thread is in the list: kept in shared memory, as it is needed once a segment and would cost
// registers in the loop over the blocks.
struct ListPlace {
  Cursor c;
  int64_t u;  // list position of the segment to load from next
  int rot;    // blocks of the run before it, modulo the teams
};
static_assert(sizeof(ListPlace) == 40, "size");

// Partials of the merge: per CTA two slots (0: a segment that began in an earlier CTA's run, 1: one that began
// in this CTA's run and goes on), [ROWS][D] unnormalised O and [ROWS][2] (m, l).
__host__ __device__ __forceinline__ size_t partial_floats(int rows, int d) { return (size_t)rows * (d + 2); }

// i modulo N for -N < i < N
template <int N>
__device__ __forceinline__ int turn(int i) {
  return i < 0 ? i + N : i;
}

// Log-sum-exp in log2 units of a row's (reference, sum): -inf where it saw nothing, NaN where it saw one
__device__ __forceinline__ float log_sum(float m, float l) {
  return l > 0.f ? m - kPShift + log2f(l) : (isnan(l) ? l : -INFINITY);
}

template <int D, bool BF16, int NT, bool SCORES>
__global__ void __launch_bounds__(Kv4Cfg<D, NT>::THREADS, Kv4Cfg<D, NT>::CTAS)
    decode_kv4_kernel(const DecodeKv4Args a, float* __restrict__ part, float* __restrict__ scores, int row_groups) {
  using C = Kv4Cfg<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;  // mma fragment coordinates
  const int team = warp / C::TEAM, half = warp % C::TEAM;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + team * C::STAGES;
  uint64_t* empty = full + C::TEAMS * C::STAGES;  // (teams of several warps) every warp has read the slot
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + C::NBAR * 8);
  volatile uint8_t* nan_seen = smem + C::OFF_BAR + C::NBAR * 8 + 4;  // [NW]
  const ErrCtx ctx{a.err, abort_flag};
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int w = 0; w < C::NW; ++w) nan_seen[w] = 0;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    for (int s = 0; s < C::NBAR; ++s) mbar_init(bars + s, s < C::TEAMS * C::STAGES ? 1 : C::TEAM);
    fence_barrier_init();
  }
  __syncthreads();

  asm volatile("griddepcontrol.launch_dependents;");
  const WorkList wl{a.lens, a.b, a.hkv * row_groups, a.capacity};
  const int64_t total = wl.total(a.b);
  const int G = runs_of(total, gridDim.x);
  if ((int)blockIdx.x >= G) return;
  const int64_t u0 = run_start(total, blockIdx.x, G), u1 = run_start(total, blockIdx.x + 1, G);
  const int R = (a.h / a.hkv) * a.nq;  // query rows of a key/value head
  const float scale_log2 = a.scale * kLog2e;

  // Blocks go to the teams in turn: of a segment's blocks [first, end) in this run, team (rot + i) % TEAMS takes
  // first + i, where rot counts the run's blocks before.  A team's i-th block of the run is in slot i % STAGES.
  uint8_t* ring = smem + C::OFF_RING + team * C::STAGES * C::BLOCK;
  Cursor here = wl.find(u0);
  ListPlace* lists = reinterpret_cast<ListPlace*>(smem + C::OFF_LIST);
  int loads = 0, uses = 0;
  const bool loader = half == 0 && lane == 0;
  bool ok = true;
  if (loader) lists[team] = ListPlace{here, u0, 0};
  bool load_ok = true;  // (when a wait of the loader runs out, the teams' waits for their blocks run out too)
  const uint8_t* load_src = nullptr;  // the block loaded last, and how many blocks of its segment's part follow it
  int load_left = 0;
  auto load_next = [&]() {
    if (!loader || !load_ok) return;
    if (load_left >= C::TEAMS) {
      load_src += C::TEAMS * C::BLOCK;
      load_left -= C::TEAMS;
    } else {
      load_left = -1;
      ListPlace& at = lists[team];
      while (load_left < 0 && at.u < u1) {
        const Place p = wl.at(at.c, at.u);
        int first, end;
        run_blocks(p.seg, p.nb, u0, u1, &first, &end);
        at.u = p.seg + WorkList::positions(p.nb);
        const int mine = first + turn<C::TEAMS>(team - at.rot);
        at.rot = (at.rot + end - first) % C::TEAMS;
        if (mine < end) {
          const int hk = p.hr / row_groups;
          load_src = a.cache + (((int64_t)p.b * a.hkv + hk) * (a.capacity / kKv4Block) + mine) * C::BLOCK;
          load_left = end - 1 - mine;
        }
      }
      if (load_left < 0) return;  // nothing left in the run
    }
    const int s = loads % C::STAGES;
    if (C::TEAM > 1 && loads >= C::STAGES)
      load_ok = mbar_wait(empty + s, (uint32_t)(loads / C::STAGES - 1) & 1, ctx, kSiteKv4Empty);
    if (load_ok) {
      mbar_arrive_expect_tx(full + s, C::BLOCK);
      // read once, so first to leave L2: 222 -> 214 us for 1.21 GB
      bulk_load_once(ring + s * C::BLOCK, load_src, C::BLOCK, full + s);
      ++loads;
    }
  };
  for (int s = 0; s < C::STAGES; ++s) load_next();

  float o_acc[D / 16][NT][4];  // tile 4 gr + i: channels 64 gr + 8 g + 2 i (+ 1), rows 2t (+ 1)
  // pairs: rows 2t, 2t + 1.  P = 2^(S + off), off = 8 - m for the m in use
  float2 off[NT], l_run[NT], corr[C::GROUPS][NT];
  uint32_t qf[D / 16][NT][2];
  float2 qsum[C::GROUPS][NT], cf[NT];
  const int kap = (g >> 1) + (g & 1) * 4;  // token of operand row g: rows 2t, 2t + 1 are tokens t, t + 4
  float* ml = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* obuf = reinterpret_cast<float*>(smem + C::OFF_O);

  int rot = 0;
  for (int64_t seg_u = u0; seg_u < u1;) {
    // the segment (sequence, head, row group) at seg_u, as far as this CTA's run goes
    const Place sp = wl.at(here, seg_u);
    seg_u = sp.seg + WorkList::positions(sp.nb);
    int blk0, blk1;
    run_blocks(sp.seg, sp.nb, u0, u1, &blk0, &blk1);
    if (blk0 >= blk1) continue;
    const int hk = sp.hr / row_groups, rg = sp.hr - hk * row_groups;
    const int row0 = rg * C::ROWS;  // first query row of the group among the R
    // Q rows of this group: rows row0 .. row0 + ROWS of the key/value head, zero past R
    const int64_t q_row0 = ((int64_t)sp.b * a.hkv + hk) * R + row0;  // rows of Q, O, L in [B][H][Nq] order
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + g;
      const bool there = row0 + row < R;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (q_row0 + row) * D);
      uint4 raw[D / 32];
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks) {
        // channels (ks / 2) * 64 + t * 16 + (ks % 2) * 8 .. + 8
        raw[ks] = there ? src[(ks / 2) * 8 + t * 2 + (ks % 2)] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {raw[ks].x, raw[ks].y, raw[ks].z, raw[ks].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<BF16>(w[i]);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // scaled by 2^(14 - ex), the row's largest element lies in [2^14, 2^15)
      const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 120);
      const float up = __uint_as_float((uint32_t)(141 - ex) << 23);
      const float factor = __uint_as_float((uint32_t)(113 + ex) << 23) * (scale_log2 * 0x1p24f);  // (codes count 2^-24)
      cf[nt] = make_float2(__shfl_sync(0xffffffffu, factor, (2 * t) * 4),
                           __shfl_sync(0xffffffffu, factor, (2 * t + 1) * 4));
#pragma unroll
      for (int gr = 0; gr < C::GROUPS; ++gr) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int ks = gr * 2 + j;
          float2 f[4] = {unpack2<BF16>(raw[ks].x), unpack2<BF16>(raw[ks].y), unpack2<BF16>(raw[ks].z),
                         unpack2<BF16>(raw[ks].w)};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[i] = fmul2(f[i], make_float2(up, up));
            sum += f[i].x + f[i].y;
          }
          // (odd codes count 16 times as much)
          qf[ks * 2][nt][0] = pack2<false>(f[0].x, f[2].x);                          // channels 0, 4 of the eight
          qf[ks * 2][nt][1] = pack2<false>(f[0].y * 0.0625f, f[2].y * 0.0625f);      // 1, 5
          qf[ks * 2 + 1][nt][0] = pack2<false>(f[1].x, f[3].x);                      // 2, 6
          qf[ks * 2 + 1][nt][1] = pack2<false>(f[1].y * 0.0625f, f[3].y * 0.0625f);  // 3, 7
        }
        // sum over the group's channels (the four t) of row g, then for this lane's rows 2t, 2t + 1
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= 0x1p-24f;
        qsum[gr][nt] = make_float2(__shfl_sync(0xffffffffu, sum, (2 * t) * 4),
                                   __shfl_sync(0xffffffffu, sum, (2 * t + 1) * 4));
      }
    }
    int last[NT][2];  // one past the newest slot that rows 2t, 2t + 1 see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = row0 + nt * 8 + 2 * t + e;
        last[nt][e] = a.causal ? sp.len - a.nq + row % a.nq + 1 : sp.len;
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      off[nt] = make_float2(kNoScore, kNoScore);
      l_run[nt] = make_float2(0.f, 0.f);
#pragma unroll
      for (int gr = 0; gr < C::GROUPS; ++gr) corr[gr][nt] = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o_acc[i][nt][e] = 0.f;

    // corr, which the lanes hold for tokens of their own, into the sums of O (in units of 2^-24 and 2^-20)
    auto fold = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int gr = 0; gr < C::GROUPS; ++gr) {
          float2 c = corr[gr][nt];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            c = fadd2(c, make_float2(__shfl_xor_sync(0xffffffffu, c.x, o), __shfl_xor_sync(0xffffffffu, c.y, o)));
          const float2 even = fmul2(c, make_float2(0x1p-24f, 0x1p-24f)), odd = fmul2(c, make_float2(0x1p-20f, 0x1p-20f));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float(&x)[4] = o_acc[gr * 4 + i][nt];
            const float2 a = fadd2(make_float2(x[0], x[1]), even), b = fadd2(make_float2(x[2], x[3]), odd);
            x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
          }
          corr[gr][nt] = make_float2(0.f, 0.f);
        }
    };

    for (int blk = blk0 + turn<C::TEAMS>(team - rot); ok && blk < blk1; blk += C::TEAMS) {
      const int s = uses % C::STAGES;
      ok = __all_sync(0xffffffffu, mbar_wait(full + s, (uint32_t)(uses / C::STAGES) & 1, ctx, kSiteKv4Full));
      if (!ok) break;
      ++uses;
      uint8_t* blkp = ring + s * C::BLOCK;
      // not every slot of this block is inside every row's range
      const bool edge = blk * kKv4Block + kKv4Block > sp.len - (a.causal ? a.nq - 1 : 0);
      if (edge) {
        // V parameters of slots behind the sequence to zero: v_hat = 0 whatever lies there.  NaN in a slot that
        // some rows do not see (0 x NaN is not 0 to them) too: the other rows get theirs behind the loop.
        for (int i = lane; i < C::TOK * C::GROUPS; i += 32) {
          const int slot = blk * kKv4Block + half * C::TOK + i / C::GROUPS;
          uint32_t* par = reinterpret_cast<uint32_t*>(blkp + kv4_params_at(D, 1)) + half * C::TOK * C::GROUPS + i;
          const bool nan = slot > sp.len - a.nq && (*par & 0x7FFFu) > 0x7C00u;
          if (nan && slot < sp.len && a.causal) nan_seen[warp] = 1;
          if (slot >= sp.len || (nan && a.causal)) *par = 0u;
        }
        __syncwarp();
      }
      const uint32_t* kpar = reinterpret_cast<const uint32_t*>(blkp + kv4_params_at(D, 0));
      const uint32_t* vpar = reinterpret_cast<const uint32_t*>(blkp + kv4_params_at(D, 1));
      // log2 P up to which no product can be too large: from the largest V step of this warp's tokens (fp16 bits of
      // numbers >= 0 order like the numbers; below 2^(exponent + 1))
      float most;
      {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < C::TOK * C::GROUPS / 32; ++i)
          top = max(top, vpar[half * C::TOK * C::GROUPS + i * 32 + lane] & 0x7FFFu);
        most = kMostProduct - 1.f - (float)((int)(__reduce_max_sync(0xffffffffu, top) >> 10) - 15);
      }
#pragma unroll 1
      for (int step = 0; step < C::TOK / 32; ++step) {
        const int tok0 = half * C::TOK + step * 32;  // first of this step's 32 tokens in the block
        // ---- S^T of 2 x 16 tokens
        float2 sc[2][NT][2];  // [token tile][row tile][token of this lane, the one 8 behind], rows 2t, 2t + 1
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const int ta = tok0 + mt * 16 + kap;  // this lane's tokens: ta and ta + 8
          const uint8_t* ka = blkp + kv4_codes_at(D, 0) + ta * (D / 2) + t * 8;
#pragma unroll
          for (int gr = 0; gr < C::GROUPS; ++gr) {
            const uint2 wa = *reinterpret_cast<const uint2*>(ka + gr * 32);
            const uint2 wb = *reinterpret_cast<const uint2*>(ka + gr * 32 + 8 * (D / 2));
            float acc[NT][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t xa[4], xb[4];
              code_pairs(j ? wa.y : wa.x, xa);
              code_pairs(j ? wb.y : wb.x, xb);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t af[4] = {xa[2 * k], xb[2 * k], xa[2 * k + 1], xb[2 * k + 1]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  if (j == 0 && k == 0)
                    mma_f16_first(acc[nt], af, qf[gr * 4][nt][0], qf[gr * 4][nt][1]);
                  else
                    mma_f16(acc[nt], af, qf[gr * 4 + j * 2 + k][nt][0], qf[gr * 4 + j * 2 + k][nt][1]);
                }
              }
            }
            const float2 p0 = unpack2<false>(kpar[ta * C::GROUPS + gr]);
            const float2 p1 = unpack2<false>(kpar[(ta + 8) * C::GROUPS + gr]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float st = e ? p1.x : p0.x, md = fmaf(-8.f, st, e ? p1.y : p0.y);
                const float2 mid = gr == 0 ? fmul2(qsum[0][nt], make_float2(md, md)) : ffma2(qsum[gr][nt], md, sc[mt][nt][e]);
                sc[mt][nt][e] = ffma2(make_float2(acc[nt][2 * e], acc[nt][2 * e + 1]), st, mid);
              }
          }
        }
        // ---- mask, running maximum (log2 units), exponentials
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (edge) {
            asm volatile("");  // a branch, not eight selections for every block
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int slot = blk * kKv4Block + tok0 + mt * 16 + kap + e * 8;
                if (slot >= last[nt][0]) sc[mt][nt][e].x = -INFINITY;
                if (slot >= last[nt][1]) sc[mt][nt][e].y = -INFINITY;
              }
          }
          if constexpr (SCORES) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + 2 * t;
                float* dst = scores + (q_row0 + row) * a.capacity + blk * kKv4Block + tok0 + mt * 16 + kap + e * 8;
                if (row0 + row < R) dst[0] = sc[mt][nt][e].x * cf[nt].x;
                if (row0 + row + 1 < R) dst[a.capacity] = sc[mt][nt][e].y * cf[nt].y;
              }
          }
          float2 mx = make_float2(fmaxf(max3(sc[0][nt][0].x, sc[0][nt][1].x, sc[1][nt][0].x), sc[1][nt][1].x),
                                  fmaxf(max3(sc[0][nt][0].y, sc[0][nt][1].y, sc[1][nt][0].y), sc[1][nt][1].y));
          const float2 z = ffma2v(mx, cf[nt], off[nt]);
          if (__any_sync(0xffffffffu, fmaxf(z.x, z.y) > most)) {
            // largest score and largest product (log2, without the reference) of the step
            float2 prod = make_float2(-INFINITY, -INFINITY);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float st = 0.f;
#pragma unroll
                for (int gr = 0; gr < C::GROUPS; ++gr)  // (a NaN is left out)
                  st = fmaxf(st, unpack2<false>(vpar[(tok0 + mt * 16 + kap + e * 8) * C::GROUPS + gr]).x);
                st = __log2f(st);
                prod.x = fmaxf(prod.x, fmaf(sc[mt][nt][e].x, cf[nt].x, st));
                prod.y = fmaxf(prod.y, fmaf(sc[mt][nt][e].y, cf[nt].y, st));
              }
            mx = fmul2(mx, cf[nt]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              mx.x = fmaxf(mx.x, __shfl_xor_sync(0xffffffffu, mx.x, o));
              mx.y = fmaxf(mx.y, __shfl_xor_sync(0xffffffffu, mx.y, o));
              prod.x = fmaxf(prod.x, __shfl_xor_sync(0xffffffffu, prod.x, o));
              prod.y = fmaxf(prod.y, __shfl_xor_sync(0xffffffffu, prod.y, o));
            }
            const float2 next = make_float2(lowered(off[nt].x, prod.x, mx.x), lowered(off[nt].y, prod.y, mx.y));
            const float2 alpha = make_float2(ex2(next.x - off[nt].x), ex2(next.y - off[nt].y));
            off[nt] = next;
            l_run[nt] = fmul2(l_run[nt], alpha);
#pragma unroll
            for (int gr = 0; gr < C::GROUPS; ++gr) corr[gr][nt] = fmul2(corr[gr][nt], alpha);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o_acc[i][nt][0] *= alpha.x;
              o_acc[i][nt][1] *= alpha.y;
              o_acc[i][nt][2] *= alpha.x;
              o_acc[i][nt][3] *= alpha.y;
            }
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 x = ffma2v(sc[mt][nt][e], cf[nt], off[nt]);
              sc[mt][nt][e] = make_float2(ex2(x.x), ex2(x.y));
              l_run[nt] = fadd2(l_run[nt], sc[mt][nt][e]);
            }
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const int ta = tok0 + mt * 16 + kap;
          const uint8_t* vb = blkp + kv4_codes_at(D, 1) + (tok0 + mt * 16 + t) * (D / 2) + g * 4;
#pragma unroll
          for (int gr = 0; gr < C::GROUPS; ++gr) {
            // tokens t, t + 4, t + 8, t + 12: operand columns 2t, 2t + 1, 2t + 8, 2t + 9
            uint32_t c[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) c[q] = *reinterpret_cast<const uint32_t*>(vb + q * 4 * (D / 2) + gr * 32);
            const float2 p0 = unpack2<false>(vpar[ta * C::GROUPS + gr]);
            const float2 p1 = unpack2<false>(vpar[(ta + 8) * C::GROUPS + gr]);
            uint32_t pf[NT][2], pl[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float st = e ? p1.x : p0.x, md = e ? p1.y : p0.y;
                corr[gr][nt] = ffma2(sc[mt][nt][e], md, corr[gr][nt]);
                const float2 y = fmul2(sc[mt][nt][e], make_float2(st, st));
                const uint32_t h = pack2<false>(y.x, y.y);
                // the codes' offset of 8, times what the codes are multiplied with
                const float2 back = unpack2<false>(h);
                corr[gr][nt] = ffma2(BF16 ? back : y, -8.f, corr[gr][nt]);
                pf[nt][e] = movmatrix(h);
                if constexpr (!BF16) {
                  pl[nt][e] = movmatrix(pack2<false>(y.x - back.x, y.y - back.y));
                }
              }
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              const uint32_t sel = hi ? 0x7632u : 0x5410u;
              uint32_t lo4[4], hi4[4];
              code_pairs(__byte_perm(c[0], c[1], sel), lo4);
              code_pairs(__byte_perm(c[2], c[3], sel), hi4);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                // operand rows g, g + 8: channels 64 gr + 8 g + 4 hi + 2 k and + 1
                const uint32_t af[4] = {lo4[2 * k], lo4[2 * k + 1], hi4[2 * k], hi4[2 * k + 1]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma_f16(o_acc[gr * 4 + hi * 2 + k][nt], af, pf[nt][0], pf[nt][1]);
                  if constexpr (!BF16) mma_f16(o_acc[gr * 4 + hi * 2 + k][nt], af, pl[nt][0], pl[nt][1]);
                }
              }
            }
          }
        }
      }
      // the block is read: its slot takes the team's next one
      if (edge) fence_proxy_async_smem();  // the zeroed parameters come before the next copy into the slot
      __syncwarp();
      if (C::TEAM > 1 && lane == 0) mbar_arrive(empty + s);
      load_next();
      if (uses % (kFold / C::TOK) == 0) fold();
    }

    if (nan_seen[warp]) {  // rows that see one of the newest slots that hold NaN
      const int64_t block0 = ((int64_t)sp.b * a.hkv + hk) * (a.capacity / kKv4Block);
      for (int slot = max(blk0 * kKv4Block, sp.len - a.nq + 1); slot < min(blk1 * kKv4Block, sp.len); ++slot) {
        const uint32_t* par = reinterpret_cast<const uint32_t*>(a.cache + (block0 + slot / kKv4Block) * C::BLOCK +
                                                                kv4_params_at(D, 1)) + slot % kKv4Block * C::GROUPS;
#pragma unroll
        for (int gr = 0; gr < C::GROUPS; ++gr)
          if ((par[gr] & 0x7FFFu) > 0x7C00u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (slot < last[nt][0]) corr[gr][nt].x = __int_as_float(0x7FC00000);
              if (slot < last[nt][1]) corr[gr][nt].y = __int_as_float(0x7FC00000);
            }
      }
      __syncwarp();
      nan_seen[warp] = 0;
    }

    // ---- join the warps: rows' maxima and sums, then O 64 channels at a time
    fold();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = e ? l_run[nt].y : l_run[nt].x;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o_acc[i][nt][e] *= 0x1p24f;
          o_acc[i][nt][e + 2] *= 0x1p20f;
        }
        const float r = e ? off[nt].y : off[nt].x;
        const float ref = r == kNoScore ? -INFINITY : kPShift - r;  // m of this warp's exponentials
        if (g == 0)
          *reinterpret_cast<float2*>(ml + (warp * C::ROWS + nt * 8 + 2 * t + e) * 2) = make_float2(ref, l);
      }
    // (a warp whose team had none of these blocks has m = -inf, l = 0 and is left out of the sums of O)
    const int nblk = blk1 - blk0;
    auto active = [&](int w) { return turn<C::TEAMS>(w / C::TEAM - rot) < nblk; };
    __syncthreads();
    float* fac = obuf + C::NW * C::ROWS * C::OSTRIDE;  // [NW][ROWS] weight of each warp's sums, then [ROWS][2] (m, l)
    float* mlt = fac + C::NW * C::ROWS;
    if (threadIdx.x < C::NW * C::ROWS) {
      const int row = threadIdx.x % C::ROWS, w = threadIdx.x / C::ROWS;
      float M = -INFINITY;
#pragma unroll
      for (int i = 0; i < C::NW; ++i) M = fmaxf(M, ml[(i * C::ROWS + row) * 2]);
      // (a row whose scores were all NaN has no maximum, but its sums are NaN)
      const float m = ml[threadIdx.x / C::ROWS * C::ROWS * 2 + row * 2];
      fac[w * C::ROWS + row] = m == -INFINITY ? 1.f : ex2(m - M);
      if (w == 0) {
        float l = 0.f;
        for (int i = 0; i < C::NW; ++i) {
          const float2 v = *reinterpret_cast<const float2*>(ml + (i * C::ROWS + row) * 2);
          l += v.y * (v.x == -INFINITY ? 1.f : ex2(v.x - M));
        }
        *reinterpret_cast<float2*>(mlt + row * 2) = make_float2(M, l);
      }
    }
    const bool whole = nblk == sp.nb;
    float* slot = part + ((size_t)blockIdx.x * 2 + (blk0 == 0 ? 1 : 0)) * partial_floats(C::ROWS, D);
#pragma unroll 1
    for (int cc = 0; cc < D / C::OCH; ++cc) {
      if (active(warp)) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          if (i / (C::OCH / 16) != cc) continue;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<float2*>(obuf + (warp * C::ROWS + nt * 8 + 2 * t + e) * C::OSTRIDE +
                                         (i / 4 * 64) % C::OCH + g * 8 + (i % 4) * 2) = make_float2(o_acc[i][nt][e], o_acc[i][nt][2 + e]);
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < C::ROWS * (C::OCH / 2); i += C::THREADS) {
        const int row = i / (C::OCH / 2), c2 = i % (C::OCH / 2);  // channel pair
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::NW; ++w)
          if (active(w)) {
            const float f = fac[w * C::ROWS + row];
            const float2 x = *reinterpret_cast<const float2*>(obuf + (w * C::ROWS + row) * C::OSTRIDE + c2 * 2);
            v.x = fmaf(x.x, f, v.x);
            v.y = fmaf(x.y, f, v.y);
          }
        const int ch = cc * C::OCH + c2 * 2;
        if (row0 + row < R) {
          const float2 st = *reinterpret_cast<const float2*>(mlt + row * 2);
          if (whole) {
            const float inv = st.y > 0.f ? 1.f / st.y : 0.f;
            reinterpret_cast<uint32_t*>(a.o)[((q_row0 + row) * D + ch) / 2] = pack2<BF16>(v.x * inv, v.y * inv);
            if (cc == 0 && c2 == 0) a.lse[q_row0 + row] = log_sum(st.x, st.y) * kLn2;
          } else {
            *reinterpret_cast<float2*>(slot + row * D + ch) = v;
            if (cc == 0 && c2 == 0) *reinterpret_cast<float2*>(slot + C::ROWS * D + row * 2) = st;
          }
        }
      }
      __syncthreads();
    }
    rot = (rot + nblk) % C::TEAMS;
    if (*abort_flag) break;
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

// Where a segment's partials are: those of CTAs g0 .. g1 (g0 == g1: finished by that CTA)
template <int D, int ROWS>
struct Partials {
  const float* part;
  int g0, g1;
  __device__ __forceinline__ const float* of(int g) const {
    return part + ((size_t)g * 2 + (g == g0 ? 1 : 0)) * partial_floats(ROWS, D);
  }
};

constexpr int kFinishThreads = 256;
constexpr int kWeightSlots = 4 * kFinishThreads;  // slots of a head whose weights a block of the finish adds up
constexpr int kMaxRuns = 640;  // CTAs of the decode kernel, at most
constexpr int kAhead = 8;      // partials of O that a thread loads before their weights are known
constexpr int kJoinAtOnce = 64;  // partials whose weights are in shared memory
// channels of a segment that a block of the finish joins: four for each thread
template <int D, int NT>
constexpr int finish_channels() {
  return NT == 1 ? (D < 128 ? D : 128) : 64;
}

// What is left when the runs are done.  Blocks [0, segments x D / finish_channels): the segments that several CTAs'
// runs cut are joined from their partials, in the order of the CTAs, and the rows of empty sequences are
// written.  What it costs is a chain of latencies, so all that hangs on the lengths alone is done before
// the runs are over and the partials are loaded with the numbers that weigh them (8 sequences, d = 256: 26 us a
// call -> 23; 80 registers, as blocks that need more find room only when two of the runs are over: 26 with 64
// and their spills).  Further blocks, when weights are asked for, kWeightSlots slots of a head each: weights_out =
// weights_in + sum over the head's rows of 2^(S - L log2e).
template <int D, bool BF16, int NT, bool SCORES>
__global__ void __launch_bounds__(kFinishThreads, 3)
    decode_kv4_finish(const DecodeKv4Args a, const float* __restrict__ part, const float* __restrict__ scores,
                      int row_groups, int ctas) {
  constexpr int ROWS = 8 * NT;
  constexpr int CH = finish_channels<D, NT>(), SPLIT = D / CH;
  static_assert(ROWS * CH / 4 <= kFinishThreads, "four channels of a row for each thread");
  const int hr_count = a.hkv * row_groups;
  const int joins = a.b * hr_count * SPLIT;  // blocks that join
  const int R = (a.h / a.hkv) * a.nq;
  const WorkList wl{a.lens, a.b, hr_count, a.capacity};
  const int64_t total = wl.total(a.b);
  const int G = runs_of(total, ctas);
  __shared__ float fac[ROWS][kJoinAtOnce];
  __shared__ float2 stat[ROWS];
  auto partials = [&](int64_t before, int nb, int hr) {
    const int64_t first = before + (int64_t)hr * WorkList::positions(nb) + kSegCost;
    return Partials<D, ROWS>{part, run_of(total, first, G), run_of(total, first + nb - 1, G)};
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // The lengths are older than the runs (the decode kernel itself started only when all before it was
  // done), so only what follows has to wait for them.
  if ((int)blockIdx.x < joins) {
    const int seg = blockIdx.x / SPLIT, ch0 = (blockIdx.x - seg * SPLIT) * CH;
    const int b = seg / hr_count, hr = seg - b * hr_count;
    const int hk = hr / row_groups, rg = hr - hk * row_groups;
    const int rows = min(ROWS, R - rg * ROWS);
    const int64_t row0 = ((int64_t)b * a.hkv + hk) * R + rg * ROWS;
    if (hr == 0 && ch0 == 0 && threadIdx.x == 0 && clamp_len(a.lens[b], a.capacity) != a.lens[b])
      report_error(a.err, DERR_BAD_ARG, kSiteKv4Len);
    const int nb = wl.blocks(b);
    const int64_t before = wl.total(b);
    Partials<D, ROWS> P{part, 0, 0};
    if (nb > 0) {
      P = partials(before, nb, hr);
      // nothing to join (the first block stays, so that this launch is not over before the decode kernel is)
      if (P.g0 == P.g1 && blockIdx.x > 0) return;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int row = threadIdx.x / (CH / 4), ch = ch0 + threadIdx.x % (CH / 4) * 4;  // this thread's four channels
    uint2* dst = reinterpret_cast<uint2*>(a.o) + ((row0 + row) * D + ch) / 4;
    if (nb == 0) {
      if (row < rows) *dst = make_uint2(0u, 0u);
      if (ch0 == 0 && (int)threadIdx.x < rows) a.lse[row0 + threadIdx.x] = -INFINITY;
      return;
    }
    if (P.g0 == P.g1) return;
    const int n = P.g1 - P.g0 + 1;
    float4 x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (row < rows && j < n) x[j] = *reinterpret_cast<const float4*>(P.of(P.g0 + j) + row * D + ch);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& y, float f) {
      o.x = fmaf(y.x, f, o.x), o.y = fmaf(y.y, f, o.y), o.z = fmaf(y.z, f, o.z), o.w = fmaf(y.w, f, o.w);
    };
    for (int base = 0; base < n; base += kJoinAtOnce) {
      // each row's reference and sum, and each partial's weight: one warp a row
      const int count = min(n - base, kJoinAtOnce);
      for (int r = warp; r < rows; r += kFinishThreads / 32) {
        const auto ml = [&](int j) { return *reinterpret_cast<const float2*>(P.of(P.g0 + j) + ROWS * D + r * 2); };
        float2 v = make_float2(-INFINITY, 0.f);
        if (lane < count) v = ml(base + lane);
        float M = v.x, l = 0.f;
        if (base == 0) {
          for (int j = lane + 32; j < n; j += 32) M = fmaxf(M, ml(j).x);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        } else {
          M = stat[r].x;
        }
        for (int j = lane; j < count; j += 32) {
          if (j >= 32) v = ml(base + j);
          const float f = v.x == -INFINITY ? 1.f : ex2(v.x - M);  // (no maximum: nothing seen, or only NaN)
          fac[r][j] = f;
          l = fmaf(v.y, f, l);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) stat[r] = make_float2(M, base == 0 ? l : stat[r].y + l);
      }
      __syncthreads();
      if (row < rows) {
        if (base == 0) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            if (j < n) add(x[j], fac[row][j]);
        }
#pragma unroll 4
        for (int j = base == 0 ? kAhead : 0; j < count; ++j)
          add(*reinterpret_cast<const float4*>(P.of(P.g0 + base + j) + row * D + ch), fac[row][j]);
      }
      if (base + kJoinAtOnce < n) __syncthreads();
    }
    if (ch0 == 0 && (int)threadIdx.x < rows)
      a.lse[row0 + threadIdx.x] = log_sum(stat[threadIdx.x].x, stat[threadIdx.x].y) * kLn2;
    if (row >= rows) return;
    const float l = stat[row].y, inv = l > 0.f ? 1.f / l : 0.f;
    *dst = make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
    return;
  }
  // ---- weights
  if constexpr (SCORES) {
    const int tiles = (a.capacity + kWeightSlots - 1) / kWeightSlots;
    const int wb = (int)blockIdx.x - joins;
    const int bh = wb / tiles, b = bh / a.hkv, hk = bh - b * a.hkv;
    const int slot0 = (wb - bh * tiles) * kWeightSlots + threadIdx.x;  // this thread's slots: slot0 + i * kFinishThreads
    const int len = clamp_len(a.lens[b], a.capacity);
    if (slot0 - (int)threadIdx.x >= len) return;
    const int nb = blocks_of(len);
    const int64_t before = wl.total(b);
    Partials<D, ROWS> P = partials(before, nb, hk * row_groups);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int WT = kWeightSlots / kFinishThreads;
    constexpr int RT = 4;  // rows whose scores are loaded together
    const int64_t at = (int64_t)bh * a.capacity + slot0;
    float w[WT], w_in[WT], x[RT][WT];
#pragma unroll
    for (int i = 0; i < WT; ++i) {
      w[i] = 0.f;
      w_in[i] = a.w_in && slot0 + i * kFinishThreads < len ? a.w_in[at + i * kFinishThreads] : 0.f;
    }
    const float* s = scores + (int64_t)bh * R * a.capacity + slot0;
    auto load = [&](int row0, int rows) {  // scores of rows [row0, row0 + RT) of the head, those below row0 + rows
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < WT; ++i)
          x[r][i] = r < rows && slot0 + i * kFinishThreads < len
                        ? s[(int64_t)(row0 + r) * a.capacity + i * kFinishThreads] : -INFINITY;
    };
    for (int rg = 0; rg < row_groups; ++rg) {
      // the group's log-sum-exps, from the partials where several CTAs have them (O's block writes L only now)
      if (rg > 0) P = partials(before, nb, hk * row_groups + rg);
      const int rows = min(ROWS, R - rg * ROWS), n = P.g1 - P.g0 + 1;
      load(rg * ROWS, rows);
      __syncthreads();
      for (int row = warp; row < rows; row += kFinishThreads / 32) {
        float L;
        if (n == 1) {
          L = a.lse[(int64_t)bh * R + rg * ROWS + row] * kLog2e;
        } else {
          float2 v = make_float2(-INFINITY, 0.f);
          if (lane < n) v = *reinterpret_cast<const float2*>(P.of(P.g0 + lane) + ROWS * D + row * 2);
          float M = v.x, l = 0.f;
          for (int j = lane + 32; j < n; j += 32) M = fmaxf(M, P.of(P.g0 + j)[ROWS * D + row * 2]);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
          for (int j = lane; j < n; j += 32) {
            if (j >= 32) v = *reinterpret_cast<const float2*>(P.of(P.g0 + j) + ROWS * D + row * 2);
            l = fmaf(v.y, v.x == -INFINITY ? 1.f : ex2(v.x - M), l);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
          L = log_sum(M, l);
        }
        if (lane == 0) stat[row].x = L;
      }
      __syncthreads();
      for (int r0 = 0; r0 < rows; r0 += RT) {
        if (r0 > 0) load(rg * ROWS + r0, rows - r0);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if (r0 + r >= rows) break;
          const float L = stat[r0 + r].x;
          if (L == -INFINITY) continue;
#pragma unroll
          for (int i = 0; i < WT; ++i) w[i] += x[r][i] == -INFINITY ? 0.f : ex2(x[r][i] - L);  // (unseen: not NaN with L)
        }
      }
    }
#pragma unroll
    for (int i = 0; i < WT; ++i)
      if (slot0 + i * kFinishThreads < len) a.w_out[at + i * kFinishThreads] = w_in[i] + w[i];
  }
}

// Groups of 8 query rows that a CTA takes together: two when there are more than 8 rows, so that the cache is
// read once for 16; d = 256 has no registers for two (768 bytes of spills).
int row_tiles(int h, int hkv, int nq, int d) { return ((h / hkv) * nq > 8 && d < 256) ? 2 : 1; }

// CTAs of the decode kernel: as many as run at once, no more than there can be blocks
int grid_size(int b, int hkv, int row_groups, int capacity, int ctas) {
  const int64_t most = (int64_t)b * hkv * row_groups * (capacity / kKv4Block);
  return (int)std::min<int64_t>(most, std::min(ctas * device_sm_count(), kMaxRuns));
}
template <int D, bool BF16, int NT>
cudaError_t launch_nt(const DecodeKv4Args& a) {
  using C = Kv4Cfg<D, NT>;
  const int R = (a.h / a.hkv) * a.nq;
  const int row_groups = (R + C::ROWS - 1) / C::ROWS;
  const int G = grid_size(a.b, a.hkv, row_groups, a.capacity, C::CTAS);
  float* part = static_cast<float*>(a.ws);
  float* scores = part + (size_t)G * 2 * partial_floats(C::ROWS, D);
  auto kern = a.w_out ? decode_kv4_kernel<D, BF16, NT, true> : decode_kv4_kernel<D, BF16, NT, false>;
  static std::atomic<unsigned long long> allowed[2];  // context in which the kernel may have its shared memory
  cudaError_t e = allow_smem(kern, C::SMEM, &allowed[a.w_out ? 1 : 0]);
  if (e != cudaSuccess) return e;
  kern<<<G, C::THREADS, C::SMEM, a.stream>>>(a, part, scores, row_groups);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // launched while the runs are still going (it waits for them before it reads anything)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.b * a.hkv * row_groups) * (D / finish_channels<D, NT>()));
  if (a.w_out) cfg.gridDim.x += (unsigned)((a.capacity + kWeightSlots - 1) / kWeightSlots) * a.b * a.hkv;
  cfg.blockDim = dim3(kFinishThreads);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto finish = a.w_out ? decode_kv4_finish<D, BF16, NT, true> : decode_kv4_finish<D, BF16, NT, false>;
  return cudaLaunchKernelEx(&cfg, finish, a, (const float*)part, (const float*)scores,
                            row_groups, G);
}

template <int D>
cudaError_t launch_d(const DecodeKv4Args& a) {
  const bool bf = a.dtype == DT_BF16;
  if (row_tiles(a.h, a.hkv, a.nq, D) == 1) return bf ? launch_nt<D, true, 1>(a) : launch_nt<D, false, 1>(a);
  if constexpr (D < 256) return bf ? launch_nt<D, true, 2>(a) : launch_nt<D, false, 2>(a);
  return cudaErrorNotSupported;
}

}  // namespace

size_t decode_kv4_workspace_bytes(int b, int h, int hkv, int nq, int capacity, int d, bool weights) {
  const int nt = row_tiles(h, hkv, nq, d), rows = 8 * nt;
  const int ctas = nt == 1 ? (d == 256 ? Kv4Cfg<256, 1>::CTAS : Kv4Cfg<128, 1>::CTAS) : Kv4Cfg<128, 2>::CTAS;
  const int R = (h / hkv) * nq;
  const int row_groups = (R + rows - 1) / rows;
  size_t n = (size_t)grid_size(b, hkv, row_groups, capacity, ctas) * 2 * partial_floats(rows, d);
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
