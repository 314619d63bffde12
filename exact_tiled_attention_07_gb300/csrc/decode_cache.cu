// Decode attention over 16-bit key/value caches of sequences of different lengths, with a sliding window and sinks, or behind
// a prefix that all sequences share (bf16/fp16, head dims 64/128/256; sm_103a: TMA, tcgen05, TMEM).
//
// What it computes: sequence b has lens[b] keys and values in its cache, the newest of which are those of its Nq new rows;
// row i sees slots j < hi = lens[b] - Nq + i + 1, with a window only those with j >= hi - window or j < sinks; with a prefix
// every row sees all of its P keys as well.  O = softmax(tau Q K^T) V and L = m + ln l over what a row sees.
//
// Bound: HBM for the caches (a key and a value are used by the H / Hkv x Nq rows of a head only); the prefix is read once
// for up to 128 rows of all sequences and is bound by matrix products and exponentials where there are more.
//
// Work: entries of (rows, keys): for the prefix (key/value head, 128 of the B x group x Nq rows that read it), for the
// caches (sequence, key/value head, 128 of its group x Nq rows).  An entry is cut into tiles of 128 keys (64 at d = 256),
// and the tiles of all entries form one list, found on the device from the lengths, of which each CTA (one an SM) takes an
// equal run.  What lies of an entry in one run is a segment.  A window's tiles begin at its first key, not at a
// multiple of the tile; the sinks in front of it have tiles of their own; a tile's loads end behind its last key (in steps
// of 16 rows).
// An entry that lies inside one run, and has no prefix, is finished there; the segments of the others (O and row statistics of
// each, unnormalised, in the workspace) are joined by a second launch, decode_cache_finish, which starts under the first one.
// Slots need no bookkeeping: along the list each new segment has either the next entry or the next CTA, so entry + CTA
// numbers them.
//
// A CTA is a chain of warps that run ahead of one another across segments:
//   producer  walks the list, publishes segments in a ring, loads K and V tiles into a ring that takes the shared memory;
//   MMA warp  S = Q K^T (Q in TMEM) two tiles ahead of O += P V (P in TMEM, over S), also across the end of a segment;
//   softmax   (4 warps, a thread a row) as in the forward kernel: exp2, lazy rescaling by 2^8.  With 32 rows or fewer
//             the rows stand in all four lane quarters and each takes a quarter of the tile's columns, as if they were
//             other pieces of the keys (two halves for up to 64 rows);
//   drain     (4 warps) the next segment's Q into TMEM, a finished segment's O out of it (copies of a row joined), so that
//             the softmax goes on with the next segment's scores meanwhile.
// Measured (one GB300, d = 128, 4 rows a head): 32 x 8 heads of 32,768 slots (4.3 GB) 597 us, 7.2 TB/s, above the measured copy
// rate; 64 x 8 of 2,048 slots 97 us (5.5 TB/s); d = 64 and 256 6.8 and 7.1 TB/s on 2.1 and 4.3 GB.  Around that: 5 us until the first
// scores, of which 1.5 are index arithmetic and the rest latencies (launch, lengths, Q, first keys), one behind the other;
// 2.5 to 3 us for a segment of one tile (the drain's work on it: 150 us for 512 x 8 heads of 100 slots); 0.9 us for a tile of
// the prefix with 128 rows, one softmax warp a scheduler, twice the matrix instructions' time.  Steps (16 sequences with a
// window of 4,096; 64 behind a prefix of 32,768): segments' copies joined by the second launch 60, 142 us; joined here, index
// arithmetic in 32 bits, the next segment's Q not waited for while a P V is due 50, 146; the prefix in pieces 50, 130; a warp a
// row in the second launch 49, 124.
#include <cuda.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"
#include "tmap.h"

namespace fa {
namespace {

constexpr int BM = 128;  // rows of a tile (TMEM lanes)
constexpr float kRescaleThreshold = 8.0f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kLoadRows = 16;   // rows of the loads that end a tile early
// What a segment's start and end cost, in tiles.  Counted as 2, 3, 4, 6: 12 sequences of up to 2,047 slots behind 20,001 shared
// tokens 48, 44, 42, 44 us; 64 of up to 3,943 behind 32,768 130, 130, 134, 142; without a prefix the same within 2 %.
constexpr int kSegCost = 3;
constexpr int kSegs = 4;        // published segments, and row statistics, in flight
constexpr int kFinishThreads = 128;
constexpr int kListed = 64;  // slots of partial results that a warp lists at a time (a multiple of 32)
constexpr int kAhead = 8;    // partial results whose loads a warp has in flight
constexpr int kMostCtas = 512;
constexpr int kFewSequences = 512;
constexpr int kDrainBarrier = 1;  // named barrier of the four drain warps

template <int D>
struct CacheCfg {
  static constexpr int BN = D == 256 ? 64 : 128;  // keys of a tile
  static constexpr int KB = D / 64;               // 64-column (128-byte) blocks of a row
  static constexpr int TILE_BYTES = BN * D * 2;
  static constexpr int STAGES = D == 64 ? 12 : 6;
  static constexpr int PRODUCER_WARP = 4, MMA_WARP = 5, DRAIN_WARP0 = 6;
  static constexpr int THREADS = 320;
  static constexpr int READERS = 9;  // warps that read a published segment: MMA, softmax, drain
  // TMEM columns: S double buffer, O, Q (two buffers; one at d = 256, where they fill the 512)
  static constexpr int S_COL0 = 0, S_COL1 = BN, O_COL = 256;
  static constexpr int QBUFS = D == 256 ? 1 : 2;
  static constexpr int Q_COL = D == 256 ? 2 * BN : O_COL + D;
  static_assert(D == 256 ? Q_COL + D / 2 <= O_COL : Q_COL + D <= 512, "TMEM columns");
  static constexpr int OFF_BAR = STAGES * TILE_BYTES;
  static constexpr int NBAR = 2 * STAGES + 2 * kSegs + QBUFS + 2 + 2 + kSegs + 4;
  static constexpr int OFF_SEG = OFF_BAR + NBAR * 8 + 16;  // [kSegs] Seg
  static constexpr int OFF_STAT = OFF_SEG + kSegs * 64;    // [kSegs][128] (m, l)
  static constexpr int OFF_RED = OFF_STAT + kSegs * BM * 8;
  // copies of rows meet here, 32 columns at a time (rows of 36 floats: no two of a quarter warp in one bank)
  static constexpr int XROW = 36;
  static constexpr int OFF_X = (OFF_RED + 16 * 8 + 15) & ~15;
  static constexpr int SMEM = OFF_X + (D == 256 ? 0 : BM * (XROW + 1) * 4);  // and the weights of copies
  static_assert(STAGES >= 4, "the products run two tiles ahead");
  static_assert(SMEM <= 232448 && OFF_SEG % 8 == 0 && OFF_STAT % 8 == 0 && OFF_RED % 8 == 0, "shared memory");
};

// x / y of numbers that are not negative: a division of 64 bits takes a hundred instructions, of 32 bits a fifth of that.
__device__ __forceinline__ int64_t div(int64_t x, int64_t y) {
  return (x | y) >> 32 == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// What lies of an entry in a CTA's run.
struct Seg {
  int rows;     // of the entry's 128 (0: no more segments)
  int prefix;
  int b, kvh, rt;
  int head;     // of the tensor map
  int t0, nt;   // tiles [t0, t0 + nt) of the entry
  int ns, sk;   // its first ns tiles hold the sinks, keys [0, sk)
  int lo, end;  // the others keys [lo, end)
  int slot;     // of the partial results
  int whole;    // all there is for its rows: O and L are final
};
static_assert(sizeof(Seg) <= 64, "Seg");

// The list of tiles.  Offsets count tiles and kSegCost for each entry.
struct List {
  const int32_t* lens;
  int b, hkv, nq, capacity, p, log_bn;  // (log2 of a tile's keys: divisions by it are shifts)
  int rt_own, rt_pre;  // row tiles of a sequence's head, of the prefix' head
  int window, sinks;

  __device__ int tiles_of(int keys) const { return (int)(((unsigned)keys + (1u << log_bn) - 1) >> log_bn); }
  // keys of a sequence: sinks [0, sk), the rest [lo, len)
  struct Keys {
    int len, lo, sk, ns, tiles;
  };
  __device__ Keys keys(int len) const {
    Keys k;
    k.len = len;
    k.lo = 0;
    if (window > 0) {
      const int64_t lo = (int64_t)len - nq + 1 - window;  // the first row's
      k.lo = lo > 0 ? (int)lo : 0;
    }
    k.sk = sinks < k.lo ? sinks : k.lo;
    k.ns = tiles_of(k.sk);
    k.tiles = k.ns + tiles_of(len - k.lo);
    return k;
  }
  __device__ int len_of(int s) const { return min(max(lens[s], 0), capacity); }
  __device__ static int64_t cost(int tiles) { return tiles > 0 ? tiles + kSegCost : 0; }
  __device__ int prefix_tiles() const { return tiles_of(p); }
  __device__ int64_t own_total(int s) const { return (int64_t)hkv * rt_own * cost(keys(len_of(s)).tiles); }
};

// The prefix' entries: (key/value head, piece of the keys, row tile), pieces of `piece` tiles.  One piece where a head has one row
// tile; with several, pieces as long as a CTA's run: neighbouring CTAs then read the same keys for different rows at the
// same time, and L2 hands out what HBM was read for once (without pieces eight row tiles read a prefix of 134 MB seven
// times from HBM).  A run is at least as long as all the prefix' tiles by all CTAs, so there are not more than 4/3 grid + hkv
// rt_pre entries.
struct Prefix {
  int tiles, piece, pieces, entries;
  __device__ void set(const List& list, int64_t own, int grid) {
    tiles = piece = list.prefix_tiles();
    pieces = entries = 0;
    if (tiles == 0) return;
    if (list.rt_pre > 1) {
      const int64_t run = div(own + (int64_t)list.hkv * list.rt_pre * tiles + grid - 1, grid);
      const int n = max(1, (int)div(tiles + run / 2, run));
      piece = (tiles + n - 1) / n;  // (two or more: at least 3/4 of a run)
    }
    pieces = (tiles + piece - 1) / piece;
    entries = list.hkv * pieces * list.rt_pre;
  }
  __device__ int64_t cost() const { return piece + kSegCost; }
  __device__ int64_t total() const { return entries * cost(); }
  __device__ int tiles_of(int x) const { return min(piece, tiles - x * piece); }
};
// CTA c of n takes [start(c), start(c + 1)) of a list.
__device__ __forceinline__ int64_t run_start(int64_t total, int c, int n) { return div(total * c, n); }
__device__ __forceinline__ int run_of(int64_t total, int64_t at, int n) { return (int)div((at + 1) * n - 1, total); }
__device__ __forceinline__ int runs_of(int64_t total, int grid) { return total < grid ? (int)total : grid; }

// Partial results: for the prefix' segments, then the caches', [slots][D / 4][lanes] float4 and [slots][lanes] (m, l), a lane for
// each row; then the lists' offset of each sequence.
struct Partials {
  float4 *pre_o, *own_o;
  float2 *pre_ml, *own_ml;
  int64_t* offsets;  // [b + 2]: of each sequence's first entry, then the total, and the caches' part of it
  int pre_lanes, own_lanes;
};

int cache_grid() { return std::min(kMostCtas, device_sm_count()); }
int row_copies(int d, int64_t rows) { return d == 256 || rows > 64 ? 1 : (rows > 32 ? 2 : 4); }

struct Shape {  // of a launch
  int gn, rt_own, rt_pre, r_own, r_pre, own_lanes, pre_lanes;
  int64_t pre_slots, own_slots;
  Shape(int b, int h, int hkv, int nq, int p, int d, int grid) {
    gn = h / hkv * nq;
    const int64_t all = (int64_t)b * gn;
    rt_own = (gn + BM - 1) / BM;
    rt_pre = p > 0 ? (int)((all + BM - 1) / BM) : 0;
    r_own = row_copies(d, gn);
    r_pre = row_copies(d, all);
    own_lanes = std::min(gn, BM);
    pre_lanes = (int)std::min<int64_t>(all, BM);
    pre_slots = p > 0 ? (int64_t)hkv * rt_pre + 3 * grid : 0;
    own_slots = (int64_t)b * hkv * rt_own + grid;
  }
  size_t bytes(int b, int d) const {
    const size_t lanes = (size_t)pre_slots * pre_lanes + (size_t)own_slots * own_lanes;
    return lanes * ((size_t)d * 4 + 8) + ((size_t)b + 2) * 8;
  }
  Partials carve(void* ws, int d) const {
    Partials w;
    char* at = static_cast<char*>(ws);
    w.pre_o = reinterpret_cast<float4*>(at);
    at += (size_t)pre_slots * pre_lanes * d * 4;
    w.own_o = reinterpret_cast<float4*>(at);
    at += (size_t)own_slots * own_lanes * d * 4;
    w.pre_ml = reinterpret_cast<float2*>(at);
    at += (size_t)pre_slots * pre_lanes * 8;
    w.own_ml = reinterpret_cast<float2*>(at);
    at += (size_t)own_slots * own_lanes * 8;
    w.offsets = reinterpret_cast<int64_t*>(at);
    w.pre_lanes = pre_lanes;
    w.own_lanes = own_lanes;
    return w;
  }
};

struct CacheParams {
  const void* q;
  void* o;
  float* lse;
  List list;
  Partials ws;
  int gn;
  int r_own, r_pre;  // copies of a row
  float scale_log2;
  unsigned long long* err;
  unsigned long long* counter;
};

// Where a TMEM lane's row is: copy cp of R, row rit of the tile.
__device__ __forceinline__ void lane_row(int R, int quarter, int lane, int* cp, int* rit) {
  const int quarters = 4 / R;  // lane quarters of a copy
  *cp = quarter / quarters;
  *rit = (quarter % quarters) * 32 + lane;
}

// One tile of a segment for one row (copy): scores of columns [col0, col0 + BN / R) in, weights out; hi, lo, top: the columns
// c < hi with c >= lo or c < top are visible (relative to col0).
template <int BN, bool BF16, int R>
__device__ __forceinline__ void softmax_tile(uint32_t tbase, uint32_t lane_base, uint32_t s_col, int cp, int hi, int lo,
                                             int top, float scale_log2, float& m, float& l, float& alpha, bool& rescale) {
  constexpr int COLS = BN / R;
  const int col0 = cp * COLS;
  uint32_t sr[COLS / 32][32];
#pragma unroll
  for (int c = 0; c < COLS / 32; ++c) tmem_ld32(tmem_addr(tbase, lane_base, s_col + col0 + c * 32), sr[c]);
  tmem_wait_ld();
#pragma unroll
  for (int c = 0; c < COLS / 32; ++c) reg_fence(sr[c]);
  float s[COLS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) s[c] = __uint_as_float(sr[c / 32][c % 32]);
  hi -= col0, lo -= col0, top -= col0;
  if (hi < COLS || (lo > 0 && top < COLS)) {
#pragma unroll
    for (int c = 0; c < COLS; ++c)
      if (c >= hi || (c < lo && c >= top)) s[c] = -INFINITY;
  }
  const float m_blk = row_max3(s) * scale_log2;
  alpha = 1.f;
  rescale = false;
  if (m == -INFINITY) {
    m = m_blk;  // first tile with a visible key for this row (O is still zero)
    alpha = 0.f;
  } else if (m_blk > m + kRescaleThreshold) {
    alpha = ex2(m - m_blk);
    m = m_blk;
    rescale = true;
  }
  const float neg_m = m == -INFINITY ? 0.f : -m;
  float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int g = 0; g < COLS / 32; ++g) {
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 x = ffma2(make_float2(s[g * 32 + 2 * i], s[g * 32 + 2 * i + 1]), scale_log2, neg_m);
      const float2 p = make_float2(ex2(x.x), ex2(x.y));
      part[i & 1] = fadd2(part[i & 1], p);
      pk[i] = pack2<BF16>(p.x, p.y);
    }
    tmem_st16(tmem_addr(tbase, lane_base, s_col + col0 / 2 + g * 16), pk);
  }
  if constexpr (R > 1) {
    // the other copies' columns contribute nothing to this copy's rows
    const uint32_t zero[16] = {};
#pragma unroll
    for (int g = 0; g < BN / 32; ++g)
      if (g / (COLS / 32) != cp) tmem_st16(tmem_addr(tbase, lane_base, s_col + g * 16), zero);
  }
  l = l * alpha + ((part[0].x + part[1].x) + (part[0].y + part[1].y));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(CacheCfg<D>::THREADS, 1)
    decode_cache_kernel(const __grid_constant__ CacheParams a, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k16,
                        const __grid_constant__ CUtensorMap tm_v16, const __grid_constant__ CUtensorMap tm_kp,
                        const __grid_constant__ CUtensorMap tm_vp, const __grid_constant__ CUtensorMap tm_kp16,
                        const __grid_constant__ CUtensorMap tm_vp16) {
  using C = CacheCfg<D>;
  constexpr int BN = C::BN;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const List& list = a.list;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = kv_full + C::STAGES;
  uint64_t* seg_full = kv_empty + C::STAGES;  // [kSegs] a segment is published in this place
  uint64_t* seg_empty = seg_full + kSegs;     // [kSegs] every reader has it
  uint64_t* q_full = seg_empty + kSegs;       // [QBUFS] a segment's Q is in TMEM
  uint64_t* s_full = q_full + C::QBUFS;       // [2]
  uint64_t* p_full = s_full + 2;              // [2] one for each S buffer: the softmax is never two phases ahead
  uint64_t* stat_full = p_full + 2;           // [kSegs] row statistics of a segment are written
  uint64_t* pv_done = stat_full + kSegs;      // P V of a tile is done
  uint64_t* o_full = pv_done + 1;             // O of a segment is final
  uint64_t* o_empty = o_full + 1;             // and has been read
  uint64_t* drain = o_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Seg* segs = reinterpret_cast<Seg*>(smem + C::OFF_SEG);
  float2* stats = reinterpret_cast<float2*>(smem + C::OFF_STAT);
  int64_t* red = reinterpret_cast<int64_t*>(smem + C::OFF_RED);
  const ErrCtx ctx{a.err, abort_flag};

  asm volatile("griddepcontrol.launch_dependents;");
  if (warp == C::PRODUCER_WARP && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_k16);
    tma_prefetch_desc(&tm_v16);
    if (list.p > 0) {
      tma_prefetch_desc(&tm_kp);
      tma_prefetch_desc(&tm_vp);
    }
  }
  if (threadIdx.x == 0) {
    if ((smem_u32(smem) & 1023u) != 0) report_error(a.err, DERR_BAD_SMEM_ALIGN, 400);
    *abort_flag = (smem_u32(smem) & 1023u) != 0;
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(kv_full + s, 1);
      mbar_init(kv_empty + s, 1);
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(seg_full + s, 1);
      mbar_init(seg_empty + s, C::READERS);
      mbar_init(stat_full + s, 128);
    }
    for (int i = 0; i < C::QBUFS; ++i) mbar_init(q_full + i, 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
    }
    mbar_init(pv_done, 1);
    mbar_init(o_full, 1);
    mbar_init(o_empty, 128);
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // the first 32 sequences' part of the list, summed up to each of them, for the producer's search
  int64_t first32 = 0;
  auto sum_up = [&](int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    return v;
  };
  if (warp == C::PRODUCER_WARP) first32 = sum_up(lane < list.b ? list.own_total(lane) : 0);
  // the list's length: every thread adds up some sequences; CTA 0 leaves each one's offset for the finishing launch
  int64_t sum = 0;
  for (int s = threadIdx.x; s < list.b; s += C::THREADS) {
    if (blockIdx.x == 0 && list.lens[s] != list.len_of(s)) report_error(a.err, DERR_BAD_ARG, 401);
    sum += list.own_total(s);
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) red[warp] = sum;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t own_all = 0;
#pragma unroll
  for (int w = 0; w < C::THREADS / 32; ++w) own_all += red[w];
  Prefix pre;
  pre.set(list, own_all, gridDim.x);
  const int64_t pre_total = pre.total(), total = pre_total + own_all;
  if (blockIdx.x == 0 && warp == C::DRAIN_WARP0) {
    int64_t at = pre_total;
    for (int s0 = 0; s0 < list.b; s0 += 32) {
      const int64_t mine = s0 + lane < list.b ? list.own_total(s0 + lane) : 0, v = sum_up(mine);
      if (s0 + lane < list.b) a.ws.offsets[s0 + lane] = at + v - mine;
      at += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) a.ws.offsets[list.b] = total, a.ws.offsets[list.b + 1] = own_all;
    __syncwarp();
  }
  const uint32_t tbase = *tmem_slot;
  const int runs = runs_of(total, gridDim.x);
  const bool start_ok = *abort_flag == 0 && (int)blockIdx.x < runs;

  // one warp's read of segment s; `good` turns false (and rows 0) when the bounded wait ran out
  auto read_seg = [&](int s, bool& good) {
    const int at = s % kSegs;
    good = __all_sync(0xffffffffu, mbar_wait(seg_full + at, (uint32_t)(s / kSegs) & 1, ctx, 410)) && good;
    Seg g;
    const volatile int* from = reinterpret_cast<const volatile int*>(segs + at);
    int* to = reinterpret_cast<int*>(&g);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Seg) / 4); ++i) to[i] = from[i];
    if (!good) g.rows = 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty + at);
    return g;
  };
  // a tile's first key and how many of the keys behind it are the segment's
  auto tile_keys = [&](const Seg& g, int t, int* keys) {
    const int base = t < g.ns ? t * BN : g.lo + (t - g.ns) * BN;
    *keys = min(BN, (t < g.ns ? g.sk : g.end) - base);
    return base;
  };

  if (warp == C::PRODUCER_WARP) {
    // ------------------------------------------------------------------ producer
    if (start_ok) {
      const int64_t u0 = run_start(total, blockIdx.x, runs), u1 = run_start(total, blockIdx.x + 1, runs);
      // the sequence that the run begins in, or the first one behind the prefix (the whole warp), and its offset
      int b = 0;
      int64_t b_off = pre_total;
      const int64_t from = max(u0, pre_total);
      for (int s0 = 0; s0 < list.b && u1 > pre_total; s0 += 32) {
        const int64_t v = s0 == 0 ? first32 : sum_up(s0 + lane < list.b ? list.own_total(s0 + lane) : 0);
        const unsigned past = __ballot_sync(0xffffffffu, b_off + v > from);
        if (past) {
          const int f = __ffs(past) - 1;
          b = s0 + f;
          const int64_t before = __shfl_sync(0xffffffffu, v, f > 0 ? f - 1 : 0);
          if (f > 0) b_off += before;
          break;
        }
        b_off += __shfl_sync(0xffffffffu, v, 31);
      }
      if (lane == 0) {
        int n_segs = 0;
        uint32_t pos = 0;  // loads issued
        bool ok = true;
        auto publish = [&](const Seg& g) {
          const int at = n_segs % kSegs;
          if (n_segs >= kSegs && !mbar_wait(seg_empty + at, (uint32_t)(n_segs / kSegs - 1) & 1, ctx, 411)) return false;
          volatile int* to = reinterpret_cast<volatile int*>(segs + at);
          const int* from_ = reinterpret_cast<const int*>(&g);
#pragma unroll
          for (int i = 0; i < (int)(sizeof(Seg) / 4); ++i) to[i] = from_[i];
          mbar_arrive(seg_full + at);
          ++n_segs;
          return true;
        };
        // the entry at u0, then one after the other
        Seg g;
        int tiles, len_next = 0;
        int64_t off;
        List::Keys keys{};
        auto begin_own = [&](int entry) {  // entry of sequence b
          g.prefix = 0;
          g.b = b;
          g.kvh = entry / list.rt_own;
          g.rt = entry - g.kvh * list.rt_own;
          g.ns = keys.ns;
          g.sk = keys.sk;
          g.lo = keys.lo;
          g.end = keys.len;
          tiles = keys.tiles;
        };
        auto next_len = [&]() { len_next = b + 1 < list.b ? list.lens[b + 1] : 0; };
        int piece = 0;  // of the prefix' keys
        auto begin_pre = [&]() {
          g.lo = piece * pre.piece * BN;
          tiles = pre.tiles_of(piece);
          g.end = min(list.p, g.lo + tiles * BN);
        };
        if (u0 < pre_total) {
          const int c = (int)pre.cost();
          const int e = (int)div(u0, c);
          off = (int64_t)e * c;
          g.prefix = 1;
          g.b = 0;
          g.kvh = e / (pre.pieces * list.rt_pre);
          piece = e / list.rt_pre - g.kvh * pre.pieces;
          g.rt = e % list.rt_pre;
          g.ns = g.sk = 0;
          begin_pre();
          if (u1 > pre_total) keys = list.keys(list.len_of(b));
        } else {
          keys = list.keys(list.len_of(b));
          const int64_t c = List::cost(keys.tiles), in = u0 - b_off;
          const int e = (int)div(in, c);
          off = b_off + e * c;
          begin_own(e);
        }
        next_len();
        while (ok) {
          g.head = g.prefix ? g.kvh : g.b * list.hkv + g.kvh;
          g.rows = min(BM, (g.prefix ? list.b * a.gn : a.gn) - g.rt * BM);
          g.slot = (g.prefix ? (g.kvh * pre.pieces + piece) * list.rt_pre : g.head * list.rt_own) + g.rt + (int)blockIdx.x;
          // its tiles in this run
          g.t0 = (int)max((int64_t)0, u0 - off - kSegCost);
          const int t1 = (int)min((int64_t)tiles, u1 - off - kSegCost);
          g.nt = t1 - g.t0;
          g.whole = list.p == 0 && g.nt == tiles;
          if (g.nt > 0 && !(ok = publish(g))) break;
          for (int t = g.t0; ok && t < t1; ++t) {
            int n;
            const int base = tile_keys(g, t, &n);
            if (!(ok = debug_check(n > 0 && base >= 0 && g.head >= 0 && g.head < (g.prefix ? list.hkv : list.b * list.hkv), ctx, 420)))
              break;
            for (int v = 0; ok && v < 2; ++v, ++pos) {
              const int slot = pos % C::STAGES;
              const uint32_t use = pos / C::STAGES;
              if (use > 0 && !(ok = mbar_wait(kv_empty + slot, (use - 1) & 1, ctx, 412))) break;
              uint8_t* dst = smem + slot * C::TILE_BYTES;
              if (n == BN) {
                const CUtensorMap* tm = g.prefix ? (v ? &tm_vp : &tm_kp) : (v ? &tm_v : &tm_k);
                mbar_arrive_expect_tx(kv_full + slot, C::TILE_BYTES);
                for (int kb = 0; kb < C::KB; ++kb) {
                  if (g.prefix) tma_load_3d(dst + kb * (BN * 128), tm, kv_full + slot, kb * 64, base, g.head);
                  else tma_load_3d_once(dst + kb * (BN * 128), tm, kv_full + slot, kb * 64, base, g.head);
                }
              } else {
                const CUtensorMap* tm = g.prefix ? (v ? &tm_vp16 : &tm_kp16) : (v ? &tm_v16 : &tm_k16);
                const int boxes = (n + kLoadRows - 1) / kLoadRows;
                mbar_arrive_expect_tx(kv_full + slot, boxes * kLoadRows * D * 2);
                for (int x = 0; x < boxes; ++x)
                  for (int kb = 0; kb < C::KB; ++kb)
                    tma_load_3d(dst + kb * (BN * 128) + x * kLoadRows * 128, tm, kv_full + slot, kb * 64,
                                base + x * kLoadRows, g.head);
              }
            }
          }
          // the next entry
          off += g.prefix ? pre.cost() : tiles + kSegCost;
          if (off >= u1) break;
          if (++g.rt < (g.prefix ? list.rt_pre : list.rt_own)) continue;
          g.rt = 0;
          if (g.prefix) {
            if (++piece == pre.pieces) {
              piece = 0;
              if (++g.kvh == list.hkv) {  // the sequences follow (b is the first one with something in its cache)
                begin_own(0);
                continue;
              }
            }
            begin_pre();
            continue;
          }
          if (++g.kvh < list.hkv) continue;
          do {
            ++b;
            if (b >= list.b) break;
            keys = list.keys(min(max(len_next, 0), list.capacity));
            next_len();
          } while (keys.tiles == 0);
          if (b >= list.b) break;
          begin_own(0);
        }
        Seg none{};
        if (ok) publish(none);
        // every copy this thread started must land before the CTA may exit
        ErrCtx nctx = ctx;
        int no_abort = 0;
        nctx.abort = &no_abort;
        for (int64_t i = (int64_t)pos - 1; i >= 0 && i >= (int64_t)pos - C::STAGES; --i)
          mbar_wait(kv_full + i % C::STAGES, (uint32_t)(i / C::STAGES) & 1, nctx, 413);
      }
    }
    __syncwarp();
  } else if (warp == C::MMA_WARP) {
    // ------------------------------------------------------------------ MMA issuer (converged, one lane issues)
    if (start_ok) {
      const bool leader = elect_one_sync();
      const uint32_t idesc_qk = make_idesc_f16(BM, BN, BF16, false, false);
      const uint32_t idesc_pv = make_idesc_f16(BM, D, BF16, false, true);
      const uint32_t ring = smem_u32(smem);
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctx, site));
      };
      auto commit = [&](uint64_t* bar) {
        if (leader) umma_commit(bar);
        __syncwarp();
      };
      bool ok = true;
      int sq = 0, t = 0;  // the segment and the tile of it whose S is next
      Seg g = read_seg(0, ok);
      uint32_t g_qk = 0, g_pv = 0;  // tiles whose S, whose P V has been issued
      // of the (at most two) tiles between S and P V: first of its segment (and the segment), last, keys
      int first_[2] = {-1, -1}, last_[2] = {0, 0}, keys_[2] = {0, 0};
      while (ok) {
        while (ok && g.rows > 0 && g_qk < g_pv + 2) {
          // (one Q buffer: the next segment's Q arrives when the last one's O is final)
          if (C::QBUFS == 1 && t == 0 && g_qk > g_pv) break;
          // (with two it may be on its way still: the P V of what is there does not wait for it)
          if (C::QBUFS == 2 && t == 0 && g_qk > g_pv &&
              !__all_sync(0xffffffffu, mbar_test_wait(q_full + (sq & 1), (uint32_t)(sq >> 1) & 1)))
            break;
          const uint32_t pos = 2 * g_qk, slot = pos % C::STAGES;
          const int qb = C::QBUFS == 2 ? (sq & 1) : 0;
          if (t == 0 && !(ok = wait(q_full + qb, (uint32_t)(sq / C::QBUFS) & 1, 420))) break;
          if (!(ok = wait(kv_full + slot, (pos / C::STAGES) & 1, 421))) break;
          tc_fence_after();
          const uint32_t kt = ring + slot * C::TILE_BYTES;
          const uint32_t q_col = C::Q_COL + qb * (D / 2), s_col = (g_qk & 1) ? C::S_COL1 : C::S_COL0;
          uint64_t bd[D / 16];
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            bd[kk] = make_sdesc_sw128(kt + (kk * 16 / 64) * (BN * 128) + (kk * 16 % 64) * 2, 16, 1024);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_ts(tbase + s_col, tbase + q_col + kk * 8, bd[kk], idesc_qk, kk > 0 ? 1u : 0u);
            umma_commit(s_full + (g_qk & 1));
            umma_commit(kv_empty + slot);
          }
          __syncwarp();
          int n;
          tile_keys(g, g.t0 + t, &n);
          const int fi = t == 0 ? sq : -1, la = t + 1 == g.nt;
          if (g_qk & 1) first_[1] = fi, last_[1] = la, keys_[1] = n;
          else first_[0] = fi, last_[0] = la, keys_[0] = n;
          ++g_qk;
          if (++t == g.nt) {
            t = 0;
            g = read_seg(++sq, ok);
          }
        }
        if (!ok || g_pv == g_qk) break;
        const int i = g_pv & 1;
        const int first = i ? first_[1] : first_[0], last = i ? last_[1] : last_[0], n = i ? keys_[1] : keys_[0];
        const uint32_t pos = 2 * g_pv + 1, slot = pos % C::STAGES;
        if (!(ok = wait(kv_full + slot, (pos / C::STAGES) & 1, 422))) break;
        const int steps = (n + 15) / 16;  // of 16 keys
        if (n < steps * 16) {
          // V rows behind the segment's keys (another sequence's, or what the place held before): zero, since 0 x NaN is NaN
          uint8_t* vt = smem + slot * C::TILE_BYTES;
          for (int x = n * 8 + lane; x < steps * 128; x += 32)
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
              *reinterpret_cast<uint4*>(vt + kb * (BN * 128) + x * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!(ok = wait(p_full + i, (g_pv >> 1) & 1, 423))) break;
        // the first P V of a segment overwrites O: the last segment's must have been read
        if (first > 0 && !(ok = wait(o_empty, (uint32_t)(first - 1) & 1, 424))) break;
        tc_fence_after();
        const uint32_t vt = ring + slot * C::TILE_BYTES, p_col = i ? C::S_COL1 : C::S_COL0;
        uint64_t bd[BN / 16];
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) bd[kk] = make_sdesc_sw128(vt + kk * 2048, BN * 128, 1024);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            if (kk < steps) umma_ts(tbase + C::O_COL, tbase + p_col + kk * 8, bd[kk], idesc_pv, (first < 0 || kk > 0) ? 1u : 0u);
          umma_commit(pv_done);
          umma_commit(kv_empty + slot);
          if (last) umma_commit(o_full);
        }
        __syncwarp();
        ++g_pv;
      }
      // all MMAs complete before TMEM is released
      ErrCtx nctx = ctx;
      int no_abort = 0;
      nctx.abort = &no_abort;
      commit(drain);
      mbar_wait(drain, 0, nctx, 425);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------------ softmax (one TMEM lane per thread)
    const uint32_t lane_base = warp * 32;
    bool ok = start_ok;
    uint32_t gt = 0;  // tiles (all segments)
    for (int s = 0; ok; ++s) {
      const Seg g = read_seg(s, ok);
      if (g.rows == 0) break;
      const int R = g.prefix ? a.r_pre : a.r_own;
      int cp, rit;
      lane_row(R, warp, lane, &cp, &rit);
      // this row's keys: [lo, hi) and those below sinks
      int hi = g.end, lo = 0, sinks = 0;
      if (!g.prefix) {
        hi = g.end - list.nq + (g.rt * BM + rit) % list.nq + 1;
        if (list.window > 0) {
          lo = hi > list.window ? hi - list.window : 0;
          sinks = list.sinks;
        }
      }
      const bool any = (warp % (4 / R)) * 32 < g.rows;  // the warp holds rows
      float m = -INFINITY, l = 0.f;
      for (int t = 0; ok && t < g.nt; ++t, ++gt) {
        const uint32_t s_col = (gt & 1) ? C::S_COL1 : C::S_COL0;
        ok = __all_sync(0xffffffffu, mbar_wait(s_full + (gt & 1), (gt >> 1) & 1, ctx, 430));
        if (!ok) break;
        if (any) {
          tc_fence_after();
          int n;
          const int base = tile_keys(g, g.t0 + t, &n);
          const int h = min(hi - base, n), w = lo - base, top = sinks - base;
          float alpha;
          bool rescale;
          if constexpr (D == 256) {
            softmax_tile<BN, BF16, 1>(tbase, lane_base, s_col, 0, h, w, top, a.scale_log2, m, l, alpha, rescale);
          } else {
            if (R == 4) softmax_tile<BN, BF16, 4>(tbase, lane_base, s_col, cp, h, w, top, a.scale_log2, m, l, alpha, rescale);
            else if (R == 2) softmax_tile<BN, BF16, 2>(tbase, lane_base, s_col, cp, h, w, top, a.scale_log2, m, l, alpha, rescale);
            else softmax_tile<BN, BF16, 1>(tbase, lane_base, s_col, 0, h, w, top, a.scale_log2, m, l, alpha, rescale);
          }
          if (__any_sync(0xffffffffu, rescale)) {
            // O row *= alpha once the P V of the tile before has completed (a first tile has nothing to rescale)
            ok = __all_sync(0xffffffffu, mbar_wait(pv_done, (gt - 1) & 1, ctx, 431));
            if (!ok) break;
            tc_fence_after();
            const float f = rescale ? alpha : 1.f;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t r[32];
              const uint32_t ta = tmem_addr(tbase, lane_base, C::O_COL + c * 32);
              tmem_ld32(ta, r);
              tmem_wait_ld();
              reg_fence(r);
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
              tmem_st32(ta, r);
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        mbar_arrive(p_full + (gt & 1));
      }
      stats[(s % kSegs) * BM + threadIdx.x] = make_float2(m, l);
      mbar_arrive(stat_full + s % kSegs);
    }
  } else {
    // ------------------------------------------------------------------ drain: Q in, O out
    const int quarter = warp & 3;
    const uint32_t lane_base = quarter * 32;
    bool ok = start_ok;
    // Q of a segment into TMEM as 16-bit pairs (lanes without a row: zeros)
    auto load_q = [&](const Seg& g, int s) {
      int cp, rit;
      lane_row(g.prefix ? a.r_pre : a.r_own, quarter, lane, &cp, &rit);
      const int r = g.rt * BM + rit;
      const int64_t row = g.prefix ? ((int64_t)(r / a.gn) * list.hkv + g.kvh) * a.gn + r % a.gn
                                   : ((int64_t)g.b * list.hkv + g.kvh) * a.gn + r;
      const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + row * D);
      const uint32_t q_col = C::Q_COL + (C::QBUFS == 2 ? (s & 1) : 0) * (D / 2);
      constexpr int BLOCKS = D == 64 ? 1 : 2;  // 64-column blocks whose loads are in flight together
#pragma unroll 1
      for (int c = 0; c < D / 64; c += BLOCKS) {
        uint32_t x[BLOCKS][32];
#pragma unroll
        for (int k = 0; k < BLOCKS; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 u = rit < g.rows ? from[(c + k) * 8 + i] : make_uint4(0u, 0u, 0u, 0u);
            x[k][4 * i] = u.x, x[k][4 * i + 1] = u.y, x[k][4 * i + 2] = u.z, x[k][4 * i + 3] = u.w;
          }
#pragma unroll
        for (int k = 0; k < BLOCKS; ++k) tmem_st32(tmem_addr(tbase, lane_base, q_col + (c + k) * 32), x[k]);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(q_full + (C::QBUFS == 2 ? (s & 1) : 0));
    };
    // O of segment s out of TMEM; false when a wait ran out
    auto store_o = [&](const Seg& g, int s) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(o_full, s & 1, ctx, 440));
      ok = ok && __all_sync(0xffffffffu, mbar_wait(stat_full + s % kSegs, (uint32_t)(s / kSegs) & 1, ctx, 441));
      if (!(ok = named_bar_and(kDrainBarrier, 128, ok))) return false;
      tc_fence_after();
      int cp, rit;
      const int R = g.prefix ? a.r_pre : a.r_own;
      lane_row(R, quarter, lane, &cp, &rit);
      const float2* stat = stats + (s % kSegs) * BM;
      float2 ml = stat[quarter * 32 + lane];
      const int lanes = g.prefix ? a.ws.pre_lanes : a.ws.own_lanes;
      const bool mine = rit < g.rows;
      float4* out = (g.prefix ? a.ws.pre_o : a.ws.own_o) + (int64_t)g.slot * (D / 4) * lanes;
      const int64_t row0 = ((int64_t)g.b * list.hkv + g.kvh) * a.gn + g.rt * BM;  // (whole) of O
      uint16_t* final_o = static_cast<uint16_t*>(a.o) + row0 * D;
      // the copies of a row joined: their common maximum and sum, this copy's weight
      float f = 1.f;
      float* weight = reinterpret_cast<float*>(smem + C::OFF_X) + BM * C::XROW;  // [copy][row]
      if (R > 1) {
        float2 c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = k < R ? stat[k * (BM / R) + rit] : make_float2(-INFINITY, 0.f);
        const float M = fmaxf(fmaxf(c[0].x, c[1].x), fmaxf(c[2].x, c[3].x));
        float l = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) l += c[k].x == -INFINITY ? c[k].y : ex2(c[k].x - M) * c[k].y;  // (NaN scores: m = -inf, l = NaN)
        f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - M);
        ml = make_float2(M, l);
      }
      if (g.whole && !(ml.y == 0.f)) f *= 1.f / ml.y;
      float* xs = reinterpret_cast<float*>(smem + C::OFF_X);
      const int copies = R * g.rows;  // rows of the exchange, which takes 128 of 32 columns: 128 / copies pieces of the rows at a time
      const int pieces = R == 1 ? D / 32 : BM / copies;
#pragma unroll 1
      for (int c = 0, at = 0; c < D / 32; ++c) {
        if (R > 1 && at == 0) named_bar_sync(kDrainBarrier, 128);  // what was exchanged before has been read
        uint32_t r[32];
        tmem_ld32(tmem_addr(tbase, lane_base, C::O_COL + c * 32), r);
        tmem_wait_ld();
        reg_fence(r);
        if (R == 1 && g.whole && ml.y == 0.f) {  // a row that sees nothing: 0, also where V is not finite (0 x NaN)
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0u;
        }
        if (c == D / 32 - 1) {  // all of O is in registers or gone: the next segment may overwrite it
          tc_fence_before();
          mbar_arrive(o_empty);
        }
        if (R == 1) {
          if (mine && g.whole) {
            uint4* dst = reinterpret_cast<uint4*>(final_o + rit * D + c * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t pk[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                pk[k] = pack2<BF16>(__uint_as_float(r[8 * i + 2 * k]) * f, __uint_as_float(r[8 * i + 2 * k + 1]) * f);
              dst[i] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          } else if (mine) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              out[(c * 8 + i) * lanes + rit] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                                           __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
          }
        } else if constexpr (D < 256) {
          if (mine) {
            float4* to = reinterpret_cast<float4*>(xs + (at * copies + cp * g.rows + rit) * C::XROW);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              to[i] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]), __uint_as_float(r[4 * i + 2]),
                                  __uint_as_float(r[4 * i + 3]));
            if (at == 0) weight[cp * g.rows + rit] = f;
          }
          if (++at < pieces && c < D / 32 - 1) continue;
          named_bar_sync(kDrainBarrier, 128);
          const int first = c + 1 - at;
#pragma unroll 1
          for (int e = quarter * 32 + lane; e < g.rows * 8 * at; e += 128) {
            const int i = e & 7, pr = e >> 3, piece = pr / g.rows, row = pr - piece * g.rows;
            const float* from = xs + (piece * copies + row) * C::XROW + 4 * i;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k < R) {
                const float fk = weight[k * g.rows + row];
                const float4 x = *reinterpret_cast<const float4*>(from + k * g.rows * C::XROW);
                if (fk != 0.f)  // (not a copy that saw nothing)
                  sum.x = fmaf(fk, x.x, sum.x), sum.y = fmaf(fk, x.y, sum.y), sum.z = fmaf(fk, x.z, sum.z), sum.w = fmaf(fk, x.w, sum.w);
              }
            }
            const int col = (first + piece) * 8 + i;
            if (g.whole)
              *reinterpret_cast<uint2*>(final_o + row * D + 4 * col) = make_uint2(pack2<BF16>(sum.x, sum.y), pack2<BF16>(sum.z, sum.w));
            else
              out[col * lanes + row] = sum;
          }
          at = 0;
        }
      }
      if (mine && cp == 0) {
        if (g.whole) a.lse[row0 + rit] = ml.y == 0.f ? -INFINITY : (ml.x + log2f(ml.y)) * kLn2;
        else (g.prefix ? a.ws.pre_ml : a.ws.own_ml)[(int64_t)g.slot * lanes + rit] = ml;
      }
      if (a.counter && quarter == 0 && lane == 0) atomicAdd(a.counter, (unsigned long long)g.nt);
      return true;
    };
    // The four warps meet at named barriers, which no limit of time ends: whether there is a segment, and whether its O came,
    // they decide together (a reducing barrier), and between that and their last barrier nothing waits for anything else.
    // (What runs once a segment is kept short: its instructions come from L2 or memory, and unrolled over all columns they
    // cost more than a short segment.)
    Seg g{}, next{};  // the segment whose O is due, the one behind it
    auto advance = [&](int s) {
      next = read_seg(s, ok);
      if (ok && next.rows > 0) load_q(next, s);
    };
    for (int s = -1; start_ok; ++s, g = next) {
      if (s >= 0 && !named_bar_and(kDrainBarrier, 128, ok && g.rows > 0)) break;
      if constexpr (C::QBUFS == 2) {  // the S that read this Q buffer are those of the segment before, whose O was final
        advance(s + 1);
        if (s >= 0 && !store_o(g, s)) break;
      } else {
        if (s >= 0 && !store_o(g, s)) break;
        advance(s + 1);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Joins the segments of rows that have several: O = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s, L = (M + log2 of the latter) ln 2, in
// the list's order; rows that see nothing get O = 0, L = -inf; rows with one segment are finished.  A warp takes a row (or
// several one after the other, where there are many): a lane four columns (at d = 64 half a warp every second partial
// result, at d = 256 a lane eight columns), kAhead partial results in flight.  Against a block a row with four results side by
// side: 124 against 130 us for 2,048 rows behind a prefix, the same for few rows.  (Held to 80 registers, so that blocks stand beside the
// first launch's CTAs and wait there, they slow those down: 44 against 39 us for 768 rows, 126 against 124.)
template <int D, bool BF16>
__global__ void __launch_bounds__(kFinishThreads)
    decode_cache_finish(const __grid_constant__ CacheParams a, int grid, int rows, int rows_per_warp) {
  constexpr int WARPS = kFinishThreads / 32, CH = D / 4;
  constexpr int WAYS = CH < 32 ? 32 / CH : 1, PER = CH > 32 ? CH / 32 : 1;  // results side by side, float4 columns of a lane
  constexpr int AHEAD = kAhead / PER;
  __shared__ int64_t part[2][WARPS];
  __shared__ int slot_list[WARPS][kListed];
  const List& list = a.list;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = lane % (CH < 32 ? CH : 32), way = lane / (CH < 32 ? CH : 32);
  int* slots = slot_list[warp];
  const int first = ((int)blockIdx.x * WARPS + warp) * rows_per_warp, end = min(rows, first + rows_per_warp);
  const int b_block = (int)blockIdx.x * WARPS * rows_per_warp / a.gn / list.hkv;  // sequence of the block's first row
  int64_t total = 0, own_off = 0;
  Prefix pre{};
  // The list of few sequences is looked at again here, before the wait for the kernel that wrote it down.
  const bool alone = list.b <= kFewSequences;
  if (alone) {
    int64_t all = 0, before = 0;
    for (int s = threadIdx.x; s < list.b; s += kFinishThreads) {
      const int64_t x = list.own_total(s);
      all += x;
      if (s < b_block) before += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if (lane == 0) part[0][warp] = all, part[1][warp] = before;
    __syncthreads();
    all = before = 0;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) all += part[0][k], before += part[1][k];
    if (list.p > 0) pre.set(list, all, grid);
    total = pre.total() + all;
    own_off = pre.total() + before;
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    total = a.ws.offsets[list.b];
    if (list.p > 0) pre.set(list, a.ws.offsets[list.b + 1], grid);
  }
  const int runs = runs_of(total, grid);
  bool waited = !alone;
  int b_at = b_block;  // (alone) own_off is this sequence's offset
  for (int row = first; row < end; ++row) {
    const int bh = row / a.gn;  // sequence and key/value head
    const int w = row - bh * a.gn;
    const int b = bh / list.hkv, kvh = bh - b * list.hkv;
    if (alone) {
      for (; b_at < b; ++b_at) own_off += list.own_total(b_at);
    } else {
      own_off = a.ws.offsets[b];
    }
    // The segments of an entry: CTAs c0 to c1 have one each, in slots from the entry's number + c0 on; those of the prefix'
    // pieces come first, in their order.
    const int rt = (b * a.gn + w) / BM;
    int n_pre = 0;
    auto list_slots = [&](int base) {  // slots of the prefix' partial results base .. base + kListed - 1; how many there are in all
      int n = 0;
      for (int x0 = 0; x0 < pre.pieces; x0 += 32) {
        const int x = x0 + lane, e = (kvh * pre.pieces + x) * list.rt_pre + rt;
        int c0 = 0, mine = 0;
        if (x < pre.pieces) {
          const int64_t off = e * pre.cost() + kSegCost;
          c0 = run_of(total, off, runs);
          mine = run_of(total, off + pre.tiles_of(x) - 1, runs) - c0 + 1;
        }
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        for (int k = 0; k < mine; ++k) {
          const int i = n + upto - mine + k - base;
          if (i >= 0 && i < kListed) slots[i] = e + c0 + k;
        }
        n += __shfl_sync(0xffffffffu, upto, 31);
      }
      __syncwarp();
      return n;
    };
    if (list.p > 0) n_pre = list_slots(0);
    int own_n = 0, own_slot = 0;
    const int tiles = list.keys(list.len_of(b)).tiles;
    if (tiles > 0) {
      const int e = kvh * list.rt_own + w / BM;
      const int64_t off = own_off + e * List::cost(tiles) + kSegCost;
      const int c0 = run_of(total, off, runs);
      own_n = run_of(total, off + tiles - 1, runs) - c0 + 1;
      own_slot = b * list.hkv * list.rt_own + e + c0;
    }
    if (!waited) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      waited = true;
    }
    const int n = n_pre + own_n;  // partial results
    if (n == 1 && list.p == 0) continue;
    const int pre_at = (b * a.gn + w) % BM, own_at = w % BM;
    float M = -INFINITY, l = 0.f;
    float4 acc[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = 0; base < n; base += 32) {
      // (the list holds kListed slots of the prefix)
      if (base > 0 && base % kListed == 0 && base < n_pre) {
        __syncwarp();
        list_slots(base);
      }
      const int m = min(32, n - base);
      auto o_at = [&](int i) {  // O of result base + i, this lane's first column
        i += base;
        const bool own = i >= n_pre;
        const int64_t slot = own ? own_slot + i - n_pre : slots[i % kListed];
        const int lanes = own ? a.ws.own_lanes : a.ws.pre_lanes;
        return (own ? a.ws.own_o : a.ws.pre_o) + (slot * CH + col) * lanes + (own ? own_at : pre_at);
      };
      // the first results' O on the way while the statistics of all come
      float4 x[AHEAD][PER];
      auto load = [&](int i0) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          const int i = i0 + j * WAYS + way;
          if (i < m) {
            const float4* o = o_at(i);
            const int lanes = base + i >= n_pre ? a.ws.own_lanes : a.ws.pre_lanes;
#pragma unroll
            for (int k = 0; k < PER; ++k) x[j][k] = o[(int64_t)32 * k * lanes];
          }
        }
      };
      load(0);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < m) {
        const int i = base + lane;
        const bool own = i >= n_pre;
        const int64_t slot = own ? own_slot + i - n_pre : slots[i % kListed];
        ml = own ? a.ws.own_ml[slot * a.ws.own_lanes + own_at] : a.ws.pre_ml[slot * a.ws.pre_lanes + pre_at];
      }
      float top = fmaxf(M, ml.x);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
      const float old = M == -INFINITY ? 1.f : ex2(M - top);  // (nothing yet: sums of 0, or of NaN)
      M = top;
      // what saw nothing (m = -inf, l = 0) is left out, whatever its O holds; a row of NaN scores has m = -inf and l = NaN
      const unsigned there = __ballot_sync(0xffffffffu, ml.x != -INFINITY || !(ml.y == 0.f));
      const float f = ml.x == -INFINITY ? 1.f : ex2(ml.x - top);
      float add = f * ml.y;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) add += __shfl_xor_sync(0xffffffffu, add, s);
      l = l * old + add;
#pragma unroll
      for (int k = 0; k < PER; ++k) acc[k].x *= old, acc[k].y *= old, acc[k].z *= old, acc[k].w *= old;
      for (int i0 = 0; i0 < m; i0 += AHEAD * WAYS) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          const int i = i0 + j * WAYS + way;
          const float fi = __shfl_sync(0xffffffffu, f, i & 31);
          if (i < m && ((there >> i) & 1)) {
#pragma unroll
            for (int k = 0; k < PER; ++k)
              acc[k].x = fmaf(fi, x[j][k].x, acc[k].x), acc[k].y = fmaf(fi, x[j][k].y, acc[k].y),
              acc[k].z = fmaf(fi, x[j][k].z, acc[k].z), acc[k].w = fmaf(fi, x[j][k].w, acc[k].w);
          }
        }
      }
    }
    if constexpr (WAYS == 2) {
      acc[0].x += __shfl_xor_sync(0xffffffffu, acc[0].x, 16), acc[0].y += __shfl_xor_sync(0xffffffffu, acc[0].y, 16);
      acc[0].z += __shfl_xor_sync(0xffffffffu, acc[0].z, 16), acc[0].w += __shfl_xor_sync(0xffffffffu, acc[0].w, 16);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;  // (nothing visible: O = 0)
    uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + (int64_t)row * D);
    if (way == 0) {
#pragma unroll
      for (int k = 0; k < PER; ++k)
        dst[col + 32 * k] = make_uint2(pack2<BF16>(acc[k].x * inv, acc[k].y * inv), pack2<BF16>(acc[k].z * inv, acc[k].w * inv));
    }
    if (lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
    __syncwarp();  // (the next row's slots)
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D, bool BF16>
cudaError_t launch_d(const CacheDecodeArgs& a) {
  using C = CacheCfg<D>;
  const int grid = cache_grid();
  const Shape shape(a.b, a.h, a.hkv, a.nq, a.p, D, grid);
  CacheParams p{};
  p.q = a.q;
  p.o = a.o;
  p.lse = a.lse;
  p.list = List{a.lens, a.b, a.hkv, a.nq, a.capacity, a.p, D == 256 ? 6 : 7, shape.rt_own, shape.rt_pre, a.window, a.window > 0 ? a.sinks : 0};
  p.ws = shape.carve(a.ws, D);
  p.gn = shape.gn;
  p.r_own = shape.r_own;
  p.r_pre = shape.r_pre;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.err = a.err;
  p.counter = a.counter;
  CUtensorMap tk, tv, tk16, tv16, tkp, tvp, tkp16, tvp16;
  const uint64_t heads = (uint64_t)a.b * a.hkv;
  if (!make_tmap_16bit_3d(&tk, a.k, BF16, D, a.capacity, heads, C::BN) ||
      !make_tmap_16bit_3d(&tv, a.v, BF16, D, a.capacity, heads, C::BN) ||
      !make_tmap_16bit_3d(&tk16, a.k, BF16, D, a.capacity, heads, kLoadRows) ||
      !make_tmap_16bit_3d(&tv16, a.v, BF16, D, a.capacity, heads, kLoadRows))
    return cudaErrorInvalidValue;
  tkp = tk, tvp = tv, tkp16 = tk16, tvp16 = tv16;
  if (a.p > 0 && (!make_tmap_16bit_3d(&tkp, a.kp, BF16, D, a.p, a.hkv, C::BN) ||
                  !make_tmap_16bit_3d(&tvp, a.vp, BF16, D, a.p, a.hkv, C::BN) ||
                  !make_tmap_16bit_3d(&tkp16, a.kp, BF16, D, a.p, a.hkv, kLoadRows) ||
                  !make_tmap_16bit_3d(&tvp16, a.vp, BF16, D, a.p, a.hkv, kLoadRows)))
    return cudaErrorInvalidValue;
  auto kern = decode_cache_kernel<D, BF16>;
  static std::atomic<unsigned long long> allowed;
  cudaError_t e = allow_smem(kern, C::SMEM, &allowed);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::THREADS, C::SMEM, a.stream>>>(p, tk, tv, tk16, tv16, tkp, tvp, tkp16, tvp16);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // launched while the runs are still going (it waits for them before it reads what they write)
  // (several rows a warp only where single ones would be many more warps than the GPU holds)
  const int rows = a.b * a.h * a.nq, per_warp = std::max(1, std::min(16, rows / (grid * 64)));
  const int per_block = per_warp * (kFinishThreads / 32);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((rows + per_block - 1) / per_block));
  cfg.blockDim = dim3(kFinishThreads);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_cache_finish<D, BF16>, p, grid, rows, per_warp);
}

}  // namespace

size_t decode_cache_workspace_bytes(int b, int h, int hkv, int nq, int p, int d) {
  return Shape(b, h, hkv, nq, p, d, cache_grid()).bytes(b, d);
}

cudaError_t launch_decode_cache(const CacheDecodeArgs& a) {
  const bool bf = a.dtype == DT_BF16;
  switch (a.d) {
    case 64: return bf ? launch_d<64, true>(a) : launch_d<64, false>(a);
    case 128: return bf ? launch_d<128, true>(a) : launch_d<128, false>(a);
    case 256: return bf ? launch_d<256, true>(a) : launch_d<256, false>(a);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace fa
