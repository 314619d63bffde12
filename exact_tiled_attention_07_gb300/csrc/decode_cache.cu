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
// The joining of segments (O and row statistics of each, unnormalised, in the workspace) is a second launch,
// decode_cache_finish.  Slots need no bookkeeping: along the list each new segment has either the next entry or the next CTA, so
// entry + CTA numbers them.
//
// A CTA is a chain of warps that run ahead of one another across segments:
//   producer  walks the list, publishes segments in a ring, loads K and V tiles into a ring that takes the shared memory;
//   MMA warp  S = Q K^T (Q in TMEM) two tiles ahead of O += P V (P in TMEM, over S), also across the end of a segment;
//   softmax   (4 warps, a thread a row) as in the forward kernel: exp2, lazy rescaling by 2^8.  With 32 rows or fewer
//             the rows stand in all four lane quarters and each takes a quarter of the tile's columns, as if they were
//             other pieces of the keys (two halves for up to 64 rows);
//   drain     (4 warps) the next segment's Q into TMEM, a finished segment's O out of it, so that the softmax goes on
//             with the next segment's scores meanwhile.
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
constexpr int kSegCost = 2;     // what a segment's start and end cost, in tiles
constexpr int kSegs = 4;        // published segments, and row statistics, in flight
constexpr int kFinishThreads = 256;

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
  static constexpr int SMEM = OFF_RED + 16 * 8;
  static_assert(STAGES >= 4, "the products run two tiles ahead");
  static_assert(SMEM <= 232448 && OFF_SEG % 8 == 0 && OFF_STAT % 8 == 0 && OFF_RED % 8 == 0, "shared memory");
};

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
};
static_assert(sizeof(Seg) <= 64, "Seg");

// The list of tiles.  Offsets count tiles and kSegCost for each entry.
struct List {
  const int32_t* lens;
  int b, hkv, nq, capacity, p, bn;
  int rt_own, rt_pre;  // row tiles of a sequence's head, of the prefix' head
  int window, sinks;

  // keys of a sequence: sinks [0, sk), the rest [lo, len)
  struct Keys {
    int len, lo, sk, ns, tiles;
  };
  __host__ __device__ Keys keys(int len) const {
    Keys k;
    k.len = len;
    k.lo = 0;
    if (window > 0) {
      const int64_t lo = (int64_t)len - nq + 1 - window;  // the first row's
      k.lo = lo > 0 ? (int)lo : 0;
    }
    k.sk = sinks < k.lo ? sinks : k.lo;
    k.ns = (k.sk + bn - 1) / bn;
    k.tiles = k.ns + (int)(((int64_t)len - k.lo + bn - 1) / bn);
    return k;
  }
  __device__ int len_of(int s) const { return min(max(lens[s], 0), capacity); }
  __host__ __device__ static int64_t cost(int tiles) { return tiles > 0 ? tiles + kSegCost : 0; }
  __host__ __device__ int prefix_tiles() const { return (int)(((int64_t)p + bn - 1) / bn); }
  __host__ __device__ int prefix_entries() const { return p > 0 ? hkv * rt_pre : 0; }
  __host__ __device__ int64_t prefix_total() const { return prefix_entries() * cost(prefix_tiles()); }
  __device__ int64_t own_total(int s) const { return (int64_t)hkv * rt_own * cost(keys(len_of(s)).tiles); }
};
// CTA c of n takes [start(c), start(c + 1)) of a list.
__device__ __forceinline__ int64_t run_start(int64_t total, int c, int n) { return total * c / n; }
__device__ __forceinline__ int run_of(int64_t total, int64_t at, int n) { return (int)(((at + 1) * n - 1) / total); }
__device__ __forceinline__ int runs_of(int64_t total, int grid) { return total < grid ? (int)total : grid; }

// Partial results: for the prefix' segments, then the caches', [slots][D / 4][lanes] float4 and [slots][lanes] (m, l); then the
// lists' offset of each sequence.  A lane is a row, or one of a row's copies.
struct Partials {
  float4 *pre_o, *own_o;
  float2 *pre_ml, *own_ml;
  int64_t* offsets;  // [b + 1]: of each sequence's first entry, then the total
  int pre_lanes, own_lanes;
};

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
    own_lanes = r_own * std::min(gn, BM);
    pre_lanes = r_pre * (int)std::min<int64_t>(all, BM);
    pre_slots = p > 0 ? (int64_t)hkv * rt_pre + grid : 0;
    own_slots = (int64_t)b * hkv * rt_own + grid;
  }
  size_t bytes(int b, int d) const {
    const size_t lanes = (size_t)pre_slots * pre_lanes + (size_t)own_slots * own_lanes;
    return lanes * ((size_t)d * 4 + 8) + ((size_t)b + 2) * 8 + 64;
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
  List list;
  Partials ws;
  int h, gn;
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
  int64_t total = list.prefix_total();
#pragma unroll
  for (int w = 0; w < C::THREADS / 32; ++w) total += red[w];
  if (blockIdx.x == 0 && warp == C::DRAIN_WARP0) {
    int64_t at = list.prefix_total();
    for (int s0 = 0; s0 < list.b; s0 += 32) {
      int64_t v = s0 + lane < list.b ? list.own_total(s0 + lane) : 0;
      const int64_t mine = v;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (s0 + lane < list.b) a.ws.offsets[s0 + lane] = at + v - mine;
      at += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) a.ws.offsets[list.b] = total;
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
      const int64_t pre_total = list.prefix_total();
      // the sequence that the run begins in (the whole warp), and its offset
      int b = 0;
      int64_t b_off = pre_total;
      if (u1 > pre_total) {
        const int64_t from = max(u0, pre_total);
        for (int s0 = 0; s0 < list.b; s0 += 32) {
          int64_t v = s0 + lane < list.b ? list.own_total(s0 + lane) : 0;
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
          }
          const unsigned past = __ballot_sync(0xffffffffu, b_off + v > from);
          if (past) {
            const int f = __ffs(past) - 1;
            b = s0 + f;
            if (f > 0) b_off += __shfl_sync(0xffffffffu, v, f - 1);
            break;
          }
          b_off += __shfl_sync(0xffffffffu, v, 31);
        }
      }
      if (lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        int n_segs = 0;
        uint32_t pos = 0;  // loads issued
        bool ok = true;
        auto publish = [&](const Seg& g) {
          const int at = n_segs % kSegs;
          if (n_segs >= kSegs && !mbar_wait(seg_empty + at, (uint32_t)(n_segs / kSegs - 1) & 1, ctx, 411)) return false;
          volatile int* to = reinterpret_cast<volatile int*>(segs + at);
          const int* from = reinterpret_cast<const int*>(&g);
#pragma unroll
          for (int i = 0; i < (int)(sizeof(Seg) / 4); ++i) to[i] = from[i];
          mbar_arrive(seg_full + at);
          ++n_segs;
          return true;
        };
        int64_t u = u0;
        List::Keys keys = list.keys(b < list.b ? list.len_of(b) : 0);
        while (ok && u < u1) {
          // the entry at u: its offset, tiles and rows
          Seg g;
          int64_t off;
          int tiles;
          if (u < pre_total) {
            const int64_t c = List::cost(list.prefix_tiles());
            const int e = (int)(u / c);
            off = e * c;
            tiles = list.prefix_tiles();
            g.prefix = 1;
            g.kvh = e / list.rt_pre;
            g.rt = e - g.kvh * list.rt_pre;
            g.b = 0;
            g.head = g.kvh;
            g.rows = min(BM, list.b * a.gn - g.rt * BM);
            g.ns = g.sk = g.lo = 0;
            g.end = list.p;
            g.slot = e + (int)blockIdx.x;
          } else {
            const int entries = list.hkv * list.rt_own;
            while (b < list.b && u >= b_off + entries * List::cost(keys.tiles)) {
              b_off += entries * List::cost(keys.tiles);
              ++b;
              keys = list.keys(b < list.b ? list.len_of(b) : 0);
            }
            if (b >= list.b) break;
            const int64_t c = List::cost(keys.tiles);
            const int e = (int)((u - b_off) / c);
            off = b_off + e * c;
            tiles = keys.tiles;
            g.prefix = 0;
            g.b = b;
            g.kvh = e / list.rt_own;
            g.rt = e - g.kvh * list.rt_own;
            g.head = b * list.hkv + g.kvh;
            g.rows = min(BM, a.gn - g.rt * BM);
            g.ns = keys.ns;
            g.sk = keys.sk;
            g.lo = keys.lo;
            g.end = keys.len;
            g.slot = b * entries + e + (int)blockIdx.x;
          }
          // its tiles in this run
          g.t0 = (int)max((int64_t)0, u - off - kSegCost);
          const int t1 = (int)min((int64_t)tiles, u1 - off - kSegCost);
          g.nt = t1 - g.t0;
          u = min(u1, off + tiles + kSegCost);
          if (g.nt <= 0) continue;
          if (!(ok = publish(g))) break;
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
        if (n < BN) {
          // V rows behind the segment's keys (another sequence's, or what the place held before): zero, since 0 x NaN is NaN
          uint8_t* vt = smem + slot * C::TILE_BYTES;
          for (int x = n * 8 + lane; x < BN * 8; x += 32)
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
            umma_ts(tbase + C::O_COL, tbase + p_col + kk * 8, bd[kk], idesc_pv, (first < 0 || kk > 0) ? 1u : 0u);
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
          lo = max(0, hi - list.window);
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
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 u = rit < g.rows ? from[c * 8 + i] : make_uint4(0u, 0u, 0u, 0u);
          w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
        tmem_st32(tmem_addr(tbase, lane_base, q_col + c * 32), w);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(q_full + (C::QBUFS == 2 ? (s & 1) : 0));
    };
    if (ok) {
      Seg g = read_seg(0, ok);
      if (g.rows > 0) load_q(g, 0);
      for (int s = 0; ok && g.rows > 0; ++s) {
        // (with two Q buffers the S that read this one are those of the segment before, whose O was final)
        Seg next{};
        if (C::QBUFS == 2) {
          next = read_seg(s + 1, ok);
          if (ok && next.rows > 0) load_q(next, s + 1);
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(o_full, s & 1, ctx, 440));
        ok = ok && __all_sync(0xffffffffu, mbar_wait(stat_full + s % kSegs, (uint32_t)(s / kSegs) & 1, ctx, 441));
        if (!ok) break;
        tc_fence_after();
        int cp, rit;
        const int R = g.prefix ? a.r_pre : a.r_own;
        lane_row(R, quarter, lane, &cp, &rit);
        const float2 ml = stats[(s % kSegs) * BM + quarter * 32 + lane];
        const int lanes = g.prefix ? a.ws.pre_lanes : a.ws.own_lanes;
        const int to = cp * (lanes / R) + rit;
        const bool mine = rit < g.rows;
        const bool any = (quarter % (4 / R)) * 32 < g.rows;
        float4* out = (g.prefix ? a.ws.pre_o : a.ws.own_o) + (int64_t)g.slot * (D / 4) * lanes + to;
        constexpr int HALF = D == 256 ? 128 : D;  // columns held in registers at a time
#pragma unroll 1
        for (int h = 0; h < D / HALF; ++h) {
          uint32_t r[HALF / 32][32];
          if (any) {
#pragma unroll
            for (int c = 0; c < HALF / 32; ++c) tmem_ld32(tmem_addr(tbase, lane_base, C::O_COL + h * HALF + c * 32), r[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < HALF / 32; ++c) reg_fence(r[c]);
          }
          if (h == D / HALF - 1) {  // O is in registers: the next segment may overwrite it
            tc_fence_before();
            mbar_arrive(o_empty);
          }
          if (mine) {
#pragma unroll
            for (int c = 0; c < HALF / 4; ++c)
              out[(int64_t)(h * (HALF / 4) + c) * lanes] =
                  make_float4(__uint_as_float(r[c / 8][c % 8 * 4]), __uint_as_float(r[c / 8][c % 8 * 4 + 1]),
                              __uint_as_float(r[c / 8][c % 8 * 4 + 2]), __uint_as_float(r[c / 8][c % 8 * 4 + 3]));
          }
        }
        if (mine) (g.prefix ? a.ws.pre_ml : a.ws.own_ml)[(int64_t)g.slot * lanes + to] = ml;
        if (a.counter && quarter == 0 && lane == 0) atomicAdd(a.counter, (unsigned long long)g.nt);
        if (C::QBUFS == 1) {
          next = read_seg(s + 1, ok);
          if (ok && next.rows > 0) load_q(next, s + 1);
        }
        g = next;
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

// Joins the segments of each row: O = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s, L = (M + log2 of the latter) ln 2, in the list's
// order.  A warp takes a row; a lane its columns, four at a time.
template <int D, bool BF16>
__global__ void __launch_bounds__(kFinishThreads)
    decode_cache_finish(const __grid_constant__ CacheParams a, void* __restrict__ out, float* __restrict__ lse, int64_t rows, int grid) {
  const List& list = a.list;
  const int lane = threadIdx.x & 31;
  const int64_t row = ((int64_t)blockIdx.x * kFinishThreads + threadIdx.x) >> 5;
  const int64_t bh = row / a.gn;  // sequence and key/value head
  const int w = (int)(row - bh * a.gn);
  const int b = (int)(bh / list.hkv), kvh = (int)(bh - (int64_t)b * list.hkv);
  const bool valid = row < rows;
  const int tiles = valid ? list.keys(list.len_of(b)).tiles : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!valid) return;
  const int64_t total = a.ws.offsets[list.b];
  const int runs = runs_of(total, grid);
  // the segments of an entry: CTAs [c0, c0 + n) have one each, in slots from first + c0 on
  struct Part {
    const float4* o;
    const float2* ml;
    int n, lanes, copies, lane;
  } part[2];
  auto entry = [&](int64_t e, int64_t off, int t, const float4* o, const float2* ml, int lanes, int copies, int r) {
    Part x;
    const int c0 = run_of(total, off + kSegCost, runs), c1 = run_of(total, off + kSegCost + t - 1, runs);
    x.n = c1 - c0 + 1;
    x.lanes = lanes;
    x.copies = copies;
    x.lane = r;
    x.o = o + (e + c0) * (D / 4) * lanes;
    x.ml = ml + (e + c0) * lanes;
    return x;
  };
  part[0].n = part[1].n = 0;
  part[0].copies = part[1].copies = 1;
  if (list.p > 0) {
    const int64_t r = (int64_t)b * a.gn + w;
    const int rt = (int)(r / BM);
    const int64_t e = (int64_t)kvh * list.rt_pre + rt;
    part[0] = entry(e, e * List::cost(list.prefix_tiles()), list.prefix_tiles(), a.ws.pre_o, a.ws.pre_ml, a.ws.pre_lanes, a.r_pre,
                    (int)(r % BM));
  }
  if (tiles > 0) {
    const int64_t e = (int64_t)kvh * list.rt_own + w / BM;
    part[1] = entry((int64_t)b * list.hkv * list.rt_own + e, a.ws.offsets[b] + e * List::cost(tiles), tiles, a.ws.own_o,
                    a.ws.own_ml, a.ws.own_lanes, a.r_own, w % BM);
  }
  const int n0 = part[0].n * part[0].copies, n = n0 + part[1].n * part[1].copies;  // partial results
  auto place = [&](int i, const float4** o, int* lanes) {
    const Part& x = i < n0 ? part[0] : part[1];
    if (i >= n0) i -= n0;
    const int seg = i / x.copies, at = (i - seg * x.copies) * (x.lanes / x.copies) + x.lane;
    *o = x.o + (int64_t)seg * (D / 4) * x.lanes + at;
    *lanes = x.lanes;
    return x.ml + (int64_t)seg * x.lanes + at;
  };
  constexpr int CH = D / 4;                          // float4 columns of a row
  constexpr int PER = CH > 32 ? CH / 32 : 1;         // of a lane
  constexpr int WAYS = CH < 32 ? 32 / CH : 1;        // partial results side by side (d = 64)
  const int col = lane % (CH < 32 ? CH : 32), way = lane / (CH < 32 ? CH : 32);
  float M = -INFINITY, l = 0.f;
  float4 acc[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += 32) {
    // 32 results' statistics at once, then their O
    const float4* o = nullptr;
    int lanes = 0;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (i0 + lane < n) ml = *place(i0 + lane, &o, &lanes);
    float mx = ml.x;
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    const float top = fmaxf(M, mx);
    const float old = M == -INFINITY ? 0.f : ex2(M - top);
    M = top;
    // (a row of NaN scores has m = -inf and l = NaN)
    const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - top);
    const bool there = ml.x != -INFINITY || ml.y != 0.f;
    l *= old;
    float add = there ? f * ml.y : 0.f;
    for (int s = 16; s > 0; s >>= 1) add += __shfl_xor_sync(0xffffffffu, add, s);
    l += add;
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[k].x *= old, acc[k].y *= old, acc[k].z *= old, acc[k].w *= old;
    const unsigned present = __ballot_sync(0xffffffffu, there);
    const int m = min(32, n - i0);
#pragma unroll 4
    for (int i = 0; i < m; i += WAYS) {
      const int mine = i + way;
      const float fi = __shfl_sync(0xffffffffu, f, mine & 31);
      if (mine < m && ((present >> mine) & 1)) {
        place(i0 + mine, &o, &lanes);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const float4 x = o[(int64_t)(col + 32 * k) * lanes];
          acc[k].x = fmaf(fi, x.x, acc[k].x), acc[k].y = fmaf(fi, x.y, acc[k].y);
          acc[k].z = fmaf(fi, x.z, acc[k].z), acc[k].w = fmaf(fi, x.w, acc[k].w);
        }
      }
    }
  }
  if constexpr (WAYS > 1) {
    acc[0].x += __shfl_xor_sync(0xffffffffu, acc[0].x, 16), acc[0].y += __shfl_xor_sync(0xffffffffu, acc[0].y, 16);
    acc[0].z += __shfl_xor_sync(0xffffffffu, acc[0].z, 16), acc[0].w += __shfl_xor_sync(0xffffffffu, acc[0].w, 16);
  }
  static_assert(WAYS <= 2, "two results side by side");
  const float inv = l == 0.f ? 0.f : 1.f / l;  // (nothing visible: O = 0)
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + row * D);
  if (way == 0) {
#pragma unroll
    for (int k = 0; k < PER; ++k)
      dst[col + 32 * k] = make_uint2(pack2<BF16>(acc[k].x * inv, acc[k].y * inv), pack2<BF16>(acc[k].z * inv, acc[k].w * inv));
  }
  if (lane == 0) lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

template <int D, bool BF16>
cudaError_t launch_d(const CacheDecodeArgs& a) {
  using C = CacheCfg<D>;
  const int grid = device_sm_count();
  const Shape shape(a.b, a.h, a.hkv, a.nq, a.p, D, grid);
  CacheParams p{};
  p.q = a.q;
  p.list = List{a.lens, a.b, a.hkv, a.nq, a.capacity, a.p, C::BN, shape.rt_own, shape.rt_pre, a.window, a.window > 0 ? a.sinks : 0};
  p.ws = shape.carve(a.ws, D);
  p.h = a.h;
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
  const int64_t rows = (int64_t)a.b * a.h * a.nq;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((rows * 32 + kFinishThreads - 1) / kFinishThreads));
  cfg.blockDim = dim3(kFinishThreads);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_cache_finish<D, BF16>, p, a.o, a.lse, rows, grid);
}

}  // namespace

size_t decode_cache_workspace_bytes(int b, int h, int hkv, int nq, int p, int d) {
  return Shape(b, h, hkv, nq, p, d, device_sm_count()).bytes(b, d);
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
