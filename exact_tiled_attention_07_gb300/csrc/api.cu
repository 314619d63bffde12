// C ABI (include/fa.h): argument validation, workspace carving, kernel selection.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "fa.h"
#include "kernels.h"
#include "ptx.cuh"

namespace fa {
namespace {

// Device error word written by kernels (see ptx.cuh) and the tile counter.
__device__ unsigned long long g_err_word;
__device__ unsigned long long g_tile_counter;

thread_local char t_msg[512] = "";

fa_status fail(fa_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_msg, sizeof(t_msg), fmt, ap);
  va_end(ap);
  return s;
}

struct DeviceSyms {
  unsigned long long* err = nullptr;
  unsigned long long* counter = nullptr;
  unsigned long long ctx = 0;  // id of the context the addresses belong to
};

constexpr int kMaxDevices = 64;
DeviceSyms g_syms[kMaxDevices];
std::mutex g_syms_mu;

// Device addresses of the file-scope device symbols for the current device, looked up again
// whenever the current context is not the one they were taken in (a device reset destroys the
// primary context, and the next one may place the library's module elsewhere).
fa_status device_syms(DeviceSyms* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(FA_ERR_UNSUPPORTED, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_syms_mu);
  DeviceSyms& s = g_syms[dev];
  const unsigned long long ctx = current_context_id();
  if (!s.err || ctx == 0 || ctx != s.ctx) {
    void* p = nullptr;
    if ((e = cudaGetSymbolAddress(&p, g_err_word)) != cudaSuccess)
      return fail(FA_ERR_CUDA, "cudaGetSymbolAddress(error word): %s", cudaGetErrorString(e));
    void* c = nullptr;
    if ((e = cudaGetSymbolAddress(&c, g_tile_counter)) != cudaSuccess)
      return fail(FA_ERR_CUDA, "cudaGetSymbolAddress(tile counter): %s", cudaGetErrorString(e));
    s.counter = static_cast<unsigned long long*>(c);
    s.err = static_cast<unsigned long long*>(p);
    s.ctx = current_context_id();  // the lookup made the device's context current if none was
  }
  *out = s;
  return FA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shared shape/pointer checks. Returns FA_OK and sets *empty when there is nothing to do.
fa_status check_common(int B, int H, int N, int d, fa_dtype dt, bool* empty) {
  *empty = false;
  if (dt != FA_BF16 && dt != FA_FP16 && dt != FA_FP32) return fail(FA_ERR_UNSUPPORTED, "unknown dtype %d", (int)dt);
  if (B < 0 || H < 0 || N < 0) return fail(FA_ERR_INVALID_ARG, "negative size B=%d H=%d N=%d", B, H, N);
  if (d < 1 || d > 256) return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d outside [1, 256]", d);
  const int64_t bh = (int64_t)B * H;
  if (bh > INT32_MAX) return fail(FA_ERR_INVALID_ARG, "B*H=%lld too large", (long long)bh);
  if ((int64_t)N > (int64_t)INT32_MAX - 128) return fail(FA_ERR_INVALID_ARG, "N=%d too large", N);
  const int64_t npad = padded_rows(N);
  if (bh > 0 && npad > 0 && (double)bh * (double)npad * (double)(d + 2) * 4.0 > 9.0e18)
    return fail(FA_ERR_INVALID_ARG, "problem too large");
  if (bh == 0 || N == 0) *empty = true;
  return FA_OK;
}

fa_status check_ptrs(std::initializer_list<const void*> ptrs, const char* what) {
  int i = 0;
  for (const void* p : ptrs) {
    if (!p) return fail(FA_ERR_INVALID_ARG, "%s: pointer %d is null", what, i);
    if (!aligned16(p)) return fail(FA_ERR_INVALID_ARG, "%s: pointer %d is not 16-byte aligned", what, i);
    ++i;
  }
  return FA_OK;
}

fa_status check_scale(float scale) {
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  return FA_OK;
}

fa_status launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  t_msg[0] = 0;
  return FA_OK;
}

// A 16-bit call that had no tensor-core kernel and ran on the CUDA-core kernels: it succeeded,
// and the calling thread's message says which path ran (nothing changes backend silently).
fa_status note_cuda_core_path(fa_status st, const char* pass, fa_dtype dtype, int d) {
  if (st == FA_OK && dtype != FA_FP32)
    snprintf(t_msg, sizeof(t_msg),
             "notice: the %s %s pass at d=%d ran on the CUDA-core kernels (fp32 arithmetic): no tensor-core "
             "kernel for this head dimension",
             dtype == FA_BF16 ? "bf16" : "fp16", pass, d);
  return st;
}

// after the per-row vectors and the dQ accumulator: the backward's work-item queue counters
constexpr size_t kSchedBytes = 256;

size_t workspace_bytes_for(int B, int H, int N, int d) {
  const size_t bh = (size_t)B * H, npad = (size_t)padded_rows(N);
  return bh * npad * 4 * (2 + (size_t)d) + kSchedBytes;
}

fa_status carve(BwdArgs* a, void* ws, size_t ws_bytes, int B, int H, int N, int d) {
  const size_t need = workspace_bytes_for(B, H, N, d);
  if (ws_bytes < need) return fail(FA_ERR_INVALID_ARG, "workspace of %zu bytes < %zu required", ws_bytes, need);
  const size_t rows = (size_t)B * H * padded_rows(N);
  float* base = static_cast<float*>(ws);
  a->delta = base;
  a->lse2 = base + rows;
  a->dq_acc = base + 2 * rows;
  a->sched = reinterpret_cast<unsigned*>(base + rows * (2 + (size_t)d));
  return FA_OK;
}

// 4-bit cache arguments (include/fa.h).
fa_status check_kv4(int B, int Hkv, int capacity, int d, bool* empty) {
  *empty = false;
  if (B < 0) return fail(FA_ERR_INVALID_ARG, "negative size B=%d", B);
  if (Hkv < 1) return fail(FA_ERR_INVALID_ARG, "Hkv=%d key/value heads: at least one", Hkv);
  if (d != 64 && d != 128 && d != 256)
    return fail(FA_ERR_UNSUPPORTED, "the 4-bit cache supports d in {64, 128, 256}, got %d", d);
  if (capacity < 64 || capacity % 64 != 0)
    return fail(FA_ERR_INVALID_ARG, "capacity=%d is not a positive multiple of 64", capacity);
  // (kernels count slots in 32 bits, up to a block's share of them behind the last)
  if (capacity > INT32_MAX - 4096 || (int64_t)B * Hkv > INT32_MAX / 4 || (int64_t)Hkv * (capacity / 64) > INT32_MAX ||
      (double)B * Hkv * capacity * d > 4.0e15)
    return fail(FA_ERR_INVALID_ARG, "cache too large: B=%d Hkv=%d capacity=%d", B, Hkv, capacity);
  if (B == 0) *empty = true;
  return FA_OK;
}

// Arrays of 32-bit integers or floats that need their natural alignment only.
fa_status check_words(std::initializer_list<const void*> ptrs, const char* what) {
  for (const void* p : ptrs)
    if (!p || (reinterpret_cast<uintptr_t>(p) & 3u) != 0)
      return fail(FA_ERR_INVALID_ARG, "%s: a 32-bit array is null or not 4-byte aligned", what);
  return FA_OK;
}

// Rows that lie over one another cannot all be written: one dimension's rows have to end before the other's next step.
fa_status check_output_rows(int tokens, int64_t token_stride, int heads, int64_t head_stride, int d, const char* what) {
  const int64_t small = std::min(token_stride, head_stride), large = std::max(token_stride, head_stride);
  const int along = token_stride < head_stride ? tokens : heads;  // rows `small` apart
  if (small < d) return fail(FA_ERR_INVALID_ARG, "%s: an output stride of %lld elements < d=%d", what, (long long)small, d);
  if (tokens > 1 && heads > 1 && (double)(along - 1) * (double)small + d > (double)large)
    return fail(FA_ERR_INVALID_ARG, "%s: output rows overlap (strides of %lld and %lld elements)", what,
                (long long)token_stride, (long long)head_stride);
  return FA_OK;
}

struct Bytes {
  const void* p;
  size_t n;
};
bool overlap(const Bytes& a, const Bytes& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}

// Token and head strides of a packed [T][heads][d] tensor: rows may lie apart (a slice of a fused
// projection) but each starts on 16 bytes.
fa_status check_strides(std::initializer_list<int64_t> strides, int elem_bytes, const char* what) {
  for (int64_t s : strides)
    if (s < 0 || s >= ((int64_t)1 << 38) || (s * elem_bytes) % 16 != 0)
      return fail(FA_ERR_INVALID_ARG, "%s: a stride of %lld elements is negative, too large or not a multiple of 16 bytes",
                  what, (long long)s);
  return FA_OK;
}

// A [B][N][heads][d] tensor of rows: where it lies and its strides in elements.
struct RowTensor {
  const char* name;
  const void* p;
  NormRopeStrides st;
  int heads;
};

// Whether rows lie apart: from the smallest stride up, a dimension's rows end before the next one's first step.
bool rows_apart(const NormRopeStrides& st, int64_t heads, int B, int N, int d) {
  struct Dim {
    int64_t stride, n;
  } dims[3] = {{st.batch, B}, {st.token, N}, {st.head, heads}};
  std::sort(dims, dims + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  double extent = d;
  for (const Dim& x : dims) {
    if (x.n <= 1) continue;
    if ((double)x.stride < extent) return false;
    extent += (double)(x.n - 1) * (double)x.stride;
  }
  return true;
}
fa_status check_rows_apart(const RowTensor& t, int B, int N, int d, const char* what) {
  if (!rows_apart(t.st, t.heads, B, N, d))
    return fail(FA_ERR_INVALID_ARG, "%s: rows of %s overlap (strides of %lld, %lld and %lld elements)", what, t.name,
                (long long)t.st.batch, (long long)t.st.token, (long long)t.st.head);
  return FA_OK;
}

// An output and another tensor (of one element size) do not meet if they lie apart in memory, are heads of one tensor, or
// lie side by side inside a token.
bool rows_meet(const RowTensor& a, const RowTensor& b, int B, int N, int d, int eb) {
  auto bytes = [&](const RowTensor& t) {
    return (size_t)((B - 1) * t.st.batch + (N - 1) * t.st.token + (t.heads - 1) * t.st.head + d) * eb;
  };
  if (!overlap({a.p, bytes(a)}, {b.p, bytes(b)})) return false;
  if ((B > 1 && a.st.batch != b.st.batch) || (N > 1 && a.st.token != b.st.token)) return true;
  const bool a_first = reinterpret_cast<uintptr_t>(a.p) <= reinterpret_cast<uintptr_t>(b.p);
  const RowTensor &lo = a_first ? a : b, &hi = a_first ? b : a;
  const int64_t off = (int64_t)((reinterpret_cast<uintptr_t>(hi.p) - reinterpret_cast<uintptr_t>(lo.p)) / eb);
  const int64_t lo_end = (lo.heads - 1) * lo.st.head + d, hi_end = off + (hi.heads - 1) * hi.st.head + d;
  if (off < lo_end) return true;
  // heads of one tensor (the stride of one head alone is open: the other's, or where both are alone what lies between them)
  if (lo.heads == 1 || hi.heads == 1 || lo.st.head == hi.st.head) {
    NormRopeStrides st = lo.st;
    st.head = lo.heads > 1 ? lo.st.head : (hi.heads > 1 ? hi.st.head : off);
    if (st.head > 0 && off % st.head == 0 && off / st.head >= lo.heads && rows_apart(st, off / st.head + hi.heads, B, N, d)) return false;
  }
  // the smaller step of the token and the batch dimension repeats the pattern; the larger one has to leave room for it
  int64_t small = INT64_MAX, large = INT64_MAX;
  int n_small = 1;
  if (N > 1) small = a.st.token, n_small = N;
  if (B > 1 && a.st.batch < small) {
    large = small;
    small = a.st.batch;
    n_small = B;
  } else if (B > 1) {
    large = a.st.batch;
  }
  if (small != INT64_MAX && hi_end > small) return true;
  return large != INT64_MAX && (double)(n_small - 1) * (double)small + hi_end > (double)large;
}
bool same_rows(const RowTensor& a, const RowTensor& b, int B, int N) {
  return a.p == b.p && a.heads == b.heads && (B <= 1 || a.st.batch == b.st.batch) && (N <= 1 || a.st.token == b.st.token) &&
         (a.heads <= 1 || a.st.head == b.st.head);
}

}  // namespace

unsigned long long current_context_id() {
  static PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
  static PFN_cuCtxGetId_v12000 get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 4000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
    p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(p);
  });
  if (!get_current || !get_id) return 0;
  CUcontext c = nullptr;
  if (get_current(&c) != CUDA_SUCCESS || !c) return 0;
  unsigned long long id = 0;
  return get_id(c, &id) == CUDA_SUCCESS ? id : 0;
}

int device_sm_count() {
  static int cached[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return kSmCount;
  if (cached[dev] == 0) {
    int v = 0;
    cached[dev] = (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0) ? v : kSmCount;
  }
  return cached[dev];
}

int set_last_error(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_msg, sizeof(t_msg), fmt, ap);
  va_end(ap);
  return status;
}

}  // namespace fa

using namespace fa;

namespace {

// Query heads H share key/value heads Hkv (H a multiple of Hkv); Hkv == H is plain attention.
fa_status check_heads(int H, int Hkv) {
  if (Hkv < 1 || H % Hkv != 0)
    return fail(FA_ERR_INVALID_ARG, "H=%d query heads must be a positive multiple of Hkv=%d key/value heads", H, Hkv);
  return FA_OK;
}

// Masks beyond causal: a window (keys with |i - j| >= window hidden; 0 = none) and a block
// mask of bytes [mask_heads][nb][nb] over 128 x 128 score blocks (NULL = none).
struct MaskSpec {
  int window = 0;
  const uint8_t* block_mask = nullptr;
  int mask_heads = 0;
  bool band = false;  // causal with `window` and the first `sinks` keys always visible
  int sinks = 0;
  bool any() const { return window > 0 || block_mask != nullptr; }
};

fa_status check_band(int window, int sinks, const char* what) {
  if (window < 1) return fail(FA_ERR_INVALID_ARG, "%s: window must be >= 1, got %d", what, window);
  if (sinks < 0) return fail(FA_ERR_INVALID_ARG, "%s: sinks must be >= 0, got %d", what, sinks);
  return FA_OK;
}

fa_status check_mask(const MaskSpec& m, int H, int Hkv, int N, int d, fa_dtype dtype, bool backward) {
  if (m.window < 0) return fail(FA_ERR_INVALID_ARG, "window must be >= 0 (0: none), got %d", m.window);
  if (m.block_mask) {
    if (m.mask_heads != 1 && m.mask_heads != H)
      return fail(FA_ERR_INVALID_ARG, "mask_heads must be 1 or H=%d, got %d", H, m.mask_heads);
  } else if (m.mask_heads != 0) {
    return fail(FA_ERR_INVALID_ARG, "mask_heads=%d without a block mask (must be 0)", m.mask_heads);
  }
  if (m.band) {
    const fa_status st = check_band(m.window, m.sinks, backward ? "fa_bwd_window" : "fa_fwd_window");
    if (st != FA_OK) return st;
    if (!fwd_tc_supported((int)dtype, d))
      return fail(FA_ERR_UNSUPPORTED, "windows with sinks run on the tensor-core kernels (bf16/fp16, d in {64, 128, 256})");
    return FA_OK;
  }
  if (!m.any()) return FA_OK;
  const bool tc = backward ? bwd_tc_supported((int)dtype, d) : fwd_tc_supported((int)dtype, d);
  if (!tc)
    return fail(FA_ERR_UNSUPPORTED, "block and window masks run on the tensor-core kernels (bf16/fp16, d in %s)",
                backward ? "{64, 128}" : "{64, 128, 256}");
  const bool fits = backward ? bwd_masked_fits(H / Hkv, N, d) : fwd_masked_fits(N, d);
  if (!fits) return fail(FA_ERR_UNSUPPORTED, "masked problem too long for the kernels' tile lists (N=%d)", N);
  return FA_OK;
}

fa_status fwd_impl(const void* Q, const void* K, const void* V, void* O, float* L, int B, int H, int Hkv, int N,
                   int d, float scale, int causal, fa_dtype dtype, void* stream, const char* name,
                   const MaskSpec& mask = MaskSpec()) {
  bool empty;
  fa_status st = check_common(B, H, N, d, dtype, &empty);
  if (st != FA_OK || empty) return st;
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  if ((st = check_ptrs({Q, K, V, O, L}, name)) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if ((st = check_mask(mask, H, Hkv, N, d, dtype, false)) != FA_OK) return st;
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  FwdArgs a{Q, K, V, O, L, B * H, N, d, scale, causal ? 1 : 0, (int)dtype, syms.err, syms.counter,
            static_cast<cudaStream_t>(stream)};
  a.group = H / Hkv;
  a.window = std::min(mask.window, N);  // (a longer one hides nothing more; kernels add it to row numbers in 32 bits)
  a.block_mask = mask.block_mask;
  a.mask_heads = mask.mask_heads;
  a.heads = H;
  a.band = mask.band;
  a.sinks = mask.sinks;
  if (fwd_tc_supported(a.dtype, d)) return launched(launch_fwd_tc(a), "forward (tensor-core kernel)");
  return note_cuda_core_path(launched(launch_fwd_simt(a), "forward (CUDA-core kernel)"), "forward", dtype, d);
}

fa_status bwd_main_impl(const void* Q, const void* K, const void* V, const void* dO, void* dK, void* dV,
                        void* workspace, size_t workspace_bytes, int B, int H, int Hkv, int N, int d, float scale,
                        int causal, fa_dtype dtype, void* stream, const char* name, const MaskSpec& mask = MaskSpec()) {
  bool empty;
  fa_status st = check_common(B, H, N, d, dtype, &empty);
  if (st != FA_OK || empty) return st;
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  if ((st = check_ptrs({Q, K, V, dO, dK, dV, workspace}, name)) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if ((st = check_mask(mask, H, Hkv, N, d, dtype, true)) != FA_OK) return st;
  BwdArgs a{};
  if ((st = carve(&a, workspace, workspace_bytes, B, H, N, d)) != FA_OK) return st;
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  a.q = Q;
  a.k = K;
  a.v = V;
  a.dout = dO;
  a.dk = dK;
  a.dv = dV;
  a.bh = B * H;
  a.n = N;
  a.d = d;
  a.scale = scale;
  a.causal = causal ? 1 : 0;
  a.dtype = (int)dtype;
  a.err = syms.err;
  a.counter = syms.counter;
  a.stream = static_cast<cudaStream_t>(stream);
  a.group = H / Hkv;
  a.window = std::min(mask.window, N);  // (a longer one hides nothing more; kernels add it to row numbers in 32 bits)
  a.block_mask = mask.block_mask;
  a.mask_heads = mask.mask_heads;
  a.heads = H;
  a.band = mask.band;
  a.sinks = mask.sinks;
  if (bwd_tc_supported(a.dtype, d)) return launched(launch_bwd_tc(a), "backward (tensor-core kernel)");
  return note_cuda_core_path(launched(launch_bwd_simt(a), "backward (CUDA-core kernels)"), "backward", dtype, d);
}

fa_status bwd_pre_impl(const void* O, const void* dO, const float* L, void* workspace, size_t workspace_bytes, int B, int H,
                       int N, int d, fa_dtype dtype, void* stream, const char* name, int delta_rows = 0) {
  bool empty;
  fa_status st = check_common(B, H, N, d, dtype, &empty);
  if (st != FA_OK || empty) return st;
  if ((st = check_ptrs({O, dO, L, workspace}, name)) != FA_OK) return st;
  BwdArgs a{};
  if ((st = carve(&a, workspace, workspace_bytes, B, H, N, d)) != FA_OK) return st;
  a.o = O;
  a.dout = dO;
  a.lse = L;
  a.bh = B * H;
  a.n = N;
  a.d = d;
  a.dtype = (int)dtype;
  a.delta_rows = delta_rows;
  a.stream = static_cast<cudaStream_t>(stream);
  return launched(launch_bwd_pre(a), name);
}

// (window) D of a sequence's first `delta_rows` rows; in front of bwd_pre_impl with the same number.
fa_status window_delta_impl(const void* Q, const void* K, const void* V, const void* dO, const float* L, void* workspace,
                            size_t workspace_bytes, int B, int H, int Hkv, int N, int d, float scale, int window, int sinks,
                            fa_dtype dtype, void* stream, int delta_rows) {
  BwdArgs a{};
  const fa_status st = carve(&a, workspace, workspace_bytes, B, H, N, d);
  if (st != FA_OK) return st;
  a.q = Q;
  a.k = K;
  a.v = V;
  a.dout = dO;
  a.lse = L;
  a.bh = B * H;
  a.n = N;
  a.d = d;
  a.scale = scale;
  a.dtype = (int)dtype;
  a.stream = static_cast<cudaStream_t>(stream);
  a.group = H / Hkv;
  a.window = std::min(window, N);
  a.sinks = sinks;
  a.delta_rows = delta_rows;
  return launched(launch_window_delta(a), "fa_bwd_window");
}

}  // namespace

extern "C" {

fa_status fa_fwd(const void* Q, const void* K, const void* V, void* O, float* L, int B, int H, int N, int d,
                 float scale, int causal, fa_dtype dtype, void* stream) {
  return fwd_impl(Q, K, V, O, L, B, H, H, N, d, scale, causal, dtype, stream, "fa_fwd");
}

fa_status fa_fwd_gqa(const void* Q, const void* K, const void* V, void* O, float* L, int B, int H, int Hkv, int N,
                     int d, float scale, int causal, fa_dtype dtype, void* stream) {
  return fwd_impl(Q, K, V, O, L, B, H, Hkv, N, d, scale, causal, dtype, stream, "fa_fwd_gqa");
}

size_t fa_bwd_workspace_size(int B, int H, int N, int d) {
  bool empty;
  if (check_common(B, H, N, d, FA_FP32, &empty) != FA_OK) return 0;
  return workspace_bytes_for(B, H, N, d);
}

fa_status fa_bwd_preprocess(const void* O, const void* dO, const float* L, void* workspace, size_t workspace_bytes,
                            int B, int H, int N, int d, fa_dtype dtype, void* stream) {
  return bwd_pre_impl(O, dO, L, workspace, workspace_bytes, B, H, N, d, dtype, stream, "fa_bwd_preprocess");
}

fa_status fa_bwd_main(const void* Q, const void* K, const void* V, const void* dO, void* dK, void* dV,
                      void* workspace, size_t workspace_bytes, int B, int H, int N, int d, float scale, int causal,
                      fa_dtype dtype, void* stream) {
  return bwd_main_impl(Q, K, V, dO, dK, dV, workspace, workspace_bytes, B, H, H, N, d, scale, causal, dtype, stream,
                       "fa_bwd_main");
}

fa_status fa_bwd_dq_convert(const void* workspace, size_t workspace_bytes, void* dQ, int B, int H, int N, int d,
                            float scale, fa_dtype dtype, void* stream) {
  bool empty;
  fa_status st = check_common(B, H, N, d, dtype, &empty);
  if (st != FA_OK || empty) return st;
  if ((st = check_ptrs({workspace, dQ}, "fa_bwd_dq_convert")) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  BwdArgs a{};
  if ((st = carve(&a, const_cast<void*>(workspace), workspace_bytes, B, H, N, d)) != FA_OK) return st;
  a.dq = dQ;
  a.bh = B * H;
  a.n = N;
  a.d = d;
  a.scale = scale;
  a.dtype = (int)dtype;
  a.stream = static_cast<cudaStream_t>(stream);
  return launched(launch_dq_convert(a), "fa_bwd_dq_convert");
}

fa_status fa_bwd_gqa(const void* Q, const void* K, const void* V, const void* O, const void* dO, const float* L,
                     void* dQ, void* dK, void* dV, void* workspace, size_t workspace_bytes, int B, int H, int Hkv,
                     int N, int d, float scale, int causal, fa_dtype dtype, void* stream) {
  bool empty;
  fa_status st = check_common(B, H, N, d, dtype, &empty);
  if (st != FA_OK || empty) return st;
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  if ((st = check_ptrs({Q, K, V, O, dO, L, dQ, dK, dV, workspace}, "fa_bwd")) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if ((st = fa_bwd_preprocess(O, dO, L, workspace, workspace_bytes, B, H, N, d, dtype, stream)) != FA_OK) return st;
  if ((st = bwd_main_impl(Q, K, V, dO, dK, dV, workspace, workspace_bytes, B, H, Hkv, N, d, scale, causal, dtype,
                          stream, "fa_bwd")) != FA_OK)
    return st;
  st = fa_bwd_dq_convert(workspace, workspace_bytes, dQ, B, H, N, d, scale, dtype, stream);
  return bwd_tc_supported((int)dtype, d) ? st : note_cuda_core_path(st, "backward", dtype, d);
}

fa_status fa_fwd_masked(const void* Q, const void* K, const void* V, void* O, float* L, int B, int H, int Hkv, int N,
                        int d, float scale, int causal, int window, const uint8_t* block_mask, int mask_heads,
                        fa_dtype dtype, void* stream) {
  MaskSpec m;
  m.window = window;
  m.block_mask = block_mask;
  m.mask_heads = mask_heads;
  return fwd_impl(Q, K, V, O, L, B, H, Hkv, N, d, scale, causal, dtype, stream, "fa_fwd_masked", m);
}

fa_status fa_bwd_masked(const void* Q, const void* K, const void* V, const void* O, const void* dO, const float* L,
                        void* dQ, void* dK, void* dV, void* workspace, size_t workspace_bytes, int B, int H, int Hkv,
                        int N, int d, float scale, int causal, int window, const uint8_t* block_mask, int mask_heads,
                        fa_dtype dtype, void* stream) {
  MaskSpec m;
  m.window = window;
  m.block_mask = block_mask;
  m.mask_heads = mask_heads;
  bool empty;
  fa_status st = check_common(B, H, N, d, dtype, &empty);
  if (st != FA_OK || empty) return st;
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  if ((st = check_ptrs({Q, K, V, O, dO, L, dQ, dK, dV, workspace}, "fa_bwd_masked")) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if ((st = check_mask(m, H, Hkv, N, d, dtype, true)) != FA_OK) return st;
  if ((st = fa_bwd_preprocess(O, dO, L, workspace, workspace_bytes, B, H, N, d, dtype, stream)) != FA_OK) return st;
  if ((st = bwd_main_impl(Q, K, V, dO, dK, dV, workspace, workspace_bytes, B, H, Hkv, N, d, scale, causal, dtype,
                          stream, "fa_bwd_masked", m)) != FA_OK)
    return st;
  return fa_bwd_dq_convert(workspace, workspace_bytes, dQ, B, H, N, d, scale, dtype, stream);
}

fa_status fa_fwd_window(const void* Q, const void* K, const void* V, void* O, float* L, int B, int H, int Hkv, int N, int d,
                        float scale, int window, int sinks, fa_dtype dtype, void* stream) {
  MaskSpec m;
  m.band = true;
  m.window = window;
  m.sinks = sinks;
  return fwd_impl(Q, K, V, O, L, B, H, Hkv, N, d, scale, 1, dtype, stream, "fa_fwd_window", m);
}

fa_status fa_bwd_window(const void* Q, const void* K, const void* V, const void* O, const void* dO, const float* L,
                        void* dQ, void* dK, void* dV, void* workspace, size_t workspace_bytes, int B, int H, int Hkv,
                        int N, int d, float scale, int window, int sinks, fa_dtype dtype, void* stream) {
  MaskSpec m;
  m.band = true;
  m.window = window;
  m.sinks = sinks;
  bool empty;
  fa_status st = check_common(B, H, N, d, dtype, &empty);
  if (st != FA_OK || empty) return st;
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  if ((st = check_ptrs({Q, K, V, O, dO, L, dQ, dK, dV, workspace}, "fa_bwd_window")) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if ((st = check_mask(m, H, Hkv, N, d, dtype, true)) != FA_OK) return st;
  const int delta_rows = window_delta_rows(N, window, sinks);
  if ((st = window_delta_impl(Q, K, V, dO, L, workspace, workspace_bytes, B, H, Hkv, N, d, scale, window, sinks, dtype, stream,
                              delta_rows)) != FA_OK)
    return st;
  if ((st = bwd_pre_impl(O, dO, L, workspace, workspace_bytes, B, H, N, d, dtype, stream, "fa_bwd_window", delta_rows)) != FA_OK)
    return st;
  if ((st = bwd_main_impl(Q, K, V, dO, dK, dV, workspace, workspace_bytes, B, H, Hkv, N, d, scale, 1, dtype, stream,
                          "fa_bwd_window", m)) != FA_OK)
    return st;
  return fa_bwd_dq_convert(workspace, workspace_bytes, dQ, B, H, N, d, scale, dtype, stream);
}

fa_status fa_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO, const float* L,
                 void* dQ, void* dK, void* dV, void* workspace, size_t workspace_bytes, int B, int H, int N, int d,
                 float scale, int causal, fa_dtype dtype, void* stream) {
  return fa_bwd_gqa(Q, K, V, O, dO, L, dQ, dK, dV, workspace, workspace_bytes, B, H, H, N, d, scale, causal, dtype,
                    stream);
}

// Effective number of cache splits: 0 or less picks automatically (for the kernel that runs);
// never more than Nk.
static int decode_splits(int B, int H, int Hkv, int Nq, int Nk, int d, int splits, bool tc) {
  int s = splits > 0 ? splits
                     : (tc ? decode_tc_auto_splits(B, H, Hkv, Nq, Nk, d) : decode_auto_splits(B, H, Hkv, Nq, Nk));
  if (s > Nk) s = Nk;
  if (s > 4096) s = 4096;
  return s < 1 ? 1 : s;
}

static fa_status check_decode(int B, int H, int Hkv, int Nq, int Nk, int d, fa_dtype dtype, bool* empty) {
  *empty = false;
  if (dtype != FA_BF16 && dtype != FA_FP16 && dtype != FA_FP32)
    return fail(FA_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (B < 0 || H < 0 || Nq < 0 || Nk < 0) return fail(FA_ERR_INVALID_ARG, "negative size");
  if (d != 64 && d != 128 && d != 256) return fail(FA_ERR_UNSUPPORTED, "decode supports d in {64, 128, 256}, got %d", d);
  if ((int64_t)B * H * Nq == 0) {
    *empty = true;
    return FA_OK;
  }
  fa_status st = check_heads(H, Hkv);
  if (st != FA_OK) return st;
  if (Nk < 1) return fail(FA_ERR_INVALID_ARG, "decode needs at least one cached key (Nk=%d)", Nk);
  if ((double)B * Hkv * Nk * d > 4.0e15 || (double)B * H * Nq * d > 4.0e15)
    return fail(FA_ERR_INVALID_ARG, "problem too large");
  return FA_OK;
}

size_t fa_decode_workspace_size(int B, int H, int Hkv, int Nq, int Nk, int d, int splits) {
  bool empty;
  if (check_decode(B, H, Hkv, Nq, Nk, d, FA_BF16, &empty) != FA_OK || empty) return 0;
  // enough for either kernel (the size does not depend on the dtype)
  const int s = std::max(decode_splits(B, H, Hkv, Nq, Nk, d, splits, true), decode_splits(B, H, Hkv, Nq, Nk, d, splits, false));
  return decode_workspace_bytes(B, H, Nq, d, s);
}

fa_status fa_decode(const void* Q, const void* K, const void* V, void* O, float* L, int B, int H, int Hkv, int Nq,
                    int Nk, int d, float scale, int splits, fa_dtype dtype, void* workspace, size_t workspace_bytes,
                    void* stream) {
  bool empty;
  fa_status st = check_decode(B, H, Hkv, Nq, Nk, d, dtype, &empty);
  if (st != FA_OK || empty) return st;
  if ((st = check_ptrs({Q, K, V, O, L}, "fa_decode")) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  DecodeArgs a{};
  a.q = Q;
  a.k = K;
  a.v = V;
  a.o = O;
  a.lse = L;
  a.b = B;
  a.h = H;
  a.hkv = Hkv;
  a.nq = Nq;
  a.nk = Nk;
  a.d = d;
  a.scale = scale;
  const bool tc = decode_tc_supported((int)dtype, d, (int64_t)B * H * Nq);
  a.splits = decode_splits(B, H, Hkv, Nq, Nk, d, splits, tc);
  a.dtype = (int)dtype;
  a.stream = static_cast<cudaStream_t>(stream);
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  a.err = syms.err;
  a.counter = syms.counter;
  const size_t need = decode_workspace_bytes(B, H, Nq, d, a.splits);
  if (need > 0) {
    if (!workspace || !aligned16(workspace))
      return fail(FA_ERR_INVALID_ARG, "fa_decode: %d splits need a 16-byte-aligned workspace", a.splits);
    if (workspace_bytes < need)
      return fail(FA_ERR_INVALID_ARG, "fa_decode: workspace of %zu bytes < %zu required", workspace_bytes, need);
    a.ws = static_cast<float*>(workspace);
  }
  return launched(tc ? launch_decode_tc(a) : launch_decode(a), "fa_decode");
}

fa_status fa_quantize_fp8(const void* X, void* X8, float* scales, int B, int H, int N, int d, fa_dtype dtype,
                          void* stream) {
  bool empty;
  fa_status st = check_common(B, H, N, d, dtype, &empty);
  if (st != FA_OK || empty) return st;
  if (d != 64 && d != 128 && d != 256)
    return fail(FA_ERR_UNSUPPORTED, "fa_quantize_fp8 supports d in {64, 128, 256}, got %d", d);
  if ((st = check_ptrs({X, X8, scales}, "fa_quantize_fp8")) != FA_OK) return st;
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  QuantArgs a{X, X8, scales, B * H, N, d, (int)dtype, static_cast<cudaStream_t>(stream)};
  a.err = syms.err;
  return launched(launch_quantize_fp8(a), "fa_quantize_fp8");
}

fa_status fa_fwd_fp8_gqa(const void* Q8, const void* K8, const void* V8, const float* q_scales,
                         const float* k_scales, const float* v_scales, void* O, float* L, int B, int H, int Hkv, int N,
                         int d, float scale, int causal, fa_dtype out_dtype, void* stream) {
  if (out_dtype != FA_BF16 && out_dtype != FA_FP16)
    return fail(FA_ERR_UNSUPPORTED, "fa_fwd_fp8 writes O as bf16 or fp16, not dtype %d", (int)out_dtype);
  bool empty;
  fa_status st = check_common(B, H, N, d, out_dtype, &empty);
  if (st != FA_OK || empty) return st;
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  if (!fwd_fp8_supported(d)) return fail(FA_ERR_UNSUPPORTED, "fa_fwd_fp8 supports d in {64, 128, 256}, got %d", d);
  if ((st = check_ptrs({Q8, K8, V8, q_scales, k_scales, v_scales, O, L}, "fa_fwd_fp8")) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  Fp8FwdArgs a{};
  a.q8 = Q8;
  a.k8 = K8;
  a.v8 = V8;
  a.q_scales = q_scales;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.o = O;
  a.lse = L;
  a.bh = B * H;
  a.n = N;
  a.d = d;
  a.scale = scale;
  a.causal = causal ? 1 : 0;
  a.out_dtype = (int)out_dtype;
  a.err = syms.err;
  a.counter = syms.counter;
  a.stream = static_cast<cudaStream_t>(stream);
  a.group = H / Hkv;
  return launched(launch_fwd_fp8(a), "fa_fwd_fp8");
}

fa_status fa_fwd_fp8(const void* Q8, const void* K8, const void* V8, const float* q_scales, const float* k_scales,
                     const float* v_scales, void* O, float* L, int B, int H, int N, int d, float scale, int causal,
                     fa_dtype out_dtype, void* stream) {
  return fa_fwd_fp8_gqa(Q8, K8, V8, q_scales, k_scales, v_scales, O, L, B, H, H, N, d, scale, causal, out_dtype,
                        stream);
}

static fa_status varlen_impl(const void* Q, const void* K, const void* V, void* O, float* L, const int32_t* cu_seqlens, int S,
                             int T, int H, int Hkv, int d, int64_t q_token_stride, int64_t q_head_stride,
                             int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                             int64_t o_token_stride, int64_t o_head_stride, float scale, int causal, int window, int sinks,
                             fa_dtype dtype, void* stream, const char* name) {
  if (dtype != FA_BF16 && dtype != FA_FP16)
    return fail(FA_ERR_UNSUPPORTED, "%s takes bf16 or fp16, not dtype %d", name, (int)dtype);
  if (S < 0 || T < 0 || H < 0) return fail(FA_ERR_INVALID_ARG, "negative size S=%d T=%d H=%d", S, T, H);
  if (!fwd_tc_supported((int)dtype, d))
    return fail(FA_ERR_UNSUPPORTED, "%s supports d in {64, 128, 256}, got %d", name, d);
  if (S == 0 || T == 0 || H == 0) return FA_OK;
  fa_status st = check_heads(H, Hkv);
  if (st != FA_OK) return st;
  if ((double)H * ((double)T / 128 + S) > 1.0e9 || T > INT32_MAX - 512)
    return fail(FA_ERR_INVALID_ARG, "problem too large: S=%d T=%d H=%d", S, T, H);
  if ((st = check_ptrs({Q, K, V, O}, name)) != FA_OK) return st;
  if ((st = check_words({L, cu_seqlens}, name)) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  const int64_t strides[] = {q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                             v_token_stride, v_head_stride, o_token_stride, o_head_stride};
  for (int64_t v : strides) {
    if ((st = check_strides({v}, 2, name)) != FA_OK) return st;
    if (v < d) return fail(FA_ERR_INVALID_ARG, "%s: a stride of %lld elements < d=%d", name, (long long)v, d);
  }
  if ((st = check_output_rows(T, o_token_stride, H, o_head_stride, d, name)) != FA_OK) return st;
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  VarlenFwdArgs a{Q, K, V, O, L, cu_seqlens, S, T, H, H / Hkv, d, q_token_stride, q_head_stride, k_token_stride,
                  k_head_stride, v_token_stride, v_head_stride, o_token_stride, o_head_stride, scale, causal ? 1 : 0,
                  (int)dtype, syms.err, syms.counter, static_cast<cudaStream_t>(stream), window, sinks};
  return launched(launch_fwd_varlen(a), name);
}

fa_status fa_fwd_varlen(const void* Q, const void* K, const void* V, void* O, float* L, const int32_t* cu_seqlens, int S,
                        int T, int H, int Hkv, int d, int64_t q_token_stride, int64_t q_head_stride,
                        int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                        int64_t o_token_stride, int64_t o_head_stride, float scale, int causal, fa_dtype dtype,
                        void* stream) {
  return varlen_impl(Q, K, V, O, L, cu_seqlens, S, T, H, Hkv, d, q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                     v_token_stride, v_head_stride, o_token_stride, o_head_stride, scale, causal, 0, 0, dtype, stream,
                     "fa_fwd_varlen");
}

fa_status fa_fwd_varlen_window(const void* Q, const void* K, const void* V, void* O, float* L, const int32_t* cu_seqlens,
                               int S, int T, int H, int Hkv, int d, int64_t q_token_stride, int64_t q_head_stride,
                               int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                               int64_t v_head_stride, int64_t o_token_stride, int64_t o_head_stride, float scale,
                               int window, int sinks, fa_dtype dtype, void* stream) {
  const fa_status st = check_band(window, sinks, "fa_fwd_varlen_window");
  if (st != FA_OK) return st;
  return varlen_impl(Q, K, V, O, L, cu_seqlens, S, T, H, Hkv, d, q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                     v_token_stride, v_head_stride, o_token_stride, o_head_stride, scale, 1, window, sinks, dtype, stream,
                     "fa_fwd_varlen_window");
}

static fa_status kv4_rows(bool read, const void* K, const void* V, const int32_t* cu_seqlens, const int32_t* lens,
                          void* cache, float* weights, int B, int T, int Hkv, int capacity, int d,
                          int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                          int64_t v_head_stride, fa_dtype dtype, void* stream, const char* name) {
  bool empty;
  fa_status st = check_kv4(B, Hkv, capacity, d, &empty);
  if (st != FA_OK) return st;
  if (dtype != FA_BF16 && dtype != FA_FP16 && dtype != FA_FP32)
    return fail(FA_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (T < 0) return fail(FA_ERR_INVALID_ARG, "%s: negative row count T=%d", name, T);
  if (empty || T == 0) return FA_OK;
  if ((st = check_ptrs({K, V, cache}, name)) != FA_OK) return st;
  if ((st = check_words({cu_seqlens, lens}, name)) != FA_OK) return st;
  if (weights && (st = check_words({weights}, name)) != FA_OK) return st;
  const int eb = dtype == FA_FP32 ? 4 : 2;
  if ((st = check_strides({k_token_stride, k_head_stride, v_token_stride, v_head_stride}, eb, name)) != FA_OK) return st;
  if (read) {
    if ((st = check_output_rows(T, k_token_stride, Hkv, k_head_stride, d, name)) != FA_OK) return st;
    if ((st = check_output_rows(T, v_token_stride, Hkv, v_head_stride, d, name)) != FA_OK) return st;
  }
  if (T > INT32_MAX - 64 || (int64_t)Hkv * (d / 8) > 65535 * 32)
    return fail(FA_ERR_INVALID_ARG, "%s: T=%d rows of %d heads are too many for one call", name, T, Hkv);
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  Kv4RowArgs a{K, V, cu_seqlens, lens, static_cast<uint8_t*>(cache), weights, B, T, Hkv, capacity, d,
               k_token_stride, k_head_stride, v_token_stride, v_head_stride, (int)dtype, syms.err,
               static_cast<cudaStream_t>(stream)};
  return launched(read ? launch_kv4_read(a) : launch_kv4_append(a), name);
}

fa_status fa_kv4_append(const void* K, const void* V, const int32_t* cu_seqlens, const int32_t* lens, void* cache,
                        float* weights, int B, int T, int Hkv, int capacity, int d, int64_t k_token_stride,
                        int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, fa_dtype dtype,
                        void* stream) {
  return kv4_rows(false, K, V, cu_seqlens, lens, cache, weights, B, T, Hkv, capacity, d, k_token_stride, k_head_stride,
                  v_token_stride, v_head_stride, dtype, stream, "fa_kv4_append");
}

fa_status fa_kv4_read(const void* cache, const int32_t* cu_seqlens, const int32_t* lens, void* K, void* V, int B, int T,
                      int Hkv, int capacity, int d, int64_t k_token_stride, int64_t k_head_stride,
                      int64_t v_token_stride, int64_t v_head_stride, fa_dtype dtype, void* stream) {
  return kv4_rows(true, K, V, cu_seqlens, lens, const_cast<void*>(cache), nullptr, B, T, Hkv, capacity, d,
                  k_token_stride, k_head_stride, v_token_stride, v_head_stride, dtype, stream, "fa_kv4_read");
}

static fa_status check_decode_kv4(int B, int H, int Hkv, int Nq, int capacity, int d, bool* empty) {
  fa_status st = check_kv4(B, Hkv, capacity, d, empty);
  if (st != FA_OK) return st;
  if (H < 0 || Nq < 0) return fail(FA_ERR_INVALID_ARG, "negative size H=%d Nq=%d", H, Nq);
  if (*empty || H == 0 || Nq == 0) {
    *empty = true;
    return FA_OK;
  }
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  // rows of one key/value head, and its blocks times groups of eight of them, are counted in 32 bits
  const int64_t rows = (int64_t)(H / Hkv) * Nq;
  if (rows > INT32_MAX / 64 || (double)B * Hkv * ((rows + 7) / 8) > 1.0e9 ||
      (double)Hkv * ((rows + 7) / 8) * (capacity / 64 + 64) > 2.0e9 || (double)B * Hkv * (capacity / 64) > 2.0e9 ||
      (double)B * Hkv * rows * capacity > 2.0e18)
    return fail(FA_ERR_INVALID_ARG, "problem too large");
  return FA_OK;
}

size_t fa_decode_kv4_workspace_size(int B, int H, int Hkv, int Nq, int capacity, int d, int weights) {
  bool empty;
  if (check_decode_kv4(B, H, Hkv, Nq, capacity, d, &empty) != FA_OK || empty) return 0;
  return decode_kv4_workspace_bytes(B, H, Hkv, Nq, capacity, d, weights != 0);
}

fa_status fa_decode_kv4(const void* Q, const void* cache, const int32_t* lens, void* O, float* L,
                        const float* weights_in, float* weights_out, int B, int H, int Hkv, int Nq, int capacity, int d,
                        float scale, int causal, fa_dtype dtype, void* workspace, size_t workspace_bytes,
                        void* stream) {
  bool empty;
  fa_status st = check_decode_kv4(B, H, Hkv, Nq, capacity, d, &empty);
  if (st != FA_OK) return st;
  if (dtype != FA_BF16 && dtype != FA_FP16)
    return fail(FA_ERR_UNSUPPORTED, "fa_decode_kv4 takes bf16 or fp16 queries, not dtype %d", (int)dtype);
  if (empty && B > 0 && weights_out && weights_in != weights_out)
    return fail(FA_ERR_INVALID_ARG, "fa_decode_kv4: weights without query rows");
  if (empty) return FA_OK;
  if ((st = check_ptrs({Q, cache, O, workspace}, "fa_decode_kv4")) != FA_OK) return st;
  if ((st = check_words({lens, L}, "fa_decode_kv4")) != FA_OK) return st;
  if (weights_in && !weights_out)
    return fail(FA_ERR_INVALID_ARG, "fa_decode_kv4: weights_in without weights_out");
  if (weights_out && (st = check_words({weights_out}, "fa_decode_kv4")) != FA_OK) return st;
  if (weights_in && (st = check_words({weights_in}, "fa_decode_kv4")) != FA_OK) return st;
  const size_t nw = (size_t)B * Hkv * capacity * 4;
  if (weights_in && weights_in != weights_out && overlap({weights_in, nw}, {weights_out, nw}))
    return fail(FA_ERR_INVALID_ARG, "fa_decode_kv4: weights_in overlaps weights_out without being it");
  if ((st = check_scale(scale)) != FA_OK) return st;
  const size_t need = decode_kv4_workspace_bytes(B, H, Hkv, Nq, capacity, d, weights_out != nullptr);
  if (workspace_bytes < need)
    return fail(FA_ERR_INVALID_ARG, "fa_decode_kv4: workspace of %zu bytes < %zu required", workspace_bytes, need);
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  DecodeKv4Args a{Q, static_cast<const uint8_t*>(cache), lens, O, L, weights_in, weights_out, workspace, B, H, Hkv, Nq,
                  capacity, d, scale, causal ? 1 : 0, (int)dtype, syms.err, static_cast<cudaStream_t>(stream)};
  return launched(launch_decode_kv4(a), "fa_decode_kv4");
}

fa_status fa_kv4_evict(const void* cache, const float* weights, const int32_t* lens, int keep, int recent,
                       void* out_cache, float* out_weights, int32_t* out_lens, int32_t* kept, int B, int Hkv,
                       int capacity, int out_capacity, int d, void* stream) {
  bool empty;
  fa_status st = check_kv4(B, Hkv, capacity, d, &empty);
  if (st != FA_OK) return st;
  if ((st = check_kv4(B, Hkv, out_capacity, d, &empty)) != FA_OK) return st;
  if (keep < 1 || keep > out_capacity)
    return fail(FA_ERR_INVALID_ARG, "fa_kv4_evict: keep=%d outside [1, out_capacity=%d]", keep, out_capacity);
  if (recent < 0 || recent > keep)
    return fail(FA_ERR_INVALID_ARG, "fa_kv4_evict: recent=%d outside [0, keep=%d]", recent, keep);
  if (empty) return FA_OK;
  if ((st = check_ptrs({cache, out_cache}, "fa_kv4_evict")) != FA_OK) return st;
  if ((st = check_words({weights, lens, out_weights, out_lens, kept}, "fa_kv4_evict")) != FA_OK) return st;
  // what is read while other blocks write; out_lens may be lens
  const size_t heads = (size_t)B * Hkv;
  const Bytes in[] = {{cache, heads * (capacity / 64) * 72 * d}, {weights, heads * capacity * 4}, {lens, (size_t)B * 4}};
  const Bytes out[] = {{out_cache, heads * (out_capacity / 64) * 72 * d}, {out_weights, heads * out_capacity * 4},
                       {kept, heads * keep * 4}, {out_lens, (size_t)B * 4}};
  for (int i = 0; i < 4; ++i) {
    for (const Bytes& r : in)
      if (overlap(out[i], r) && !(i == 3 && out_lens == lens && r.p == lens))
        return fail(FA_ERR_INVALID_ARG, "fa_kv4_evict: the kept rows go into another cache, not into their own");
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j]))
        return fail(FA_ERR_INVALID_ARG, "fa_kv4_evict: an output lies in another one");
  }
  if ((double)B * Hkv * ((keep + 63) / 64) > (double)INT32_MAX)
    return fail(FA_ERR_INVALID_ARG, "fa_kv4_evict: too many rows for one call");
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  Kv4EvictArgs a{static_cast<const uint8_t*>(cache), weights, lens, static_cast<uint8_t*>(out_cache), out_weights,
                 out_lens, kept, B, Hkv, capacity, out_capacity, d, keep, recent, syms.err,
                 static_cast<cudaStream_t>(stream)};
  return launched(launch_kv4_evict(a), "fa_kv4_evict");
}

static fa_status check_decode_cache(int B, int H, int Hkv, int Nq, int P, int capacity, int d, bool* empty, const char* name) {
  *empty = false;
  if (B < 0 || H < 0 || Nq < 0 || P < 0)
    return fail(FA_ERR_INVALID_ARG, "%s: negative size B=%d H=%d Nq=%d P=%d", name, B, H, Nq, P);
  if (d != 64 && d != 128 && d != 256)
    return fail(FA_ERR_UNSUPPORTED, "%s supports d in {64, 128, 256}, got %d", name, d);
  if (capacity < 1) return fail(FA_ERR_INVALID_ARG, "%s: capacity=%d slots: at least one", name, capacity);
  if ((int64_t)B * H * Nq == 0) {
    *empty = true;
    return FA_OK;
  }
  const fa_status st = check_heads(H, Hkv);
  if (st != FA_OK) return st;
  // rows, entries and, some tiles behind the last, keys are counted in 32 bits
  if ((double)B * H * Nq > 2.0e8 || (double)B * Hkv > 1.0e8 || capacity > INT32_MAX - 4096 || P > INT32_MAX - 4096 ||
      (double)B * Hkv * capacity * d > 4.0e15 || (double)Hkv * P * d > 4.0e15)
    return fail(FA_ERR_INVALID_ARG, "%s: problem too large: B=%d H=%d Hkv=%d Nq=%d P=%d capacity=%d", name, B, H, Hkv, Nq, P,
                capacity);
  return FA_OK;
}

static fa_status decode_cache_impl(CacheDecodeArgs* a, size_t workspace_bytes, const char* name) {
  bool empty;
  fa_status st = check_decode_cache(a->b, a->h, a->hkv, a->nq, a->p, a->capacity, a->d, &empty, name);
  if (st != FA_OK) return st;
  if (a->dtype != FA_BF16 && a->dtype != FA_FP16)
    return fail(FA_ERR_UNSUPPORTED, "%s takes bf16 or fp16, not dtype %d", name, a->dtype);
  if (empty) return FA_OK;
  if ((st = check_ptrs({a->q, a->k, a->v, a->o, a->ws}, name)) != FA_OK) return st;
  if (a->p > 0 && (st = check_ptrs({a->kp, a->vp}, name)) != FA_OK) return st;
  if ((st = check_words({a->lens, a->lse}, name)) != FA_OK) return st;
  if ((st = check_scale(a->scale)) != FA_OK) return st;
  const size_t need = decode_cache_workspace_bytes(a->b, a->h, a->hkv, a->nq, a->p, a->d);
  if (workspace_bytes < need)
    return fail(FA_ERR_INVALID_ARG, "%s: workspace of %zu bytes < %zu required", name, workspace_bytes, need);
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  a->err = syms.err;
  a->counter = syms.counter;
  return launched(launch_decode_cache(*a), name);
}

size_t fa_decode_window_workspace_size(int B, int H, int Hkv, int Nq, int capacity, int d) {
  bool empty;
  if (check_decode_cache(B, H, Hkv, Nq, 0, capacity, d, &empty, "fa_decode_window") != FA_OK || empty) return 0;
  return decode_cache_workspace_bytes(B, H, Hkv, Nq, 0, d);
}

fa_status fa_decode_window(const void* Q, const void* K, const void* V, const int32_t* lens, void* O, float* L, int B, int H,
                           int Hkv, int Nq, int capacity, int d, float scale, int window, int sinks, fa_dtype dtype,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (window < 0) return fail(FA_ERR_INVALID_ARG, "fa_decode_window: window must be >= 0 (0: none), got %d", window);
  if (sinks < 0 || (sinks > 0 && window == 0))
    return fail(FA_ERR_INVALID_ARG, "fa_decode_window: sinks=%d: >= 0, and 0 without a window", sinks);
  CacheDecodeArgs a{Q, K, V, nullptr, nullptr, lens, O, L, workspace, B, H, Hkv, Nq, capacity, 0, d, window, sinks, scale,
                    (int)dtype, nullptr, nullptr, static_cast<cudaStream_t>(stream)};
  return decode_cache_impl(&a, workspace_bytes, "fa_decode_window");
}

size_t fa_decode_prefix_workspace_size(int B, int H, int Hkv, int Nq, int P, int capacity, int d) {
  bool empty;
  if (check_decode_cache(B, H, Hkv, Nq, P, capacity, d, &empty, "fa_decode_prefix") != FA_OK || empty) return 0;
  return decode_cache_workspace_bytes(B, H, Hkv, Nq, P, d);
}

fa_status fa_decode_prefix(const void* Q, const void* KP, const void* VP, const void* K, const void* V, const int32_t* lens,
                           void* O, float* L, int B, int H, int Hkv, int Nq, int P, int capacity, int d, float scale,
                           fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  CacheDecodeArgs a{Q, K, V, KP, VP, lens, O, L, workspace, B, H, Hkv, Nq, capacity, P, d, 0, 0, scale,
                    (int)dtype, nullptr, nullptr, static_cast<cudaStream_t>(stream)};
  return decode_cache_impl(&a, workspace_bytes, "fa_decode_prefix");
}

// The checks of fa_qk_norm_rope and fa_qk_norm_rope_bwd. `in` and `out` hold the queries' and the keys' tensors by turns.
static fa_status norm_rope_impl(NormRopeArgs* a, std::initializer_list<RowTensor> in, std::initializer_list<RowTensor> out,
                                const char* name) {
  if (a->dtype != FA_BF16 && a->dtype != FA_FP16 && a->dtype != FA_FP32)
    return fail(FA_ERR_UNSUPPORTED, "unknown dtype %d", a->dtype);
  if (a->wdtype != FA_FP32 && a->wdtype != a->dtype)
    return fail(FA_ERR_UNSUPPORTED, "%s: weights are fp32 or of the rows' dtype", name);
  if (a->b < 0 || a->n < 0 || a->h < 0 || a->hkv < 0)
    return fail(FA_ERR_INVALID_ARG, "%s: negative size B=%d N=%d H=%d Hkv=%d", name, a->b, a->n, a->h, a->hkv);
  if (a->d < 8 || a->d > 256 || a->d % 8 != 0)
    return fail(FA_ERR_UNSUPPORTED, "%s: d=%d is not a multiple of 8 in [8, 256]", name, a->d);
  if (a->rotary < 0 || a->rotary > a->d || a->rotary % 8 != 0)
    return fail(FA_ERR_INVALID_ARG, "%s: rotary=%d is not a multiple of 8 in [0, d=%d]", name, a->rotary, a->d);
  if (!std::isfinite(a->eps) || a->eps < 0.f) return fail(FA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", name);
  // units of work are counted in 32 bits, up to a grid's share behind the last
  if ((double)a->b * a->n * ((double)a->h + a->hkv) > 1.0e9)
    return fail(FA_ERR_INVALID_ARG, "%s: B=%d N=%d H=%d Hkv=%d: too many rows for one call", name, a->b, a->n, a->h, a->hkv);
  const bool rows = (int64_t)a->b * a->n > 0;
  const int eb = a->dtype == FA_FP32 ? 4 : 2;
  fa_status st;
  if (rows && a->h + a->hkv > 0) {
    for (const auto* list : {&in, &out})
      for (const RowTensor& t : *list) {
        if (t.heads == 0) continue;
        if ((st = check_ptrs({t.p}, name)) != FA_OK) return st;
        if ((st = check_strides({t.st.batch, t.st.token, t.st.head}, eb, name)) != FA_OK) return st;
        if ((double)(a->b - 1) * t.st.batch + (double)(a->n - 1) * t.st.token + (double)(t.heads - 1) * t.st.head > 1.0e18)
          return fail(FA_ERR_INVALID_ARG, "%s: %s reaches too far", name, t.name);
      }
    for (auto o = out.begin(); o != out.end(); ++o) {
      if (o->heads == 0) continue;
      if ((st = check_rows_apart(*o, a->b, a->n, a->d, name)) != FA_OK) return st;
      const int kind = (int)(o - out.begin()) & 1;
      for (auto i = in.begin(); i != in.end(); ++i)
        if (i->heads && !(((int)(i - in.begin()) & 1) == kind && same_rows(*o, *i, a->b, a->n)) &&
            rows_meet(*o, *i, a->b, a->n, a->d, eb))
          return fail(FA_ERR_INVALID_ARG, "%s: %s overlaps %s", name, o->name, i->name);
      for (auto o2 = out.begin(); o2 != o; ++o2)
        if (o2->heads && rows_meet(*o, *o2, a->b, a->n, a->d, eb))
          return fail(FA_ERR_INVALID_ARG, "%s: %s overlaps %s", name, o->name, o2->name);
    }
    if (a->rotary > 0) {
      if ((st = check_ptrs({a->table}, name)) != FA_OK) return st;
      if (a->table_len < 1) return fail(FA_ERR_INVALID_ARG, "%s: an empty table", name);
      if (a->positions) {
        if ((st = check_words({a->positions}, name)) != FA_OK) return st;
      } else if (a->n > a->table_len) {
        return fail(FA_ERR_INVALID_ARG, "%s: N=%d positions but table_len=%d", name, a->n, a->table_len);
      }
    }
  }
  for (const void* w : {a->wq, a->wk, (const void*)a->dwq, (const void*)a->dwk})
    if (!aligned16(w)) return fail(FA_ERR_INVALID_ARG, "%s: a weight is not 16-byte aligned", name);
  return FA_OK;
}

static NormRopeStrides strides_at(const int64_t* s, int i) { return {s[3 * i], s[3 * i + 1], s[3 * i + 2]}; }

fa_status fa_qk_norm_rope(const void* Q, const void* K, const void* wq, const void* wk, const float* table,
                          const int32_t* positions, void* Qo, void* Ko, const int64_t* strides, int B, int N, int H, int Hkv,
                          int d, int rotary, int adjacent, int table_len, float eps, fa_dtype dtype, fa_dtype weight_dtype,
                          void* stream) {
  if (!strides) return fail(FA_ERR_INVALID_ARG, "fa_qk_norm_rope: strides is null");
  NormRopeArgs a{};
  a.q = Q, a.k = K, a.wq = wq, a.wk = wk, a.table = table, a.positions = positions, a.qo = Qo, a.ko = Ko;
  a.q_st = strides_at(strides, 0), a.k_st = strides_at(strides, 1);
  a.qo_st = strides_at(strides, 2), a.ko_st = strides_at(strides, 3);
  a.b = B, a.n = N, a.h = H, a.hkv = Hkv, a.d = d, a.rotary = rotary, a.adjacent = adjacent ? 1 : 0;
  a.table_len = table_len, a.eps = eps, a.dtype = (int)dtype, a.wdtype = (int)weight_dtype;
  a.stream = static_cast<cudaStream_t>(stream);
  fa_status st = norm_rope_impl(&a, {{"Q", Q, a.q_st, H}, {"K", K, a.k_st, Hkv}},
                                {{"Qo", Qo, a.qo_st, H}, {"Ko", Ko, a.ko_st, Hkv}}, "fa_qk_norm_rope");
  if (st != FA_OK || (int64_t)B * N == 0 || H + Hkv == 0) return st;
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  a.err = syms.err;
  return launched(launch_norm_rope(a), "fa_qk_norm_rope");
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d) {
  // a row of sums for each block, for as many as the current device takes at once
  return d < 8 || d > 256 || d % 8 != 0 ? 0 : (size_t)norm_rope_bwd_blocks() * d * 4;
}

fa_status fa_qk_norm_rope_bwd(const void* dQo, const void* dKo, const void* Q, const void* K, const void* wq,
                              const void* wk, const float* table, const int32_t* positions, void* dQ, void* dK, void* dwq,
                              void* dwk, void* workspace, size_t workspace_bytes, const int64_t* strides, int B, int N,
                              int H, int Hkv, int d, int rotary, int adjacent, int table_len, float eps, fa_dtype dtype,
                              fa_dtype weight_dtype, void* stream) {
  if (!strides) return fail(FA_ERR_INVALID_ARG, "fa_qk_norm_rope_bwd: strides is null");
  NormRopeArgs a{};
  a.q = Q, a.k = K, a.wq = wq, a.wk = wk, a.table = table, a.positions = positions, a.qo = dQo, a.ko = dKo;
  a.dq = dQ, a.dk = dK, a.dwq = dwq, a.dwk = dwk;
  a.qo_st = strides_at(strides, 0), a.ko_st = strides_at(strides, 1);
  a.q_st = strides_at(strides, 2), a.k_st = strides_at(strides, 3);
  a.dq_st = strides_at(strides, 4), a.dk_st = strides_at(strides, 5);
  a.b = B, a.n = N, a.h = H, a.hkv = Hkv, a.d = d, a.rotary = rotary, a.adjacent = adjacent ? 1 : 0;
  a.table_len = table_len, a.eps = eps, a.dtype = (int)dtype, a.wdtype = (int)weight_dtype, a.backward = 1;
  a.stream = static_cast<cudaStream_t>(stream);
  fa_status st = norm_rope_impl(
      &a, {{"dQo", dQo, a.qo_st, H}, {"dKo", dKo, a.ko_st, Hkv}, {"Q", Q, a.q_st, H}, {"K", K, a.k_st, Hkv}},
      {{"dQ", dQ, a.dq_st, H}, {"dK", dK, a.dk_st, Hkv}}, "fa_qk_norm_rope_bwd");
  if (st != FA_OK) return st;
  const bool rows = (int64_t)B * N > 0 && H + Hkv > 0;
  if (!rows && !dwq && !dwk) return FA_OK;
  const size_t nw = (size_t)d * (weight_dtype == FA_FP32 ? 4 : 2);
  if (dwq && dwk && overlap({dwq, nw}, {dwk, nw})) return fail(FA_ERR_INVALID_ARG, "fa_qk_norm_rope_bwd: dwq overlaps dwk");
  if ((st = check_ptrs({workspace}, "fa_qk_norm_rope_bwd")) != FA_OK) return st;
  DeviceSyms syms;
  if ((st = device_syms(&syms)) != FA_OK) return st;
  a.err = syms.err;
  const size_t need = fa_qk_norm_rope_bwd_workspace_size(d);
  if (workspace_bytes < need)
    return fail(FA_ERR_INVALID_ARG, "fa_qk_norm_rope_bwd: workspace of %zu bytes < %zu required", workspace_bytes, need);
  a.partials = static_cast<float*>(workspace);
  return launched(launch_norm_rope(a), "fa_qk_norm_rope_bwd");
}

fa_status fa_check_device_error(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "stream synchronize: %s", cudaGetErrorString(e));
  DeviceSyms syms;
  fa_status st = device_syms(&syms);
  if (st != FA_OK) return st;
  unsigned long long w = 0;
  if ((e = cudaMemcpy(&w, syms.err, sizeof(w), cudaMemcpyDeviceToHost)) != cudaSuccess)
    return fail(FA_ERR_CUDA, "reading the device error word: %s", cudaGetErrorString(e));
  if (w == 0) {
    t_msg[0] = 0;
    return FA_OK;
  }
  const unsigned long long zero = 0;
  cudaMemcpy(syms.err, &zero, sizeof(zero), cudaMemcpyHostToDevice);
  const unsigned code = (unsigned)(w >> 56), site = (unsigned)((w >> 40) & 0xFFFF);
  const unsigned long long block = w & 0xFFFFFFFFFFull;
  if (code == DERR_TIMEOUT)
    return fail(FA_ERR_TIMEOUT, "a bounded wait expired (site %u, block %llu)", site, block);
  if (code == DERR_BOUNDS)
    return fail(FA_ERR_DEVICE, "device index check failed (site %u, block %llu)", site, block);
  return fail(FA_ERR_DEVICE, "device check %u failed (site %u, block %llu)", code, site, block);
}

fa_status fa_selftest_bounded_wait(int timeout_ms, int arrive, void* stream) {
  if (timeout_ms < 1 || timeout_ms > 1000)
    return fail(FA_ERR_INVALID_ARG, "fa_selftest_bounded_wait: timeout_ms must be in [1, 1000], got %d", timeout_ms);
  DeviceSyms syms;
  fa_status st = device_syms(&syms);
  if (st != FA_OK) return st;
  return launched(launch_bounded_wait_selftest(syms.err, timeout_ms, arrive ? 1 : 0, static_cast<cudaStream_t>(stream)),
                  "fa_selftest_bounded_wait");
}

fa_status fa_selftest_debug_check(int index, int limit, void* stream) {
  if (!FA_DEBUG_CHECKS) return fail(FA_ERR_UNSUPPORTED, "fa_selftest_debug_check: library built without FA_DEBUG");
  DeviceSyms syms;
  fa_status st = device_syms(&syms);
  if (st != FA_OK) return st;
  return launched(launch_debug_check_selftest(syms.err, index, limit, static_cast<cudaStream_t>(stream)),
                  "fa_selftest_debug_check");
}

int fa_debug_build(void) { return FA_DEBUG_CHECKS; }

fa_status fa_sm_clock_sample(unsigned long long* out, int blocks, void* stream) {
  if (!out || !aligned16(out)) return fail(FA_ERR_INVALID_ARG, "fa_sm_clock_sample: null or misaligned output");
  if (blocks < 1 || blocks > device_sm_count())
    return fail(FA_ERR_INVALID_ARG, "fa_sm_clock_sample: blocks=%d outside [1, %d]", blocks, device_sm_count());
  return launched(launch_sm_clock_sample(out, blocks, static_cast<cudaStream_t>(stream)), "fa_sm_clock_sample");
}

fa_status fa_tile_counter(void* stream, unsigned long long* value, int reset) {
  if (!value) return fail(FA_ERR_INVALID_ARG, "fa_tile_counter: null output");
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "stream synchronize: %s", cudaGetErrorString(e));
  DeviceSyms syms;
  fa_status st = device_syms(&syms);
  if (st != FA_OK) return st;
  if ((e = cudaMemcpy(value, syms.counter, sizeof(*value), cudaMemcpyDeviceToHost)) != cudaSuccess)
    return fail(FA_ERR_CUDA, "reading the tile counter: %s", cudaGetErrorString(e));
  if (reset) {
    const unsigned long long zero = 0;
    if ((e = cudaMemcpy(syms.counter, &zero, sizeof(zero), cudaMemcpyHostToDevice)) != cudaSuccess)
      return fail(FA_ERR_CUDA, "resetting the tile counter: %s", cudaGetErrorString(e));
  }
  return FA_OK;
}

int fa_uses_tensor_cores(int pass, fa_dtype dtype, int d) {
  return pass == 0 ? (int)fwd_tc_supported((int)dtype, d) : (int)bwd_tc_supported((int)dtype, d);
}

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported dtype or head dimension";
    case FA_ERR_CUDA: return "CUDA error";
    case FA_ERR_TIMEOUT: return "device wait timed out";
    case FA_ERR_DEVICE: return "device-side check failed";
  }
  return "unknown status";
}

const char* fa_last_error_message(void) { return t_msg; }

}  // extern "C"
