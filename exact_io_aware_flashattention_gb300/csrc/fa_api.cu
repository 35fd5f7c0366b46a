// C-ABI layer of libfa_gb300.so: argument validation, TMA tensor maps,
// kernel launches and the device status words.  See include/fa.h for the
// contract of every entry point.
#include "fa.h"

#include <cudaTypedefs.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <initializer_list>
#include <mutex>
#include <utility>

#include "fa_internal.h"
#include "fa_paged.h"
#include "fa_paged4.h"

namespace {

// Most recent CUDA runtime error behind an FA_ERR_LAUNCH / FA_ERR_CUDA return
// on this thread (see fa_last_cuda_error).
thread_local cudaError_t t_last_cuda_error = cudaSuccess;

fa_status launch_status(cudaError_t e) {
  if (e == cudaSuccess) return FA_OK;
  t_last_cuda_error = e;
  return FA_ERR_LAUNCH;
}

// Records a failing runtime call and returns FA_ERR_CUDA.
fa_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return FA_OK;
  t_last_cuda_error = e;
  return FA_ERR_CUDA;
}

#define FA_TRY(x)                   \
  do {                              \
    fa_status _s = (x);             \
    if (_s != FA_OK) return _s;     \
  } while (0)

#define FA_TRY_CUDA(x)                                \
  do {                                                \
    const cudaError_t _e = (x);                       \
    if (_e != cudaSuccess) return cuda_status(_e);    \
  } while (0)

// First device-side error: code, block, wait site, thread, and the first
// failed drain (site, block).  Read and cleared by fa_last_device_status.
__device__ int g_status_words[fa::kStatusWords];

// Named range around each public call, for timeline tools (a no-op unless a
// tool is attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

__global__ void wait_selftest_kernel(fa::DevStatus st) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    fa::mbar_init(&bar, 1);
    abort_flag = 0;
    fa::mbar_fence_init();
  }
  __syncthreads();
  // Nothing ever arrives on `bar`: the bounded wait must give up and record
  // FA_ERR_DEVICE_TIMEOUT.
  if (threadIdx.x == 0) fa::mbar_wait(&bar, 0, st, &abort_flag, 99);
  __syncthreads();
}

// The same with the drain wait a kernel does on its way out: nothing ever
// completes `bar`, so the drain gives up and records its site (98).
__global__ void drain_selftest_kernel(fa::DevStatus st) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    fa::mbar_init(&bar, 1);
    fa::mbar_fence_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) fa::mbar_wait_drain(&bar, 0, st, 98);
  __syncthreads();
}

constexpr int kMaxDevices = 64;

struct DeviceState {
  bool ready = false;
  std::atomic<bool> paged_ready{false};   // the paged-cache and rotary kernels too
  std::atomic<bool> paged4_ready{false};  // and those of the norms and the 4-bit cache
  bool unusable = false;   // a kernel's drain gave up: no further launches on this device
  int num_sms = 0;
  int* status = nullptr;
};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

unsigned long long default_timeout_ns() {
  static unsigned long long t = [] {
    const char* s = std::getenv("FA_WAIT_TIMEOUT_NS");
    unsigned long long v = s ? std::strtoull(s, nullptr, 10) : 0ull;
    return v ? v : 2000000000ull;  // 2 s: far above any single wait of a correct run
  }();
  return t;
}

// Per-device state, set up once with the device current: its SM count, the
// status words' address, the kernels' shared-memory attributes and the
// forward kernel's register check.  With `launch`, a device on which a drain
// has failed is refused.
fa_status device_state(DeviceState** out, bool launch = true) {
  int dev = -1;
  FA_TRY_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= kMaxDevices) return FA_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState& s = g_dev[dev];
  if (launch && s.unusable) return FA_ERR_DEVICE_DRAIN;
  if (!s.ready) {
    int major = 0, minor = 0, sms = 0;
    FA_TRY_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
    FA_TRY_CUDA(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
    FA_TRY_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    if (major != 10 || minor != 3) return FA_ERR_UNSUPPORTED_DEVICE;
    void* p = nullptr;
    FA_TRY_CUDA(cudaGetSymbolAddress(&p, g_status_words));
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
              cudaSuccess ||
          q != cudaDriverEntryPointSuccess || fn == nullptr)
        return FA_ERR_CUDA;
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    {
      const cudaError_t e = fa::configure_kernels();
      if (e != cudaSuccess) return launch_status(e);
    }
    s.num_sms = sms;
    s.status = static_cast<int*>(p);
    s.ready = true;
  }
  *out = &s;
  return FA_OK;
}

fa::DevStatus dev_status(const DeviceState* s) { return fa::DevStatus{s->status, default_timeout_ns()}; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

fa_status check_shape(int B, int Hq, int Hkv, int N, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || N < 1) return FA_ERR_BAD_SHAPE;
  if (Hq % Hkv != 0) return FA_ERR_BAD_SHAPE;
  if (B > 65535 || N > 65535 * 128) return FA_ERR_BAD_SHAPE;
  if ((long long)((N + 127) / 128) * Hq * B >= (1LL << 31)) return FA_ERR_BAD_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_HEADDIM;
  return FA_OK;
}

fa_status check_scale(int causal, float scale) {
  if (causal != 0 && causal != 1) return FA_ERR_BAD_ARGUMENT;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_BAD_ARGUMENT;
  return FA_OK;
}

struct Range {
  uintptr_t lo, hi;
};
Range range(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + bytes};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

size_t elems(int B, int H, int N, int d) { return (size_t)B * H * N * d; }

fa_status check_shape_ex(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  FA_TRY(check_shape(B, Hq, Hkv, Nq, d));
  return check_shape(B, Hq, Hkv, Nk, d);
}

// How the forward tiles a problem: per-head 128-row query tiles, or, for few
// query rows (Nq < 128, Hq/Hkv * Nq <= 128, Hq > Hkv), one tile holding the
// rows of all query heads of a kv group; the key tiles split into chunks.
struct FwdGeometry {
  int packed, nqt, units, splits, split_tiles;
};
FwdGeometry fwd_geometry(int B, int Hq, int Hkv, int Nq, int Nk, int num_splits) {
  FwdGeometry g;
  const int G = Hq / Hkv;
  g.packed = (G > 1 && Nq < 128 && G * Nq <= 128) ? 1 : 0;
  g.nqt = g.packed ? 1 : (Nq + 127) / 128;
  g.units = g.packed ? B * Hkv : B * Hq;
  const int ntk = (Nk + 127) / 128;
  g.split_tiles = (ntk + num_splits - 1) / num_splits;
  g.splits = (ntk + g.split_tiles - 1) / g.split_tiles;
  return g;
}

// Split forward workspace: per-split O, fp32 [S, B*Hq*Nq, d], then per-split
// LSE, fp32 [S, B*Hq*Nq], each 256-byte aligned.
struct FwdWsLayout {
  size_t o_off, lse_off, total;
};
FwdWsLayout fwd_ws_layout(int B, int Hq, int Nq, int d, int num_splits) {
  const size_t rows = (size_t)B * Hq * Nq;
  FwdWsLayout w;
  w.o_off = 0;
  w.lse_off = align256((size_t)num_splits * rows * d * 4);
  w.total = w.lse_off + align256((size_t)num_splits * rows * 4);
  return w;
}

// Backward workspace: fp32 dQ accumulator [B,Hq,N,d], then LSE*log2(e) and
// D = rowsum(dO*O), each fp32 [B*Hq, ntp] with ntp = ceil(N/128)*128.
struct WsLayout {
  size_t dq_off, lse2_off, dr_off, total;
};
WsLayout ws_layout(int B, int Hq, int N, int d) {
  const size_t ntp = (size_t)((N + 127) / 128) * 128;
  WsLayout w;
  w.dq_off = 0;
  w.lse2_off = align256(elems(B, Hq, N, d) * 4);
  w.dr_off = w.lse2_off + align256((size_t)B * Hq * ntp * 4);
  w.total = w.dr_off + align256((size_t)B * Hq * ntp * 4);
  return w;
}

// Tensor maps are a pure function of (kind, base address, sizes): a small
// per-thread cache saves re-encoding them when the same buffers come back.
struct TmapKey {
  const void* base;
  int kind, B, H, N, d;
  bool operator==(const TmapKey& o) const {
    return base == o.base && kind == o.kind && B == o.B && H == o.H && N == o.N && d == o.d;
  }
};
struct TmapSlot {
  TmapKey key{nullptr, -1, 0, 0, 0, 0};
  CUtensorMap map;   // the encoded map of either rank
};
constexpr int kTmapSlots = 32;
thread_local TmapSlot t_tmaps[kTmapSlots];

int tmap_slot(const TmapKey& k) {
  uint64_t h = reinterpret_cast<uintptr_t>(k.base) >> 8;
  h = h * 0x9E3779B97F4A7C15ull + (uint64_t)k.kind;
  h = h * 0x9E3779B97F4A7C15ull + (uint64_t)(uint32_t)k.N;
  h = h * 0x9E3779B97F4A7C15ull + (uint64_t)(uint32_t)(k.B * 131 + k.H * 7 + k.d);
  return (int)((h >> 40) % kTmapSlots);
}

template <typename Encode>
fa_status cached_tmap(CUtensorMap* m, const TmapKey& key, Encode encode) {
  TmapSlot& slot = t_tmaps[tmap_slot(key)];
  if (slot.key == key) {
    *m = slot.map;
    return FA_OK;
  }
  const fa_status st = encode(m);
  if (st == FA_OK) {
    slot.key = key;
    slot.map = *m;
  }
  return st;
}

fa_status tmap_bf16_encode(CUtensorMap* m, const void* base, int B, int H, int N, int d) {  // rank 4
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)H, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)N * d * 2, (cuuint64_t)H * N * d * 2};
  cuuint32_t box[4] = {64, 128, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_LAUNCH;
}

// Q (or O) [B, Hq, Nq, d] viewed as {d, Hq*Nq, B}: a 128-row box may start at
// any row of a batch (a tile of one head, or the rows of a group of heads).
fa_status tmap_rows_bf16_encode(CUtensorMap* m, const void* base, int B, int H, int N, int d) {  // rank 3
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H * N, (cuuint64_t)B};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)H * N * d * 2};
  cuuint32_t box[3] = {64, 128, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_LAUNCH;
}

// fp32 dQ accumulator [B*Hq, N, d] viewed as {d, N, B*Hq} with a {32, 128, 1}
// box and 128-byte swizzle, the target of the tiled TMA reduce-add.
fa_status tmap_dq_accum_encode(CUtensorMap* m, void* base, int B, int Hq, int N, int d) {  // rank 3
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)B * Hq};
  cuuint64_t strides[2] = {(cuuint64_t)d * 4, (cuuint64_t)N * d * 4};
  cuuint32_t box[3] = {32, 128, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_LAUNCH;
}

// [B, H, N, d] bf16 as {d, N, H, B}, {64, 128, 1, 1} boxes.
fa_status tmap_bf16(fa::TmaMap4* m, const void* base, int B, int H, int N, int d) {
  return cached_tmap(&m->m, TmapKey{base, 0, B, H, N, d},
                     [&](CUtensorMap* x) { return tmap_bf16_encode(x, base, B, H, N, d); });
}
fa_status tmap_rows_bf16(fa::TmaMap3* m, const void* base, int B, int H, int N, int d) {
  return cached_tmap(&m->m, TmapKey{base, 1, B, H, N, d},
                     [&](CUtensorMap* x) { return tmap_rows_bf16_encode(x, base, B, H, N, d); });
}
fa_status tmap_dq_accum(fa::TmaMap3* m, void* base, int B, int Hq, int N, int d) {
  return cached_tmap(&m->m, TmapKey{base, 2, B, Hq, N, d},
                     [&](CUtensorMap* x) { return tmap_dq_accum_encode(x, base, B, Hq, N, d); });
}

fa_status validate_dkdv(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv, int B,
                        int Hq, int Hkv, int N, int d, int causal, float scale, const void* workspace,
                        size_t workspace_bytes) {
  if (!q || !k || !v || !dO || !dk || !dv || !workspace) return FA_ERR_NULL_PTR;
  FA_TRY(check_shape(B, Hq, Hkv, N, d));
  FA_TRY(check_scale(causal, scale));
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dO) || !aligned16(dk) || !aligned16(dv) ||
      !aligned16(workspace))
    return FA_ERR_MISALIGNED;
  if (workspace_bytes < ws_layout(B, Hq, N, d).total) return FA_ERR_WORKSPACE_TOO_SMALL;
  const size_t qb = elems(B, Hq, N, d) * 2, kb = elems(B, Hkv, N, d) * 2;
  const Range ins[] = {range(q, qb), range(k, kb), range(v, kb), range(dO, qb)};
  const Range outs[] = {range(dk, kb), range(dv, kb), range(workspace, ws_layout(B, Hq, N, d).total)};
  for (const Range& o : outs)
    for (const Range& i : ins)
      if (overlap(o, i)) return FA_ERR_ALIASING;
  if (overlap(outs[0], outs[1]) || overlap(outs[0], outs[2]) || overlap(outs[1], outs[2])) return FA_ERR_ALIASING;
  return FA_OK;
}

fa_status dkdv(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv, int B, int Hq, int Hkv,
               int N, int d, int causal, int window, int with_dq, float scale, void* workspace,
               size_t workspace_bytes, void* stream) {
  FA_TRY(validate_dkdv(q, k, v, dO, dk, dv, B, Hq, Hkv, N, d, causal, scale, workspace, workspace_bytes));
  DeviceState* ds = nullptr;
  FA_TRY(device_state(&ds));
  fa::TmaMap4 tq, tk, tv, tdo;
  fa::TmaMap3 tdq;
  const WsLayout w = ws_layout(B, Hq, N, d);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  FA_TRY(tmap_bf16(&tq, q, B, Hq, N, d));
  FA_TRY(tmap_bf16(&tk, k, B, Hkv, N, d));
  FA_TRY(tmap_bf16(&tv, v, B, Hkv, N, d));
  FA_TRY(tmap_bf16(&tdo, dO, B, Hq, N, d));
  FA_TRY(tmap_dq_accum(&tdq, ws + w.dq_off, B, Hq, N, d));
  fa::BwdArgs a;
  a.lse2 = reinterpret_cast<const float*>(ws + w.lse2_off);
  a.drow = reinterpret_cast<const float*>(ws + w.dr_off);
  a.dq_accum = reinterpret_cast<float*>(ws + w.dq_off);
  a.dk = dk;
  a.dv = dv;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.N = N;
  a.causal = causal;
  a.window = window;
  a.with_dq = with_dq;
  a.v8 = ((reinterpret_cast<uintptr_t>(dk) | reinterpret_cast<uintptr_t>(dv)) & 31u) == 0;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  return launch_status(
      fa::launch_bwd_dkdv(d, tq, tk, tv, tdo, tdq, a, dev_status(ds), ds->num_sms, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int fa_version(void) { return 101; }

const char* fa_last_cuda_error(void) { return cudaGetErrorString(t_last_cuda_error); }

const char* fa_strerror(fa_status s) {
  switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_NULL_PTR: return "a required pointer is NULL";
    case FA_ERR_BAD_SHAPE:
      return "bad shape (B, Hq, Hkv, N must be >= 1, Hq % Hkv == 0, B <= 65535, N <= 8388480, "
             "ceil(N/128)*Hq*B < 2^31)";
    case FA_ERR_UNSUPPORTED_HEADDIM: return "unsupported head dimension (d must be 64 or 128)";
    case FA_ERR_MISALIGNED: return "a pointer is not 16-byte aligned";
    case FA_ERR_WORKSPACE_TOO_SMALL: return "workspace smaller than fa_bwd_workspace_bytes()";
    case FA_ERR_UNSUPPORTED_DEVICE: return "current device is not compute capability 10.3 (GB300)";
    case FA_ERR_LAUNCH: return "kernel launch or tensor-map encoding failed";
    case FA_ERR_DEVICE_TIMEOUT: return "a device-side bounded wait ran out";
    case FA_ERR_CUDA: return "CUDA runtime error";
    case FA_ERR_BAD_ARGUMENT: return "bad argument (scale must be finite and > 0, causal 0 or 1)";
    case FA_ERR_ALIASING: return "an output overlaps an input or another output";
    case FA_ERR_SCRATCH_LIMIT:
      return "problem needs more scratch than fa_bwd_noalloc's built-in buffer (FA_NOALLOC_SCRATCH_BYTES) holds";
    case FA_ERR_DEVICE_DRAIN:
      return "a kernel exited with its own copies or MMAs possibly in flight after a device-side timeout; "
             "no further launches on this device in this process";
    case FA_ERR_BAD_INDEX:
      return "a kernel read a page number, length, offset or axis out of range and skipped the access";
  }
  return "unknown status";
}

size_t fa_bwd_workspace_bytes(int B, int Hq, int Hkv, int N, int d) {
  if (check_shape(B, Hq, Hkv, N, d) != FA_OK) return 0;
  return ws_layout(B, Hq, N, d).total;
}

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int N,
                 int d, int causal, float scale, void* stream) {
  return fa_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, N, N, d, causal, 0, 1, scale, nullptr, 0, stream);
}

size_t fa_fwd_ex_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d, int num_splits) {
  if (check_shape_ex(B, Hq, Hkv, Nq, Nk, d) != FA_OK || num_splits < 1) return 0;
  if (num_splits == 1) return 0;
  return fwd_ws_layout(B, Hq, Nq, d, num_splits).total;
}

int fa_fwd_ex_default_splits(int B, int Hq, int Hkv, int Nq, int Nk, int d, int causal, int window) {
  if (check_shape_ex(B, Hq, Hkv, Nq, Nk, d) != FA_OK) return 1;
  DeviceState* ds = nullptr;
  if (device_state(&ds) != FA_OK) return 1;
  const FwdGeometry g = fwd_geometry(B, Hq, Hkv, Nq, Nk, 1);
  const long long units = (long long)g.units * g.nqt;
  int ntk = (Nk + 127) / 128;
  if (causal && window > 0) ntk = std::min(ntk, (window + 127) / 128 + 1);
  // Key tiles on the busiest SM, counting each item's fixed cost (its Q
  // load, pipeline fill and epilogue) as about two key tiles.
  int best = 1;
  long long best_cost = -1;
  for (int s = 1; s <= std::min(64, ntk); ++s) {
    const long long rounds = (units * s + ds->num_sms - 1) / ds->num_sms;
    const long long cost = rounds * ((ntk + s - 1) / s + 2);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

fa_status fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
                    int Nk, int d, int causal, int window, int num_splits, float scale, void* workspace,
                    size_t workspace_bytes, void* stream) {
  NvtxRange nv("fa_fwd_ex");
  if (!q || !k || !v || !o || !lse) return FA_ERR_NULL_PTR;
  FA_TRY(check_shape_ex(B, Hq, Hkv, Nq, Nk, d));
  FA_TRY(check_scale(causal, scale));
  if (window < 0 || (window > 0 && !causal) || (causal && Nq > Nk) || num_splits < 1 || num_splits > 4096)
    return FA_ERR_BAD_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse)) return FA_ERR_MISALIGNED;
  const FwdGeometry g = fwd_geometry(B, Hq, Hkv, Nq, Nk, num_splits);
  if ((long long)g.nqt * g.splits * g.units >= (1LL << 31)) return FA_ERR_BAD_SHAPE;
  const size_t qb = elems(B, Hq, Nq, d) * 2, kb = elems(B, Hkv, Nk, d) * 2;
  const Range ins[] = {range(q, qb), range(k, kb), range(v, kb)};
  const Range ro = range(o, qb), rl = range(lse, (size_t)B * Hq * Nq * 4);
  for (const Range& i : ins)
    if (overlap(ro, i) || overlap(rl, i)) return FA_ERR_ALIASING;
  if (overlap(ro, rl)) return FA_ERR_ALIASING;
  FwdWsLayout w{};
  if (g.splits > 1) {
    w = fwd_ws_layout(B, Hq, Nq, d, num_splits);
    if (!workspace) return FA_ERR_NULL_PTR;
    if (!aligned16(workspace)) return FA_ERR_MISALIGNED;
    if (workspace_bytes < w.total) return FA_ERR_WORKSPACE_TOO_SMALL;
    const Range rw = range(workspace, w.total);
    for (const Range& i : ins)
      if (overlap(rw, i)) return FA_ERR_ALIASING;
    if (overlap(rw, ro) || overlap(rw, rl)) return FA_ERR_ALIASING;
  }

  DeviceState* ds = nullptr;
  FA_TRY(device_state(&ds));
  fa::TmaMap3 tq;
  fa::TmaMap4 tk, tv, to;
  FA_TRY(tmap_rows_bf16(&tq, q, B, Hq, Nq, d));
  FA_TRY(tmap_bf16(&tk, k, B, Hkv, Nk, d));
  FA_TRY(tmap_bf16(&tv, v, B, Hkv, Nk, d));
  FA_TRY(tmap_bf16(&to, o, B, Hq, Nq, d));
  fa::FwdArgs a;
  a.o = o;
  a.lse = lse;
  a.o_part = g.splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.o_off) : nullptr;
  a.lse_part = g.splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.lse_off) : nullptr;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.Nq = Nq;
  a.Nk = Nk;
  a.causal = causal;
  a.window = window;
  a.packed = g.packed;
  a.nqt = g.nqt;
  a.units = g.units;
  a.splits = g.splits;
  a.split_tiles = g.split_tiles;
  a.scale_log2 = scale * 1.4426950408889634f;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  FA_TRY(launch_status(fa::launch_fwd(d, tq, tk, tv, to, a, dev_status(ds), ds->num_sms, st)));
  if (g.splits > 1) FA_TRY(launch_status(fa::launch_fwd_merge(d, a, ds->num_sms, st)));
  return FA_OK;
}

fa_status fa_bwd_preprocess(const void* o, const void* dO, const float* lse, int B, int Hq, int Hkv, int N, int d,
                            void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nv("fa_bwd_preprocess");
  if (!o || !dO || !lse || !workspace) return FA_ERR_NULL_PTR;
  FA_TRY(check_shape(B, Hq, Hkv, N, d));
  if (!aligned16(o) || !aligned16(dO) || !aligned16(lse) || !aligned16(workspace)) return FA_ERR_MISALIGNED;
  const WsLayout w = ws_layout(B, Hq, N, d);
  if (workspace_bytes < w.total) return FA_ERR_WORKSPACE_TOO_SMALL;
  const size_t qb = elems(B, Hq, N, d) * 2;
  const Range rw = range(workspace, w.total);
  if (overlap(rw, range(o, qb)) || overlap(rw, range(dO, qb)) || overlap(rw, range(lse, (size_t)B * Hq * N * 4)))
    return FA_ERR_ALIASING;
  DeviceState* ds = nullptr;
  FA_TRY(device_state(&ds));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return launch_status(fa::launch_bwd_preprocess(
      d, o, dO, lse, reinterpret_cast<float*>(ws + w.lse2_off), reinterpret_cast<float*>(ws + w.dr_off),
      reinterpret_cast<float*>(ws + w.dq_off), (long long)B * Hq, N, ds->num_sms, static_cast<cudaStream_t>(stream)));
}

fa_status fa_bwd_dkdv(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv, int B, int Hq,
                      int Hkv, int N, int d, int causal, float scale, void* workspace, size_t workspace_bytes,
                      void* stream) {
  NvtxRange nv("fa_bwd_dkdv");
  return dkdv(q, k, v, dO, dk, dv, B, Hq, Hkv, N, d, causal, 0, 1, scale, workspace, workspace_bytes, stream);
}



fa_status fa_bwd_dq_convert(void* dq, int B, int Hq, int Hkv, int N, int d, float scale, const void* workspace,
                            size_t workspace_bytes, void* stream) {
  NvtxRange nv("fa_bwd_dq_convert");
  if (!dq || !workspace) return FA_ERR_NULL_PTR;
  FA_TRY(check_shape(B, Hq, Hkv, N, d));
  FA_TRY(check_scale(0, scale));
  if (!aligned16(dq) || !aligned16(workspace)) return FA_ERR_MISALIGNED;
  const WsLayout w = ws_layout(B, Hq, N, d);
  if (workspace_bytes < w.total) return FA_ERR_WORKSPACE_TOO_SMALL;
  if (overlap(range(dq, elems(B, Hq, N, d) * 2), range(workspace, w.total))) return FA_ERR_ALIASING;
  DeviceState* ds = nullptr;
  FA_TRY(device_state(&ds));
  const uint8_t* ws = static_cast<const uint8_t*>(workspace);
  return launch_status(fa::launch_bwd_dq_convert(reinterpret_cast<const float*>(ws + w.dq_off), dq, scale,
                                                 (long long)elems(B, Hq, N, d), ds->num_sms,
                                                 static_cast<cudaStream_t>(stream)));
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                 void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int d, int causal, float scale,
                 void* workspace, size_t workspace_bytes, void* stream) {
  return fa_bwd_ex(q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, N, d, causal, 0, 0, scale, workspace,
                   workspace_bytes, stream);
}

fa_status fa_bwd_ex(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                    void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int d, int causal, int window,
                    int deterministic, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nv("fa_bwd_ex");
  if (!o || !dq || !lse) return FA_ERR_NULL_PTR;
  if (window < 0 || (window > 0 && !causal) || (deterministic != 0 && deterministic != 1)) return FA_ERR_BAD_ARGUMENT;
  FA_TRY(validate_dkdv(q, k, v, dO, dk, dv, B, Hq, Hkv, N, d, causal, scale, workspace, workspace_bytes));
  if (!aligned16(o) || !aligned16(dq) || !aligned16(lse)) return FA_ERR_MISALIGNED;
  const size_t qb = elems(B, Hq, N, d) * 2, kb = elems(B, Hkv, N, d) * 2;
  const Range rdq = range(dq, qb);
  const Range others[] = {range(q, qb),  range(k, kb),  range(v, kb),  range(o, qb), range(dO, qb),
                          range(lse, (size_t)B * Hq * N * 4), range(dk, kb), range(dv, kb),
                          range(workspace, ws_layout(B, Hq, N, d).total)};
  for (const Range& r : others)
    if (overlap(rdq, r)) return FA_ERR_ALIASING;
  const Range ro = range(o, qb);
  const Range rl = range(lse, (size_t)B * Hq * N * 4), rw = range(workspace, ws_layout(B, Hq, N, d).total);
  if (overlap(ro, range(dk, kb)) || overlap(ro, range(dv, kb)) || overlap(ro, rw)) return FA_ERR_ALIASING;
  if (overlap(rl, range(dk, kb)) || overlap(rl, range(dv, kb)) || overlap(rl, rw)) return FA_ERR_ALIASING;
  if (!deterministic) {
    FA_TRY(fa_bwd_preprocess(o, dO, lse, B, Hq, Hkv, N, d, workspace, workspace_bytes, stream));
    FA_TRY(dkdv(q, k, v, dO, dk, dv, B, Hq, Hkv, N, d, causal, window, 1, scale, workspace, workspace_bytes, stream));
    return fa_bwd_dq_convert(dq, B, Hq, Hkv, N, d, scale, workspace, workspace_bytes, stream);
  }
  // Deterministic: LSE*log2(e) and D only (no accumulator), dK/dV without
  // dQ partials, then dQ per query tile in a fixed order.
  DeviceState* ds = nullptr;
  FA_TRY(device_state(&ds));
  const WsLayout w = ws_layout(B, Hq, N, d);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  FA_TRY(launch_status(fa::launch_bwd_preprocess(d, o, dO, lse, reinterpret_cast<float*>(ws + w.lse2_off),
                                                 reinterpret_cast<float*>(ws + w.dr_off), nullptr, (long long)B * Hq,
                                                 N, ds->num_sms, st)));
  FA_TRY(dkdv(q, k, v, dO, dk, dv, B, Hq, Hkv, N, d, causal, window, 0, scale, workspace, workspace_bytes, stream));
  fa::TmaMap4 tq, tk, tv, tdo;
  FA_TRY(tmap_bf16(&tq, q, B, Hq, N, d));
  FA_TRY(tmap_bf16(&tk, k, B, Hkv, N, d));
  FA_TRY(tmap_bf16(&tv, v, B, Hkv, N, d));
  FA_TRY(tmap_bf16(&tdo, dO, B, Hq, N, d));
  fa::DqArgs a;
  a.lse2 = reinterpret_cast<const float*>(ws + w.lse2_off);
  a.drow = reinterpret_cast<const float*>(ws + w.dr_off);
  a.dq = dq;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.N = N;
  a.causal = causal;
  a.window = window;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  return launch_status(fa::launch_bwd_dq(d, tq, tk, tv, tdo, a, dev_status(ds), ds->num_sms, st));
}

fa_status fa_last_device_status(void* stream, int* detail) {
  NvtxRange nv("fa_last_device_status");
  FA_TRY_CUDA(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
  DeviceState* ds = nullptr;
  FA_TRY(device_state(&ds, false));
  int words[fa::kStatusWords] = {};
  FA_TRY_CUDA(cudaMemcpy(words, ds->status, sizeof(words), cudaMemcpyDeviceToHost));
  const int zero[fa::kStatusWords] = {};
  FA_TRY_CUDA(cudaMemcpy(ds->status, zero, sizeof(zero), cudaMemcpyHostToDevice));
  if (words[4] != 0 || ds->unusable) {
    // A block exited with copies or MMAs possibly still in flight: nothing
    // more is launched on this device by this process.
    {
      std::lock_guard<std::mutex> lock(g_mu);
      ds->unusable = true;
    }
    if (detail && words[4] != 0) {
      detail[0] = words[5];
      detail[1] = words[4];
      detail[2] = -1;
    }
    return FA_ERR_DEVICE_DRAIN;
  }
  if (detail) {
    detail[0] = words[1];
    detail[1] = words[2];
    detail[2] = words[3];
  }
  return static_cast<fa_status>(words[0]);
}

fa_status fa_selftest_wait_timeout(unsigned long long timeout_ns, void* stream) {
  if (timeout_ns < 1000ull || timeout_ns > 10000000000ull) return FA_ERR_BAD_ARGUMENT;
  DeviceState* ds = nullptr;
  FA_TRY(device_state(&ds));
  fa::DevStatus st{ds->status, timeout_ns};
  wait_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(st);
  return launch_status(cudaGetLastError());
}

fa_status fa_selftest_drain_timeout(unsigned long long timeout_ns, void* stream) {
  if (timeout_ns < 1000ull || timeout_ns > 10000000000ull) return FA_ERR_BAD_ARGUMENT;
  DeviceState* ds = nullptr;
  FA_TRY(device_state(&ds));
  fa::DevStatus st{ds->status, timeout_ns};
  drain_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(st);
  return launch_status(cudaGetLastError());
}

}  // extern "C"

// ---------------------------------------------------------------------------
// fa_bwd_noalloc: fa_bwd with its scratch in a buffer compiled into the
// library, for callers that cannot allocate device memory.
// ---------------------------------------------------------------------------
namespace {

// The scratch lives here, in the library's own device image: every device
// that loads the library holds these FA_NOALLOC_SCRATCH_BYTES until exit.
// In host code this name is only a stand-in for the symbol, not a device
// address; the address comes from cudaGetSymbolAddress below.
static __device__ __align__(256) unsigned char g_noalloc_scratch[FA_NOALLOC_SCRATCH_BYTES];

std::mutex g_noalloc_mu;
void* g_noalloc_ptr[kMaxDevices] = {};

// Device address of the scratch on the current device, looked up once per
// device with that device current.
fa_status noalloc_scratch(void** out) {
  int dev = -1;
  FA_TRY_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= kMaxDevices) return FA_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    FA_TRY_CUDA(cudaGetSymbolAddress(&p, g_noalloc_scratch));
    if (p == nullptr) return FA_ERR_CUDA;
    g_noalloc_ptr[dev] = p;
  }
  *out = g_noalloc_ptr[dev];
  return FA_OK;
}

}  // namespace

extern "C" fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dO,
                                    const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N,
                                    int d, int causal, float scale, void* stream) {
  NvtxRange nv("fa_bwd_noalloc");
  FA_TRY(check_shape(B, Hq, Hkv, N, d));
  if (ws_layout(B, Hq, N, d).total > (size_t)FA_NOALLOC_SCRATCH_BYTES) return FA_ERR_SCRATCH_LIMIT;
  if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return FA_ERR_NULL_PTR;
  FA_TRY(check_scale(causal, scale));
  DeviceState* ds = nullptr;
  FA_TRY(device_state(&ds));
  void* scratch = nullptr;
  FA_TRY(noalloc_scratch(&scratch));
  // fa_bwd clears the dQ accumulator in its first kernel, so whatever the
  // previous call left in the scratch does not matter.
  return fa_bwd(q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale, scratch,
                (size_t)FA_NOALLOC_SCRATCH_BYTES, stream);
}

// ---------------------------------------------------------------------------
// Rotary positions and the paged cache
// ---------------------------------------------------------------------------
namespace {

constexpr long long kMaxSpan = 1LL << 46;   // elements one dimension may span

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Rows of `row` contiguous elements over up to three strided dimensions, in
// bytes; dimensions of size 1 are dropped, the others sorted by stride, the
// largest first.
struct View {
  uintptr_t base = 0;
  unsigned long long row = 0;
  int n = 0;
  unsigned long long size[3] = {}, stride[3] = {};

  // First byte past the last row of dimensions [from, n).
  unsigned long long extent(int from = 0) const {
    unsigned long long e = row;
    for (int i = from; i < n; ++i) e += (size[i] - 1) * stride[i];
    return e;
  }
  // Every dimension's steps clear what lies inside it, so no two rows meet.
  bool distinct() const {
    for (int i = 0; i < n; ++i)
      if (stride[i] < extent(i + 1)) return false;
    return true;
  }
};

View view(const void* p, long long row, int elem, std::initializer_list<std::pair<long long, long long>> dims) {
  View v;
  v.base = reinterpret_cast<uintptr_t>(p);
  v.row = (unsigned long long)row * elem;
  for (const auto& d : dims)
    if (d.first > 1) {
      int i = v.n++;
      for (; i > 0 && v.stride[i - 1] < (unsigned long long)d.second * elem; --i) {
        v.size[i] = v.size[i - 1];
        v.stride[i] = v.stride[i - 1];
      }
      v.size[i] = (unsigned long long)d.first;
      v.stride[i] = (unsigned long long)d.second * elem;
    }
  return v;
}
View bytes_view(const void* p, size_t n) { return view(p, (long long)n, 1, {}); }

// Whether no byte of a's rows is one of b's: their address ranges are apart,
// or both step alike through their outer dimensions and are apart inside one
// step (the q, k and v parts of one projection's output).
bool apart(const View& a, const View& b) {
  if (a.base + a.extent() <= b.base || b.base + b.extent() <= a.base) return true;
  const uintptr_t lo = std::min(a.base, b.base);
  for (int outer = 1; outer <= a.n && outer <= b.n; ++outer) {
    const int i = outer - 1;
    if (a.stride[i] != b.stride[i]) return false;
    const uintptr_t ea = a.base + a.extent(outer), eb = b.base + b.extent(outer);
    // The span of both inside one step must fit the step, and the steps of
    // this level must fit one step of the level outside it (the larger count).
    const unsigned long long span = std::max(ea, eb) - lo;
    if (i > 0 && std::max(a.size[i], b.size[i]) * a.stride[i] > a.stride[i - 1]) return false;
    if (span <= a.stride[i] && (ea <= b.base || eb <= a.base)) return true;
  }
  return false;
}

// Strides of the dimensions larger than 1: none negative, all multiples of 8
// elements, and small enough that no address computation overflows.
fa_status check_strides(std::initializer_list<std::pair<long long, long long>> dims) {
  for (const auto& d : dims)
    if (d.first > 1) {
      if (d.second < 0 || d.second > kMaxSpan / d.first) return FA_ERR_BAD_ARGUMENT;
      if (d.second % 8) return FA_ERR_MISALIGNED;
    }
  return FA_OK;
}

long long stride_of(long long size, long long stride) { return size > 1 ? stride : 0; }

// In place: every row is written where it is read.  (The same rows in another
// order, as with two dimensions exchanged, would be read after they are lost.)
bool in_place(const fa::RowView& out, const fa::RowView& in) {
  return out.p == in.p && out.sb == in.sb && out.sh == in.sh && out.sn == in.sn;
}

fa_status check_rotary(const fa_rotary* r, int d) {
  if (!r->positions || !r->inv_freq || !r->axes) return FA_ERR_NULL_PTR;
  if (r->rot < 16 || r->rot > d || r->rot % 16 || r->n_axes < 1 || r->n_axes > 1024 || (r->interleaved != 0 && r->interleaved != 1) ||
      r->axis_stride < 0 || r->axis_stride > kMaxSpan / 1024 || r->batch_stride < 0 || r->batch_stride > (1LL << 31))
    return FA_ERR_BAD_ARGUMENT;
  if (!aligned(r->positions, 4) || !aligned(r->inv_freq, 8) || !aligned(r->axes, 4)) return FA_ERR_MISALIGNED;
  return FA_OK;
}

fa::RotaryArgs rotary_args(const fa_rotary* r, int inverse) {
  return fa::RotaryArgs{r->positions, r->axis_stride, r->batch_stride, r->inv_freq, r->axes,
                        r->n_axes,    r->rot,         r->interleaved,  inverse};
}

fa_status check_dtype(int dtype) { return dtype == FA_BF16 || dtype == FA_FP16 ? FA_OK : FA_ERR_BAD_ARGUMENT; }

View kv_view(const fa_paged_kv* kv, const void* p) {
  return view(p, kv->d, 2,
              {{kv->num_pages, kv->page_stride}, {kv->Hkv, kv->head_stride}, {kv->page_size, kv->slot_stride}});
}

fa_status check_kv(const fa_paged_kv* kv) {
  if (!kv || !kv->k || !kv->v) return FA_ERR_NULL_PTR;
  FA_TRY(check_dtype(kv->dtype));
  if (kv->num_pages < 1 || kv->Hkv < 1 || kv->page_size < 16 || kv->page_size > 65536 || kv->page_size % 16)
    return FA_ERR_BAD_SHAPE;
  if (kv->d != 64 && kv->d != 128) return FA_ERR_UNSUPPORTED_HEADDIM;
  FA_TRY(check_strides({{kv->num_pages, kv->page_stride}, {kv->Hkv, kv->head_stride}, {kv->page_size, kv->slot_stride}}));
  if (!aligned16(kv->k) || !aligned16(kv->v)) return FA_ERR_MISALIGNED;
  return kv_view(kv, kv->k).distinct() ? FA_OK : FA_ERR_BAD_ARGUMENT;
}

View scores_view(const fa_paged_kv* kv, const float* s) {
  return bytes_view(s, (size_t)kv->num_pages * kv->Hkv * kv->page_size * 4);
}

fa_status check_table(const fa_page_table* t, int B, int page_size) {
  if (!t || !t->pages) return FA_ERR_NULL_PTR;
  if (t->max_pages < 1 || (long long)t->max_pages * page_size > (1LL << 30)) return FA_ERR_BAD_SHAPE;
  if (B > 1 && (t->stride < 0 || t->stride > (1LL << 31))) return FA_ERR_BAD_ARGUMENT;
  return aligned(t->pages, 4) ? FA_OK : FA_ERR_MISALIGNED;
}

View table_view(const fa_page_table* t, int B) { return view(t->pages, t->max_pages, 4, {{B, t->stride}}); }

fa::PagedKv kv_args(const fa_paged_kv* kv) {
  return fa::PagedKv{kv->k,
                     kv->v,
                     stride_of(kv->num_pages, kv->page_stride),
                     stride_of(kv->Hkv, kv->head_stride),
                     stride_of(kv->page_size, kv->slot_stride),
                     kv->num_pages,
                     kv->page_size,
                     kv->Hkv,
                     kv->d};
}

fa::PageTable table_args(const fa_page_table* t) { return fa::PageTable{t->pages, t->stride, t->max_pages}; }

// K or V pool as {d, page_size, Hkv, num_pages} with a 16-slot box.  The
// stride of a dimension of size 1 is never stepped: any valid value does.
fa_status tmap_pool(fa::TmaMap4* m, const fa_paged_kv* kv, const void* base) {
  auto bytes = [&](long long size, long long stride) { return (cuuint64_t)(size > 1 ? stride : kv->d) * 2; };
  cuuint64_t dims[4] = {(cuuint64_t)kv->d, (cuuint64_t)kv->page_size, (cuuint64_t)kv->Hkv, (cuuint64_t)kv->num_pages};
  cuuint64_t strides[3] = {bytes(kv->page_size, kv->slot_stride), bytes(kv->Hkv, kv->head_stride),
                           bytes(kv->num_pages, kv->page_stride)};
  cuuint32_t box[4] = {64, 16, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = g_encode(&m->m, kv->dtype == FA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                              4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_LAUNCH;
}

// Decode workspace: the CTAs' parts, what they left of cut units with its
// (max, sum), and, with scores, the LSE and every key's scores.
struct DecodeWs {
  size_t parts, part, ml, lse2, stash, total;
};
DecodeWs decode_ws(int B, int Hq, int d, int page_size, int max_pages, bool with_scores) {
  DecodeWs w{};
  const size_t slots = (size_t)fa::kDecodeMaxParts * 2 * 16;
  w.parts = 0;
  w.part = align256((size_t)fa::kDecodeMaxParts * sizeof(fa::DecodePart));
  w.ml = w.part + slots * d * 4;
  w.lse2 = w.ml + slots * 8;
  w.stash = w.lse2 + (with_scores ? align256((size_t)B * Hq * 4) : 0);
  w.total = w.stash + (with_scores ? align256((size_t)B * Hq * page_size * max_pages * 4) : 0);
  return w;
}

// CTAs of the cluster that takes a unit of at most `tiles` tiles, where `units`
// of them are decoded by clusters, or 0 for equal parts of all tiles, which
// take a second kernel to join them and a scan of the lengths at the start,
// 3-5 us together, the time of about 4 tiles of a CTA.  So clusters, as large as
// the `slots` CTAs that run at a time allow, where the busiest CTA gets no more
// than 4 tiles above an equal part, and no more than 12: lengths that differ
// leave CTAs idle, equal parts don't.  (With scores the weights of a kv head
// must be summed in one place, so its heads must be one unit's.  Calls on a
// stream, pages of 16, 32 q and 8 kv heads, d = 128, tiles of 64 keys, us by
// clusters | equal parts: 1 sequence of 2000 keys 7.7 | 9.0, of 4000 11.1 | 10.1;
// 8 of 1000 9.0 | 12.5, of 2000 15.0 | 18.9; 64 of 250 18.7 | 19.4; 128 of 250 35.8 |
// 30.1; lengths from 0 to 2000 in equal steps, 8 sequences 11.6 | 12.7, 32 33.1 |
// 30.3; 32 from 0 to 1000, 16 tiles a CTA, 19.1 | 21.6, with scores 23.6 | 24.2; 8
// from 0 to 8000, d = 64, 16 tiles, with scores, 28.7 | 22.8.  128 q heads, 8 of
// 1000 12.0 | 19.2.  The 4-bit cache, tiles of 128 keys, in a graph: 1 sequence of 2000
// keys 7.4 | 10.8, of 8000, 8 tiles a CTA, 12.6 | 13.5; 4 of 2000 9.0 | 13.7; 16 of 1000
// 11.2 | 15.4; 64 of 600 23.2 | 24.6; 32 of up to 4096, 16 heads a group, 16 tiles a CTA,
// 26.8 | 25.2.)
int decode_cluster(long long units, long long tiles, int slots) {
  int c = 1;
  while (c < fa::kMaxCluster && units * c * 2 <= slots && c < tiles) c *= 2;
  if (units * c > 2 * slots) return 0;
  const long long waves = (units * c + slots - 1) / slots, busiest = (tiles + c - 1) / c;
  return busiest <= 12 && waves * busiest <= (units * tiles + slots - 1) / slots + 4 ? c : 0;
}

// device_state, with the kernels of this section set up (on their first use,
// so that callers of the attention alone do not wait for it).
fa_status paged_device_state(DeviceState** out) {
  FA_TRY(device_state(out));
  if ((*out)->paged_ready) return FA_OK;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!(*out)->paged_ready) {
    const cudaError_t e = fa::configure_paged_kernels();
    if (e != cudaSuccess) return launch_status(e);
    (*out)->paged_ready = true;
  }
  return FA_OK;
}

// Each output apart from every input and every other output.
template <size_t NO, size_t NI>
bool outputs_apart(const View (&outs)[NO], const View (&ins)[NI]) {
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = 0; j < NI; ++j)
      if (!apart(outs[i], ins[j])) return false;
    for (size_t j = 0; j < i; ++j)
      if (!apart(outs[i], outs[j])) return false;
  }
  return true;
}

}  // namespace

extern "C" {

fa_status fa_rope(const void* q, const long long* q_strides, void* q_out, const long long* q_out_strides, const void* k,
                  const long long* k_strides, void* k_out, const long long* k_out_strides, int B, int Hq, int Hk, int N,
                  int d, int dtype, const fa_rotary* rotary, int inverse, void* stream) {
  NvtxRange nv("fa_rope");
  if (!q || !q_strides || !q_out || !q_out_strides || !rotary) return FA_ERR_NULL_PTR;
  if (Hk != 0 && (!k || !k_strides || !k_out || !k_out_strides)) return FA_ERR_NULL_PTR;
  if (Hk < 0 || (Hk == 0 && (k || k_out))) return FA_ERR_BAD_SHAPE;
  if (B < 1 || Hq < 1 || N < 1 || (long long)B * N >= (1LL << 31) || (long long)Hq + Hk > 65535) return FA_ERR_BAD_SHAPE;
  if (d < 16 || d > 256 || d % 16) return FA_ERR_UNSUPPORTED_HEADDIM;
  FA_TRY(check_dtype(dtype));
  if (inverse != 0 && inverse != 1) return FA_ERR_BAD_ARGUMENT;
  FA_TRY(check_rotary(rotary, d));
  const void* ptrs[4] = {q, q_out, k, k_out};
  const long long* strides[4] = {q_strides, q_out_strides, k_strides, k_out_strides};
  fa::RowView rows[4] = {};
  View views[4];
  const int n = Hk ? 4 : 2;
  for (int i = 0; i < n; ++i) {
    const int H = i < 2 ? Hq : Hk;
    const long long* s = strides[i];
    FA_TRY(check_strides({{B, s[0]}, {H, s[1]}, {N, s[2]}}));
    if (!aligned16(ptrs[i])) return FA_ERR_MISALIGNED;
    rows[i] = fa::RowView{const_cast<void*>(ptrs[i]), stride_of(B, s[0]), stride_of(H, s[1]), stride_of(N, s[2])};
    views[i] = view(ptrs[i], d, 2, {{B, s[0]}, {H, s[1]}, {N, s[2]}});
  }
  const View tables[3] = {
      view(rotary->positions, N, 4, {{rotary->n_axes, rotary->axis_stride}, {B, rotary->batch_stride}}),
      bytes_view(rotary->inv_freq, (size_t)rotary->rot / 2 * 8), bytes_view(rotary->axes, (size_t)rotary->rot / 2 * 4)};
  for (int i = 1; i < n; i += 2) {
    if (!views[i].distinct()) return FA_ERR_ALIASING;
    for (int j = 0; j < n; ++j)
      if (j != i && !(j == i - 1 && in_place(rows[i], rows[j])) && !apart(views[i], views[j])) return FA_ERR_ALIASING;
    for (const View& t : tables)
      if (!apart(views[i], t)) return FA_ERR_ALIASING;
  }
  DeviceState* ds = nullptr;
  FA_TRY(paged_device_state(&ds));
  const fa::RopeArgs a{rows[0], rows[1], rows[2], rows[3], B, Hq, Hk, N, d, rotary_args(rotary, inverse)};
  return launch_status(fa::launch_rope(dtype, a, dev_status(ds), ds->num_sms, static_cast<cudaStream_t>(stream)));
}

fa_status fa_paged_append(const fa_paged_kv* kv, const fa_page_table* table, const int* seq_lens, const int* cu_seqlens,
                          int B, int T, const void* k, const long long* k_strides, const void* v,
                          const long long* v_strides, const void* q, const long long* q_strides, void* q_out,
                          const long long* q_out_strides, int Hq, const fa_rotary* rotary, float* scores, void* stream) {
  NvtxRange nv("fa_paged_append");
  FA_TRY(check_kv(kv));
  if (!seq_lens || !k_strides || !v_strides || (T != 0 && (!k || !v))) return FA_ERR_NULL_PTR;
  if (B < 1 || T < 0 || (!cu_seqlens && T != B)) return FA_ERR_BAD_SHAPE;
  FA_TRY(check_table(table, B, kv->page_size));
  if (!aligned(seq_lens, 4) || !aligned(cu_seqlens, 4) || !aligned16(scores)) return FA_ERR_MISALIGNED;
  if (q && !rotary) return FA_ERR_BAD_ARGUMENT;
  if (q ? (!q_out || !q_strides || !q_out_strides) : q_out != nullptr) return FA_ERR_NULL_PTR;
  if (q ? Hq < 1 : Hq != 0) return FA_ERR_BAD_SHAPE;
  if ((long long)Hq + 2LL * kv->Hkv > 65535) return FA_ERR_BAD_SHAPE;
  if (rotary) FA_TRY(check_rotary(rotary, kv->d));
  if (T == 0) return FA_OK;
  const void* ptrs[4] = {k, v, q, q_out};
  const long long* strides[4] = {k_strides, v_strides, q_strides, q_out_strides};
  fa::RowView rows[4] = {};
  View views[4];
  const int n = q ? 4 : 2;
  for (int i = 0; i < n; ++i) {
    const int H = i < 2 ? kv->Hkv : Hq;
    const long long* s = strides[i];
    FA_TRY(check_strides({{T, s[0]}, {H, s[1]}}));
    if (!aligned16(ptrs[i])) return FA_ERR_MISALIGNED;
    rows[i] = fa::RowView{const_cast<void*>(ptrs[i]), 0, stride_of(H, s[1]), stride_of(T, s[0])};
    views[i] = view(ptrs[i], kv->d, 2, {{T, s[0]}, {H, s[1]}});
  }
  View small[6];
  int ns = 0;
  small[ns++] = table_view(table, B);
  small[ns++] = bytes_view(seq_lens, (size_t)B * 4);
  if (cu_seqlens) small[ns++] = bytes_view(cu_seqlens, (size_t)(B + 1) * 4);
  if (rotary) {
    small[ns++] = view(rotary->positions, T, 4, {{rotary->n_axes, rotary->axis_stride}});
    small[ns++] = bytes_view(rotary->inv_freq, (size_t)rotary->rot / 2 * 8);
    small[ns++] = bytes_view(rotary->axes, (size_t)rotary->rot / 2 * 4);
  }
  View outs[4] = {kv_view(kv, kv->k), kv_view(kv, kv->v)};
  int no = 2;
  if (scores) outs[no++] = scores_view(kv, scores);
  const int qo = q ? no : -1;
  if (q) outs[no++] = views[3];
  for (int i = 0; i < no; ++i) {
    if (!outs[i].distinct()) return FA_ERR_ALIASING;
    for (int j = 0; j < (q ? 3 : 2); ++j)
      if (!(i == qo && j == 2 && in_place(rows[3], rows[2])) && !apart(outs[i], views[j])) return FA_ERR_ALIASING;
    for (int j = 0; j < i; ++j)
      if (!apart(outs[i], outs[j])) return FA_ERR_ALIASING;
    for (int j = 0; j < ns; ++j)
      if (!apart(outs[i], small[j])) return FA_ERR_ALIASING;
  }
  DeviceState* ds = nullptr;
  FA_TRY(paged_device_state(&ds));
  fa::AppendArgs a{};
  a.k = rows[0];
  a.v = rows[1];
  a.q = rows[2];
  a.q_out = rows[3];
  a.kv = kv_args(kv);
  a.table = table_args(table);
  a.seq_lens = seq_lens;
  a.cu = cu_seqlens;
  a.scores = scores;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  if (rotary) a.r = rotary_args(rotary, 0);
  return launch_status(fa::launch_append(kv->dtype, a, dev_status(ds), ds->num_sms, static_cast<cudaStream_t>(stream)));
}

size_t fa_paged_decode_workspace_bytes(int B, int Hq, int Hkv, int d, int page_size, int max_pages, int with_scores) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || (d != 64 && d != 128) || page_size < 16 || page_size > 65536 ||
      page_size % 16 || max_pages < 1 || (long long)max_pages * page_size > (1LL << 30) ||
      (long long)B * Hq >= (1LL << 31))
    return 0;
  return decode_ws(B, Hq, d, page_size, max_pages, with_scores != 0).total;
}

fa_status fa_paged_decode(const void* q, const long long* q_strides, const fa_paged_kv* kv, const fa_page_table* table,
                          const int* seq_lens, void* o, float* lse, float* scores, int B, int Hq, int window,
                          float scale, void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nv("fa_paged_decode");
  FA_TRY(check_kv(kv));
  if (!q || !q_strides || !seq_lens || !o || !lse || !workspace) return FA_ERR_NULL_PTR;
  if (B < 1 || Hq < 1 || Hq % kv->Hkv || (long long)B * Hq >= (1LL << 31)) return FA_ERR_BAD_SHAPE;
  FA_TRY(check_table(table, B, kv->page_size));
  FA_TRY(check_scale(0, scale));
  if (window < 0) return FA_ERR_BAD_ARGUMENT;
  FA_TRY(check_strides({{B, q_strides[0]}, {Hq, q_strides[1]}}));
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || !aligned16(scores) || !aligned16(workspace) ||
      !aligned(seq_lens, 4))
    return FA_ERR_MISALIGNED;
  const size_t need =
      fa_paged_decode_workspace_bytes(B, Hq, kv->Hkv, kv->d, kv->page_size, table->max_pages, scores ? 1 : 0);
  if (need == 0) return FA_ERR_BAD_SHAPE;
  if (workspace_bytes < need) return FA_ERR_WORKSPACE_TOO_SMALL;
  const View ins[] = {view(q, kv->d, 2, {{B, q_strides[0]}, {Hq, q_strides[1]}}), kv_view(kv, kv->k), kv_view(kv, kv->v),
                      table_view(table, B), bytes_view(seq_lens, (size_t)B * 4)};
  const View outs[] = {bytes_view(o, (size_t)B * Hq * kv->d * 2), bytes_view(lse, (size_t)B * Hq * 4),
                       bytes_view(workspace, need), scores ? scores_view(kv, scores) : bytes_view(nullptr, 0)};
  if (!outputs_apart(outs, ins)) return FA_ERR_ALIASING;
  DeviceState* ds = nullptr;
  FA_TRY(paged_device_state(&ds));
  fa::DecodeArgs a{};
  a.q = q;
  a.q_sb = stride_of(B, q_strides[0]);
  a.q_sh = stride_of(Hq, q_strides[1]);
  a.kv = kv_args(kv);
  a.table = table_args(table);
  a.seq_lens = seq_lens;
  a.o = o;
  a.lse = lse;
  a.scores = scores;
  a.B = B;
  a.Hq = Hq;
  a.window = window;
  a.scale_log2 = scale * 1.4426950408889634f;
  const int G = Hq / kv->Hkv;
  a.unit_heads = G <= 8 ? 8 : 16;
  const DecodeWs w = decode_ws(B, Hq, kv->d, kv->page_size, table->max_pages, scores != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.parts = reinterpret_cast<fa::DecodePart*>(ws + w.parts);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.lse2 = scores ? reinterpret_cast<float*>(ws + w.lse2) : nullptr;
  a.stash = scores ? reinterpret_cast<float*>(ws + w.stash) : nullptr;
  a.stash_keys = (long long)kv->page_size * table->max_pages;
  const long long units = (long long)B * kv->Hkv * ((G + a.unit_heads - 1) / a.unit_heads);
  const int keys = fa::decode_tile_keys(kv->d);
  long long unit_tiles = (a.stash_keys + keys - 1) / keys;           // at most
  if (window > 0) unit_tiles = std::min(unit_tiles, (window - 1LL) / keys + 2);
  // Two CTAs per SM, but no more than there can be tiles.
  int parts = (int)std::min<long long>(units * unit_tiles, std::min(2 * ds->num_sms, fa::kDecodeMaxParts));
  if (!scores || G <= a.unit_heads) {
    const int c = decode_cluster(units, unit_tiles, 2 * ds->num_sms);
    a.cluster = c;
    if (c) parts = (int)units * c;
  }
  fa::TmaMap4 tk, tv;
  FA_TRY(tmap_pool(&tk, kv, kv->k));
  FA_TRY(tmap_pool(&tv, kv, kv->v));
  return launch_status(fa::launch_paged_decode(kv->dtype, tk, tv, a, dev_status(ds), parts,
                                               static_cast<cudaStream_t>(stream)));
}

fa_status fa_paged_evict(const fa_paged_kv* kv, float* scores, const fa_page_table* table, const int* seq_lens,
                         const fa_page_table* dst, int* new_lens, int* kept, int B, int budget, int recent, int sinks,
                         void* stream) {
  NvtxRange nv("fa_paged_evict");
  FA_TRY(check_kv(kv));
  if (!scores || !seq_lens || !new_lens || !kept) return FA_ERR_NULL_PTR;
  // Grids: up to 8 CTAs, and a block per 32 kept keys, for each (sequence, kv head).
  if (B < 1 || (long long)B * kv->Hkv >= (1LL << 27) ||
      (long long)B * kv->Hkv * (((long long)budget + 31) / 32) >= (1LL << 31))
    return FA_ERR_BAD_SHAPE;
  FA_TRY(check_table(table, B, kv->page_size));
  FA_TRY(check_table(dst, B, kv->page_size));
  if (budget < 1 || recent < 0 || sinks < 0 || (long long)recent + sinks > budget ||
      (long long)dst->max_pages * kv->page_size < budget)
    return FA_ERR_BAD_ARGUMENT;
  if (!aligned16(scores) || !aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(kept, 4)) return FA_ERR_MISALIGNED;
  const View ins[] = {table_view(table, B), bytes_view(seq_lens, (size_t)B * 4), table_view(dst, B)};
  const View outs[] = {kv_view(kv, kv->k), kv_view(kv, kv->v), scores_view(kv, scores), bytes_view(new_lens, (size_t)B * 4),
                       bytes_view(kept, (size_t)B * kv->Hkv * budget * 4)};
  if (!outputs_apart(outs, ins) || dst->pages == table->pages) return FA_ERR_ALIASING;
  DeviceState* ds = nullptr;
  FA_TRY(paged_device_state(&ds));
  fa::EvictArgs a{};
  a.kv = kv_args(kv);
  a.scores = scores;
  a.table = table_args(table);
  a.dst = table_args(dst);
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.kept = kept;
  a.B = B;
  a.budget = budget;
  a.recent = recent;
  a.sinks = sinks;
  return launch_status(fa::launch_paged_evict(a, dev_status(ds), ds->num_sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Norms with rotary positions, and the 4-bit cache
// ---------------------------------------------------------------------------
namespace {

fa_status check_norm(const fa_qk_norm* n) {
  if ((n->weights_fp32 != 0 && n->weights_fp32 != 1) || !(n->eps >= 0.f) || std::isinf(n->eps)) return FA_ERR_BAD_ARGUMENT;
  const size_t by = n->weights_fp32 ? 4 : 16;
  if (!aligned(n->q_weight, by) || !aligned(n->k_weight, by)) return FA_ERR_MISALIGNED;
  return FA_OK;
}

fa::NormArgs norm_args(const fa_qk_norm* n) {
  return n ? fa::NormArgs{n->q_weight, n->k_weight, n->weights_fp32, 1, n->eps} : fa::NormArgs{};
}

// What a call reads by element: the rotation's arrays (three), the norm's weights (two),
// and an append's table, lengths and offsets.
struct Tables {
  View v[3 + 2 + 3];
  int n = 0;
  void add(const View& x) { v[n++] = x; }
  void rotary(const fa_rotary* r, int B, int N) {
    if (!r) return;
    add(view(r->positions, N, 4, {{r->n_axes, r->axis_stride}, {B, r->batch_stride}}));
    add(bytes_view(r->inv_freq, (size_t)r->rot / 2 * 8));
    add(bytes_view(r->axes, (size_t)r->rot / 2 * 4));
  }
  void norm(const fa_qk_norm* n_, int d) {
    if (!n_) return;
    const size_t bytes = (size_t)d * (n_->weights_fp32 ? 4 : 2);
    if (n_->q_weight) add(bytes_view(n_->q_weight, bytes));
    if (n_->k_weight) add(bytes_view(n_->k_weight, bytes));
  }
  bool apart_from(const View& out) const {
    for (int i = 0; i < n; ++i)
      if (!apart(out, v[i])) return false;
    return true;
  }
};

fa_status check_rows(int B, int Hq, int Hk, int N, int d, int dtype) {
  if (B < 1 || Hq < 1 || Hk < 0 || N < 1 || (long long)B * N >= (1LL << 31) || (long long)Hq + Hk > 65535)
    return FA_ERR_BAD_SHAPE;
  if (d < 16 || d > 256 || d % 16) return FA_ERR_UNSUPPORTED_HEADDIM;
  return check_dtype(dtype);
}

// [B,H,N,d] rows of a call.
fa_status rows_of(const void* p, const long long* s, int B, int H, int N, int d, fa::RowView& r, View& v) {
  FA_TRY(check_strides({{B, s[0]}, {H, s[1]}, {N, s[2]}}));
  if (!aligned16(p)) return FA_ERR_MISALIGNED;
  r = fa::RowView{const_cast<void*>(p), stride_of(B, s[0]), stride_of(H, s[1]), stride_of(N, s[2])};
  v = view(p, d, 2, {{B, s[0]}, {H, s[1]}, {N, s[2]}});
  return FA_OK;
}

View kv4_view(const fa_paged4_kv* kv) {
  return view(kv->data, (long long)kv->page_size * (kv->d + kv->d / 8), 1,
              {{kv->num_pages, kv->page_stride}, {kv->Hkv, kv->head_stride}});
}

fa_status check_kv4(const fa_paged4_kv* kv) {
  if (!kv || !kv->data) return FA_ERR_NULL_PTR;
  FA_TRY(check_dtype(kv->dtype));
  if (kv->num_pages < 1 || kv->Hkv < 1 || kv->page_size < 16 || kv->page_size > 65536 || kv->page_size % 16)
    return FA_ERR_BAD_SHAPE;
  if (kv->d != 64 && kv->d != 128) return FA_ERR_UNSUPPORTED_HEADDIM;
  for (const auto& d : {std::pair<long long, long long>{kv->num_pages, kv->page_stride}, {kv->Hkv, kv->head_stride}})
    if (d.first > 1) {
      if (d.second < 0 || d.second > kMaxSpan / d.first) return FA_ERR_BAD_ARGUMENT;
      if (d.second % 16) return FA_ERR_MISALIGNED;
    }
  if (!aligned16(kv->data)) return FA_ERR_MISALIGNED;
  return kv4_view(kv).distinct() ? FA_OK : FA_ERR_BAD_ARGUMENT;
}

fa::PagedKv kv4_args(const fa_paged4_kv* kv) {
  return fa::PagedKv{kv->data,
                     kv->data,
                     stride_of(kv->num_pages, kv->page_stride),
                     stride_of(kv->Hkv, kv->head_stride),
                     0,
                     kv->num_pages,
                     kv->page_size,
                     kv->Hkv,
                     kv->d};
}

// As paged_device_state, for the kernels of this section.
fa_status paged4_device_state(DeviceState** out) {
  FA_TRY(device_state(out));
  if ((*out)->paged4_ready) return FA_OK;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!(*out)->paged4_ready) {
    const cudaError_t e = fa::configure_paged4_kernels();
    if (e != cudaSuccess) return launch_status(e);
    (*out)->paged4_ready = true;
  }
  return FA_OK;
}

}  // namespace

extern "C" {

fa_status fa_qk_norm_rope(const void* q, const long long* q_strides, void* q_out, const long long* q_out_strides,
                          const void* k, const long long* k_strides, void* k_out, const long long* k_out_strides, int B,
                          int Hq, int Hk, int N, int d, int dtype, const fa_qk_norm* norm, const fa_rotary* rotary,
                          void* stream) {
  NvtxRange nv("fa_qk_norm_rope");
  if (!q || !q_strides || !q_out || !q_out_strides || !norm) return FA_ERR_NULL_PTR;
  if (Hk != 0 && (!k || !k_strides || !k_out || !k_out_strides)) return FA_ERR_NULL_PTR;
  if (Hk == 0 && (k || k_out)) return FA_ERR_BAD_SHAPE;
  FA_TRY(check_rows(B, Hq, Hk, N, d, dtype));
  FA_TRY(check_norm(norm));
  if (rotary) FA_TRY(check_rotary(rotary, d));
  fa::RowView rows[4] = {};
  View views[4];
  FA_TRY(rows_of(q, q_strides, B, Hq, N, d, rows[0], views[0]));
  FA_TRY(rows_of(q_out, q_out_strides, B, Hq, N, d, rows[1], views[1]));
  if (Hk) {
    FA_TRY(rows_of(k, k_strides, B, Hk, N, d, rows[2], views[2]));
    FA_TRY(rows_of(k_out, k_out_strides, B, Hk, N, d, rows[3], views[3]));
  }
  Tables tables;
  tables.rotary(rotary, B, N);
  tables.norm(norm, d);
  const int n = Hk ? 4 : 2;
  for (int i = 1; i < n; i += 2) {
    if (!views[i].distinct() || !tables.apart_from(views[i])) return FA_ERR_ALIASING;
    for (int j = 0; j < n; ++j)
      if (j != i && !(j == i - 1 && in_place(rows[i], rows[j])) && !apart(views[i], views[j])) return FA_ERR_ALIASING;
  }
  DeviceState* ds = nullptr;
  FA_TRY(paged4_device_state(&ds));
  const fa::NormRopeArgs a{rows[0], rows[1], rows[2], rows[3], B, Hq, Hk, N, d,
                           rotary ? rotary_args(rotary, 0) : fa::RotaryArgs{}, norm_args(norm)};
  return launch_status(fa::launch_norm_rope(dtype, a, dev_status(ds), ds->num_sms, static_cast<cudaStream_t>(stream)));
}

size_t fa_qk_norm_rope_bwd_workspace_bytes(int d) {
  return d < 16 || d > 256 || d % 16 ? 0 : (size_t)fa::kNormBwdMaxBlocks * d * 4;
}

fa_status fa_qk_norm_rope_bwd(const void* dq_out, const long long* dq_out_strides, const void* q, const long long* q_strides,
                              void* dq, const long long* dq_strides, const void* dk_out, const long long* dk_out_strides,
                              const void* k, const long long* k_strides, void* dk, const long long* dk_strides,
                              float* dq_weight, float* dk_weight, int B, int Hq, int Hk, int N, int d, int dtype,
                              const fa_qk_norm* norm, const fa_rotary* rotary, void* workspace, size_t workspace_bytes,
                              void* stream) {
  NvtxRange nv("fa_qk_norm_rope_bwd");
  if (!dq_out || !dq_out_strides || !q || !q_strides || !dq || !dq_strides || !norm) return FA_ERR_NULL_PTR;
  if (Hk != 0 && (!dk_out || !dk_out_strides || !k || !k_strides || !dk || !dk_strides)) return FA_ERR_NULL_PTR;
  if (Hk == 0 && (dk_out || k || dk || dk_weight)) return FA_ERR_BAD_SHAPE;
  FA_TRY(check_rows(B, Hq, Hk, N, d, dtype));
  FA_TRY(check_norm(norm));
  if (rotary) FA_TRY(check_rotary(rotary, d));
  const bool weights = dq_weight || dk_weight;
  if (weights && !workspace) return FA_ERR_NULL_PTR;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned16(workspace)) return FA_ERR_MISALIGNED;
  const size_t need = fa_qk_norm_rope_bwd_workspace_bytes(d);
  if (weights && workspace_bytes < need) return FA_ERR_WORKSPACE_TOO_SMALL;
  fa::NormRopeBwdArgs a{};
  View in[4], out[5];
  FA_TRY(rows_of(dq_out, dq_out_strides, B, Hq, N, d, a.dy[0], in[0]));
  FA_TRY(rows_of(q, q_strides, B, Hq, N, d, a.x[0], in[1]));
  FA_TRY(rows_of(dq, dq_strides, B, Hq, N, d, a.dx[0], out[0]));
  if (Hk) {
    FA_TRY(rows_of(dk_out, dk_out_strides, B, Hk, N, d, a.dy[1], in[2]));
    FA_TRY(rows_of(k, k_strides, B, Hk, N, d, a.x[1], in[3]));
    FA_TRY(rows_of(dk, dk_strides, B, Hk, N, d, a.dx[1], out[1]));
  }
  Tables tables;
  tables.rotary(rotary, B, N);
  tables.norm(norm, d);
  const int ni = Hk ? 4 : 2;
  int no = Hk ? 2 : 1;
  const int rows = no;
  if (dq_weight) out[no++] = bytes_view(dq_weight, (size_t)d * 4);
  if (dk_weight) out[no++] = bytes_view(dk_weight, (size_t)d * 4);
  if (weights) out[no++] = bytes_view(workspace, need);
  for (int i = 0; i < no; ++i) {
    if (!out[i].distinct() || !tables.apart_from(out[i])) return FA_ERR_ALIASING;
    for (int j = 0; j < ni; ++j)
      if (!(i < rows && j == 2 * i && in_place(a.dx[i], a.dy[i])) && !apart(out[i], in[j])) return FA_ERR_ALIASING;
    for (int j = 0; j < i; ++j)
      if (!apart(out[i], out[j])) return FA_ERR_ALIASING;
  }
  DeviceState* ds = nullptr;
  FA_TRY(paged4_device_state(&ds));
  a.H[0] = Hq;
  a.H[1] = Hk;
  a.B = B;
  a.N = N;
  a.d = d;
  if (rotary) a.r = rotary_args(rotary, 1);
  a.n = norm_args(norm);
  a.dw[0] = dq_weight;
  a.dw[1] = dk_weight;
  a.part = static_cast<float*>(workspace);
  return launch_status(fa::launch_norm_rope_bwd(dtype, a, dev_status(ds), ds->num_sms, static_cast<cudaStream_t>(stream)));
}

fa_status fa_paged4_append(const fa_paged4_kv* kv, const fa_page_table* table, const int* seq_lens, const int* cu_seqlens,
                           int B, int T, const void* k, const long long* k_strides, const void* v,
                           const long long* v_strides, const void* q, const long long* q_strides, void* q_out,
                           const long long* q_out_strides, int Hq, const fa_qk_norm* norm, const fa_rotary* rotary,
                           void* stream) {
  NvtxRange nv("fa_paged4_append");
  FA_TRY(check_kv4(kv));
  if (!seq_lens || !k_strides || !v_strides || (T != 0 && (!k || !v))) return FA_ERR_NULL_PTR;
  if (B < 1 || T < 0 || (!cu_seqlens && T != B)) return FA_ERR_BAD_SHAPE;
  FA_TRY(check_table(table, B, kv->page_size));
  if (!aligned(seq_lens, 4) || !aligned(cu_seqlens, 4)) return FA_ERR_MISALIGNED;
  if (q && !rotary && !norm) return FA_ERR_BAD_ARGUMENT;
  if (q ? (!q_out || !q_strides || !q_out_strides) : q_out != nullptr) return FA_ERR_NULL_PTR;
  if (q ? Hq < 1 : Hq != 0) return FA_ERR_BAD_SHAPE;
  if ((long long)Hq + 2LL * kv->Hkv > 65535) return FA_ERR_BAD_SHAPE;
  if (rotary) FA_TRY(check_rotary(rotary, kv->d));
  if (norm) FA_TRY(check_norm(norm));
  if (T == 0) return FA_OK;
  fa::Append4Args a{};
  View in[3], out[2] = {kv4_view(kv)};
  const long long ks[3] = {0, k_strides[1], k_strides[0]}, vs[3] = {0, v_strides[1], v_strides[0]};
  FA_TRY(rows_of(k, ks, 1, kv->Hkv, T, kv->d, a.k, in[0]));
  FA_TRY(rows_of(v, vs, 1, kv->Hkv, T, kv->d, a.v, in[1]));
  if (q) {
    const long long qs[3] = {0, q_strides[1], q_strides[0]}, os[3] = {0, q_out_strides[1], q_out_strides[0]};
    FA_TRY(rows_of(q, qs, 1, Hq, T, kv->d, a.q, in[2]));
    FA_TRY(rows_of(q_out, os, 1, Hq, T, kv->d, a.q_out, out[1]));
  }
  Tables tables;
  tables.add(table_view(table, B));
  tables.add(bytes_view(seq_lens, (size_t)B * 4));
  if (cu_seqlens) tables.add(bytes_view(cu_seqlens, (size_t)(B + 1) * 4));
  tables.rotary(rotary, 1, T);
  tables.norm(norm, kv->d);
  for (int i = 0; i < (q ? 2 : 1); ++i) {
    if (!out[i].distinct() || !tables.apart_from(out[i])) return FA_ERR_ALIASING;
    for (int j = 0; j < (q ? 3 : 2); ++j)
      if (!(i == 1 && j == 2 && in_place(a.q_out, a.q)) && !apart(out[i], in[j])) return FA_ERR_ALIASING;
  }
  if (q && !apart(out[0], out[1])) return FA_ERR_ALIASING;
  DeviceState* ds = nullptr;
  FA_TRY(paged4_device_state(&ds));
  a.kv = kv4_args(kv);
  a.table = table_args(table);
  a.seq_lens = seq_lens;
  a.cu = cu_seqlens;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  if (rotary) a.r = rotary_args(rotary, 0);
  a.n = norm_args(norm);
  return launch_status(fa::launch_append4(kv->dtype, a, dev_status(ds), ds->num_sms, static_cast<cudaStream_t>(stream)));
}

fa_status fa_paged4_read(const fa_paged4_kv* kv, const fa_page_table* table, const int* seq_lens, void* k,
                         const long long* k_strides, void* v, const long long* v_strides, int B, int N, void* stream) {
  NvtxRange nv("fa_paged4_read");
  FA_TRY(check_kv4(kv));
  if (!seq_lens || !k || !k_strides || !v || !v_strides) return FA_ERR_NULL_PTR;
  if (B < 1 || N < 1 || N > (1 << 30)) return FA_ERR_BAD_SHAPE;
  FA_TRY(check_table(table, B, kv->page_size));
  if (!aligned(seq_lens, 4)) return FA_ERR_MISALIGNED;
  fa::Read4Args a{};
  View out[2];
  FA_TRY(rows_of(k, k_strides, B, kv->Hkv, N, kv->d, a.k, out[0]));
  FA_TRY(rows_of(v, v_strides, B, kv->Hkv, N, kv->d, a.v, out[1]));
  const View in[] = {kv4_view(kv), table_view(table, B), bytes_view(seq_lens, (size_t)B * 4)};
  if (!out[0].distinct() || !out[1].distinct() || !outputs_apart(out, in)) return FA_ERR_ALIASING;
  DeviceState* ds = nullptr;
  FA_TRY(paged4_device_state(&ds));
  a.kv = kv4_args(kv);
  a.table = table_args(table);
  a.seq_lens = seq_lens;
  a.B = B;
  a.N = N;
  return launch_status(fa::launch_read4(kv->dtype, a, dev_status(ds), ds->num_sms, static_cast<cudaStream_t>(stream)));
}

size_t fa_paged4_decode_workspace_bytes(int B, int Hq, int Hkv, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || (d != 64 && d != 128) || (long long)B * Hq >= (1LL << 31)) return 0;
  return decode_ws(B, Hq, d, 16, 1, false).total;
}

fa_status fa_paged4_decode(const void* q, const long long* q_strides, const fa_paged4_kv* kv, const fa_page_table* table,
                           const int* seq_lens, void* o, float* lse, int B, int Hq, int window, float scale,
                           void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nv("fa_paged4_decode");
  FA_TRY(check_kv4(kv));
  if (!q || !q_strides || !seq_lens || !o || !lse || !workspace) return FA_ERR_NULL_PTR;
  if (B < 1 || Hq < 1 || Hq % kv->Hkv || (long long)B * Hq >= (1LL << 31)) return FA_ERR_BAD_SHAPE;
  FA_TRY(check_table(table, B, kv->page_size));
  FA_TRY(check_scale(0, scale));
  if (window < 0) return FA_ERR_BAD_ARGUMENT;
  FA_TRY(check_strides({{B, q_strides[0]}, {Hq, q_strides[1]}}));
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || !aligned16(workspace) || !aligned(seq_lens, 4))
    return FA_ERR_MISALIGNED;
  const size_t need = fa_paged4_decode_workspace_bytes(B, Hq, kv->Hkv, kv->d);
  if (workspace_bytes < need) return FA_ERR_WORKSPACE_TOO_SMALL;
  const View ins[] = {view(q, kv->d, 2, {{B, q_strides[0]}, {Hq, q_strides[1]}}), kv4_view(kv), table_view(table, B),
                      bytes_view(seq_lens, (size_t)B * 4)};
  const View outs[] = {bytes_view(o, (size_t)B * Hq * kv->d * 2), bytes_view(lse, (size_t)B * Hq * 4),
                       bytes_view(workspace, need)};
  if (!outputs_apart(outs, ins)) return FA_ERR_ALIASING;
  DeviceState* ds = nullptr;
  FA_TRY(paged4_device_state(&ds));
  fa::DecodeArgs a{};
  a.q = q;
  a.q_sb = stride_of(B, q_strides[0]);
  a.q_sh = stride_of(Hq, q_strides[1]);
  a.kv = kv4_args(kv);
  a.table = table_args(table);
  a.seq_lens = seq_lens;
  a.o = o;
  a.lse = lse;
  a.B = B;
  a.Hq = Hq;
  a.window = window;
  a.scale_log2 = scale * 1.4426950408889634f;
  const int G = Hq / kv->Hkv;
  a.unit_heads = G <= 8 ? 8 : 16;
  const DecodeWs w = decode_ws(B, Hq, kv->d, kv->page_size, table->max_pages, false);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.parts = reinterpret_cast<fa::DecodePart*>(ws + w.parts);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  const long long units = (long long)B * kv->Hkv * ((G + a.unit_heads - 1) / a.unit_heads);
  auto tiles_of = [&](int keys) {                  // of a unit, at most
    const long long n = ((long long)kv->page_size * table->max_pages + keys - 1) / keys;
    return window > 0 ? std::min(n, (window - 1LL) / keys + 2) : n;
  };
  // As many CTAs as run at a time, but no more than there can be tiles.
  const int slots = std::min(fa::decode4_ctas_per_sm(a.unit_heads) * ds->num_sms, fa::kDecodeMaxParts);
  int parts = (int)std::min<long long>(units * tiles_of(fa::kDecode4TileKeys), slots);
  a.cluster = decode_cluster(units, tiles_of(fa::kDecode4ClusterKeys), slots);
  if (a.cluster) parts = (int)units * a.cluster;
  return launch_status(fa::launch_decode4(kv->dtype, a, dev_status(ds), parts, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
