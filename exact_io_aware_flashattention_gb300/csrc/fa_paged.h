// Internal launcher interface of rotary positions and the paged cache
// (fa_rope.cu, fa_paged.cu, fa_evict.cu), between the C-ABI layer (fa_api.cu)
// and the kernels.  Nothing here is exported from the shared library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "sm103a.cuh"

namespace fa {

// Loads a kernel ahead of its first launch, which may be inside a stream
// capture, where loading is not safe.
template <typename K>
cudaError_t preload_kernel(K* k) {
  cudaFuncAttributes attr;
  return cudaFuncGetAttributes(&attr, k);
}

// Programmatic dependent launch.  Every kernel of this section is launched so
// that its blocks may start while the kernel in front of it finishes, which
// hides the launch and the set-up (2 us a call on a busy stream: 134 MB of
// rotary rows 26.6 -> 24.2 us); each lets the next one do so at once, and each
// block waits, before it touches global memory, until everything in front is
// complete and visible.
#ifdef __CUDACC__
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*k)(P...), dim3 grid, int block, size_t smem, int cluster, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// Barrier of a cluster, and loads from the shared memory of one of its CTAs.
constexpr int kMaxCluster = 8;
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ int ld_cluster(const int* p, int rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ int2 ld_cluster2(const int* p, int rank) {
  uint32_t a;
  int2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(const float2* p, int rank) {
  const int2 v = ld_cluster2(reinterpret_cast<const int*>(p), rank);
  return make_float2(__int_as_float(v.x), __int_as_float(v.y));
}
#endif

// Wait-site ids / index-check sites of these kernels in the status words.
enum : int { kSiteAxis = 41, kSiteAppend = 42, kSiteDecodeLen = 43, kSiteDecodePage = 44, kSiteEvictLen = 45, kSiteEvictPage = 46 };
constexpr int kErrBadIndex = 14;   // == FA_ERR_BAD_INDEX

// Rows of d elements: (b, h, n) at b * sb + h * sh + n * sn elements from p.
struct RowView {
  void* p;
  long long sb, sh, sn;
};

struct RotaryArgs {
  const int* pos;            // [n_axes, B, N] with strides (pos_axis, pos_batch, 1)
  long long pos_axis, pos_batch;
  const double* inv_freq;    // [rot / 2] radians per position
  const int* axes;           // [rot / 2] axis of each pair
  int n_axes, rot;           // rot = 0: nothing is rotated
  int interleaved;           // pair i = elements (2i, 2i+1) instead of (i, i + rot/2)
  int inverse;               // angles negated (the gradient)
};

struct RopeArgs {
  RowView q, q_out, k, k_out;
  int B, Hq, Hk, N, d;
  RotaryArgs r;
};

// A pool of pages: (page, kv head, slot) at page * s_page + g * s_head + slot * s_slot elements.
struct PagedKv {
  void* k;
  void* v;
  long long s_page, s_head, s_slot;
  int num_pages, page_size, Hkv, d;
};

// Row b lists the pages of sequence b.
struct PageTable {
  const int* pages;
  long long stride;
  int cols;
};

struct AppendArgs {
  RowView q, q_out, k, v;    // tokens as N (sb unused); q.p NULL: no q
  PagedKv kv;
  PageTable table;
  const int* seq_lens;       // [B] lengths with the new tokens
  const int* cu;             // [B + 1] first new token of each sequence, NULL: token b belongs to sequence b
  float* scores;             // [num_pages, Hkv, page_size] or NULL
  int B, T, Hq;
  RotaryArgs r;
};

cudaError_t launch_rope(int dtype, const RopeArgs& a, const DevStatus& st, int num_sms, cudaStream_t stream);
cudaError_t launch_append(int dtype, const AppendArgs& a, const DevStatus& st, int num_sms, cudaStream_t stream);

// What a CTA of the decode kernel worked on: `left` tiles (decode_tile_keys
// keys each) from `tile` of unit (b, col) on.  The first unit is spread over
// the CTAs i0 .. i1, the last one (if it is another) over this one .. last_i1.
struct DecodePart {
  int b, col, tile, left, i0, i1, last_i1, pad;
};

struct DecodeArgs {
  const void* q;             // (b, h) at b * q_sb + h * q_sh elements
  long long q_sb, q_sh;
  PagedKv kv;
  PageTable table;
  const int* seq_lens;
  void* o;                   // [B, Hq, d]
  float* lse;                // [B, Hq]
  float* scores;             // [num_pages, Hkv, page_size] or NULL
  int B, Hq, window;
  float scale_log2;
  int unit_heads;            // query heads of a kv group that share a unit: 8 or 16
  int cluster;               // CTAs of a cluster that takes one unit, 0: equal parts of all tiles
  // Workspace
  DecodePart* parts;         // [kDecodeMaxParts]
  float* part;               // [kDecodeMaxParts][2][16][d] unnormalised O of units cut over CTAs
  float2* part_ml;           // [kDecodeMaxParts][2][16] their maximum (log2 units) and sum
  float* lse2;               // [B, Hq] log-sum-exp in log2 units (with scores)
  float* stash;              // [B, Hkv, stash_keys, G] scores in log2 units (with scores)
  long long stash_keys;
};

constexpr int kDecodeMaxParts = 320;   // CTAs of the decode kernel at most
constexpr int decode_tile_keys(int d) { return d == 64 ? 128 : 64; }

// `tk`, `tv` view the pools as {d, page_size, Hkv, num_pages}; `parts` CTAs.
cudaError_t launch_paged_decode(int dtype, const TmaMap4& tk, const TmaMap4& tv, const DecodeArgs& a, const DevStatus& st,
                                int parts, cudaStream_t stream);

struct EvictArgs {
  PagedKv kv;
  float* scores;
  PageTable table, dst;
  const int* seq_lens;
  int* new_lens;             // [B]
  int* kept;                 // [B, Hkv, budget], -1 past the new length
  int B, budget, recent, sinks;
  unsigned page_mul;         // division by page_size (set by the launcher)
  int page_shift;
};

cudaError_t launch_paged_evict(EvictArgs a, const DevStatus& st, int num_sms, cudaStream_t stream);

// One-time set-up of the current device (see configure_kernels).
cudaError_t configure_rope_kernels();
cudaError_t configure_decode_kernels();
cudaError_t configure_evict_kernels();

inline cudaError_t configure_paged_kernels() {
  cudaError_t e = configure_rope_kernels();
  if (e == cudaSuccess) e = configure_decode_kernels();
  if (e == cudaSuccess) e = configure_evict_kernels();
  return e;
}

}  // namespace fa
