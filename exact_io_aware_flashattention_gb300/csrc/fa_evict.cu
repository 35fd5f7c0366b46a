// Eviction from a paged key / value cache by accumulated attention weight.
//
// For each (sequence b, kv head g) of len keys, m = min(len, budget) keys
// stay: all of them if len <= budget, else the first `sinks`, the last
// `recent`, and of the rest the budget - sinks - recent with the largest
// score, equal scores going to the lowest index.  The kept keys are written in
// their order to slots 0 .. m-1 of the pages dst names (K, V and score);
// the source pages are not written.
//
// Bound by HBM: 4 bytes per key to choose, 2 (4 d + 4) bytes per kept row to
// move, nearly all of it the second, so two kernels: the choice, which is
// short, and a copy whose rows are spread evenly over the GPU whatever was
// chosen.
//
// fa_evict_select_kernel.  One cluster of 1, 2, 4 or 8 CTAs per (b, g), each
// with an equal run of the keys, held in shared memory as order-preserving
// integers.  The need-th largest is found 11, 11 and 10 bits at a time: every
// CTA counts its keys that match the digits found so far into a histogram,
// reads the others' histograms through distributed shared memory, and all
// reach the same digit; three passes over shared memory replace a sort.  It
// stops early when the digit's bin is wanted whole.  The kept indices then go
// out in order by one block scan and the counts of the CTAs before.
//
// fa_evict_copy_kernel.  A warp takes 32 (or 8) consecutive kept keys: each
// lane looks one up (index, source page, target page) and moves its score,
// then the rows go 16 bytes a lane, eight loads in flight.
#include "fa_internal.h"
#include "sm103a.cuh"

namespace fa {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxCached = 49 * kThreads;     // keys in shared memory: 196 KB with the histograms

// Order-preserving map of scores to unsigned: larger score, larger key;
// -0 counts as +0 and NaN as the smallest.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster(const int* p, int rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct Select {
  int hist[3][kBins];
  int warp_sums[kWarps];
  int counts[2];          // this CTA's keys: above the threshold or protected, equal to it
  int bin, left, whole;
};

// Inclusive sum over the block; total to every thread.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();                    // the last scan's sums have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int s = warp_sums[lane];
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return x + (warp > 0 ? before : 0);
}

__global__ void __launch_bounds__(kThreads) fa_evict_select_kernel(const EvictArgs a, int cluster, int cap, const DevStatus st) {
  extern __shared__ __align__(16) uint8_t smem[];
  Select& sh = *reinterpret_cast<Select*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + sizeof(Select));     // [cap]
  launch_dependents();
  const int unit = blockIdx.x / cluster, rank = blockIdx.x - unit * cluster;
  const int b = unit / a.kv.Hkv, g = unit - b * a.kv.Hkv;
  const int ps = a.kv.page_size, tid = threadIdx.x;
  int len = a.seq_lens[b];
  if (len < 0 || len > (long long)a.table.cols * ps) {
    if (tid == 0) record_error(st, kErrBadIndex, kSiteEvictLen);
    len = 0;
  }
  const int m = min(len, a.budget);
  if (g == 0 && rank == 0 && tid == 0) a.new_lens[b] = m;
  int* kept = a.kept + (long long)unit * a.budget;
  for (int i = m + rank * kThreads + tid; i < a.budget; i += cluster * kThreads) kept[i] = -1;
  if (len <= a.budget) {
    for (int i = rank * kThreads + tid; i < m; i += cluster * kThreads) kept[i] = i;
    return;                            // the whole cluster does
  }
  // Candidates are [lo, hi); the others are protected.
  const int lo = a.sinks, hi = len - a.recent;
  int need = m - a.sinks - a.recent;
  const int run = (len + cluster - 1) / cluster, j0 = min(len, rank * run), j1 = min(len, j0 + run);
  const bool cached = run <= cap;
  const int* pages = a.table.pages + b * a.table.stride;
  auto key_at = [&](int j) -> uint32_t {
    const int c = j / ps, p = pages[c];
    if (p < 0 || p >= a.kv.num_pages) {
      record_error(st, kErrBadIndex, kSiteEvictPage);
      return 0u;
    }
    return score_key(a.scores[((long long)p * a.kv.Hkv + g) * ps + (j - c * ps)]);
  };
  // Keys [from, from + n) of the run into shared memory.
  auto load = [&](int from, int n) {
#pragma unroll 4
    for (int i = tid; i < n; i += kThreads) keys[i] = key_at(from + i);
  };
  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  if (cached) load(j0, j1 - j0);
  __syncthreads();

  uint32_t prefix = 0, mask = 0;
  if (need > 0)
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      int* hist = sh.hist[pass];
      for (int i = tid; i < j1 - j0; i += kThreads) {
        const int j = j0 + i;
        if (j < lo || j >= hi) continue;
        const uint32_t k = cached ? keys[i] : key_at(j);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
      }
      if (cluster > 1) cluster_sync(); else __syncthreads();
      // Two bins a thread, the largest first: where the running count reaches
      // `need` is the digit.
      const int top = kBins - 1 - 2 * tid;
      int n0 = 0, n1 = 0;
      if (cluster == 1) {
        n0 = hist[top];
        n1 = hist[top - 1];
      } else {
        for (int r = 0; r < cluster; ++r) {
          n0 += ld_cluster(&hist[top], r);
          n1 += ld_cluster(&hist[top - 1], r);
        }
      }
      int total;
      const int upto = block_scan(n0 + n1, sh.warp_sums, total);
      const int before = upto - n0 - n1;
      if (before < need && upto >= need) {
        const bool first = before + n0 >= need;
        sh.bin = first ? top : top - 1;
        sh.left = need - before - (first ? 0 : n0);
        sh.whole = sh.left == (first ? n0 : n1);
      }
      __syncthreads();
      prefix |= (uint32_t)sh.bin << shift;
      mask |= ((1u << bits) - 1) << shift;
      need = sh.left;
      if (sh.whole) break;             // every key with these digits stays
    }
  // A key stays if it is protected, its digits are above the threshold's, or
  // they are equal and it is among the first `need` such keys.
  auto classify = [&](int j, uint32_t k, int& keep, int& eq) {
    const bool safe = j < lo || j >= hi;
    keep = safe || (mask != 0 && (k & mask) > prefix);
    eq = !safe && mask != 0 && (k & mask) == prefix;
  };
  int keep_before = 0, eq_before = 0;
  if (cluster > 1) {
    int keep = 0, eq = 0;
    for (int i = tid; i < j1 - j0; i += kThreads) {
      int x, y;
      classify(j0 + i, cached ? keys[i] : key_at(j0 + i), x, y);
      keep += x;
      eq += y;
    }
    int total_keep, total_eq;
    block_scan(keep, sh.warp_sums, total_keep);
    block_scan(eq, sh.warp_sums, total_eq);
    if (tid == 0) {
      sh.counts[0] = total_keep;
      sh.counts[1] = total_eq;
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      keep_before += ld_cluster(&sh.counts[0], r);
      eq_before += ld_cluster(&sh.counts[1], r);
    }
    cluster_sync();                    // nobody exits while its counts are read
  }
  // Each thread takes an odd number of consecutive keys (an odd stride between
  // threads meets every bank once).
  int out = keep_before + min(eq_before, need), seen = eq_before;
  for (int from = j0; from < j1; from += cap) {
    const int n = min(cap, j1 - from);
    if (!cached) {
      __syncthreads();
      load(from, n);
      __syncthreads();
    }
    const int per = ((n + kThreads - 1) / kThreads) | 1;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    int keep = 0, eq = 0;
    for (int i = i0; i < i1; ++i) {
      int x, y;
      classify(from + i, keys[i], x, y);
      keep += x;
      eq += y;
    }
    int total_eq, total;
    int rank_eq = block_scan(eq, sh.warp_sums, total_eq) - eq + seen;
    const int mine = keep + max(0, min(eq, need - rank_eq));
    int at = block_scan(mine, sh.warp_sums, total) - mine + out;
    for (int i = i0; i < i1; ++i) {
      int x, y;
      classify(from + i, keys[i], x, y);
      if (y) x = rank_eq++ < need;
      if (x) kept[at++] = from + i;
    }
    seen += total_eq;
    out += total;
  }
}

// kRows kept keys a warp, kUnroll rows' loads in flight.
template <int D, int kRows>
__global__ void __launch_bounds__(256) fa_evict_copy_kernel(const EvictArgs a, int blocks_per_unit, const DevStatus st) {
  constexpr int kVec = D / 8, kSide = 32 / (2 * kVec);   // 16-byte vectors a row; rows a warp moves at once, K and V
  constexpr int kUnroll = 8;
  static_assert(kRows % (kSide * kUnroll) == 0 || kRows == kSide * 4 || kRows == kSide * 8, "whole rounds");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / blocks_per_unit, b = unit / a.kv.Hkv, g = unit - b * a.kv.Hkv, ps = a.kv.page_size;
  const int r0 = ((blockIdx.x - unit * blocks_per_unit) * 8 + warp) * kRows;
  wait_for_previous();
  const int m = a.new_lens[b];
  if (r0 >= m) return;
  const int n = min(kRows, m - r0);
  long long from = -1, to = -1;
  if (lane < n) {
    const int i = r0 + lane, j = a.kept[(long long)unit * a.budget + i];
    const int cj = j / ps, ci = i / ps;
    const int p = a.table.pages[b * a.table.stride + cj], q = a.dst.pages[b * a.dst.stride + ci];
    if (p >= 0 && p < a.kv.num_pages && q >= 0 && q < a.kv.num_pages) {
      from = p * a.kv.s_page + g * a.kv.s_head + (long long)(j - cj * ps) * a.kv.s_slot;
      to = q * a.kv.s_page + g * a.kv.s_head + (long long)(i - ci * ps) * a.kv.s_slot;
      a.scores[((long long)q * a.kv.Hkv + g) * ps + (i - ci * ps)] =
          a.scores[((long long)p * a.kv.Hkv + g) * ps + (j - cj * ps)];
    } else {
      record_error(st, kErrBadIndex, kSiteEvictPage);
    }
  }
  const int side = lane / (2 * kVec), v = lane % kVec;
  const bool is_v = (lane / kVec) & 1;
  uint16_t* pool = static_cast<uint16_t*>(is_v ? a.kv.v : a.kv.k) + v * 8;
  constexpr int kStep = kSide * kUnroll < kRows ? kSide * kUnroll : kRows;
  for (int r = 0; r < n; r += kStep) {
    uint4 x[kStep / kSide];
#pragma unroll
    for (int u = 0; u < kStep / kSide; ++u) {
      const long long f = __shfl_sync(0xffffffffu, from, r + u * kSide + side);
      if (f >= 0) x[u] = *reinterpret_cast<const uint4*>(pool + f);
    }
#pragma unroll
    for (int u = 0; u < kStep / kSide; ++u) {
      const long long t = __shfl_sync(0xffffffffu, to, r + u * kSide + side);
      if (t >= 0) *reinterpret_cast<uint4*>(pool + t) = x[u];
    }
  }
}

template <typename... P, typename... A>
cudaError_t launch(void (*k)(P...), dim3 grid, int block, size_t smem, int cluster, bool after, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  if (after) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace

cudaError_t configure_evict_kernels() {
  return cudaFuncSetAttribute(fa_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)(sizeof(Select) + kMaxCached * 4));
}

cudaError_t launch_paged_evict(const EvictArgs& a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  const long long most = (long long)a.table.cols * a.kv.page_size;     // keys a sequence can have
  const int units = a.B * a.kv.Hkv;
  // More CTAs a unit while there are idle SMs and each still has 4 keys a thread.
  int cluster = 1;
  while (cluster < kMaxCluster && (long long)units * cluster * 2 <= num_sms && most > 4LL * kThreads * cluster) cluster *= 2;
  const long long run = (most + cluster - 1) / cluster;
  const int cap = (int)(run < kMaxCached ? (run + kThreads - 1) / kThreads * kThreads : kMaxCached);
  cudaError_t e = launch(fa_evict_select_kernel, dim3((unsigned)units * cluster), kThreads, sizeof(Select) + (size_t)cap * 4,
                         cluster, false, stream, a, cluster, cap, st);
  if (e != cudaSuccess) return e;
  // 32 rows a warp where that still gives every SM its fill of warps, else 8.
  const bool wide = (long long)units * a.budget >= 32LL * 32 * num_sms;
  const int rows = (wide ? 32 : 8) * 8;
  const int per_unit = (a.budget + rows - 1) / rows;
  const dim3 grid((unsigned)((long long)units * per_unit));
  if (a.kv.d == 64)
    return wide ? launch(fa_evict_copy_kernel<64, 32>, grid, 256, 0, 1, true, stream, a, per_unit, st)
                : launch(fa_evict_copy_kernel<64, 8>, grid, 256, 0, 1, true, stream, a, per_unit, st);
  return wide ? launch(fa_evict_copy_kernel<128, 32>, grid, 256, 0, 1, true, stream, a, per_unit, st)
              : launch(fa_evict_copy_kernel<128, 8>, grid, 256, 0, 1, true, stream, a, per_unit, st);
}

}  // namespace fa
