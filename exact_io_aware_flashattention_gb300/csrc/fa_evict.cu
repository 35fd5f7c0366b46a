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
// integers (protected ones as the largest).  The range of the others that
// holds the last key to stay is narrowed to one of 2048 equal parts, at most
// three times: every CTA counts its keys of the range into a histogram, reads
// the others' through distributed shared memory (64 sums of 32 bins first, then
// 32 bins), and all reach the same part; three passes over shared memory
// replace a sort.  (The first digits of all keys instead of their range: scores
// within a few powers of two meet in a few bins; from 1.0 to 1.01, 106.3 us
// instead of 102.9 in the first example below.)  It stops early when the part
// is wanted whole.  The kept indices then go out in order: each warp counts its
// run of keys, sums the counts of the warps and CTAs before, and writes.
//
// fa_evict_copy_kernel.  A warp takes 8 consecutive kept keys: eight lanes look
// one up each (index, source page, target page) and move its score, then the
// rows go 16 bytes a lane, all loads in flight before the first store.  (16 or
// 32 keys a warp, in rounds of 8 or 4, fill the last wave worse: 2-5 % slower.)
//
// Measured: 2 sequences of 131072 keys, 8 heads, d = 128, to 32768: 102.5 us, of
// which the selection 18 and the copy of 541 MB 82 (97 % of the 6.79 TB/s copy
// rate); 16 sequences of 0 to 8192 keys to 2048: 42.5 us, the copy of 202 MB 32;
// one of 1000 keys, 2 heads: 7.7 us.  The selection is bound by instructions
// and latencies: loads, histograms, exchanges over the cluster and the list
// take about a quarter each.
#include "fa_paged.h"
#include "sm103a.cuh"

namespace fa {

namespace {

constexpr int kThreads = 512;                 // of the selection
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCached = 49 * 1024;         // keys in shared memory: 196 KB, 222 KB with the histograms
constexpr uint32_t kProtected = 0xffffffffu;  // above every score's key, so taken first

// Order-preserving map of scores to unsigned: larger score, larger key;
// -0 counts as +0 and NaN as the smallest.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// 16 bytes from global to shared memory, without a register in between.
__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// j / page_size by a multiplication: page_size = 16 q, and with s = ceil(log2 q),
// page_mul = ceil(2^(27+s) / q) the product n page_mul / 2^(27+s) exceeds n / q
// by less than n 2^-(27+s) < 1/q for n = j / 16 < 2^27.
__device__ __forceinline__ int page_of(int j, const EvictArgs& a) {
  return (int)(((uint64_t)((uint32_t)j >> 4) * a.page_mul) >> a.page_shift);
}

struct Select {
  int hist[3][kBins];
  int coarse[3][kBins / 32];          // sums of 32 bins
  int above[kWarps], equal[kWarps];   // each warp's keys above the threshold, and equal to it
  int2 counts;                        // the CTA's
  uint32_t least[kWarps], most[kWarps];   // each warp's smallest and largest key that is not protected
  uint2 range;                        // the CTA's
  int bin, left, whole;
};

// Inclusive sum over the warp.
__device__ __forceinline__ int warp_scan(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

__global__ void __launch_bounds__(kThreads, 2)
    fa_evict_select_kernel(const EvictArgs a, int cluster, int cap, const DevStatus st) {
  extern __shared__ __align__(16) uint8_t smem[];
  Select& sh = *reinterpret_cast<Select*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + (sizeof(Select) + 15) / 16 * 16);     // [cap]
  launch_dependents();
  wait_for_previous();
  const int unit = blockIdx.x / cluster, rank = blockIdx.x - unit * cluster;
  const int b = unit / a.kv.Hkv, g = unit - b * a.kv.Hkv;
  const int ps = a.kv.page_size, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  const int lo = a.sinks, hi = len - a.recent;     // keys outside [lo, hi) are protected
  // The CTA's run of keys: a multiple of 4, so that four consecutive keys, one
  // 16-byte load, lie in one page (page sizes are multiples of 16).
  const int run = ((len + cluster - 1) / cluster + 3) & ~3;
  const int j0 = (int)min((long long)len, (long long)rank * run), n_run = min(len - j0, run);
  const bool cached = run <= cap;
  const int* pages = a.table.pages + b * a.table.stride;
  const float* pool = a.scores + (long long)g * ps;
  const long long page_scores = (long long)a.kv.Hkv * ps;
  // Keys [from, from + n) into shared memory, in fours, with the smallest and
  // largest of those that are not protected.  Past the sequence's end 0, the
  // smallest: equal keys go by index, so those never come before a key of the
  // sequence.  n rounded up to 128 is filled.
  uint32_t least = 0xffffffffu, most = 0;
  auto load = [&](int from, int n) {
    constexpr int kBatch = 8;          // page numbers, then copies, in flight per thread
    const int quads = (n + 127) / 128 * 32;
    uint4* quad = reinterpret_cast<uint4*>(keys);
    for (int i0 = tid; i0 < quads; i0 += kBatch * kThreads) {
      int p[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int j = from + 4 * (i0 + u * kThreads);
        p[u] = j < from + n ? pages[page_of(j, a)] : 0;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kThreads, j = from + 4 * i;
        if (j >= from + n) break;
        if (p[u] < 0 || p[u] >= a.kv.num_pages) {
          record_error(st, kErrBadIndex, kSiteEvictPage);
          p[u] = 0;                    // any page: what such a sequence keeps is unspecified
        }
        copy16_async(quad + i, pool + p[u] * page_scores + (j - page_of(j, a) * ps));
      }
    }
    wait_copies();
    // Each thread turns the scores it copied into keys.
    for (int i = tid; i < quads; i += kThreads) {
      const int j = from + 4 * i;
      uint4 k = make_uint4(0, 0, 0, 0);
      if (j < from + n) {
        const float4 x = reinterpret_cast<const float4*>(quad)[i];
        k = make_uint4(score_key(x.x), score_key(x.y), score_key(x.z), score_key(x.w));
        if (j >= lo && j + 4 <= hi) {
          least = min(least, min(min(k.x, k.y), min(k.z, k.w)));
          most = max(most, max(max(k.x, k.y), max(k.z, k.w)));
        } else {
          uint32_t* y = &k.x;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + e < lo || j + e >= hi) {
              y[e] = j + e < len ? kProtected : 0u;
            } else {
              least = min(least, y[e]);
              most = max(most, y[e]);
            }
        }
      }
      quad[i] = k;
    }
  };
  // body(from, n) over the run in pieces that fit shared memory.
  auto pieces = [&](auto body) {
    for (int from = j0; from < j0 + n_run; from += cap) {
      const int n = min(cap, j0 + n_run - from);
      if (!cached) {
        __syncthreads();
        load(from, n);
        __syncthreads();
      }
      body(from, n);
    }
  };
  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;

  // The range of the keys to choose from.
  for (int from = j0; from < j0 + n_run; from += cap) load(from, min(cap, j0 + n_run - from));
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    sh.least[warp] = least;
    sh.most[warp] = most;
  }
  __syncthreads();
  least = __reduce_min_sync(0xffffffffu, sh.least[lane % kWarps]);
  most = __reduce_max_sync(0xffffffffu, sh.most[lane % kWarps]);
  if (cluster > 1) {
    if (tid == 0) sh.range = make_uint2(least, most);
    cluster_sync();
    const int2 r = ld_cluster2(reinterpret_cast<const int*>(&sh.range), lane < cluster ? lane : rank);
    least = __reduce_min_sync(0xffffffffu, (uint32_t)r.x);
    most = __reduce_max_sync(0xffffffffu, (uint32_t)r.y);
  }

  // The m-th largest key lies in [base, base + span], which each pass narrows
  // to one of at most 2048 equal parts.
  uint32_t base = least, span = most - least;
  int need = m - a.sinks - a.recent;
  bool whole = need == 0;              // only the protected ones stay
  for (int pass = 0; !whole; ++pass) {
    const int shift = max(21 - __clz(span), 0);    // clz(0) = 32
    int* hist = sh.hist[pass];
    pieces([&](int, int n) {
      const int quads = (n + 3) / 4;
#pragma unroll 2
      for (int i = tid; i < quads; i += kThreads) {
        const uint4 k = reinterpret_cast<const uint4*>(keys)[i];
        const uint32_t x = k.x - base, y = k.y - base, z = k.z - base, w = k.w - base;
        if (x <= span) atomicAdd(&hist[x >> shift], 1);
        if (y <= span) atomicAdd(&hist[y >> shift], 1);
        if (z <= span) atomicAdd(&hist[z >> shift], 1);
        if (w <= span) atomicAdd(&hist[w >> shift], 1);
      }
    });
    __syncthreads();
    // Sums of 32 bins, so that the others need to read 64 of them and then 32
    // bins, not all 2048.
    for (int c = warp; c < kBins / 32; c += kWarps) {
      const int sum = __reduce_add_sync(0xffffffffu, hist[c * 32 + lane]);
      if (lane == 0) sh.coarse[pass][c] = sum;
    }
    if (cluster > 1) cluster_sync(); else __syncthreads();
    if (warp == 0) {
      // Largest first: lane l has coarse bins 63 - 2l and 62 - 2l, then bin
      // 31 - l of the coarse bin in which the running count reaches `need`.
      int n0 = 0, n1 = 0;
      if (cluster == 1) {
        n0 = sh.coarse[pass][63 - 2 * lane];
        n1 = sh.coarse[pass][62 - 2 * lane];
      } else {
        int2 v[kMaxCluster];           // all loads in flight before the first is used
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) v[r] = ld_cluster2(&sh.coarse[pass][62 - 2 * lane], r < cluster ? r : rank);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          n0 += r < cluster ? v[r].y : 0;
          n1 += r < cluster ? v[r].x : 0;
        }
      }
      int before = warp_scan(n0 + n1) - n0 - n1;
      const bool here0 = before < need && before + n0 >= need;
      const bool here1 = before + n0 < need && before + n0 + n1 >= need;
      const int src = __ffs(__ballot_sync(0xffffffffu, here0 || here1)) - 1;
      const int coarse = __shfl_sync(0xffffffffu, here0 ? 63 - 2 * lane : 62 - 2 * lane, src);
      const int rest = need - __shfl_sync(0xffffffffu, here0 ? before : before + n0, src);
      int c = 0;
      if (cluster == 1) {
        c = hist[coarse * 32 + 31 - lane];
      } else {
        int v[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) v[r] = ld_cluster(&hist[coarse * 32 + 31 - lane], r < cluster ? r : rank);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) c += r < cluster ? v[r] : 0;
      }
      before = warp_scan(c) - c;
      if (before < rest && before + c >= rest) {
        sh.bin = coarse * 32 + 31 - lane;
        sh.left = rest - before;
        sh.whole = rest - before == c;
      }
    }
    __syncthreads();
    base += (uint32_t)sh.bin << shift;
    span = min(most - base, (1u << shift) - 1);    // (never past the largest: protected keys are no candidates)
    need = sh.left;
    whole = sh.whole;                  // every key of the part stays
    if (shift == 0) break;
  }
  // A key stays if it is above `bound`, or, where only some of the equal keys
  // in the last part are wanted (ties), equal to it and among the first `need`
  // such keys.  Each warp takes a run of a piece, 128 keys at a time, four
  // consecutive ones a lane.  (Without ties base is at least 1: a base of 0
  // would mean that every key stays.)
  const bool ties = !whole;
  const uint32_t bound = ties ? base : need == 0 ? most : base - 1, below = (1u << lane) - 1;
  int above_before = 0, equal_before = 0;          // of the CTAs before, then of the pieces before
  // Keys above and equal to the bound in the warp's run of a piece, then per
  // warp in shared memory.
  auto warp_run = [&](int n, int& i0, int& i1) {
    const int per = ((n + kWarps - 1) / kWarps + 127) & ~127;
    i0 = min(n, warp * per);
    i1 = min(n, i0 + per);
  };
  auto count_run = [&](int n, int& above, int& equal) {
    int i0, i1;
    warp_run(n, i0, i1);
    for (int i = i0 + 4 * lane; i < i1; i += 128) {
      const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
      above += (k.x > bound) + (k.y > bound) + (k.z > bound) + (k.w > bound);
      if (ties)
        equal += (k.x == bound) + (k.y == bound) + (k.z == bound) + (k.w == bound);
    }
  };
  auto publish = [&](int above, int equal) {
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    __syncthreads();                   // the counts before have been read
    if (lane == 0) {
      sh.above[warp] = above;
      sh.equal[warp] = equal;
    }
    __syncthreads();
  };
  int above = 0, equal = 0;
  if (cached) {
    count_run(n_run, above, equal);
    publish(above, equal);
  }
  if (cluster > 1) {
    if (!cached) {
      pieces([&](int, int n) { count_run(n, above, equal); });
      publish(above, equal);
    }
    if (warp == 0) {
      const int x = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.above[lane] : 0);
      const int y = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.equal[lane] : 0);
      if (lane == 0) sh.counts = make_int2(x, y);
    }
    cluster_sync();
    const int2 c = lane < rank ? ld_cluster2(&sh.counts.x, lane) : make_int2(0, 0);
    above_before = __reduce_add_sync(0xffffffffu, c.x);
    equal_before = __reduce_add_sync(0xffffffffu, c.y);
    cluster_arrive();
  }
  pieces([&](int from, int n) {
    if (!cached) {
      above = equal = 0;
      count_run(n, above, equal);
      publish(above, equal);
    }
    const int aw = lane < kWarps ? sh.above[lane] : 0, ew = lane < kWarps ? sh.equal[lane] : 0;
    const int a0 = above_before + __reduce_add_sync(0xffffffffu, lane < warp ? aw : 0);
    int e0 = equal_before + __reduce_add_sync(0xffffffffu, lane < warp ? ew : 0);
    above_before += __reduce_add_sync(0xffffffffu, aw);
    equal_before += __reduce_add_sync(0xffffffffu, ew);
    int i0, i1;
    warp_run(n, i0, i1);
    // Writes the keys of the four flags a lane, in order, from `out` on.
    auto put = [&](int* out, int at, const bool (&keep)[4]) {
      int pos = 0, total = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t v = __ballot_sync(0xffffffffu, keep[e]);
        pos += __popc(v & below);
        total += __popc(v);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (keep[e]) out[pos++] = from + at + e;
      return total;
    };
    if (!ties) {
      // Past the piece's end, up to a whole 128, lie zeros, never above.
      int* out = kept + a0;
#pragma unroll 2
      for (int i = i0; i < i1; i += 128) {
        const int at = i + 4 * lane;
        const uint4 q = *reinterpret_cast<const uint4*>(keys + at);
        const bool keep[4] = {q.x > bound, q.y > bound, q.z > bound, q.w > bound};
        out += put(out, at, keep);
      }
      return;
    }
    int* out = kept + a0 + min(e0, need);
    for (int i = i0; i < i1; i += 128) {
      const int at = i + 4 * lane;
      const uint4 q = *reinterpret_cast<const uint4*>(keys + at);
      const uint32_t k[4] = {q.x, q.y, q.z, q.w};
      bool keep[4], eq[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        keep[e] = k[e] > bound && at + e < i1;
        eq[e] = k[e] == bound && at + e < i1;
      }
      const int mine = eq[0] + eq[1] + eq[2] + eq[3];
      if (__any_sync(0xffffffffu, mine)) {
        const int upto = warp_scan(mine);
        int r = e0 + upto - mine;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (eq[e]) keep[e] = r++ < need;
        e0 += __shfl_sync(0xffffffffu, upto, 31);
      }
      out += put(out, at, keep);
    }
  });
  if (cluster > 1) cluster_wait();     // nobody exits while its counts are read
}

constexpr int kRows = 8;   // kept keys a warp
constexpr int kCopyThreads = 128;
constexpr int kBlockRows = kRows * kCopyThreads / 32;

template <int D>
__global__ void __launch_bounds__(kCopyThreads, 8)
    fa_evict_copy_kernel(const EvictArgs a, int blocks_per_unit, const DevStatus st) {
  constexpr int kVec = D / 8, kSide = 32 / (2 * kVec);   // 16-byte vectors a row; rows a warp moves at once, K and V
  launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / blocks_per_unit, b = unit / a.kv.Hkv, g = unit - b * a.kv.Hkv, ps = a.kv.page_size;
  const int r0 = (blockIdx.x - unit * blocks_per_unit) * kBlockRows + warp * kRows;
  wait_for_previous();
  const int i = r0 + lane, j = lane < kRows && i < a.budget ? a.kept[(long long)unit * a.budget + i] : -1;
  if (__all_sync(0xffffffffu, j < 0)) return;
  long long from = -1, to = -1;
  if (j >= 0) {
    const int cj = page_of(j, a), ci = page_of(i, a);
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
  uint4 x[kRows / kSide];
#pragma unroll
  for (int u = 0; u < kRows / kSide; ++u) {
    const long long f = __shfl_sync(0xffffffffu, from, u * kSide + side);
    if (f >= 0) x[u] = *reinterpret_cast<const uint4*>(pool + f);
  }
#pragma unroll
  for (int u = 0; u < kRows / kSide; ++u) {
    const long long t = __shfl_sync(0xffffffffu, to, u * kSide + side);
    if (t >= 0) *reinterpret_cast<uint4*>(pool + t) = x[u];
  }
}

}  // namespace

constexpr size_t kSelectBytes = (sizeof(Select) + 15) / 16 * 16;

cudaError_t configure_evict_kernels() {
  cudaError_t e = cudaFuncSetAttribute(fa_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(kSelectBytes + kMaxCached * 4));
  if (e == cudaSuccess) e = preload_kernel(fa_evict_copy_kernel<64>);
  if (e == cudaSuccess) e = preload_kernel(fa_evict_copy_kernel<128>);
  return e;
}

cudaError_t launch_paged_evict(EvictArgs a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  const int q = a.kv.page_size / 16;
  a.page_shift = 27;
  while ((1 << (a.page_shift - 27)) < q) ++a.page_shift;
  a.page_mul = (unsigned)(((1ull << a.page_shift) + q - 1) / q);
  const long long most = (long long)a.table.cols * a.kv.page_size;     // keys a sequence can have
  const int units = a.B * a.kv.Hkv;
  // More CTAs a unit while there are SMs for them and each still has 4 keys a
  // thread (two CTAs an SM: 45.4 instead of 43.1 us for 128 units of 8192 keys).
  int cluster = 1;
  while (cluster < kMaxCluster && (long long)units * cluster * 2 <= num_sms && most > 4LL * kThreads * cluster) cluster *= 2;
  const long long run = (most + cluster - 1) / cluster;
  const int cap = (int)(run + 4 < kMaxCached ? (run + 4 + 127) / 128 * 128 : kMaxCached);
  const cudaError_t e = launch_after(fa_evict_select_kernel, dim3((unsigned)units * cluster), kThreads,
                                     kSelectBytes + (size_t)cap * 4, cluster, stream, a, cluster, cap, st);
  if (e != cudaSuccess) return e;
  const int per_unit = (a.budget + kBlockRows - 1) / kBlockRows;
  const dim3 grid((unsigned)((long long)units * per_unit));
  return a.kv.d == 64 ? launch_after(fa_evict_copy_kernel<64>, grid, kCopyThreads, 0, 1, stream, a, per_unit, st)
                      : launch_after(fa_evict_copy_kernel<128>, grid, kCopyThreads, 0, 1, stream, a, per_unit, st);
}

}  // namespace fa
