// Eviction from a paged key / value cache by accumulated attention weight.
//
// For each (sequence b, kv head g) of len keys, m = min(len, budget) keys
// stay: all of them if len <= budget, else the first `sinks`, the last
// `recent`, and of the rest the budget - sinks - recent with the largest
// score, equal scores going to the lowest index.  The kept keys are written in
// their order to slots 0 .. m-1 of the pages dst names (K, V and score);
// the source pages are not written.
#include "fa_internal.h"
#include "sm103a.cuh"

namespace fa {

namespace {

constexpr int kThreads = 1024;

// Order-preserving map of scores to unsigned: larger score, larger key;
// -0 counts as +0 and NaN as the smallest.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Inclusive sum over the block; total to every thread.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const int s = warp_sums[w];
    if (w < warp) before += s;
    total += s;
  }
  return x + before;
}

// One block per (sequence, kv head).
__global__ void __launch_bounds__(kThreads) fa_evict_kernel(const EvictArgs a, const DevStatus st) {
  __shared__ int hist[256];
  __shared__ int warp_sums[kThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int b = blockIdx.x / a.kv.Hkv, g = blockIdx.x % a.kv.Hkv;
  const int ps = a.kv.page_size, tid = threadIdx.x;
  int len = a.seq_lens[b];
  if (len < 0 || len > (long long)a.table.cols * ps) {
    if (tid == 0) record_error(st, kErrBadIndex, kSiteEvictLen);
    len = 0;
  }
  const int m = min(len, a.budget);
  if (g == 0 && tid == 0) a.new_lens[b] = m;
  const int* pages = a.table.pages + b * a.table.stride;
  auto src_page = [&](int j) {
    const int p = pages[j / ps];
    if (p >= 0 && p < a.kv.num_pages) return p;
    record_error(st, kErrBadIndex, kSiteEvictPage);
    return -1;
  };
  auto key_at = [&](int j) -> uint32_t {
    const int p = src_page(j);
    return p < 0 ? 0u : score_key(a.scores[((long long)p * a.kv.Hkv + g) * ps + j % ps]);
  };
  // The need-th largest key among the candidates [lo, hi), a byte at a time.
  const int lo = a.sinks, hi = len - a.recent;
  uint32_t prefix = 0, mask = 0;
  int need = m - a.sinks - a.recent;     // candidates to keep
  const bool all = len <= a.budget;
  if (!all && need > 0)
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kThreads) {
        const uint32_t k = key_at(j);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int bin = 255, left = need;
        while (bin > 0 && hist[bin] < left) left -= hist[bin--];
        s_prefix = prefix | ((uint32_t)bin << shift);
        s_need = left;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
      mask |= 255u << shift;
    }
  // Ordered list of the kept indices: larger keys, and the first `need` equal ones.
  int* kept = a.kept + ((long long)b * a.kv.Hkv + g) * a.budget;
  int out = 0, equal = 0;
  for (int base = 0; base < len; base += kThreads) {
    const int j = base + tid;
    int keep = 0, eq = 0;
    if (j < len) {
      if (all || j < lo || j >= hi) keep = 1;
      else if (m > a.sinks + a.recent) {
        const uint32_t k = key_at(j);
        keep = k > prefix;
        eq = k == prefix;
      }
    }
    int total;
    const int eq_rank = block_scan(eq, warp_sums, total) + equal;
    if (eq && eq_rank <= need) keep = 1;
    equal += total;
    const int at = block_scan(keep, warp_sums, total) + out;
    if (keep) kept[at - 1] = j;
    out += total;
  }
  for (int i = m + tid; i < a.budget; i += kThreads) kept[i] = -1;
  __syncthreads();
  // Copy: 16 bytes a thread.
  const int vecs = a.kv.d / 8;
  for (long long x = tid; x < (long long)m * vecs; x += kThreads) {
    const int i = (int)(x / vecs), e = (int)(x % vecs) * 8;
    const int j = kept[i], p = src_page(j), to = a.dst.pages[b * a.dst.stride + i / ps];
    if (to < 0 || to >= a.kv.num_pages) {
      record_error(st, kErrBadIndex, kSiteEvictPage);
      continue;
    }
    if (p < 0) continue;
    const long long from = p * a.kv.s_page + g * a.kv.s_head + (long long)(j % ps) * a.kv.s_slot + e;
    const long long at = to * a.kv.s_page + g * a.kv.s_head + (long long)(i % ps) * a.kv.s_slot + e;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.kv.k) + at) =
        *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.kv.k) + from);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.kv.v) + at) =
        *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.kv.v) + from);
    if (e == 0)
      a.scores[((long long)to * a.kv.Hkv + g) * ps + i % ps] = a.scores[((long long)p * a.kv.Hkv + g) * ps + j % ps];
  }
}

}  // namespace

cudaError_t launch_paged_evict(const EvictArgs& a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  fa_evict_kernel<<<a.B * a.kv.Hkv, kThreads, 0, stream>>>(a, st);
  return cudaGetLastError();
}

}  // namespace fa
