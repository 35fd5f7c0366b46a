// Attention of one new token per sequence over a paged key / value cache.
//
//   o_h = sum_j p_h(j) v_j,  p_h(j) = exp(scale q_h . k_j - lse_h),
//   lse_h = ln sum_j exp(scale q_h . k_j)
// over the visible keys j of [max(0, len - window), len); with scores, each
// visible key's accumulated weight grows by sum over the group's heads of
// p_h(j).
//
// Bound by HBM: each K and V row is read once for all query heads of its kv
// head where these are at most 16, 4 d bytes per key against 4 G d operations (G
// = Hq / Hkv heads); above that once for every 16 of them.
//
// fa_paged_decode_kernel.  The keys of all (sequence, kv head, chunk of up to
// 16 query heads) units, in tiles of 64 (d = 128) or 128 (d = 64), form one
// line that is cut into equal parts, one per CTA (two CTAs per SM), so batches
// of any lengths load the SMs evenly and one long sequence is spread over all
// of them.  A part starts and ends anywhere: a unit that lies in one CTA is
// finished there, a unit cut over several leaves one unnormalised (O, max,
// sum) per CTA in the workspace (at most two a CTA: its first and its last
// unit), which fa_paged_finish_kernel joins in a fixed order.
//   Warp 4 is the producer: it looks the pages of several tiles up at once and
// copies 16-key slices (a page is a multiple of 16, so a slice lies in one
// page) into a ring of three 32 KB tiles with TMA, 128-byte swizzled.  Warps
// 0-3 each own every fourth slice and run their own online softmax over it, so
// they meet only at a unit's end; the next unit's query rows are loaded while
// the current one is worked on.
//   Matrix products by mma.sync (m16n8k16): S^T = K Q^T takes 16 keys as rows
// and 8 heads as columns, and O^T += V^T P^T takes 16 elements of d as rows,
// so groups of up to 8 heads waste nothing on padding to 16 rows, and a
// head's maximum, sum and rescale factor sit in the lanes that hold its
// column of S^T and O^T alike.  P^T goes from accumulator to operand layout
// by one 8x8 transpose in registers.  At one query row per head the tensor
// pipe is busy 13 % of the time that the copies take, so the tcgen05 path, whose
// 128-row tiles would be filled 1/16 by a group of 8, has nothing to win here.
//
//   Few short units.  A cluster of up to 8 CTAs takes each unit, its CTAs equal
// runs of the unit's tiles; what they leave stays in their shared memory, where
// all of them join it, and with scores each adds the weights of its own keys.
// One launch, no scan of the lengths, nothing in the workspace but the stashed
// scores; but CTAs of short sequences idle, so the launcher takes it only where
// a CTA gets few tiles (decode_cluster, with both sides' times).
//
// Measured (calls in a row on three sets of tensors; of the 6.79 TB/s copy
// rate), decode and finish kernels together: 8 sequences of 32768 keys, 32 q
// and 8 kv heads, d = 128, 1074 MB: 164 us, 97 %; 64 sequences of 0 to 8192 keys,
// 16 heads, d = 64, 1000 MB: 152 us, 97 %; 16 sequences of 0 to 8192, 236 MB: 45
// us, and 51 us with scores.  About 5 us of these are the start (lengths, page
// numbers, first tiles) and the finish kernel.  One sequence of 1000 keys, by
// clusters: 5.0 us, 7.0 by equal parts.  A window of 1024 keys on the first of
// these: 8.6 us for 34 MB.
//   Larger groups, 8 sequences of 32768 keys, d = 128.  8 kv heads, 1074 MB: 8
// heads each 165 us, 96 %; 16 heads each 171 us, 92 %.  One kv head, 134 MB: 16
// heads 35.4 us; 32 heads, which read it twice, 49.7.  (9 and more heads at d =
// 128 want more than the 168 registers that two CTAs leave a thread: the query
// rows are loaded when their unit comes up, and the equal-parts kernel spills 64
// bytes.)
#include "fa_paged.h"
#include "sm103a.cuh"

#include <cuda_fp16.h>

namespace fa {

namespace {

constexpr int kConsumers = 4;                      // warps, one 16-key slice of a tile each
constexpr int kThreads = (kConsumers + 1) * 32;

// Wait-site ids.
enum : int { kSiteFull = 47, kSiteEmpty = 48, kDrainFull = 49 };

template <int D>
struct Cfg {
  static constexpr int kSl = 128 / D;                          // slices of a tile per warp
  static constexpr int kSlices = kSl * kConsumers;
  static constexpr int kKeys = 16 * kSlices;                   // keys of a tile
  static constexpr int kStages = 3;                            // 96 KB of tiles in flight per CTA
  static constexpr uint32_t kHalf = kKeys * D * 2u;            // K or V of a tile: [D/64][keys][128 bytes]
  static constexpr uint32_t kAtom = kKeys * 128u;
  static constexpr uint32_t kStage = 2u * kHalf;
  static constexpr uint32_t kBuf = kStages * kStage;           // [4 warps][8 heads][D] fp32, one head group
  static constexpr uint32_t kMl = kBuf + kConsumers * 8u * D * 4u;   // [4 warps][16 heads] (max, sum)
  static constexpr uint32_t kBar = kMl + kConsumers * 16u * 8u;
  static constexpr uint32_t kBytes = kBar + 256u;
};

struct Bars {
  uint64_t full[3], empty[3];
  uint32_t mask[3];          // slices of the stage's tile that were loaded
  int abort;
  int scan[kThreads / 32];
  int b0;                    // first sequence of this CTA's part
  long long before;          // tiles (per unit column) of the sequences before it
  long long total;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// Matrix products of 16-bit operands.  For the product with V an fp32 weight x
// becomes two values, hi + lo = x but for the rounding of lo, 2^-15 x in bf16 and
// 2^-21 x in fp16 (but no less than 2^-25): rounded to one value the weights
// made o's error 1.1-1.2 times that of rounding o alone.  The second product
// costs nothing where HBM bounds (8 sequences of 32768 keys, 32 q and 8 kv heads,
// d = 128: 165.2 us either way), 1 % at 16 heads a group (169.1 -> 170.9), 0.15
// us on one sequence of 1000 keys.  Both halves of a weight are positive, so that
// an infinite v gives an infinite o, and not the NaN of 0 or of a negative half
// times infinity.
template <typename T>
struct Mma;
template <>
struct Mma<__nv_bfloat16> {
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return cvt_bf16x2(lo, hi); }
  // hi: the upper halves of the largest floats below x (0 for 0); lo: the rest.
  static __device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    const uint32_t a = (max(__float_as_uint(x), 1u) - 1) & 0xffff0000u, b = (max(__float_as_uint(y), 1u) - 1) & 0xffff0000u;
    hi = __byte_perm(a, b, 0x7632);
    lo = pack(x - __uint_as_float(a), y - __uint_as_float(b));
  }
  static constexpr float kShift = 0.f;
};
template <>
struct Mma<__half> {
  // Weights are formed as 2^(s - m + 12): relative to the largest they would
  // vanish below 2^-25 in fp16, where many of them can still add up to
  // something; so they do below 2^-37, and the largest is 4096.  Sums and O
  // carry the factor alike.
  static constexpr float kShift = 12.f;
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  // hi: x less a little over 2^-24, the smallest step, rounded down; lo: the rest.
  static __device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    constexpr float kLess = 1.f - 0x1p-22f, kStep = 0x1p-24f;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(fmaf(y, kLess, -kStep)), "f"(fmaf(x, kLess, -kStep)));
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = pack(x - h.x, y - h.y);
  }
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Barrier among the consumer warps.
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory"); }

// Visible keys [first, len) of a sequence, as tiles [tile0, tile0 + n) of kKeys.
struct Span {
  int len, first, tile0, n;
};
template <int kKeys>
__device__ __forceinline__ Span span_of_len(const DecodeArgs& a, int len) {
  Span s;
  s.len = len;
  if (s.len < 0 || s.len > (long long)a.table.cols * a.kv.page_size) s.len = -1;   // recorded by the caller
  s.first = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
  s.tile0 = s.first / kKeys;
  s.n = s.len > 0 ? (s.len - 1) / kKeys - s.tile0 + 1 : 0;
  return s;
}
template <int kKeys>
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b) {
  return span_of_len<kKeys>(a, a.seq_lens[b]);
}

// The line of `total` tiles is cut into min(total, CTAs) parts: none is empty.
// Start of part i, and the part a tile belongs to.
__device__ __forceinline__ long long part_start(long long total, int i, int parts) { return total * i / parts; }
__device__ __forceinline__ int part_of(long long tile, long long total, int parts) {
  return (int)(((tile + 1) * parts - 1) / total);
}

// A CTA's way through its part: unit (b, column), tile within the unit.
template <int kKeys>
struct Walk {
  int b, col, tile;
  Span s;
  long long left;      // tiles of the part from here on
  // On to the unit after this one.
  __device__ __forceinline__ void next_unit(const DecodeArgs& a, int cols) {
    tile = 0;
    if (++col < cols) return;
    col = 0;
    do {
      if (++b >= a.B) {
        left = 0;
        return;
      }
      s = span_of<kKeys>(a, b);
    } while (s.n == 0);
  }
  __device__ __forceinline__ void next(const DecodeArgs& a, int cols) {
    --left;
    if (++tile == s.n && left > 0) next_unit(a, cols);
  }
};

// Query rows of unit (b, col) as the B operands of S^T = K Q^T: column = head
// lane / 4, rows = two elements of d at 2 (lane % 4), and eight further on.
template <typename T, int D, int NT>
__device__ __forceinline__ void load_q(const DecodeArgs& a, int b, int col, int chunks, uint32_t (&q)[NT][D / 16][2]) {
  const int lane = threadIdx.x & 31, G = a.Hq / a.kv.Hkv;
  const int g = col / chunks, h0 = g * G + (col - g * chunks) * 8 * NT + (lane >> 2), h1 = (g + 1) * G;
  const T* p = static_cast<const T*>(a.q) + b * a.q_sb + (lane & 3) * 2;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const bool in = h0 + n * 8 < h1;
    const T* x = p + (in ? h0 + n * 8 : h1 - 1) * a.q_sh;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) q[n][k][e] = in ? *reinterpret_cast<const uint32_t*>(x + k * 16 + e * 8) : 0u;
  }
}

// Sequences without visible keys: O = 0, LSE = -inf.  One warp of each CTA
// takes every gridDim.x-th sequence.
template <typename T, int D>
__device__ __forceinline__ void fill_empty(const DecodeArgs& a) {
  const int lane = threadIdx.x & 31;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (span_of<Cfg<D>::kKeys>(a, b).n > 0) continue;
    uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.o) + (long long)b * a.Hq * D);
    for (int i = lane; i < a.Hq * (D / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
    for (int i = lane; i < a.Hq; i += 32) a.lse[(long long)b * a.Hq + i] = -INFINITY;
  }
}

// A unit whose tiles a cluster shared: each CTA left its share's O [16][D] and
// (max, sum) [16] in its shared memory.  The threads of all CTAs take two
// elements of a head each.
template <int D>
constexpr uint32_t kClusterMl = 16u * D * 4u;
template <typename T, int D>
__device__ __forceinline__ void join_cluster(const DecodeArgs& a, const uint8_t* smem, const Walk<Cfg<D>::kKeys>& w, int rank,
                                             int h0, int h1) {
  for (int i = rank * kConsumers * 32 + threadIdx.x; i < (h1 - h0) * (D / 2); i += a.cluster * kConsumers * 32) {
    const int hh = i / (D / 2), d = i % (D / 2) * 2;
    float2 y[kMaxCluster], x[kMaxCluster];         // all loads in flight before the first is used
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      const int from = r < a.cluster ? r : rank;
      y[r] = ld_cluster2(reinterpret_cast<const float2*>(smem + kClusterMl<D>) + hh, from);
      x[r] = ld_cluster2(reinterpret_cast<const float2*>(smem + (hh * D + d) * 4), from);
    }
    float m = -INFINITY, l = 0.f;
    float2 o = make_float2(0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) m = fmaxf(m, y[r].x);
    const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < a.cluster) {
        const float f = ex2(y[r].x - mu);
        l = fmaf(f, y[r].y, l);
        o.x = fmaf(f, x[r].x, o.x);
        o.y = fmaf(f, x[r].y, o.y);
      }
    const long long row = (long long)w.b * a.Hq + h0 + hh;
    const bool none = w.s.n == 0;                  // no visible keys
    const float inv = none ? 0.f : 1.f / l;
    *reinterpret_cast<uint32_t*>(static_cast<T*>(a.o) + row * D + d) = Mma<T>::pack(o.x * inv, o.y * inv);
    if (d == 0) a.lse[row] = none ? -INFINITY : (m + (log2f(l) - Mma<T>::kShift)) * 0.69314718055994530942f;
  }
}

// The accumulated weights of the keys of this CTA's tiles [tile, tile + n) of
// the unit, whose group's heads it has all, from the scores that the CTA
// stashed.
template <typename T, int D>
__device__ __forceinline__ void add_cluster_weights(const DecodeArgs& a, const uint8_t* smem,
                                                    const Walk<Cfg<D>::kKeys>& w, int rank, int g, int G, int tile, int n) {
  constexpr int kKeys = Cfg<D>::kKeys;
  const int lane = threadIdx.x & 31;
  float2 y[kMaxCluster];               // lane h: head h of the group
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    y[r] = ld_cluster2(reinterpret_cast<const float2*>(smem + kClusterMl<D>) + min(lane, G - 1), r < a.cluster ? r : rank);
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) m = fmaxf(m, y[r].x);
  const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) l = r < a.cluster ? fmaf(ex2(y[r].x - mu), y[r].y, l) : l;
  const float lse2 = m + (log2f(l) - Mma<T>::kShift);
  const int from = max((w.s.tile0 + tile) * kKeys, w.s.first), to = min((w.s.tile0 + tile + n) * kKeys, w.s.len);
  for (int key0 = from + (threadIdx.x & ~31); key0 < to; key0 += kConsumers * 32) {
    const int key = key0 + lane, c = key / a.kv.page_size;
    const bool in = key < to;
    const int page = in ? a.table.pages[w.b * a.table.stride + c] : -1;
    const float* x = a.stash + (((long long)w.b * a.kv.Hkv + g) * a.stash_keys + (in ? key : from)) * G;
    float sum = 0.f;
    if (G % 4 == 0) {
      for (int h = 0; h < G; h += 4) {
        const float4 v = *reinterpret_cast<const float4*>(x + h);
        sum += (ex2(v.x - __shfl_sync(0xffffffffu, lse2, h)) + ex2(v.y - __shfl_sync(0xffffffffu, lse2, h + 1))) +
               (ex2(v.z - __shfl_sync(0xffffffffu, lse2, h + 2)) + ex2(v.w - __shfl_sync(0xffffffffu, lse2, h + 3)));
      }
    } else {
      for (int h = 0; h < G; ++h) sum += ex2(x[h] - __shfl_sync(0xffffffffu, lse2, h));
    }
    if (page >= 0 && page < a.kv.num_pages)
      atomicAdd(&a.scores[((long long)page * a.kv.Hkv + g) * a.kv.page_size + (key - c * a.kv.page_size)], sum);
  }
}

template <typename T, int D, int NT, bool kCluster>
__global__ void __launch_bounds__(kThreads, 2)
    fa_paged_decode_kernel(const __grid_constant__ TmaMap4 tmK, const __grid_constant__ TmaMap4 tmV, const DecodeArgs a,
                           const DevStatus st) {
  using C = Cfg<D>;
  constexpr int kSl = C::kSl;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kBar);
  volatile int* abort_flag = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  if ((smem_u32(smem) & 1023u) != 0) {
    wait_for_previous();
    if (threadIdx.x == 0) {
      record_error(st, kErrDeviceTimeout, 0);
      if (!kCluster) a.parts[blockIdx.x].left = 0;
    }
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], kConsumers);
    }
    bars->abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  wait_for_previous();
  const int G = a.Hq / a.kv.Hkv, chunks = (G + 8 * NT - 1) / (8 * NT), cols = a.kv.Hkv * chunks;
  Walk<C::kKeys> w;
  long long total = 0, t0 = 0, t1 = 0;            // the line's tiles, and this CTA's part of them
  int parts = 0, rank = 0;
  if constexpr (kCluster) {
    // The cluster's unit, and this CTA's share of its tiles (perhaps none).
    const int unit = blockIdx.x / a.cluster;
    rank = blockIdx.x - unit * a.cluster;
    w.b = unit / cols;
    w.col = unit - w.b * cols;
    w.s = span_of<C::kKeys>(a, w.b);
    w.tile = w.s.n * rank / a.cluster;
    w.left = w.s.n * (rank + 1) / a.cluster - w.tile;
    if (w.s.len < 0 && w.col == 0 && rank == 0 && threadIdx.x == 0) record_error(st, kErrBadIndex, kSiteDecodeLen);
    __syncthreads();
  } else {
    const int first_len = (int)threadIdx.x < a.B ? a.seq_lens[threadIdx.x] : 0;

    // The line: its length, and this CTA's first sequence.
    for (int round = 0; round < 2; ++round) {
      // Round 0 finds the total; round 1, for batches of more than one block's
      // worth, walks again to find the start (one block's worth is still there).
      long long before = 0, t0 = 0;
      for (int base = 0; base < a.B; base += kThreads) {
        const int b = base + threadIdx.x;
        Span s{};
        if (b < a.B) {
          s = span_of_len<C::kKeys>(a, base == 0 ? first_len : a.seq_lens[b]);
          if (s.len < 0 && round == 0 && blockIdx.x == 0) record_error(st, kErrBadIndex, kSiteDecodeLen);
        }
        int x = s.n;
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, d);
          if (lane >= d) x += y;
        }
        __syncthreads();
        if (lane == 31) bars->scan[warp] = x;
        __syncthreads();
        long long pre = before + x - s.n;
        for (int w = 0; w < kThreads / 32; ++w) {
          if (w < warp) pre += bars->scan[w];
          before += bars->scan[w];
        }
        const bool last = base + kThreads >= a.B;
        if (round == 0 && last) total = before * cols;
        const int parts = (int)min(total, (long long)gridDim.x);
        if ((last || round == 1) && blockIdx.x < parts) t0 = part_start(total, blockIdx.x, parts);
        if ((round == 1 || a.B <= kThreads) && s.n > 0 && pre * cols <= t0 && t0 < (pre + s.n) * cols) {
          bars->b0 = b;
          bars->before = pre * cols;
        }
      }
      if (a.B <= kThreads) break;
    }
    __syncthreads();
    parts = (int)min(total, (long long)gridDim.x);
    if ((int)blockIdx.x >= parts) {
      if (threadIdx.x == 0) a.parts[blockIdx.x].left = 0;
      if (warp == kConsumers) fill_empty<T, D>(a);
      return;
    }
    t0 = part_start(total, blockIdx.x, parts);
    t1 = part_start(total, blockIdx.x + 1, parts);
    w.left = t1 - t0;
    w.b = bars->b0;
    w.s = span_of<C::kKeys>(a, w.b);
    {
      const long long in = t0 - bars->before;
      w.col = (int)(in / w.s.n);
      w.tile = (int)(in - (long long)w.col * w.s.n);
    }
  }

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    // Lane l looks up slice l % kSlices of tile l / kSlices of the unit's next
    // tiles; lanes 0-15 issue one copy each: slice, K or V, 64-column block.
    constexpr int kAhead = 32 / C::kSlices;
    static_assert(C::kSlices * 2 * (D / 64) == 16, "copies of a tile");
    // The lookup of the next run of tiles is issued before the copies of this
    // one, and not repeated for the next kv head of a sequence that fits one.
    const int my_slice = lane % C::kSlices, my_tile = lane / C::kSlices;
    auto look_up = [&](const Walk<C::kKeys>& x, int& page, int& slot) {
      const int have = (int)min((long long)min(x.s.n - x.tile, kAhead), x.left);
      const int key0 = (x.s.tile0 + x.tile + my_tile) * C::kKeys + my_slice * 16;
      page = 0;
      slot = -1;                       // not visible: not copied
      if (my_tile < have && key0 < x.s.len && key0 + 16 > x.s.first) {
        const int c = key0 / a.kv.page_size;
        slot = key0 - c * a.kv.page_size;
        page = a.table.pages[x.b * a.table.stride + c];
      }
      return have;
    };
    DecodePart part{};
    part.b = w.b;
    part.col = w.col;
    part.tile = w.tile;
    part.left = (int)w.left;
    const int first_n = w.s.n;
    int it = 0, page, slot, have = look_up(w, page, slot);
    bool good = true;
    while (good && w.left > 0) {
      Walk<C::kKeys> x = w;
      x.left -= have;
      x.tile += have;
      if (x.tile == x.s.n && x.left > 0) x.next_unit(a, cols);
      int page_next = page, slot_next = slot, have_next = have;
      if (x.left > 0 && !(x.b == w.b && x.tile == w.tile && x.left >= have)) have_next = look_up(x, page_next, slot_next);
      if (slot >= 0 && (page < 0 || page >= a.kv.num_pages)) {
        record_error(st, kErrBadIndex, kSiteDecodePage);
        slot = -1;
      }
      const int g = w.col / chunks;
      for (int i = 0; i < have; ++i, ++it) {
        const int s = it % C::kStages, r = it / C::kStages;
        if (r > 0 && !mbar_wait_warp(&bars->empty[s], (r - 1) & 1, st, abort_flag, kSiteEmpty)) {
          good = false;
          break;
        }
        const int p = __shfl_sync(0xffffffffu, page, i * C::kSlices + my_slice);
        const int sl = __shfl_sync(0xffffffffu, slot, i * C::kSlices + my_slice);
        const uint32_t mask = __ballot_sync(0xffffffffu, sl >= 0) & ((1u << C::kSlices) - 1);
        if (lane == 0) {
          bars->mask[s] = mask;
          mbar_arrive_expect_tx(&bars->full[s], __popc(mask) * 2u * 16u * D * 2u);
        }
        __syncwarp();
        if (lane < 16 && sl >= 0) {
          const int kv = my_tile & 1, atom = my_tile >> 1;
          tma_load_4d(smem + s * C::kStage + kv * C::kHalf + atom * C::kAtom + my_slice * 2048u, kv ? &tmV : &tmK,
                      &bars->full[s], atom * 64, sl, g, p);
        }
      }
      w = x;
      page = page_next;
      slot = slot_next;
      have = have_next;
    }
    if (!kCluster && lane == 0) {
      DecodePart d = part;
      const long long u0 = t0 - d.tile;
      d.i0 = part_of(u0, total, parts);
      d.i1 = part_of(u0 + first_n - 1, total, parts);
      d.last_i1 = good && w.tile < w.s.n ? part_of(t1 - 1 + (w.s.n - w.tile), total, parts) : blockIdx.x;
      a.parts[blockIdx.x] = d;
    }
    if (!kCluster) fill_empty<T, D>(a);
    // Every copy issued must have landed before the CTA may exit.
    if (lane == 0)
      for (int s = 0; s < C::kStages && s < it; ++s) {
        const int last = it - 1 - ((it - 1 - s) % C::kStages);
        mbar_wait_drain(&bars->full[s], (last / C::kStages) & 1, st, kDrainFull);
      }
    if (kCluster && a.cluster > 1) {
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int qr = lane >> 2, qc = lane & 3;        // fragment row and column pair
  const uint32_t stage0 = smem_u32(smem);
  // ldmatrix row addresses: K, rows = keys (lane & 15), 16-byte half lane >> 4;
  // V transposed, rows = keys (lane & 7) + 8 (lane >> 4), half (lane >> 3) & 1.
  const int krow = warp * 16 + (lane & 15), vrow = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
  const uint32_t kbase = stage0 + krow * 128u, vbase = stage0 + C::kHalf + vrow * 128u;
  const int khalf = lane >> 4, vhalf = (lane >> 3) & 1;
  float* buf = reinterpret_cast<float*>(smem + C::kBuf);
  float2* ml = reinterpret_cast<float2*>(smem + C::kMl);
  const float sl2 = a.scale_log2;

  uint32_t q[NT][D / 16][2], q_next[NT][D / 16][2];
  float o[NT][D / 16][4], m[NT][2], l[NT][2];
  bool dead = false, fresh = true;
  const int my_tile = w.tile, my_n = (int)w.left;
  int unit_pos = w.tile;                          // tile of the unit at which this CTA entered it
  // (Where the registers for a second set of query rows are lacking they are
  // loaded when their unit comes up.)
  constexpr bool kAheadQ = NT * D <= 128;
  if constexpr (kAheadQ) load_q<T, D, NT>(a, w.b, w.col, chunks, q_next);
  int g = 0, h0 = 0, h1 = 0;                      // kv head, query heads [h0, h1) of the unit
  float* stash = nullptr;                         // this lane's first score of key 0 of the unit
  for (int it = 0; w.left > 0 || (kCluster && it == 0); ++it) {
    const bool some = !kCluster || w.left > 0;    // a CTA of a cluster may have no tile, and joins in all the same
    if (fresh) {
      fresh = false;
      unit_pos = w.tile;
      g = w.col / chunks;
      h0 = g * G + (w.col - g * chunks) * 8 * NT;
      h1 = (g + 1) * G;
      if (a.stash) stash = a.stash + ((long long)w.b * a.kv.Hkv + g) * a.stash_keys * G + h0 - g * G + qc * 2;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          if constexpr (kAheadQ) {
            q[n][k][0] = q_next[n][k][0];
            q[n][k][1] = q_next[n][k][1];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][k][e] = 0.f;
        }
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
      }
      if constexpr (!kAheadQ) {
        load_q<T, D, NT>(a, w.b, w.col, chunks, q);
      } else if (w.left > w.s.n - w.tile) {
        Walk<C::kKeys> x = w;
        x.next_unit(a, cols);
        if (x.left > 0) load_q<T, D, NT>(a, x.b, x.col, chunks, q_next);
      }
    }
    const int s = it % C::kStages;
    // After a wait that gave up the warp goes on through its part without
    // touching the tiles, so that the warps still meet at each unit's end.
    if (some && !dead && !mbar_wait_warp(&bars->full[s], (it / C::kStages) & 1, st, abort_flag, kSiteFull)) dead = true;
    // The warp's slices are warp, warp + 4, ...
    const uint32_t loaded = dead || !some ? 0u : bars->mask[s] >> warp;
    constexpr uint32_t kMine = kSl == 1 ? 1u : 0x11u;
    if (loaded & kMine) {
      const int key0 = (w.s.tile0 + w.tile) * C::kKeys + warp * 16;
      // Keys [lo, hi) of slice u are visible; of one that was not loaded none.
      int lo[kSl], hi[kSl];
      bool edge = false;
#pragma unroll
      for (int u = 0; u < kSl; ++u) {
        lo[u] = w.s.first - key0 - u * 64;
        hi[u] = loaded >> (4 * u) & 1 ? w.s.len - key0 - u * 64 : 0;
        edge |= lo[u] > 0 || hi[u] < 16;
      }
      float c[kSl][NT][2][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int u = 0; u < kSl; ++u) {
          uint32_t x[4];
          ldsm4(x, kbase + s * C::kStage + (k >> 2) * C::kAtom + u * 64 * 128u + ((((k & 3) * 2 + khalf) ^ (krow & 7)) << 4));
#pragma unroll
          for (int n = 0; n < NT; ++n) Mma<T>::mma(c[u][n][k & 1], x, q[n][k][0], q[n][k][1]);
        }
      bool in0[kSl], in1[kSl];
#pragma unroll
      for (int u = 0; u < kSl; ++u) {
        in0[u] = qr >= lo[u] && qr < hi[u];
        in1[u] = qr + 8 >= lo[u] && qr + 8 < hi[u];
      }
      uint32_t pb[kSl][NT][2][2];                  // weights as the sum of two values of T (split)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[kSl][4], mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int u = 0; u < kSl; ++u) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[u][e] = (c[u][n][0][e] + c[u][n][1][e]) * sl2;
          if (a.stash) {
            const int h = h0 + n * 8 + qc * 2;
            float* z = stash + (long long)(key0 + u * 64 + qr) * G + n * 8;
            if (G % 2 == 0) {
              if (in0[u] && h < h1) *reinterpret_cast<float2*>(z) = make_float2(x[u][0], x[u][1]);
              if (in1[u] && h < h1) *reinterpret_cast<float2*>(z + 8 * G) = make_float2(x[u][2], x[u][3]);
            } else {
              if (in0[u] && h < h1) z[0] = x[u][0];
              if (in0[u] && h + 1 < h1) z[1] = x[u][1];
              if (in1[u] && h < h1) z[8 * G] = x[u][2];
              if (in1[u] && h + 1 < h1) z[8 * G + 1] = x[u][3];
            }
          }
          if (edge) {
            if (!in0[u]) x[u][0] = x[u][1] = -INFINITY;
            if (!in1[u]) x[u][2] = x[u][3] = -INFINITY;
          }
          mx0 = fmaxf(mx0, fmaxf(x[u][0], x[u][2]));
          mx1 = fmaxf(mx1, fmaxf(x[u][1], x[u][3]));
        }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
        }
        // Relative to the exact running maximum: no weight is above 2^kShift.
        if (__any_sync(0xffffffffu, mx0 > m[n][0] || mx1 > m[n][1])) {
          const float n0 = fmaxf(m[n][0], mx0), n1 = fmaxf(m[n][1], mx1);
          const float f0 = n0 == -INFINITY ? 0.f : ex2(m[n][0] - n0), f1 = n1 == -INFINITY ? 0.f : ex2(m[n][1] - n1);
          m[n][0] = n0;
          m[n][1] = n1;
          l[n][0] *= f0;
          l[n][1] *= f1;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            o[n][k][0] *= f0;
            o[n][k][1] *= f1;
            o[n][k][2] *= f0;
            o[n][k][3] *= f1;
          }
        }
        const float u0 = m[n][0] == -INFINITY ? 0.f : m[n][0] - Mma<T>::kShift;
        const float u1 = m[n][1] == -INFINITY ? 0.f : m[n][1] - Mma<T>::kShift;
#pragma unroll
        for (int u = 0; u < kSl; ++u) {
          x[u][0] = ex2(x[u][0] - u0);
          x[u][1] = ex2(x[u][1] - u1);
          x[u][2] = ex2(x[u][2] - u0);
          x[u][3] = ex2(x[u][3] - u1);
          l[n][0] += x[u][0] + x[u][2];
          l[n][1] += x[u][1] + x[u][3];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t hi, lo;
            Mma<T>::split(x[u][2 * e], x[u][2 * e + 1], hi, lo);
            pb[u][n][0][e] = transpose8(hi);
            pb[u][n][1][e] = transpose8(lo);
          }
        }
      }
      // V rows that are not visible may hold anything, NaN included: a weight
      // of 0 does not silence them, so their operand entries become 0.
      uint32_t z0[kSl], z1[kSl];
      if (edge) {
#pragma unroll
        for (int u = 0; u < kSl; ++u) {
          const int k0 = qc * 2;
          z0[u] = (k0 >= lo[u] && k0 < hi[u] ? 0xffffu : 0u) | (k0 + 1 >= lo[u] && k0 + 1 < hi[u] ? 0xffff0000u : 0u);
          z1[u] = (k0 + 8 >= lo[u] && k0 + 8 < hi[u] ? 0xffffu : 0u) | (k0 + 9 >= lo[u] && k0 + 9 < hi[u] ? 0xffff0000u : 0u);
        }
      }
#pragma unroll
      for (int u = 0; u < kSl; ++u)
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t x[4];
          ldsm4_trans(x, vbase + s * C::kStage + (k >> 2) * C::kAtom + u * 64 * 128u +
                             ((((k & 3) * 2 + vhalf) ^ (vrow & 7)) << 4));
          if (edge) {
            x[0] &= z0[u];
            x[1] &= z0[u];
            x[2] &= z1[u];
            x[3] &= z1[u];
          }
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int n = 0; n < NT; ++n) Mma<T>::mma(o[n][k], x, pb[u][n][p][0], pb[u][n][p][1]);
        }
    }
    __syncwarp();
    if (lane == 0 && some) mbar_arrive(&bars->empty[s]);

    const bool unit_ends = w.tile + 1 == w.s.n;
    if (unit_ends || w.left <= 1) {
      // ------------------------------------------------ the unit's end here
      const bool whole = unit_ends && unit_pos == 0;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l[n][0] += __shfl_xor_sync(0xffffffffu, l[n][0], d);
          l[n][1] += __shfl_xor_sync(0xffffffffu, l[n][1], d);
        }
        if (qr == 0) {
          ml[warp * 16 + n * 8 + qc * 2] = make_float2(m[n][0], l[n][0]);
          ml[warp * 16 + n * 8 + qc * 2 + 1] = make_float2(m[n][1], l[n][1]);
        }
      }
      consumer_sync();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n > 0) consumer_sync();                // the buffer's last readers
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M = -INFINITY;
#pragma unroll
          for (int x = 0; x < kConsumers; ++x) M = fmaxf(M, ml[x * 16 + n * 8 + qc * 2 + e].x);
          f[e] = M == -INFINITY ? 0.f : ex2(m[n][e] - M);
        }
        // [warp][head][d], d xor 8 (head / 2): the eight rows and four column
        // pairs a warp stores at once fall on 32 banks.
        float* mine = buf + (warp * 8 + qc * 2) * D;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int d0 = (k * 16 + qr) ^ (qc * 8), d1 = (k * 16 + qr + 8) ^ (qc * 8);
          mine[d0] = o[n][k][0] * f[0];
          mine[D + d0] = o[n][k][1] * f[1];
          mine[d1] = o[n][k][2] * f[0];
          mine[D + d1] = o[n][k][3] * f[1];
        }
        // 16 threads a head, D / 16 elements each.  The last read of ml before
        // the barrier: behind it a warp may be past its tiles of the next unit
        // and store that unit's (max, sum) while others still sum here.
        const int hh = threadIdx.x >> 4, e0 = (threadIdx.x & 15) * (D / 16), h = h0 + n * 8 + hh;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int x = 0; x < kConsumers; ++x) M = fmaxf(M, ml[x * 16 + n * 8 + hh].x);
#pragma unroll
        for (int x = 0; x < kConsumers; ++x) {
          const float2 y = ml[x * 16 + n * 8 + hh];
          L += M == -INFINITY ? 0.f : y.y * ex2(y.x - M);
        }
        consumer_sync();
        float r[D / 16];
#pragma unroll
        for (int e = 0; e < D / 16; e += 4) {
          const float* x = buf + hh * D + ((e0 + e) ^ ((hh >> 1) * 8));
          float4 y = *reinterpret_cast<const float4*>(x);
#pragma unroll
          for (int v = 1; v < kConsumers; ++v) {
            const float4 z = *reinterpret_cast<const float4*>(x + v * 8 * D);
            y.x += z.x;
            y.y += z.y;
            y.z += z.z;
            y.w += z.w;
          }
          r[e] = y.x;
          r[e + 1] = y.y;
          r[e + 2] = y.z;
          r[e + 3] = y.w;
        }
        if constexpr (kCluster) {
          // For the join; the tiles have been read.
          float4* dst = reinterpret_cast<float4*>(smem + ((n * 8 + hh) * D + e0) * 4);
#pragma unroll
          for (int e = 0; e < D / 16; e += 4) dst[e / 4] = make_float4(r[e], r[e + 1], r[e + 2], r[e + 3]);
          if (e0 == 0) reinterpret_cast<float2*>(smem + kClusterMl<D>)[n * 8 + hh] = make_float2(M, L);
        } else if (h < h1) {
          if (whole) {
            const float inv = 1.f / L;
            uint32_t y[D / 32];
#pragma unroll
            for (int e = 0; e < D / 32; ++e) y[e] = Mma<T>::pack(r[2 * e] * inv, r[2 * e + 1] * inv);
            T* dst = static_cast<T*>(a.o) + ((long long)w.b * a.Hq + h) * D + e0;
            if constexpr (D == 128) *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
            else *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
            if (e0 == 0) {
              const float lse2 = M + (log2f(L) - Mma<T>::kShift);
              a.lse[(long long)w.b * a.Hq + h] = lse2 * 0.69314718055994530942f;
              if (a.lse2) a.lse2[(long long)w.b * a.Hq + h] = lse2;
            }
          } else {
            // Slot 1: the unit starts in this CTA and goes on; slot 0: it
            // started earlier.
            const long long at = ((long long)blockIdx.x * 2 + (unit_pos == 0 ? 1 : 0)) * 16 + n * 8 + hh;
            float4* dst = reinterpret_cast<float4*>(a.part + at * D + e0);
#pragma unroll
            for (int e = 0; e < D / 16; e += 4) dst[e / 4] = make_float4(r[e], r[e + 1], r[e + 2], r[e + 3]);
            if (e0 == 0) a.part_ml[at] = make_float2(M, L);
          }
        }
      }
      fresh = true;
    }
    w.next(a, cols);
  }
  if constexpr (kCluster) {
    if (a.cluster > 1) cluster_sync();
    else consumer_sync();
    join_cluster<T, D>(a, smem, w, rank, h0, min(h1, h0 + 8 * NT));
    if (a.stash) {
      __syncwarp();
      add_cluster_weights<T, D>(a, smem, w, rank, g, G, my_tile, my_n);
    }
    __syncwarp();
    if (a.cluster > 1) cluster_sync();             // nobody exits while its share is read
  }
}

// Where part i left head hh of a unit whose first part is i0: in the part's
// last unit if that is where the unit starts, else in its first.
__device__ __forceinline__ long long left_at(int i, int i0, int hh) {
  return ((long long)i * 2 + (i == i0 ? 1 : 0)) * 16 + hh;
}

// Joins the units that were cut:
//   O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i, m = max_i m_i.
// Only the boundaries between two parts cut units, whatever the batch:
// unit_heads / 4 blocks for each boundary.  The blocks of a unit's boundaries
// share its heads: a warp per head where there are fewer blocks than heads
// (units over few parts), else a block per head, or up to D / 32 blocks per
// head, each with a slice of D.
// Parts are taken 16 bytes of O a thread, as many at a time as the block has
// threads for its slice; the order of the sums depends on the sizes alone.
template <typename T, int D>
__device__ __forceinline__ void write_row(const DecodeArgs& a, long long row, int d0, const float4& o, float m, float l) {
  const float inv = 1.f / l;
  *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + row * D + d0) =
      make_uint2(Mma<T>::pack(o.x * inv, o.y * inv), Mma<T>::pack(o.z * inv, o.w * inv));
  if (d0 == 0) {
    const float lse2 = m + (log2f(l) - Mma<T>::kShift);
    a.lse[row] = lse2 * 0.69314718055994530942f;
    if (a.lse2) a.lse2[row] = lse2;
  }
}
__device__ __forceinline__ void add_scaled(float4& o, float f, const float4& v) {
  o.x = fmaf(f, v.x, o.x);
  o.y = fmaf(f, v.y, o.y);
  o.z = fmaf(f, v.z, o.z);
  o.w = fmaf(f, v.w, o.w);
}
template <typename T, int D>
__device__ __forceinline__ void join(const DecodeArgs& a) {
  __shared__ float sf[kDecodeMaxParts], sm[4], sl[4];
  __shared__ float4 so[128];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Y = a.unit_heads / 4, i = 1 + blockIdx.x / Y;
  const DecodePart d = a.parts[i];
  if (d.left == 0 || d.tile == 0) return;    // no such part, or it starts with a unit
  const int G = a.Hq / a.kv.Hkv, per = a.unit_heads, chunks = (G + per - 1) / per;
  const int g = d.col / chunks, hc = d.col - g * chunks, heads = min(per, G - hc * per);
  const int i0 = d.i0, n = d.i1 - i0 + 1, blocks = (n - 1) * Y, z = (i - i0 - 1) * Y + blockIdx.x % Y;
  const long long row0 = (long long)d.b * a.Hq + g * G + hc * per;
  if (blocks < heads) {
    // A warp per head, D / 4 lanes: few parts.
    const int hh = z * 4 + warp;
    if (hh >= heads) return;
    float m = -INFINITY, l = 0.f;
    for (int x = lane; x < n; x += 32) m = fmaxf(m, a.part_ml[left_at(i0 + x, i0, hh)].x);
    for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    const float mu = m == -INFINITY ? 0.f : m;
    if (lane >= D / 4) return;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = 0; x < n; ++x) {
      const long long at = left_at(i0 + x, i0, hh);
      const float2 y = a.part_ml[at];
      const float f = ex2(y.x - mu);
      l = fmaf(f, y.y, l);
      add_scaled(o, f, *reinterpret_cast<const float4*>(a.part + at * D + lane * 4));
    }
    write_row<T, D>(a, row0 + hh, lane * 4, o, m, l);
    return;
  }
  int slices = D / 32;
  while (slices > 1 && slices * heads > blocks) slices /= 2;
  if (z >= heads * slices) return;
  const int hh = z / slices, lanes = D / 4 / slices, groups = 128 / lanes;
  const int d0 = (z - hh * slices) * (D / slices) + tid % lanes * 4, group = tid / lanes;
  // Scale and sum of every part.
  float2 y[(kDecodeMaxParts + 127) / 128];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int u = 0; u < (kDecodeMaxParts + 127) / 128; ++u) {
    const int x = u * 128 + tid;
    y[u] = x < n ? a.part_ml[left_at(i0 + x, i0, hh)] : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, y[u].x);
  }
  for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  if (lane == 0) sm[warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int u = 0; u < (kDecodeMaxParts + 127) / 128; ++u) {
    const int x = u * 128 + tid;
    const float f = ex2(y[u].x - mu);
    if (x < n) sf[x] = f;
    l = fmaf(f, y[u].y, l);
  }
  for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  if (lane == 0) sl[warp] = l;
  __syncthreads();
  l = (sl[0] + sl[1]) + (sl[2] + sl[3]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int x = group; x < n; x += groups)
    add_scaled(o, sf[x], *reinterpret_cast<const float4*>(a.part + left_at(i0 + x, i0, hh) * D + d0));
  so[tid] = o;
  __syncthreads();
  if (group > 0) return;
  for (int k = 1; k < groups; ++k) add_scaled(o, 1.f, so[k * lanes + tid]);
  write_row<T, D>(a, row0 + hh, d0, o, m, l);
}

// Log-sum-exp (log2 units) of head hh0 + lane < hh0 + n of a cut unit, from its
// parts: as many parts at a time as the warp has lanes for n heads.
__device__ __forceinline__ float parts_lse2(const DecodeArgs& a, int i0, int i1, int hh0, int n, float shift) {
  const int lane = threadIdx.x & 31;
  int w = 1;
  while (w < n) w *= 2;
  const int hh = hh0 + min(lane % w, n - 1), step = 32 / w, from = i0 + lane / w;
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int x = from; x <= i1; x += step) m = fmaxf(m, a.part_ml[left_at(x, i0, hh)].x);
  for (int k = w; k < 32; k *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll 4
  for (int x = from; x <= i1; x += step) {
    const float2 y = a.part_ml[left_at(x, i0, hh)];
    l = fmaf(ex2(y.x - mu), y.y, l);
  }
  for (int k = w; k < 32; k *= 2) l += __shfl_xor_sync(0xffffffffu, l, k);
  return m + (log2f(l) - shift);
}

// Adds each visible key's weight, summed over the group's heads from the
// stashed scores (log2 units), to its accumulated weight.  kSplit blocks take
// the tiles of a part in turn, a warp a tile.  With several head chunks to a
// kv head its keys are taken once, with the first chunk's tiles.  A reduction
// at L2 rather than a load and a store, so that sequences sharing a page both
// count.
// kJoined: every LSE is there; else those of cut units come from their parts.
constexpr int kSplit = 4;
template <int kKeys, bool kJoined>
__device__ __forceinline__ void add_weights(const DecodeArgs& a, int block, float shift) {
  constexpr int kLane = kKeys / 32;    // keys a lane
  const int lane = threadIdx.x & 31, i = block / kSplit;
  int skip = (block % kSplit) * 4 + (threadIdx.x >> 5);
  const DecodePart d = a.parts[i];
  if (d.left <= skip) return;
  const int Hkv = a.kv.Hkv, G = a.Hq / Hkv, chunks = (G + a.unit_heads - 1) / a.unit_heads, cols = Hkv * chunks;
  Walk<kKeys> w;
  w.b = d.b;
  w.col = d.col;
  w.tile = d.tile;
  w.left = d.left;
  w.s = span_of<kKeys>(a, d.b);
  int i0 = d.i0, i1 = d.i1;            // parts of the unit
  bool fresh = true;
  float lse2 = 0.f;
  for (;;) {
    // `skip` tiles on, unit by unit.
    while (skip >= w.s.n - w.tile) {
      const int n = w.s.n - w.tile;
      if (w.left <= n) return;
      skip -= n;
      w.left -= n;
      w.next_unit(a, cols);
      if (w.left <= 0) return;
      i0 = i;
      i1 = w.s.n > w.left ? d.last_i1 : i;
      fresh = true;
    }
    w.tile += skip;
    w.left -= skip;
    if (w.left <= 0) return;
    skip = 4 * kSplit;
    const int g = w.col / chunks;
    if (w.col != g * chunks) continue;
    float sum[kLane] = {};
    int page[kLane], slot[kLane];
#pragma unroll
    for (int u = 0; u < kLane; ++u) {
      const int key = (w.s.tile0 + w.tile) * kKeys + u * 32 + lane;
      page[u] = -1;
      slot[u] = 0;
      if (key >= w.s.first && key < w.s.len) {
        const int c = key / a.kv.page_size;
        page[u] = a.table.pages[w.b * a.table.stride + c];
        slot[u] = key - c * a.kv.page_size;
      }
    }
    for (int h0 = 0; h0 < G; h0 += 32) {
      const int nh = min(32, G - h0);
      if (fresh || G > 32) {           // lane h holds the LSE of head h0 + h
        const bool known = kJoined || i0 == i1;
        if (known && lane < nh) lse2 = a.lse2[(long long)w.b * a.Hq + g * G + h0 + lane];
        if (!known) lse2 = parts_lse2(a, i0, i1, h0, nh, shift);
      }
#pragma unroll
      for (int u = 0; u < kLane; ++u) {
        const int key = (w.s.tile0 + w.tile) * kKeys + u * 32 + lane;
        const bool in = key >= w.s.first && key < w.s.len;
        const float* x = a.stash + (((long long)w.b * Hkv + g) * a.stash_keys + key) * G + h0;
        if (G % 4 == 0) {
          for (int h = 0; h < nh; h += 4) {
            const float l0 = __shfl_sync(0xffffffffu, lse2, h), l1 = __shfl_sync(0xffffffffu, lse2, h + 1);
            const float l2 = __shfl_sync(0xffffffffu, lse2, h + 2), l3 = __shfl_sync(0xffffffffu, lse2, h + 3);
            if (in) {
              const float4 y = *reinterpret_cast<const float4*>(x + h);
              sum[u] += (ex2(y.x - l0) + ex2(y.y - l1)) + (ex2(y.z - l2) + ex2(y.w - l3));
            }
          }
        } else {
          for (int h = 0; h < nh; ++h) {
            const float l = __shfl_sync(0xffffffffu, lse2, h);
            if (in) sum[u] += ex2(x[h] - l);
          }
        }
      }
    }
    fresh = false;
#pragma unroll
    for (int u = 0; u < kLane; ++u)
      if (page[u] >= 0 && page[u] < a.kv.num_pages)
        atomicAdd(&a.scores[((long long)page[u] * Hkv + g) * a.kv.page_size + slot[u]], sum[u]);
  }
}

// What is left after the tiles: the first blocks join, the others (with
// scores) add the weights; neither half needs the other.
template <typename T, int D, bool kScores>
__global__ void __launch_bounds__(128) fa_paged_finish_kernel(const DecodeArgs a, int joins) {
  launch_dependents();
  wait_for_previous();
  if (!kScores || blockIdx.x < joins) join<T, D>(a);
  else add_weights<Cfg<D>::kKeys, false>(a, blockIdx.x - joins, Mma<T>::kShift);
}

// The weights after every join: where a kv head's units are several (a cut
// one's parts are not known to the others), or cut so often that forming the
// LSE from the parts in every warp costs more than waiting for the joins.
template <int kKeys>
__global__ void __launch_bounds__(128) fa_paged_weights_kernel(const DecodeArgs a) {
  launch_dependents();
  wait_for_previous();
  add_weights<kKeys, true>(a, blockIdx.x, 0.f);
}

template <typename T, int D>
cudaError_t launch_decode(const TmaMap4& tk, const TmaMap4& tv, const DecodeArgs& a, const DevStatus& st, int parts,
                          cudaStream_t stream) {
  if (a.cluster)
    return launch_after(a.unit_heads == 8 ? fa_paged_decode_kernel<T, D, 1, true> : fa_paged_decode_kernel<T, D, 2, true>,
                        parts, kThreads, Cfg<D>::kBytes, a.cluster, stream, tk, tv, a, st);
  cudaError_t e =
      launch_after(a.unit_heads == 8 ? fa_paged_decode_kernel<T, D, 1, false> : fa_paged_decode_kernel<T, D, 2, false>, parts,
                   kThreads, Cfg<D>::kBytes, 1, stream, tk, tv, a, st);
  if (e != cudaSuccess) return e;
  const int joins = (parts - 1) * (a.unit_heads / 4), adds = parts * kSplit;
  // In one launch unless units are cut into more than eight or so: it saves 1-2
  // us, but every warp forms the LSE from all of a unit's parts, the slower the
  // more heads a group has.  Us in one launch | in two, d = 128, by parts a unit
  // and heads a group: 10 parts, 1 head 38.5 | 39.8, 8 heads 42.2 | 43.2, 16 heads
  // 59.6 | 60.7; 19 parts 37.9 | 39.9, 42.4 | 43.1, 58.6 | 58.9; 38 parts 30.8 | 32.9,
  // 35.3 | 35.3, 50.7 | 48.7; 152 parts 24.0 | 23.6, 31.1 | 24.9, 50.0 | 34.5.  (So few
  // heads a group would take one launch up to about 100 parts.)
  if (a.scores && a.Hq / a.kv.Hkv <= a.unit_heads && parts <= 8LL * a.B * a.kv.Hkv)
    return launch_after(fa_paged_finish_kernel<T, D, true>, joins + adds, 128, 0, 1, stream, a, joins);
  if (joins > 0) e = launch_after(fa_paged_finish_kernel<T, D, false>, joins, 128, 0, 1, stream, a, joins);
  if (e == cudaSuccess && a.scores) e = launch_after(fa_paged_weights_kernel<Cfg<D>::kKeys>, adds, 128, 0, 1, stream, a);
  return e;
}

template <typename T, int D>
cudaError_t configure_decode() {
  static_assert(Cfg<D>::kBytes <= 115712, "two CTAs per SM");
  static_assert(Cfg<D>::kKeys == decode_tile_keys(D), "tile");
  cudaError_t e = cudaSuccess;
  for (auto k : {fa_paged_decode_kernel<T, D, 1, false>, fa_paged_decode_kernel<T, D, 2, false>,
                 fa_paged_decode_kernel<T, D, 1, true>, fa_paged_decode_kernel<T, D, 2, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kBytes);
  if (e == cudaSuccess) e = preload_kernel(fa_paged_finish_kernel<T, D, false>);
  if (e == cudaSuccess) e = preload_kernel(fa_paged_finish_kernel<T, D, true>);
  if (e == cudaSuccess) e = preload_kernel(fa_paged_weights_kernel<Cfg<D>::kKeys>);
  return e;
}

}  // namespace

cudaError_t configure_decode_kernels() {
  cudaError_t e = configure_decode<__nv_bfloat16, 64>();
  if (e == cudaSuccess) e = configure_decode<__nv_bfloat16, 128>();
  if (e == cudaSuccess) e = configure_decode<__half, 64>();
  if (e == cudaSuccess) e = configure_decode<__half, 128>();
  return e;
}

cudaError_t launch_paged_decode(int dtype, const TmaMap4& tk, const TmaMap4& tv, const DecodeArgs& a, const DevStatus& st,
                                int parts, cudaStream_t stream) {
  if (dtype == 0)
    return a.kv.d == 64 ? launch_decode<__nv_bfloat16, 64>(tk, tv, a, st, parts, stream)
                        : launch_decode<__nv_bfloat16, 128>(tk, tv, a, st, parts, stream);
  return a.kv.d == 64 ? launch_decode<__half, 64>(tk, tv, a, st, parts, stream)
                      : launch_decode<__half, 128>(tk, tv, a, st, parts, stream);
}

}  // namespace fa
