// Attention of one new token per sequence over a paged key / value cache.
//
//   o_h = sum_j p_h(j) v_j,  p_h(j) = exp(scale q_h . k_j - lse_h),
//   lse_h = ln sum_j exp(scale q_h . k_j)
// over the visible keys j of [max(0, len - window), len); with scores, each
// visible key's accumulated weight grows by sum over the group's heads of
// p_h(j).
//
// Bound by HBM: each K and V row is read once for all query heads of its kv
// head, 4 d bytes per key against 4 G d operations (G = Hq / Hkv heads).
//
// fa_paged_decode_kernel.  The keys of all (sequence, kv head, chunk of up to
// 16 query heads) units, in tiles of 64, form one line that is cut into equal
// parts, one per CTA (two CTAs per SM), so batches of any lengths load the SMs
// evenly and one long sequence is spread over all of them.  A part starts and
// ends anywhere: a unit that lies in one CTA is finished there, a unit cut
// over several leaves one unnormalised (O, max, sum) per CTA in the workspace
// (at most two a CTA: its first and its last unit), which
// fa_paged_finish_kernel joins in a fixed order.
//   Warp 4 is the producer: it looks the pages of eight tiles up at once and
// copies 16-key slices (a page is a multiple of 16, so a slice lies in one
// page) into a ring of tiles with TMA, 128-byte swizzled.  Warps 0-3 each own
// one slice of every tile and run their own online softmax over it, so they
// meet only at a unit's end.
//   Matrix products by mma.sync (m16n8k16): S^T = K Q^T takes 16 keys as rows
// and 8 heads as columns, and O^T += V^T P^T takes 16 elements of d as rows,
// so groups of up to 8 heads waste nothing on padding to 16 rows, and a
// head's maximum, sum and rescale factor sit in the lanes that hold its
// column of S^T and O^T alike.  P^T goes from accumulator to operand layout
// by one 8x8 transpose in registers.  At one query row per head the tensor
// work is 1-2 % of what the copies take, so the tcgen05 path, whose 128-row
// tiles would be filled 1/16 by a group of 8, has nothing to win here.
#include "fa_internal.h"
#include "sm103a.cuh"

#include <cuda_fp16.h>

namespace fa {

namespace {

constexpr int kConsumers = 4;                      // warps, one 16-key slice of a tile each
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kTileKeys = 16 * kConsumers;

// Wait-site ids.
enum : int { kSiteFull = 47, kSiteEmpty = 48, kDrainFull = 49 };

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 3 : 6;             // 96 KB of tiles in flight per CTA
  static constexpr uint32_t kHalf = kTileKeys * D * 2u;        // K or V of a tile: [D/64][64 keys][128 bytes]
  static constexpr uint32_t kStage = 2u * kHalf;
  static constexpr uint32_t kBuf = kStages * kStage;           // [4 warps][8 heads][D] fp32, one head group
  static constexpr uint32_t kMl = kBuf + kConsumers * 8u * D * 4u;   // [4 warps][16 heads] (max, sum)
  static constexpr uint32_t kBar = kMl + kConsumers * 16u * 8u;
  static constexpr uint32_t kBytes = kBar + 256u;
};

struct Bars {
  uint64_t full[6], empty[6];
  uint32_t mask[6];          // slices of the stage's tile that were loaded
  int abort;
  int scan[kThreads / 32];
  int b0;                    // first sequence of this CTA's part
  long long before;          // tiles (per unit column) of the sequences before it
  long long total;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

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
};
template <>
struct Mma<__half> {
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

// Programmatic dependent launch: let the next kernel of the stream start its
// blocks / wait until everything of the kernel before is complete and visible.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Visible keys [first, len) of a sequence, as 64-key tiles [tile0, tile0 + n).
struct Span {
  int len, first, tile0, n;
};
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b) {
  Span s;
  s.len = a.seq_lens[b];
  if (s.len < 0 || s.len > (long long)a.table.cols * a.kv.page_size) s.len = -1;   // recorded by the caller
  s.first = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
  s.tile0 = s.first / kTileKeys;
  s.n = s.len > 0 ? (s.len - 1) / kTileKeys - s.tile0 + 1 : 0;
  return s;
}

// The line of `total` tiles is cut into min(total, CTAs) parts: none is empty.
// Start of part i, and the part a tile belongs to.
__device__ __forceinline__ long long part_start(long long total, int i, int parts) { return total * i / parts; }
__device__ __forceinline__ int part_of(long long tile, long long total, int parts) {
  return (int)(((tile + 1) * parts - 1) / total);
}

// A CTA's way through its part: unit (b, column), tile within the unit.
struct Walk {
  int b, col, tile;
  Span s;
  long long left;      // tiles of the part from here on
  __device__ __forceinline__ void next(const DecodeArgs& a, int cols) {
    --left;
    if (++tile < s.n || left == 0) return;
    tile = 0;
    if (++col < cols) return;
    col = 0;
    do {
      if (++b >= a.B) {
        left = 0;
        return;
      }
      s = span_of(a, b);
    } while (s.n == 0);
  }
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    fa_paged_decode_kernel(const __grid_constant__ TmaMap4 tmK, const __grid_constant__ TmaMap4 tmV, const DecodeArgs a,
                           const DevStatus st) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kBar);
  volatile int* abort_flag = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) record_error(st, kErrDeviceTimeout, 0);
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
  const int G = a.Hq / a.kv.Hkv, chunks = (G + 8 * NT - 1) / (8 * NT), cols = a.kv.Hkv * chunks;

  // The line: tiles before each sequence (per column; CTA 0 keeps the list for
  // the join), the total, and this CTA's first sequence.
  long long total = 0;
  for (int round = 0; round < 2; ++round) {
    // Round 0 finds the total; round 1, for batches of more than one block's
    // worth, walks again to find the start (one block's worth is still there).
    long long before = 0, t0 = 0;
    for (int base = 0; base < a.B; base += kThreads) {
      const int b = base + threadIdx.x;
      Span s{};
      if (b < a.B) {
        s = span_of(a, b);
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
      if (round == 0 && blockIdx.x == 0 && b < a.B) a.prefix[b] = pre;
      const bool last = base + kThreads >= a.B;
      if (round == 0 && last) total = before * cols;
      const int parts = (int)min(total, (long long)gridDim.x);
      if ((last || round == 1) && blockIdx.x < parts) t0 = part_start(total, blockIdx.x, parts);
      if ((round == 1 || a.B <= kThreads) && s.n > 0 && pre * cols <= t0 && t0 < (pre + s.n) * cols) {
        bars->b0 = b;
        bars->before = pre * cols;
      }
    }
    if (round == 0 && blockIdx.x == 0 && threadIdx.x == 0) a.prefix[a.B] = before;
    if (a.B <= kThreads) break;
  }
  __syncthreads();
  const int parts = (int)min(total, (long long)gridDim.x);
  if ((int)blockIdx.x >= parts) return;
  const long long t0 = part_start(total, blockIdx.x, parts), t1 = part_start(total, blockIdx.x + 1, parts);
  Walk w;
  w.left = t1 - t0;
  w.b = bars->b0;
  w.s = span_of(a, w.b);
  {
    const long long in = t0 - bars->before;
    w.col = (int)(in / w.s.n);
    w.tile = (int)(in - (long long)w.col * w.s.n);
  }

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    // Lane l looks up slice l % 4 of tile l / 4 of the next eight tiles of the
    // unit; lanes 0-15 issue one copy each: slice, K or V, 64-column block.
    constexpr int kAtoms = D / 64;
    int it = 0;
    bool good = true;
    while (good && w.left > 0) {
      const int have = (int)min((long long)min(w.s.n - w.tile, 8), w.left);
      const int key0 = (w.s.tile0 + w.tile + (lane >> 2)) * kTileKeys + (lane & 3) * 16;
      int page = -1, slot = 0;
      if ((lane >> 2) < have && key0 < w.s.len && key0 + 16 > w.s.first) {
        const int c = key0 / a.kv.page_size;
        slot = key0 - c * a.kv.page_size;
        page = a.table.pages[w.b * a.table.stride + c];
        if (page < 0 || page >= a.kv.num_pages) {
          record_error(st, kErrBadIndex, kSiteDecodePage);
          page = -1;
        }
      }
      const int g = w.col / chunks;
      for (int i = 0; i < have; ++i, ++it) {
        const int s = it % C::kStages, r = it / C::kStages;
        if (r > 0 && !mbar_wait_warp(&bars->empty[s], (r - 1) & 1, st, abort_flag, kSiteEmpty)) {
          good = false;
          break;
        }
        const int p = __shfl_sync(0xffffffffu, page, i * 4 + (lane & 3));
        const int sl = __shfl_sync(0xffffffffu, slot, i * 4 + (lane & 3));
        const uint32_t mask = __ballot_sync(0xffffffffu, p >= 0) & 15u;
        if (lane == 0) {
          bars->mask[s] = mask;
          mbar_arrive_expect_tx(&bars->full[s], __popc(mask) * 2u * 16u * D * 2u);
        }
        __syncwarp();
        if (lane < 8 * kAtoms && p >= 0) {
          const int kv = (lane >> 2) & 1, atom = lane >> 3;
          tma_load_4d(smem + s * C::kStage + kv * C::kHalf + atom * (kTileKeys * 128u) + (lane & 3) * 2048u, kv ? &tmV : &tmK,
                      &bars->full[s], atom * 64, sl, g, p);
        }
        w.next(a, cols);
      }
    }
    // Every copy issued must have landed before the CTA may exit.
    if (lane == 0)
      for (int s = 0; s < C::kStages && s < it; ++s) {
        const int last = it - 1 - ((it - 1 - s) % C::kStages);
        mbar_wait_drain(&bars->full[s], (last / C::kStages) & 1, st, kDrainFull);
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

  uint32_t q[NT][D / 16][2];
  float o[NT][D / 16][4], m[NT][2], l[NT][2];
  bool dead = false, fresh = true;
  long long unit_pos = w.tile;                    // tile of the unit at which this CTA entered it
  for (int it = 0; w.left > 0; ++it) {
    const int g = w.col / chunks, h0 = g * G + (w.col - g * chunks) * 8 * NT, h1 = (g + 1) * G;
    if (fresh) {
      fresh = false;
      unit_pos = w.tile;
      const T* qp = static_cast<const T*>(a.q) + w.b * a.q_sb;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int h = h0 + n * 8 + qr;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const T* x = qp + h * a.q_sh + k * 16 + qc * 2;
          q[n][k][0] = h < h1 ? *reinterpret_cast<const uint32_t*>(x) : 0u;
          q[n][k][1] = h < h1 ? *reinterpret_cast<const uint32_t*>(x + 8) : 0u;
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][k][e] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
      }
    }
    const int s = it % C::kStages;
    // After a wait that gave up the warp goes on through its part without
    // touching the tiles, so that the warps still meet at each unit's end.
    if (!dead && !mbar_wait_warp(&bars->full[s], (it / C::kStages) & 1, st, abort_flag, kSiteFull)) dead = true;
    if (!dead && (bars->mask[s] >> warp & 1)) {
      const int key0 = (w.s.tile0 + w.tile) * kTileKeys + warp * 16;
      // Keys [lo, hi) of the slice are visible.
      const int lo = w.s.first - key0, hi = w.s.len - key0;
      const bool edge = lo > 0 || hi < 16;
      float c[NT][2][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t x[4];
        ldsm4(x, kbase + s * C::kStage + (k >> 2) * (kTileKeys * 128u) + ((((k & 3) * 2 + khalf) ^ (krow & 7)) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) Mma<T>::mma(c[n][k & 1], x, q[n][k][0], q[n][k][1]);
      }
      const bool in0 = qr >= lo && qr < hi, in1 = qr + 8 >= lo && qr + 8 < hi;
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (c[n][0][e] + c[n][1][e]) * sl2;
        if (a.stash) {
          const int h = h0 - g * G + n * 8 + qc * 2;
          float* z = a.stash + (((long long)w.b * a.kv.Hkv + g) * a.stash_keys + key0 + qr) * G + h;
          if (in0 && h < G) z[0] = x[0];
          if (in0 && h + 1 < G) z[1] = x[1];
          if (in1 && h < G) z[8LL * G] = x[2];
          if (in1 && h + 1 < G) z[8LL * G + 1] = x[3];
        }
        if (edge) {
          if (!in0) x[0] = x[1] = -INFINITY;
          if (!in1) x[2] = x[3] = -INFINITY;
        }
        float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
        }
        // The maximum is the exact running one, so a row's largest weight is 1
        // and rounding the weights to 16 bits for the product cannot touch it;
        // the sums keep the unrounded weights.
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
        const float u0 = m[n][0] == -INFINITY ? 0.f : m[n][0], u1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
        x[0] = ex2(x[0] - u0);
        x[1] = ex2(x[1] - u1);
        x[2] = ex2(x[2] - u0);
        x[3] = ex2(x[3] - u1);
        l[n][0] += x[0] + x[2];
        l[n][1] += x[1] + x[3];
        pb[n][0] = transpose8(Mma<T>::pack(x[0], x[1]));
        pb[n][1] = transpose8(Mma<T>::pack(x[2], x[3]));
      }
      // V rows that are not visible may hold anything, NaN included: a weight
      // of 0 does not silence them, so their operand entries become 0.
      const int k0 = qc * 2;
      uint32_t z0 = 0xffffffffu, z1 = 0xffffffffu;
      if (edge) {
        z0 = (k0 >= lo && k0 < hi ? 0xffffu : 0u) | (k0 + 1 >= lo && k0 + 1 < hi ? 0xffff0000u : 0u);
        z1 = (k0 + 8 >= lo && k0 + 8 < hi ? 0xffffu : 0u) | (k0 + 9 >= lo && k0 + 9 < hi ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t x[4];
        ldsm4_trans(x, vbase + s * C::kStage + (k >> 2) * (kTileKeys * 128u) + ((((k & 3) * 2 + vhalf) ^ (vrow & 7)) << 4));
        if (edge) {
          x[0] &= z0;
          x[1] &= z0;
          x[2] &= z1;
          x[3] &= z1;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) Mma<T>::mma(o[n][k], x, pb[n][0], pb[n][1]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->empty[s]);

    const bool unit_ends = w.tile + 1 == w.s.n;
    if (unit_ends || w.left == 1) {
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
        consumer_sync();
        // 16 threads a head, D / 16 elements each.
        const int hh = threadIdx.x >> 4, e0 = (threadIdx.x & 15) * (D / 16), h = h0 + n * 8 + hh;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int x = 0; x < kConsumers; ++x) M = fmaxf(M, ml[x * 16 + n * 8 + hh].x);
#pragma unroll
        for (int x = 0; x < kConsumers; ++x) {
          const float2 y = ml[x * 16 + n * 8 + hh];
          L += M == -INFINITY ? 0.f : y.y * ex2(y.x - M);
        }
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
        if (h < h1) {
          if (whole) {
            const float inv = 1.f / L;
            uint32_t y[D / 32];
#pragma unroll
            for (int e = 0; e < D / 32; ++e) y[e] = Mma<T>::pack(r[2 * e] * inv, r[2 * e + 1] * inv);
            T* dst = static_cast<T*>(a.o) + ((long long)w.b * a.Hq + h) * D + e0;
            if constexpr (D == 128) *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
            else *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
            if (e0 == 0) {
              const float lse2 = M + log2f(L);
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
}

// The parts [i0, i1] over which head h of (b, g) is cut, and its index in them.
struct Cut {
  int i0, i1, hh;
  // Where part i left the head: its last unit if it is the unit's first part.
  __device__ __forceinline__ long long at(int i) const { return ((long long)i * 2 + (i == i0 ? 1 : 0)) * 16 + hh; }
};
__device__ __forceinline__ Cut cut_of(const DecodeArgs& a, int g, int h, long long before, long long n, long long all,
                                      int parts) {
  const int G = a.Hq / a.kv.Hkv, per = a.unit_heads, chunks = (G + per - 1) / per, cols = a.kv.Hkv * chunks;
  const int hc = h / per;
  const long long total = all * cols, t0 = before * cols + (g * chunks + hc) * n;
  parts = (int)min(total, (long long)parts);
  return Cut{part_of(t0, total, parts), part_of(t0 + n - 1, total, parts), h - hc * per};
}

// What is left after the tiles, in one launch (each half needs only the decode
// kernel): block r < B * Hq joins row r, the other blocks add the weights.
//
// Join: the parts of a unit that was cut, in order, relative to the largest
// maximum: O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i; warps take every
// fourth part.  Sequences without visible keys get O = 0, LSE = -inf.
template <typename T, int D>
__device__ __forceinline__ void join_row(const DecodeArgs& a, int parts) {
  constexpr int E = D / 32;
  __shared__ float sl[4], so[4][D];
  const long long row = blockIdx.x;
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x - b * a.Hq, G = a.Hq / a.kv.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long before = a.prefix[b], n = a.prefix[b + 1] - before, all = a.prefix[a.B];
  if (n == 0) {
    for (int e = threadIdx.x; e < D; e += 128) static_cast<T*>(a.o)[row * D + e] = (T)0.f;
    if (threadIdx.x == 0) a.lse[row] = -INFINITY;
    return;
  }
  const Cut c = cut_of(a, hq / G, hq % G, before, n, all, parts);
  if (c.i0 == c.i1) return;
  float m = -INFINITY;
  for (int i = c.i0 + lane; i <= c.i1; i += 32) m = fmaxf(m, a.part_ml[c.at(i)].x);
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float mu = m == -INFINITY ? 0.f : m;
  float l = 0.f, o[E] = {};
#pragma unroll 4
  for (int i = c.i0 + warp; i <= c.i1; i += 4) {
    const float2 y = a.part_ml[c.at(i)];
    const float f = ex2(y.x - mu);
    const float* x = a.part + c.at(i) * D + lane * E;
    l += f * y.y;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(f, x[e], o[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  if (lane == 0) sl[warp] = l;
  __syncthreads();
  l = (sl[0] + sl[1]) + (sl[2] + sl[3]);
  const float inv = 1.f / l;
  for (int e = threadIdx.x; e < D; e += 128)
    static_cast<T*>(a.o)[row * D + e] = (T)(((so[0][e] + so[1][e]) + (so[2][e] + so[3][e])) * inv);
  if (threadIdx.x == 0) a.lse[row] = (m + log2f(l)) * 0.69314718055994530942f;
}

// Log-sum-exp (log2 units) of head h of (b, g): the decode kernel's if the
// unit was whole, else from its parts.
__device__ __forceinline__ float head_lse2(const DecodeArgs& a, int b, int g, int h, long long before, long long n,
                                           long long all, int parts) {
  const Cut c = cut_of(a, g, h, before, n, all, parts);
  if (c.i0 == c.i1) return a.lse2[(long long)b * a.Hq + g * (a.Hq / a.kv.Hkv) + h];
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int i = c.i0; i <= c.i1; ++i) m = fmaxf(m, a.part_ml[c.at(i)].x);
  const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll 4
  for (int i = c.i0; i <= c.i1; ++i) {
    const float2 y = a.part_ml[c.at(i)];
    l = fmaf(ex2(y.x - mu), y.y, l);
  }
  return m + log2f(l);
}

// Weights: adds each visible key's weight, summed over the group's heads from
// the stashed scores (log2 units), to its accumulated weight.  Warps take
// equal runs of the line of tiles (a kv head's keys once, whatever its head
// chunks), two keys a lane.  A reduction at L2 rather than a load and a store,
// so that sequences sharing a page both count.
__device__ __forceinline__ void add_weights(const DecodeArgs& a, int parts) {
  const int lane = threadIdx.x & 31;
  const int first = a.B * a.Hq, warp = (blockIdx.x - first) * 4 + (threadIdx.x >> 5), warps = (gridDim.x - first) * 4;
  const int Hkv = a.kv.Hkv, G = a.Hq / Hkv;
  const long long all = a.prefix[a.B], total = all * Hkv;
  long long t = total * warp / warps;
  const long long end = total * (warp + 1) / warps;
  if (t >= end) return;
  // Last sequence with prefix * Hkv <= t, 32 samples a round.
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const int k = __popc(__ballot_sync(0xffffffffu, at < hi && a.prefix[at] * Hkv <= t));
    lo += k * step;
    hi = min(hi, lo + step);
  }
  int b = lo;
  Span s = span_of(a, b);
  long long before = a.prefix[b];
  int g = (int)((t - before * Hkv) / s.n), tile = (int)(t - before * Hkv - (long long)g * s.n);
  bool fresh = true;
  float lse2 = 0.f;
  for (; t < end; ++t) {
    // Lane h holds the LSE of head h (of the 32 heads at hand, for larger groups).
    float w[2] = {0.f, 0.f};
    int page[2] = {-1, -1};
    long long slot[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = (s.tile0 + tile) * kTileKeys + u * 32 + lane;
      if (key >= s.first && key < s.len) {
        const int c = key / a.kv.page_size;
        page[u] = a.table.pages[b * a.table.stride + c];
        slot[u] = key - c * a.kv.page_size;
      }
    }
    for (int h0 = 0; h0 < G; h0 += 32) {
      if (fresh || G > 32) lse2 = h0 + lane < G ? head_lse2(a, b, g, h0 + lane, before, s.n, all, parts) : 0.f;
      const int nh = min(32, G - h0);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int key = (s.tile0 + tile) * kTileKeys + u * 32 + lane;
        const bool in = key >= s.first && key < s.len;
        const float* x = a.stash + (((long long)b * Hkv + g) * a.stash_keys + key) * G + h0;
        if (G % 4 == 0) {
          for (int h = 0; h < nh; h += 4) {
            const float l0 = __shfl_sync(0xffffffffu, lse2, h), l1 = __shfl_sync(0xffffffffu, lse2, h + 1);
            const float l2 = __shfl_sync(0xffffffffu, lse2, h + 2), l3 = __shfl_sync(0xffffffffu, lse2, h + 3);
            if (in) {
              const float4 y = *reinterpret_cast<const float4*>(x + h);
              w[u] += (ex2(y.x - l0) + ex2(y.y - l1)) + (ex2(y.z - l2) + ex2(y.w - l3));
            }
          }
        } else {
          for (int h = 0; h < nh; ++h) {
            const float l = __shfl_sync(0xffffffffu, lse2, h);
            if (in) w[u] += ex2(x[h] - l);
          }
        }
      }
    }
    fresh = false;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (page[u] >= 0 && page[u] < a.kv.num_pages)
        atomicAdd(&a.scores[((long long)page[u] * Hkv + g) * a.kv.page_size + slot[u]], w[u]);
    if (++tile == s.n && t + 1 < end) {
      tile = 0;
      fresh = true;
      if (++g == Hkv) {
        g = 0;
        do s = span_of(a, ++b); while (s.n == 0 && b + 1 < a.B);
        before = a.prefix[b];
      }
    }
  }
}

template <typename T, int D, bool kScores>
__global__ void __launch_bounds__(128) fa_paged_finish_kernel(const DecodeArgs a, int parts) {
  wait_for_previous();
  if (!kScores || blockIdx.x < a.B * a.Hq) join_row<T, D>(a, parts);
  else add_weights(a, parts);
}

// A launch whose blocks may start before the kernel in front of it is done
// (they wait for it themselves).
template <typename... P, typename... A>
cudaError_t launch_after(void (*k)(P...), dim3 grid, dim3 block, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

template <typename T, int D>
cudaError_t launch_decode(const TmaMap4& tk, const TmaMap4& tv, const DecodeArgs& a, const DevStatus& st, int parts,
                          int num_sms, cudaStream_t stream) {
  if (a.unit_heads == 8) fa_paged_decode_kernel<T, D, 1><<<parts, kThreads, Cfg<D>::kBytes, stream>>>(tk, tv, a, st);
  else fa_paged_decode_kernel<T, D, 2><<<parts, kThreads, Cfg<D>::kBytes, stream>>>(tk, tv, a, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.B * a.Hq;
  if (!a.scores) return launch_after(fa_paged_finish_kernel<T, D, false>, (unsigned)rows, 128, stream, a, parts);
  // For the weights 16 tiles a block, up to 4 blocks an SM.
  const long long tiles = (a.stash_keys + kTileKeys - 1) / kTileKeys * a.B * a.kv.Hkv;
  const long long blocks = (tiles + 15) / 16 < 4LL * num_sms ? (tiles + 15) / 16 : 4LL * num_sms;
  return launch_after(fa_paged_finish_kernel<T, D, true>, (unsigned)(rows + blocks), 128, stream, a, parts);
}

template <typename T, int D>
cudaError_t configure_decode() {
  static_assert(Cfg<D>::kBytes <= 115712, "two CTAs per SM");
  cudaError_t e = cudaFuncSetAttribute(fa_paged_decode_kernel<T, D, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D>::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fa_paged_decode_kernel<T, D, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kBytes);
  return e;
}

}  // namespace

cudaError_t configure_paged_kernels() {
  cudaError_t e = configure_decode<__nv_bfloat16, 64>();
  if (e == cudaSuccess) e = configure_decode<__nv_bfloat16, 128>();
  if (e == cudaSuccess) e = configure_decode<__half, 64>();
  if (e == cudaSuccess) e = configure_decode<__half, 128>();
  return e;
}

cudaError_t launch_paged_decode(int dtype, const TmaMap4& tk, const TmaMap4& tv, const DecodeArgs& a, const DevStatus& st,
                                int parts, int num_sms, cudaStream_t stream) {
  if (dtype == 0)
    return a.kv.d == 64 ? launch_decode<__nv_bfloat16, 64>(tk, tv, a, st, parts, num_sms, stream)
                        : launch_decode<__nv_bfloat16, 128>(tk, tv, a, st, parts, num_sms, stream);
  return a.kv.d == 64 ? launch_decode<__half, 64>(tk, tv, a, st, parts, num_sms, stream)
                      : launch_decode<__half, 128>(tk, tv, a, st, parts, num_sms, stream);
}

}  // namespace fa
