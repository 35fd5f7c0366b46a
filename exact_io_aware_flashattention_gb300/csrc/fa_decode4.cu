// Attention of one new token per sequence over the paged cache held in 4 bits:
//   o_h = sum_j p_h(j) v_j,  p_h(j) = exp(scale q_h . k_j - lse_h),
// where k_j and v_j are the values z + s c that the cached codes stand for.
//
// Every code enters the matrix products as it is, s and z are applied in fp32
// outside: with Q_g the sum of q over group g,
//   q . k_j = sum over g of s_jg sum_i q_i c_ji + z_jg Q_g,
//   o = sum_j (s_j p_j) (c_j - 7.5) + sum_j p_j (z_j + 7.5 s_j),
// the last sum one number a head and group.  Four bits in the upper or the next
// mantissa bits of an fp16 number with exponent 0 are the subnormal c 2^-18 or c
// 2^-22: one AND for a pair of codes (and two bytes swapped give the other half of
// a word).  -7.5 times the sum of the weights, the same for all elements of a
// group, is formed by one product more and is what the others start from.  The
// tensor pipe cuts its sums instead of rounding them, which adds up over many
// keys; so products with V are summed over a tile's two slices only, and those
// sums added in fp32 (as running sums of the pipe, and of c, o was 1.2 times as far
// off at 32768 keys).
//   q, whatever its type, enters in fp16 times a power of two that brings its
// head's largest element to 2^10 (16 times that for the codes held as c 2^-22): exact
// but for elements 2^-24 times smaller than that one.  The weights s p enter times a
// power of two that brings the largest s so far to 2^6 (p is 2^8 at most), as the sum
// of two fp16 values, off by 2^-22 of themselves or 2^-31 of that s.  (The high parts
// alone, off by 2^-11, would show in o where values of opposite signs cancel.)  Up to
// four heads a group (kDup) the eight columns hold the heads twice, and the second four
// the weights' low parts, which costs no product; above that there are two products.
//
// The line of tiles, its cut into equal parts, one a CTA, and their joins are those of
// the 16-bit kernel (fa_decode.cuh, fa_paged.cu).  A unit's end counts as two tiles
// there (kEnd: 64 sequences of 0 .. 8192 keys, d = 64, 96 us with none, 84, 76 and 77 us
// with one, two and three).  A warp's slice of a tile is one record of 16 keys, and each
// of a CTA's eight warps works on two neighbouring records of a tile, fetched by untiled
// copies (one, where they lie in a page) into a ring of its own: it waits for no other
// warp before the unit's end.  (Seven warps and a producer that fetched for all left two
// of an SM's four schedulers with fewer warps: pages of 16, 126 us against 116, d = 64 142
// against 128.)  One warp also brings the next unit's query rows.  At a unit's end each
// warp leaves its sums in the place of its last tile, and fills that again once all have
// read them, while its other tiles are on their way.
//   Products by mma.sync (m16n8k16) with keys, then elements of d as rows and 8 heads as
// columns: see fa_paged.cu.  Row i of a slice's S^T is the key (i % 8) / 2 + 4 (i % 2) +
// 8 (i / 8), the pairs of keys that a word of V holds (fa_paged4.h); O^T's rows are the
// elements 8 r + t and 8 r + 4 + t of a group (lane row r, tile t).
//   A running maximum that is behind by less than 2^8 is as good as the exact
// one (weights up to 2^8, sums in fp32): the warp then neither exchanges maxima
// nor rescales.
//
// Bound by what is done to a slice: 333 instructions at d = 128, 64 of them masks, 16 byte
// swaps and 18 products.  Four warps a scheduler issue in 65 % of the cycles, the rest is
// waiting for results; the integer pipe is busy 52 %, the tensor pipe 27 %.  16 sequences
// of 32768 keys, 8 kv heads of 4 heads (604 MB): 119 us, 5.1 TB/s; the copies alone take 98
// us.  Eight heads a group, whose low parts are products of their own, take 140 us.  16
// heads a group (two column tiles, one CTA an SM with 255 registers a thread) take 224 us;
// as two units of eight heads they would take twice 140.  At 128 registers the shapes of
// equal parts, one column tile and d = 128 spill 56-80 bytes, outside the loop over tiles
// (one local load for 3800 instructions).
#include "fa_decode.cuh"
#include "fa_paged4.h"
#include "fa_rotary.cuh"
#include "sm103a.cuh"

#include <cuda_fp16.h>

namespace fa {

namespace {

enum : int { kSiteFull = 54, kSiteRead = 55, kDrainFull = 56 };

// A CTA's shape: kWarps warps, kSl slices of a tile each, and each a ring of its own
// for the records on their way.
template <int D, int NT, int W, int kSl, bool kCluster>
struct Cfg {
  static constexpr int kWarps = W, kKeys = 16 * kSl * W, kThreads = 32 * W;
  static constexpr uint32_t kSlice = Record<D>::kBytes, kStage = kSl * kSlice;
  static constexpr int kStages = (NT == 1 ? 6 : 10) * 128 / D / kSl;
  static constexpr uint32_t kRing = kStages * kStage;          // 13.5 or 22.5 KB a warp
  // At a unit's end a warp's O [8 heads][D] and (max, sum) [8 NT] take the place of the
  // last tile (in a cluster, of the ring's first records).
  static constexpr uint32_t kMl = 8u * D * 4u, kStash = kMl + NT * 64u;
  static_assert(kStash <= (kCluster ? kRing : kStage) && kStash % 8 == 0, "stash");
  static constexpr uint32_t kJoin = kStash;                    // the cluster's join, in warp 0's ring
  static_assert(kJoin + 16u * D * 4u + 128u <= kRing && kJoin % 16 == 0, "join");
  // Two of (in a cluster one): a unit's query rows, first as they are and then as operands; their sums
  // over the groups, [NT][D / 64][8 heads], and factors, [NT][8].
  static constexpr uint32_t kQ = W * kRing, kQBytes = NT * D * 16u;
  static constexpr uint32_t kQs = kQ + (kCluster ? 1 : 2) * kQBytes, kQsBytes = NT * (D / 64 + 1) * 32u;
  static constexpr uint32_t kBars = kQs + (kCluster ? 1 : 2) * kQsBytes;
};

// Tiles that a unit's end counts as in the line that is cut into equal parts.
constexpr int kEnd = 2;
__device__ __forceinline__ int cost_of(const Span& s) { return s.n > 0 ? s.n + kEnd : 0; }
// On behind the tiles up to `tile` of a unit, and its end.
template <int kKeys>
__device__ __forceinline__ void advance(Walk<kKeys>& x, int tiles, const DecodeArgs& a, int cols) {
  x.left -= tiles;
  x.tile += tiles;
  if (x.tile < x.s.n) return;
  x.left -= x.s.n + kEnd - x.tile;
  if (x.left > 0) x.next_unit(a, cols);
}

template <typename C>
struct Bars {
  uint64_t full[C::kWarps][C::kStages];
  uint64_t read;                       // a unit's stashes: every warp has read them
  Walk<C::kKeys> ahead[C::kWarps];     // of what each warp looks up next
  Walk<C::kKeys> next[2];              // the unit after this one
  int abort;
  int scan[C::kWarps];
  int b0;                    // first sequence of this CTA's part
  long long before;          // tiles (per unit column) of the sequences before it
};
template <typename C>
constexpr uint32_t kSmem = C::kBars + sizeof(Bars<C>);

using Half = Pair2<__half>;

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same starting from c0 in the columns' first, c1 in their second.
__device__ __forceinline__ void mma_from(float (&c)[4], float c0, float c1, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %10, %11};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
// Codes of two halves as c 2^-18 (of places 0 and 2) and c 2^-22 (1 and 3); places 2
// and 3 after the halves' bytes are swapped.
__device__ __forceinline__ uint32_t upper(uint32_t w) { return w & 0x03c003c0u; }
__device__ __forceinline__ uint32_t lower(uint32_t w) { return w & 0x003c003cu; }
__device__ __forceinline__ uint32_t swapped(uint32_t w) { return __byte_perm(w, w, 0x2301); }

template <typename T_, int D_, int kKeys_, int kThreads>
struct Traits {
  using T = T_;
  static constexpr int D = D_, kKeys = kKeys_, kJoinThreads = kThreads;
  static constexpr float kShift = 0.f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return Pair2<T>::down(lo, hi); }
};

// The largest power of two up to a positive normal x.
__device__ __forceinline__ float power_of(float x) { return __uint_as_float(__float_as_uint(x) & 0x7f800000u); }

// The (s, z) pairs of one row, D / 64 of them.
template <typename T, int D>
__device__ __forceinline__ void load_pars(const uint8_t* p, float2 (&x)[D / 64]) {
  if constexpr (D == 128) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    x[0] = Pair2<T>::up(w.x);
    x[1] = Pair2<T>::up(w.y);
  } else {
    x[0] = Pair2<T>::up(*reinterpret_cast<const uint32_t*>(p));
  }
}

template <typename T>
__device__ __forceinline__ float2 load_par(const uint8_t* p) {
  return Pair2<T>::up(*reinterpret_cast<const uint32_t*>(p));
}

// The query rows of unit (b, col) on their way to raw [8 NT heads][D]; a warp's work.
template <typename T, int D, int NT, bool kDup>
__device__ __forceinline__ void fetch_q(const DecodeArgs& a, int b, int col, int chunks, uint8_t* raw) {
  const int G = a.Hq / a.kv.Hkv, g = col / chunks, h0 = g * G + (col - g * chunks) * 8 * NT, h1 = (g + 1) * G;
#pragma unroll
  for (int i = threadIdx.x & 31; i < (kDup ? 4 : 8 * NT) * (D / 8); i += 32) {
    const int h = h0 + i / (D / 8);
    if (h < h1) copy16(raw + i * 16, static_cast<const T*>(a.q) + b * a.q_sb + h * a.q_sh + i % (D / 8) * 8);
  }
  copies_end();
}
// A lane's share of them: of head lane / 4 (of each eight), and of each group, the 16
// elements 16 (lane % 4) on; `heads` is the unit's number of heads.
template <int D, int NT>
struct QRows {
  uint4 x[NT][D / 64][2];
};
template <int D, int NT, bool kDup>
__device__ __forceinline__ void wait_q(const uint8_t* raw, int heads, QRows<D, NT>& q) {
  copies_wait<0>();
  __syncwarp();
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int h = n * 8 + (lane >> 2 & (kDup ? 3 : 7));
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
#pragma unroll
      for (int w = 0; w < 2; ++w)
        q.x[n][k][w] = h < heads ? *reinterpret_cast<const uint4*>(raw + h * D * 2 + k * 128 + (lane & 3) * 32 + w * 16)
                                 : make_uint4(0, 0, 0, 0);
  }
}
// The same as B operands, column = head lane / 4: at to[n][g][w][h][lane] the four
// elements 64 g + 16 (lane % 4) + 8 w + 4 h on, times the head's power of two and, the
// odd pairs, 16; sums[n][g][head] over the groups, and factors [n][head] behind them,
// both in the units of the scores (see work).
template <typename T, int D, int NT>
__device__ __forceinline__ void store_q(const QRows<D, NT>& q, float scale_log2, uint2* to, float* sums) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float top = 0x1p-100f, s[D / 64];             // the largest finite |q|
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      s[k] = 0.f;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t e[4] = {q.x[n][k][w].x, q.x[n][k][w].y, q.x[n][k][w].z, q.x[n][k][w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = Pair2<T>::up(e[i]);
          s[k] += y.x + y.y;
          top = fmaxf(top, fabsf(y.x) < INFINITY ? fabsf(y.x) : 0.f);
          top = fmaxf(top, fabsf(y.y) < INFINITY ? fabsf(y.y) : 0.f);
        }
      }
      s[k] += __shfl_xor_sync(0xffffffffu, s[k], 1);
      s[k] += __shfl_xor_sync(0xffffffffu, s[k], 2);
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float times = 1024.f / power_of(top), more = 16.f * times;
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      if ((lane & 3) == 0) sums[(n * (D / 64) + k) * 8 + (lane >> 2)] = s[k] * (times * 0x1p-18f);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint4 v = q.x[n][k][w];
        const float2 y0 = Pair2<T>::up(v.x), y1 = Pair2<T>::up(v.y), y2 = Pair2<T>::up(v.z), y3 = Pair2<T>::up(v.w);
        uint2* x = to + ((n * (D / 64) + k) * 2 + w) * 64 + lane;
        x[0] = make_uint2(Half::down(y0.x * times, y0.y * times), Half::down(y1.x * more, y1.y * more));
        x[32] = make_uint2(Half::down(y2.x * times, y2.y * times), Half::down(y3.x * more, y3.y * more));
      }
    }
    // (Not 0, which times a masked score's -inf is NaN; scores of so small factors are 0 all the same.)
    if ((lane & 3) == 0) sums[NT * (D / 64) * 8 + n * 8 + (lane >> 2)] = fmaxf(scale_log2 * 0x1p18f / times, 0x1p-126f);
  }
}

constexpr float kNone = -1e30f;      // below every score: the maximum before the first key

// mbar_wait_warp with the phase usually complete: one poll and one vote.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const DevStatus& st, volatile int* abort, int site) {
  if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity))) return true;
  return mbar_wait_warp(bar, parity, st, abort, site);
}

// A warp's work on its kSl slices of a tile, rec the first one's record, of the 16 keys
// from key0 on: S^T, its weights against the running
// maximum m and, in l, zs and o, their sums.
template <typename T, int D, int NT, bool kDup, int kSl>
__device__ __forceinline__ void work(uint8_t* rec, int key0, const Span& s, uint32_t k_at, uint32_t v_at, uint32_t kp_at,
                                     uint32_t vp_at, int ka, const float (&by)[NT][2], const uint2* q,
                                     const float (&qs)[NT][D / 64][2], float (&o)[NT][D / 16][4], float (&zs)[NT][D / 64][2],
                                     float (&m)[NT][2], float (&l)[NT][2], float (&grow)[D / 64]) {
  constexpr int kG = D / 64, kW = kDup ? 1 : 2, kStep = Record<D>::kBytes;
  // Scores, in units of log2 / by: S^T rows ka, ka + 8, columns 2 qc, 2 qc + 1.
  float x[kSl][NT][4];
  {
    uint32_t wa[kSl][kG][2], wb[kSl][kG][2];
    float c[kSl][NT][kG][4];
#pragma unroll
    for (int j = 0; j < kSl; ++j) {
      const uint8_t* r = rec + j * kStep;
      if constexpr (D == 128) {
        const uint4 ya = *reinterpret_cast<const uint4*>(r + k_at);
        const uint4 yb = *reinterpret_cast<const uint4*>(r + k_at + 8 * Record<D>::kRow);
        wa[j][0][0] = ya.x, wa[j][1][0] = ya.y, wa[j][0][1] = ya.z, wa[j][1][1] = ya.w;
        wb[j][0][0] = yb.x, wb[j][1][0] = yb.y, wb[j][0][1] = yb.z, wb[j][1][1] = yb.w;
      } else {
        const uint2 ya = *reinterpret_cast<const uint2*>(r + k_at);
        const uint2 yb = *reinterpret_cast<const uint2*>(r + k_at + 8 * Record<D>::kRow);
        wa[j][0][0] = ya.x, wa[j][0][1] = ya.y, wb[j][0][0] = yb.x, wb[j][0][1] = yb.y;
      }
    }
    // Products that follow one another are of different sums, since a product has
    // to wait for the last one of its own.
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < kG; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint2 b = q[(((n * kG + k) * 2 + u) * 2 + h) * 32];
#pragma unroll
            for (int j = 0; j < kSl; ++j) {
              const uint32_t y = h ? swapped(wa[j][k][u]) : wa[j][k][u], z = h ? swapped(wb[j][k][u]) : wb[j][k][u];
              if (u + h == 0) mma_from(c[j][n][k], 0.f, 0.f, upper(y), upper(z), lower(y), lower(z), b.x, b.y);
              else mma(c[j][n][k], upper(y), upper(z), lower(y), lower(z), b.x, b.y);
            }
          }
#pragma unroll
    for (int j = 0; j < kSl; ++j) {
      float2 pa[kG], pb[kG];
      load_pars<T, D>(rec + j * kStep + kp_at, pa);
      load_pars<T, D>(rec + j * kStep + kp_at + 8 * Record<D>::kPar, pb);
#pragma unroll
      for (int k = 0; k < kG; ++k)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2& y = e < 2 ? pa[k] : pb[k];
            x[j][n][e] = fmaf(c[j][n][k][e], y.x, k == 0 ? qs[n][k][e & 1] * y.y : fmaf(qs[n][k][e & 1], y.y, x[j][n][e]));
          }
    }
  }
  if (key0 < s.first || key0 + kSl * 16 > s.len) {
    // Keys that are not visible: their (s, z) of V, perhaps never loaded, may be
    // anything, and become 0.
#pragma unroll
    for (int j = 0; j < kSl; ++j) {
      const int key = key0 + 16 * j + ka;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (key + 8 * h < s.first || key + 8 * h >= s.len) {
#pragma unroll
          for (int n = 0; n < NT; ++n) x[j][n][2 * h] = x[j][n][2 * h + 1] = -INFINITY;
          uint32_t* par = reinterpret_cast<uint32_t*>(rec + j * kStep + vp_at + 8 * h * Record<D>::kPar);
#pragma unroll
          for (int k = 0; k < kG; ++k) par[k] = 0u;
        }
    }
    __syncwarp();
    fence_proxy_async_smem();          // before the slots' next copy
  }
  float top[NT][2], most[kG];
  bool more = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[n][e] = fmaxf(x[0][n][e], x[0][n][2 + e]);
#pragma unroll
      for (int j = 1; j < kSl; ++j) top[n][e] = fmax3(top[n][e], x[j][n][e], x[j][n][2 + e]);
      more |= fmaf(top[n][e], by[n][e], -8.f) > m[n][e];
    }
#pragma unroll
  for (int k = 0; k < kG; ++k) most[k] = 0.f;
#pragma unroll
  for (int j = 0; j < kSl; ++j) {
    float2 y[kG], z[kG];
    load_pars<T, D>(rec + j * kStep + vp_at, y);
    load_pars<T, D>(rec + j * kStep + vp_at + 8 * Record<D>::kPar, z);
#pragma unroll
    for (int k = 0; k < kG; ++k) most[k] = fmax3(most[k], y[k].x, z[k].x);
  }
#pragma unroll
  for (int k = 0; k < kG; ++k) more |= most[k] * grow[k] >= 128.f;
  if (__any_sync(0xffffffffu, more)) {
    // Maxima to the exact ones, and what was summed so far to them.
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top[n][e] = fmaxf(top[n][e], __shfl_xor_sync(0xffffffffu, top[n][e], d));
        const float to = fmaxf(m[n][e], top[n][e] * by[n][e]);
        f[e] = ex2(m[n][e] - to);
        m[n][e] = to;
        l[n][e] *= f[e];
#pragma unroll
        for (int k = 0; k < kG; ++k) zs[n][k][e] *= f[e];
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        o[n][k][0] *= f[0];
        o[n][k][1] *= f[1];
        o[n][k][2] *= f[0];
        o[n][k][3] *= f[1];
      }
    }
#pragma unroll
    for (int k = 0; k < kG; ++k) {
      // (An infinite s, of a group that reads as NaN, does not count.)
      float y = 0.f;
#pragma unroll
      for (int j = 0; j < kSl; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float z = load_par<T>(rec + j * kStep + vp_at + 8 * h * Record<D>::kPar + k * 4).x;
          y = fmaxf(y, z < INFINITY ? z : 0.f);
        }
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
      if (y * grow[k] >= 128.f) {
        const float to = 64.f / power_of(y), f = to / grow[k];
        grow[k] = to;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][k * 4 + i][e] *= f;
      }
    }
  }
  // Weights.
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < kSl; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[j][n][e] = ex2(fmaf(x[j][n][e], by[n][e & 1], -m[n][e & 1]));
      l[n][0] += x[j][n][0] + x[j][n][2];
      l[n][1] += x[j][n][1] + x[j][n][3];
    }
  // Values, group by group.
#pragma unroll
  for (int k = 0; k < kG; ++k) {
    uint32_t p[kSl][NT][kW][2];          // P^T: [high, low (kDup: in other columns)][keys 0-7, 8-15 of the fragment]
    uint32_t v[kSl][4];
#pragma unroll
    for (int j = 0; j < kSl; ++j) {
      const float2 pa = load_par<T>(rec + j * kStep + vp_at + k * 4);
      const float2 pb = load_par<T>(rec + j * kStep + vp_at + 8 * Record<D>::kPar + k * 4);
      const float sa = pa.x * grow[k], sb = pb.x * grow[k], za = fmaf(pa.x, 7.5f, pa.y), zb = fmaf(pb.x, 7.5f, pb.y);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        zs[n][k][0] = fmaf(x[j][n][0], za, fmaf(x[j][n][2], zb, zs[n][k][0]));
        zs[n][k][1] = fmaf(x[j][n][1], za, fmaf(x[j][n][3], zb, zs[n][k][1]));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float w0 = x[j][n][2 * e] * (e ? sb : sa), w1 = x[j][n][2 * e + 1] * (e ? sb : sa);
          const uint32_t high = Half::down(w0, w1);
          const float2 h = Half::up(high);
          const uint32_t low = Half::down(w0 - h.x, w1 - h.y);
          p[j][n][0][e] = transpose8(kDup && (threadIdx.x & 2) ? low : high);
          if constexpr (!kDup) p[j][n][1][e] = transpose8(low);
        }
      }
      const uint4 y = *reinterpret_cast<const uint4*>(rec + j * kStep + v_at + k * 512);
      v[j][0] = y.x, v[j][1] = y.y, v[j][2] = y.z, v[j][3] = y.w;
    }
    // What the codes are counted from: -7.5 times the sums of the weights.
    float minus[NT][2];                  // for codes c 2^-18; columns 2 qc, 2 qc + 1, all rows alike
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      constexpr uint32_t kMinus = 0x81e081e0u;                           // -7.5 2^-18
      float y[4];
#pragma unroll
      for (int j = 0; j < kSl; ++j)
#pragma unroll
        for (int h = 0; h < kW; ++h) {
          if (j + h == 0) mma_from(y, 0.f, 0.f, kMinus, kMinus, kMinus, kMinus, p[j][n][h][0], p[j][n][h][1]);
          else mma(y, kMinus, kMinus, kMinus, kMinus, p[j][n][h][0], p[j][n][h][1]);
        }
      minus[n][0] = y[0];
      minus[n][1] = y[1];
    }
    // Words: keys c, c + 4 of elements 8 r + t and 8 r + 4 + t, then keys c + 8, c + 12;
    // tiles t = 0 and 1, then with the bytes swapped 2 and 3.
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float c[NT][2][4];
#pragma unroll
      for (int j = 0; j < kSl; ++j) {
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = u ? swapped(v[j][i]) : v[j][i];
#pragma unroll
        for (int h = 0; h < kW; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t (&b)[2] = p[j][n][h];
            if (j + h == 0) {
              mma_from(c[n][0], minus[n][0], minus[n][1], upper(y[0]), upper(y[1]), upper(y[2]), upper(y[3]), b[0], b[1]);
              mma_from(c[n][1], minus[n][0] * 0x1p-4f, minus[n][1] * 0x1p-4f, lower(y[0]), lower(y[1]), lower(y[2]), lower(y[3]),
                       b[0], b[1]);
            } else {
              mma(c[n][0], upper(y[0]), upper(y[1]), upper(y[2]), upper(y[3]), b[0], b[1]);
              mma(c[n][1], lower(y[0]), lower(y[1]), lower(y[2]), lower(y[3]), b[0], b[1]);
            }
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][4 * k + 2 * u + i][e] += c[n][i][e];
    }
  }
}

template <typename T, int D, int NT, bool kDup, int W, int kSl, bool kCluster>
__global__ void __launch_bounds__(32 * W, NT == 1 && W <= 8 ? 2 : 1) fa_decode4_kernel(const DecodeArgs a, const DevStatus st) {
  using C = Cfg<D, NT, W, kSl, kCluster>;
  constexpr int kKeys = C::kKeys, kWarps = W, kThreads = C::kThreads, kG = D / 64;
  using Tr = Traits<T, D, kKeys, kThreads>;
  extern __shared__ __align__(128) uint8_t smem[];
  Bars<C>* bars = reinterpret_cast<Bars<C>*>(smem + C::kBars);
  volatile int* abort_flag = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(&bars->full[warp][s], kSl);
    if (warp == 0) {
      mbar_init(&bars->read, kWarps);
      bars->abort = 0;
    }
    mbar_fence_init();
  }
  wait_for_previous();
  const int G = a.Hq / a.kv.Hkv, chunks = (G + 8 * NT - 1) / (8 * NT), cols = a.kv.Hkv * chunks;
  Walk<kKeys> w;
  int rank = 0;
  if constexpr (kCluster) {
    // The cluster's unit, and this CTA's share of its tiles (perhaps none).
    const int unit = blockIdx.x / a.cluster;
    rank = blockIdx.x - unit * a.cluster;
    w.b = unit / cols;
    w.col = unit - w.b * cols;
    w.s = span_of<kKeys>(a, w.b);
    w.tile = w.s.n * rank / a.cluster;
    w.left = w.s.n * (rank + 1) / a.cluster - w.tile;
    if (w.s.len < 0 && w.col == 0 && rank == 0 && threadIdx.x == 0) record_error(st, kErrBadIndex, kSiteDecode4Len);
  } else {
    // The line: its length, and this CTA's first sequence.  Round 0 finds the
    // total; round 1, for batches of more than one block's worth, walks again
    // to find the start (one block's worth is still there).
    long long total = 0;
    const int first_len = (int)threadIdx.x < a.B ? a.seq_lens[threadIdx.x] : 0;
    for (int round = 0; round < 2; ++round) {
      long long before = 0, start = 0;
      for (int base = 0; base < a.B; base += kThreads) {
        const int b = base + threadIdx.x;
        Span s{};
        if (b < a.B) {
          s = span_of_len<kKeys>(a, base == 0 ? first_len : a.seq_lens[b]);
          if (s.len < 0 && round == 0 && blockIdx.x == 0) record_error(st, kErrBadIndex, kSiteDecode4Len);
        }
        int x = cost_of(s);
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, d);
          if (lane >= d) x += y;
        }
        __syncthreads();
        if (lane == 31) bars->scan[warp] = x;
        __syncthreads();
        long long pre = before + x - cost_of(s);
        for (int i = 0; i < kWarps; ++i) {
          if (i < warp) pre += bars->scan[i];
          before += bars->scan[i];
        }
        const bool last = base + kThreads >= a.B;
        if (round == 0 && last) total = before * cols;
        const int all = (int)min(total, (long long)gridDim.x);
        if ((last || round == 1) && blockIdx.x < all) start = part_start(total, blockIdx.x, all);
        if ((round == 1 || a.B <= kThreads) && s.n > 0 && pre * cols <= start && start < (pre + cost_of(s)) * cols) {
          bars->b0 = b;
          bars->before = pre * cols;
        }
      }
      if (a.B <= kThreads) break;
    }
    __syncthreads();
    const int parts = (int)min(total, (long long)gridDim.x);
    if ((int)blockIdx.x >= parts) {
      if (threadIdx.x == 0) a.parts[blockIdx.x].left = 0;
      if (warp == 0) fill_empty<Tr>(a);
      return;
    }
    const long long t0 = part_start(total, blockIdx.x, parts);
    w.left = part_start(total, blockIdx.x + 1, parts) - t0;
    w.b = bars->b0;
    w.s = span_of<kKeys>(a, w.b);
    const long long in = t0 - bars->before;
    w.col = (int)(in / cost_of(w.s));
    w.tile = (int)(in - (long long)w.col * cost_of(w.s));
    const int tile = w.tile;
    if (tile >= w.s.n) advance(w, 0, a, cols);     // a unit's end: the part starts with the next unit, if it has one
    if (w.left <= 0) {
      if (threadIdx.x == 0) a.parts[blockIdx.x].left = 0;
      if (warp == 0) fill_empty<Tr>(a);
      return;
    }
    if (threadIdx.x == 0) {
      DecodePart d{};
      d.b = w.b;
      d.col = w.col;
      d.tile = w.tile;
      d.left = (int)w.left;
      d.i0 = part_of(t0 - tile, total, parts);    // (of use where the part does not start with a unit)
      d.i1 = part_of(t0 - tile + w.s.n - 1, total, parts);
      a.parts[blockIdx.x] = d;
    }
  }

  // -------------------------------------------------------------- a warp's copies
  // Lane l holds the place and the bytes of slice l % kSl of tile l / kSl of the next ones
  // in the line (of one unit), `run` of them, `run_at` already on their way; and the page
  // and slot (-1: nothing visible) of the same slice of the run after it.
  uint8_t* ring = smem + warp * C::kRing;
  const uint8_t* from = nullptr;
  uint32_t bytes = 0;
  int run = 0, run_at = 0, flying = 0, page = 0, slot = -1;
  bool dead = false, more = true;                 // more: the run after it is not empty
  auto run_of = [](const Walk<kKeys>& x) { return (int)max(min((long long)min(x.s.n - x.tile, 32 / kSl), x.left), 0ll); };
  auto look_ahead = [&](const Walk<kKeys>& x) {
    const int key0 = (x.s.tile0 + x.tile + lane / kSl) * kKeys + (warp * kSl + lane % kSl) * 16;
    slot = -1;
    if (lane / kSl < run_of(x) && key0 < x.s.len && key0 + 16 > x.s.first) {
      const int c = key0 / a.kv.page_size;
      slot = key0 - c * a.kv.page_size;
      page = a.table.pages[x.b * a.table.stride + c];
    }
    more = x.left > 0;
    if (lane == 0) bars->ahead[warp] = x;
    __syncwarp();
  };
  auto look_up = [&] {
    Walk<kKeys> x = bars->ahead[warp];
    run = run_of(x);
    run_at = 0;
    from = nullptr;
    if (slot >= 0) {
      if (page < 0 || page >= a.kv.num_pages) record_error(st, kErrBadIndex, kSiteDecode4Page);
      else
        from = static_cast<const uint8_t*>(a.kv.k) + (x.col / chunks) * a.kv.s_head + page * a.kv.s_page +
               (long long)(slot >> 4) * C::kSlice;
    }
    bytes = from ? C::kSlice : 0u;
    if constexpr (kSl == 2) {
      // Records of one page follow one another there as here: one copy for both.
      const uint8_t* other = reinterpret_cast<const uint8_t*>(
          __shfl_xor_sync(0xffffffffu, reinterpret_cast<unsigned long long>(from), 1));
      if (from && other && (lane & 1 ? other + C::kSlice == from : from + C::kSlice == other)) bytes = lane & 1 ? 0u : 2 * C::kSlice;
    }
    advance(x, run, a, cols);
    __syncwarp();
    look_ahead(x);
  };
  // The next tile's records to stage s, whose last tile this warp has read.
  auto issue = [&](uint32_t s) {
    if (dead) return;
    if (run_at == run) {
      if (!more) return;
      look_up();
    }
    if (lane / kSl == run_at) {
      uint64_t* bar = &bars->full[warp][s];
      if (bytes) {
        mbar_arrive_expect_tx(bar, bytes);
        bulk_load(smem_u32(ring) + s * C::kStage + lane % kSl * C::kSlice, from, bytes, bar);
      } else {
        mbar_arrive(bar);
      }
    }
    ++run_at;
    ++flying;
  };
  constexpr int kQWarp = W - 1;        // prepares the units' query rows
  auto get_q = [&](const Walk<kKeys>& x, int side) { fetch_q<T, D, NT, kDup>(a, x.b, x.col, chunks, smem + C::kQ + side * C::kQBytes); };
  auto put_q = [&](const Walk<kKeys>& x, int side) {
    QRows<D, NT> rows;
    uint8_t* q = smem + C::kQ + side * C::kQBytes;
    wait_q<D, NT, kDup>(q, min(8 * NT, G - x.col % chunks * 8 * NT), rows);
    __syncwarp();
    store_q<T, D, NT>(rows, a.scale_log2, reinterpret_cast<uint2*>(q), reinterpret_cast<float*>(smem + C::kQs + side * C::kQsBytes));
  };
  look_ahead(w);
  if (warp == kQWarp) get_q(w, 0);
  for (int s = 0; s < C::kStages; ++s) issue(s);
  if (warp == kQWarp) put_q(w, 0);
  __syncthreads();

  // -------------------------------------------------------------- the units
  const int qr = lane >> 2, qc = lane & 3;        // fragment row and column pair
  const int ka = (qr >> 1) + 4 * (qr & 1);        // the keys of rows qr and qr + 8: ka and ka + 8
  const uint32_t k_at = Record<D>::k_word(ka, 2 * qc);
  const uint32_t v_at = Record<D>::kV + lane * 16;
  const uint32_t kp_at = Record<D>::kKp + ka * Record<D>::kPar, vp_at = Record<D>::kVp + ka * Record<D>::kPar;
  float qs[NT][kG][2], o[NT][D / 16][4], zs[NT][kG][2], m[NT][2], l[NT][2];
  float by[NT][2], grow[kG];                      // of S^T; brings the s of V so far to 2^7 at most
  int g = 0, h0 = 0, h1 = 0;                      // kv head, query heads [h0, h1) of the unit
  uint32_t stage = 0, phase = 0;
  int side = 0, owed = -1;              // owed: the stage of the last unit's stash, to be filled
  auto give_up = [&] {
    dead = true;
    // Every copy on its way has to land before the CTA may exit.
    if (lane == 0)
      for (uint32_t x = stage; x < stage + flying; ++x)
        mbar_wait_drain(&bars->full[warp][x % C::kStages], phase ^ (x >= C::kStages), st, kDrainFull);
    __syncwarp();
  };
  do {
    // ------------------------------------------------ one unit's tiles here
    // (A CTA of a cluster may have none, and joins in all the same.)
    const int nt = (int)min((long long)(w.s.n - w.tile), w.left);
    g = w.col / chunks;
    h0 = g * G + (w.col - g * chunks) * 8 * NT;
    h1 = (g + 1) * G;
    if (!kCluster && warp == kQWarp) {
      Walk<kKeys> x = w;
      advance(x, nt, a, cols);
      if (x.left > 0) {
        get_q(x, side ^ 1);
      }
      if (lane == 0) bars->next[side] = x;
    }
    if (!kCluster && owed >= 0) {
      // Once the others have read the last unit's stash here.
      if (!dead && !wait_warp(&bars->read, side ^ 1, st, abort_flag, kSiteRead)) give_up();
      fence_proxy_async_smem();
      issue(owed);
    }
    const uint2* q = reinterpret_cast<const uint2*>(smem + C::kQ + side * C::kQBytes);
    const float* q_sums = reinterpret_cast<const float*>(smem + C::kQs + side * C::kQsBytes);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < kG; ++k) {
        const float2 y = *reinterpret_cast<const float2*>(q_sums + (n * kG + k) * 8 + qc * 2);
        qs[n][k][0] = y.x;
        qs[n][k][1] = y.y;
      }
      const float2 y = *reinterpret_cast<const float2*>(q_sums + NT * kG * 8 + n * 8 + qc * 2);
      by[n][0] = y.x;
      by[n][1] = y.y;
    }
#pragma unroll
    for (int k = 0; k < kG; ++k) grow[k] = 0x1p107f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][k][e] = 0.f;
#pragma unroll
      for (int k = 0; k < kG; ++k) zs[n][k][0] = zs[n][k][1] = 0.f;
      m[n][0] = m[n][1] = kNone;
      l[n][0] = l[n][1] = 0.f;
    }
    uint32_t last = 0;                 // the stage of the unit's last tile
    int key0 = (w.s.tile0 + w.tile) * kKeys + warp * kSl * 16;
    for (int i = 0; i < nt; ++i, key0 += kKeys) {
      // After a wait that gave up the warp goes on through its part without
      // touching the tiles, so that the warps still meet at each unit's end.
      if (!dead && !wait_warp(&bars->full[warp][stage], phase, st, abort_flag, kSiteFull)) give_up();
      --flying;
      // (A slice whose page number is out of range was not loaded: what lies
      // there is worked on, and its sequence's outputs are unspecified.)
      if (!dead && key0 < w.s.len && key0 + kSl * 16 > w.s.first)
        work<T, D, NT, kDup, kSl>(ring + stage * C::kStage, key0, w.s, k_at, v_at, kp_at, vp_at, ka, by, q + lane, qs, o, zs, m, l,
                                  grow);
      __syncwarp();
      last = stage;
      if (kCluster || i + 1 < nt) issue(stage);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    {
      // ------------------------------------------------ the unit's end here
      const bool whole = w.tile == 0 && nt == w.s.n;
      if (!kCluster && warp == kQWarp && bars->next[side].left > 0) put_q(bars->next[side], side ^ 1);
      uint8_t* stash = smem + (kCluster ? 0 : last * C::kStage);                   // warp 0's
      float2* ml = reinterpret_cast<float2*>(stash + warp * C::kRing + C::kMl);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l[n][0] += __shfl_xor_sync(0xffffffffu, l[n][0], d);
          l[n][1] += __shfl_xor_sync(0xffffffffu, l[n][1], d);
#pragma unroll
          for (int k = 0; k < kG; ++k) {
            zs[n][k][0] += __shfl_xor_sync(0xffffffffu, zs[n][k][0], d);
            zs[n][k][1] += __shfl_xor_sync(0xffffffffu, zs[n][k][1], d);
          }
        }
        if (qr == 0) {
          ml[n * 8 + qc * 2] = make_float2(m[n][0], l[n][0]);
          ml[n * 8 + qc * 2 + 1] = make_float2(m[n][1], l[n][1]);
        }
      }
      __syncthreads();
      auto ml_of = [&](int u, int h) { return *reinterpret_cast<const float2*>(stash + u * C::kRing + C::kMl + h * 8); };
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n > 0) __syncthreads();                // the stash's last readers
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M = kNone;
#pragma unroll
          for (int u = 0; u < kWarps; ++u) M = fmaxf(M, ml_of(u, n * 8 + qc * 2 + e).x);
          f[e] = ex2(m[n][e] - M);
        }
        // [head][element], the element xor 4 (head / 2): the rows and column pairs that
        // a quarter of a warp stores at once fall on 32 banks.
        float* to = reinterpret_cast<float*>(stash + warp * C::kRing) + qc * 2 * D;
#pragma unroll
        for (int k = 0; k < kG; ++k) {
          // Codes are c 2^-18 or c 2^-22, weights s p grow; 2^22 / grow may be past fp32's range, s up to 2^124.
          const float back = 1.f / grow[k];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float z = kDup && qc >= 2 ? 0.f : zs[n][k][e & 1], s = f[e & 1];
            *reinterpret_cast<float4*>(to + (e & 1) * D + k * 64 + ((qr * 8 + (e >> 1) * 4) ^ (qc * 4))) =
                make_float4(fmaf(o[n][4 * k][e] * 0x1p18f, back, z) * s, fmaf(o[n][4 * k + 1][e] * 0x1p22f, back, z) * s,
                            fmaf(o[n][4 * k + 2][e] * 0x1p18f, back, z) * s, fmaf(o[n][4 * k + 3][e] * 0x1p22f, back, z) * s);
          }
        }
        __syncthreads();
        const int hh = threadIdx.x / (D / 4), d = threadIdx.x % (D / 4) * 4, h = h0 + n * 8 + hh;
        static_assert(kThreads >= 8 * (D / 4), "a thread for four elements of each head");
        if (hh < (kDup ? 4 : 8) && h < h1) {
          float M = kNone, L = 0.f;
#pragma unroll
          for (int u = 0; u < kWarps; ++u) M = fmaxf(M, ml_of(u, n * 8 + hh).x);
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int u = 0; u < kWarps; ++u) {
            const float2 x = ml_of(u, n * 8 + hh);
            L = fmaf(x.y, ex2(x.x - M), L);
#pragma unroll
            for (int c = 0; c < (kDup ? 8 : 4); c += 4)            // and the low parts' sums
              add_scaled(y, 1.f, *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(stash + u * C::kRing) +
                                                                  (hh + c) * D + (d ^ (hh + c >> 1) * 4)));
          }
          if constexpr (kCluster) {
            *reinterpret_cast<float4*>(smem + C::kJoin + ((n * 8 + hh) * D + d) * 4) = y;
            if (d == 0) reinterpret_cast<float2*>(smem + C::kJoin + kClusterMl<D>)[n * 8 + hh] = make_float2(M, L);
          } else {
            const long long row = (long long)w.b * a.Hq + h;
            if (whole) {
              const float inv = 1.f / L;
              *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + row * D + d) =
                  make_uint2(Tr::pack(y.x * inv, y.y * inv), Tr::pack(y.z * inv, y.w * inv));
              if (d == 0) a.lse[row] = (M + log2f(L)) * 0.69314718055994530942f;
            } else {
              // Slot 1: the unit starts in this CTA and goes on; slot 0: it
              // started earlier.
              const long long at = ((long long)blockIdx.x * 2 + (w.tile == 0 ? 1 : 0)) * 16 + n * 8 + hh;
              *reinterpret_cast<float4*>(a.part + at * D + d) = y;
              if (d == 0) a.part_ml[at] = make_float2(M, L);
            }
          }
        }
      }
    }
    if constexpr (!kCluster) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->read);
      w = bars->next[side];
      owed = last;
      side ^= 1;
    }
  } while (!kCluster && w.left > 0);
  if constexpr (kCluster) {
    if (a.cluster > 1) cluster_sync();
    else __syncthreads();
    join_cluster<Tr>(a, smem + C::kJoin, w, rank, h0, min(h1, h0 + 8 * NT));
    __syncwarp();
    if (a.cluster > 1) cluster_sync();             // nobody exits while its share is read
  } else if (warp == kQWarp) {
    fill_empty<Tr>(a);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(128) fa_decode4_join_kernel(const DecodeArgs a) {
  launch_dependents();
  wait_for_previous();
  join<Traits<T, D, kDecode4TileKeys, 128>>(a);
}

// A kernel and its CTA's shape.
template <typename T, int D, int NT, bool kDup, int W, int kSl, bool kCluster>
struct Shape {
  using C = Cfg<D, NT, W, kSl, kCluster>;
  static constexpr auto kernel = fa_decode4_kernel<T, D, NT, kDup, W, kSl, kCluster>;
  static cudaError_t launch(const DecodeArgs& a, const DevStatus& st, int ctas, cudaStream_t stream) {
    return launch_after(kernel, ctas, C::kThreads, kSmem<C>, kCluster ? a.cluster : 1, stream, a, st);
  }
  static cudaError_t configure() {
    static_assert(kSmem<C> <= (NT == 1 && W <= 8 ? 115712 : 232448), "shared memory");
    static_assert(C::kKeys == (kCluster ? kDecode4ClusterKeys : kDecode4TileKeys), "tile");
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<C>);
  }
};
// For clusters, which share few tiles, one slice of a tile a warp.
template <typename T, int D, int NT, bool kDup>
using Short = Shape<T, D, NT, kDup, 8, 1, true>;
template <typename T, int D, int NT, bool kDup>
using Long = Shape<T, D, NT, kDup, 8, 2, false>;

template <typename T, int D, int NT, bool kDup>
cudaError_t launch_shape(const DecodeArgs& a, const DevStatus& st, int parts, cudaStream_t stream) {
  if (a.cluster) return Short<T, D, NT, kDup>::launch(a, st, parts, stream);
  const cudaError_t e = Long<T, D, NT, kDup>::launch(a, st, parts, stream);
  const int joins = (parts - 1) * (a.unit_heads / 4);
  if (e != cudaSuccess || joins == 0) return e;
  return launch_after(fa_decode4_join_kernel<T, D>, joins, 128, 0, 1, stream, a);
}
template <typename T, int D>
cudaError_t launch(const DecodeArgs& a, const DevStatus& st, int parts, cudaStream_t stream) {
  if (a.unit_heads == 16) return launch_shape<T, D, 2, false>(a, st, parts, stream);
  if (a.Hq / a.kv.Hkv <= 4) return launch_shape<T, D, 1, true>(a, st, parts, stream);
  return launch_shape<T, D, 1, false>(a, st, parts, stream);
}

template <typename T, int D, int NT, bool kDup>
cudaError_t configure_shape() {
  const cudaError_t e = Short<T, D, NT, kDup>::configure();
  return e == cudaSuccess ? Long<T, D, NT, kDup>::configure() : e;
}
template <typename T, int D>
cudaError_t configure() {
  cudaError_t e = configure_shape<T, D, 1, false>();
  if (e == cudaSuccess) e = configure_shape<T, D, 1, true>();
  if (e == cudaSuccess) e = configure_shape<T, D, 2, false>();
  if (e == cudaSuccess) e = preload_kernel(fa_decode4_join_kernel<T, D>);
  return e;
}

}  // namespace

cudaError_t configure_decode4_kernels() {
  cudaError_t e = configure<__nv_bfloat16, 64>();
  if (e == cudaSuccess) e = configure<__nv_bfloat16, 128>();
  if (e == cudaSuccess) e = configure<__half, 64>();
  if (e == cudaSuccess) e = configure<__half, 128>();
  return e;
}

cudaError_t launch_decode4(int dtype, const DecodeArgs& a, const DevStatus& st, int parts, cudaStream_t stream) {
  if (dtype == 0)
    return a.kv.d == 64 ? launch<__nv_bfloat16, 64>(a, st, parts, stream) : launch<__nv_bfloat16, 128>(a, st, parts, stream);
  return a.kv.d == 64 ? launch<__half, 64>(a, st, parts, stream) : launch<__half, 128>(a, st, parts, stream);
}

}  // namespace fa
