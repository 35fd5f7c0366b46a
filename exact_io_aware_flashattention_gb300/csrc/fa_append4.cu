// New tokens stored in the 4-bit cache, and its rows read back.
//
// A row of 16-bit values (normed and turned first, if the call says so, and
// rounded to its type T as a 16-bit cache would hold it) is stored in groups of
// 64 elements: z = the smallest, s = T((largest - z) / 15), codes c = (x - z) / s
// rounded to nearest (ties to even), 0 where s is 0; it stands for z + s c.  A
// group with a value that is not finite gets a NaN s, so it reads as NaN.
// Every step is one IEEE operation, so that the same 16-bit row gives the same
// codes everywhere.
//
// Bound by HBM: 16-bit rows in, 0.5625 bytes an element out (in and out exchanged when
// reading back).  The append issues in 62 % of the cycles, on finding the groups' ends,
// quotients that round as a division does and the angles: 7357 tokens of 32 + 8 + 8
// heads, d = 128, bf16, 159 MB: 36.9 us, 4.3 TB/s.  Reading 32768 keys of 8 heads, 172 MB: 29 us,
// 5.9 TB/s (a warp a record with all its loads first; element by element 44).
#include "fa_paged4.h"
#include "fa_rotary.cuh"
#include "sm103a.cuh"

#include <algorithm>

namespace fa {

namespace {

constexpr int kThreads = 128;

// The smaller of each half, NaN if either is.
template <typename T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (sizeof(T) == 2 && Pair2<T>::kBf16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// (smallest, -largest) of a vector, as a pair whose halves grow smaller alike.
template <typename T>
__device__ __forceinline__ uint32_t ends_of(const uint4& v) {
  constexpr uint32_t kSign = 0x80008000u;
  const uint32_t lo = min2<T>(min2<T>(v.x, v.y), min2<T>(v.z, v.w));
  const uint32_t hi = min2<T>(min2<T>(v.x ^ kSign, v.y ^ kSign), min2<T>(v.z ^ kSign, v.w ^ kSign));
  return min2<T>(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
}

template <typename T>
__device__ __forceinline__ float round_to(float x) {
  return Pair2<T>::up(Pair2<T>::down(x, 0.f)).x;
}

// x / y for a correctly rounded reciprocal inv of y, as an IEEE division rounds it:
// with a quotient within a unit of the last place and its exact residual, one more
// step gives the correctly rounded quotient (Markstein's theorem).
__device__ __forceinline__ float quotient(float x, float y, float inv) {
  const float q = __fmul_rn(x, inv);
  return __fmaf_rn(__fmaf_rn(-q, y, x), inv, q);
}
// A group's s and z, from (smallest, -largest).
struct Step {
  float s, z, inv;
  bool plain;        // the residuals above are exact: s is not extremely small or large
};
template <typename T>
__device__ __forceinline__ Step step_of(uint32_t ends) {
  const float2 e = Pair2<T>::up(ends);
  const float range = __fsub_rn(-e.y, e.x);
  Step g;
  g.plain = range > 0x1p-90f && range < 0x1p90f;
  g.s = round_to<T>(g.plain ? quotient(range, 15.f, 1.f / 15.f) : __fdiv_rn(range, 15.f));
  if (!(range < INFINITY)) g.s = __int_as_float(0x7fffffff);
  g.z = e.x;
  g.inv = __frcp_rn(g.s);
  // (An s of fp16's subnormal steps may be so far from range / 15 that a quotient
  // passes 15.5; so it is not plain either.)
  g.plain = g.plain && g.s >= (Pair2<T>::kBf16 ? 0x1p-90f : 0x1p-14f);
  return g;
}
// Four codes, quotients of 0 .. 15.1, in a half: the nearest whole numbers (ties to
// even) in the last bits of their sums with 1.5 2^23, their places by products; what
// passes bit 15 of place 2 goes to bits 0 and 1.
__device__ __forceinline__ uint32_t half_of(float c0, float c1, float c2, float c3) {
  constexpr float kRound = 12582912.f;
  constexpr uint32_t kBits = 0x4b400000u;
  const uint32_t w = __float_as_uint(__fadd_rn(c0, kRound)) * 64u + __float_as_uint(__fadd_rn(c1, kRound)) * 4u +
                     __float_as_uint(__fadd_rn(c2, kRound)) * 16384u + __float_as_uint(__fadd_rn(c3, kRound)) * 1024u -
                     kBits * (64u + 4u + 16384u + 1024u);
  return (w & 0xffffu) | (w >> 16);
}
// Eight codes: in the two halves of K's word or in V's two halves.
template <typename T, bool kKeys>
__device__ __forceinline__ void encode8(const uint4& v, const Step& g, uint8_t* to) {
  float x[8];
  up8<T>(v, x);
  if (g.plain) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {               // as quotient, two at a time
      const float2 y = add2(make_float2(x[e], x[e + 1]), two(-g.z)), q = mul2(y, two(g.inv));
      const float2 c = fma2(fma2(q, two(-g.s), y), two(g.inv), q);
      x[e] = c.x;
      x[e + 1] = c.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = g.s > 0.f ? fminf(__fdiv_rn(__fsub_rn(x[e], g.z), g.s), 15.f) : 0.f;
  }
  if constexpr (kKeys) {
    *reinterpret_cast<uint32_t*>(to) = half_of(x[0], x[2], x[4], x[6]) | half_of(x[1], x[3], x[5], x[7]) << 16;
  } else {
    *reinterpret_cast<uint16_t*>(to) = (uint16_t)half_of(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<uint16_t*>(to + 4) = (uint16_t)half_of(x[4], x[5], x[6], x[7]);
  }
}

// A difference in a 16-bit value's last place may move a code by a whole step, so a
// program that forms its rows elsewhere (the prompts of a cache filled before, a check
// against elementary operations) and this kernel should agree to that place.  K's rows
// are therefore formed by fp32 operations that are rounded one by one, in an order that
// is the same for every layout of the pairs: the squares of the elements that are 32
// columns apart summed first, then neighbours; the turn without fused products, by
// angles within 2^-29.5.  (7.5 million values of K of 7357 prompt tokens against such a
// program: as in the norm's kernel 2.5 codes a call differed, so none in twelve calls;
// 40.5 -> 42.3 us.)
// Of a row whose lane c has the elements 8 c .. 8 c + 7 and D / 2 more:
template <int D>
__device__ __forceinline__ float plain_sum_of_squares(const float (&a)[8], const float (&b)[8], int c) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = __fmul_rn(a[i], a[i]), q = __fmul_rn(b[i], b[i]);
    if constexpr (D == 128) {
      // (b's are 64 columns further, the lane's four off 32.)
      const float po = __shfl_xor_sync(0xffffffffu, p, 4), qo = __shfl_xor_sync(0xffffffffu, q, 4);
      s[i] = __fadd_rn(__fadd_rn(__fadd_rn(c < 4 ? p : po, c < 4 ? po : p), c < 4 ? q : qo), c < 4 ? qo : q);
    } else {
      s[i] = __fadd_rn(p, q);
    }
  }
  const float r = __fadd_rn(__fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3])),
                            __fadd_rn(__fadd_rn(s[4], s[5]), __fadd_rn(s[6], s[7])));
  return sum_over(r, 4);
}
template <bool kInter>
__device__ __forceinline__ void plain_turn8(float (&a)[8], float (&b)[8], const float (&cs)[8], const float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& x = kInter ? (i < 4 ? a[2 * i] : b[2 * i - 8]) : a[i];
    float& y = kInter ? (i < 4 ? a[2 * i + 1] : b[2 * i - 7]) : b[i];
    const float t = __fsub_rn(__fmul_rn(x, cs[i]), __fmul_rn(y, sn[i]));
    y = __fadd_rn(__fmul_rn(y, cs[i]), __fmul_rn(x, sn[i]));
    x = t;
  }
}

// Which lane of a row has vector v of it (8 elements), as its first or second one, where
// the lanes have the chunks of chunk_of.
__device__ __forceinline__ int2 place_of(int v, const RotaryArgs& r) {
  if (r.interleaved || v >= r.rot / 8) return make_int2(v / 2, v % 2);
  return v < r.rot / 16 ? make_int2(v, 0) : make_int2(v - r.rot / 16, 1);
}

// One row of K or V, two vectors a thread, into its record: codes to the addresses of
// the vectors, (s, z) to par.  All lanes of a row take part.  own: a thread's vectors
// are of the group of its four lanes.
template <typename T, int D, bool kKeys>
__device__ __forceinline__ void store_row(const uint4& va, const uint4& vb, const Chunk& ck, bool own, uint8_t* ca, uint8_t* cb,
                                          uint8_t* par, int c, bool live) {
  constexpr uint32_t kNone = Pair2<T>::kBf16 ? 0x7f807f80u : 0x7c007c00u;         // infinities
  const uint32_t pa = ends_of<T>(va), pb = ends_of<T>(vb);
  if (own) {
    uint32_t p = min2<T>(pa, pb);
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) p = min2<T>(p, __shfl_xor_sync(0xffffffffu, p, d));
    if (!live) return;
    const Step g = step_of<T>(p);
    encode8<T, kKeys>(va, g, ca);
    encode8<T, kKeys>(vb, g, cb);
    if ((c & 3) == 0) *reinterpret_cast<uint32_t*>(par + c) = Pair2<T>::down(g.s, g.z);
    return;
  }
  if constexpr (D == 128) {
    const int ga = ck.e0 / 64, gb = ck.e1 / 64;
    uint32_t p[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      p[k] = min2<T>(k == ga ? pa : kNone, k == gb ? pb : kNone);
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) p[k] = min2<T>(p[k], __shfl_xor_sync(0xffffffffu, p[k], d));
    }
    if (!live) return;
    const Step a = step_of<T>(p[ga]), b = step_of<T>(p[gb]);
    encode8<T, kKeys>(va, a, ca);
    encode8<T, kKeys>(vb, b, cb);
    // Some lane has a vector of each group; lane 0's first is of group 0.
    if (c == 0) *reinterpret_cast<uint32_t*>(par) = Pair2<T>::down(a.s, a.z);
    if (c == 7) *reinterpret_cast<uint32_t*>(par + 4) = Pair2<T>::down(b.s, b.z);
  }
}

// grid: x over groups of kThreads / (D/16) tokens, y over groups of hpb heads of v,
// then k, then q: those whose rows take longest start first (7357 tokens 43.1 -> 41.2 us,
// one token each 4.8 -> 4.3).  The first rows are on their way while the slot is looked up and
// the angles are formed.
constexpr int kSlots = 3;
// kHalves: a lane has eight neighbours of each half of a row of q and K, as
// plain_sum_of_squares takes them (rows turned whole by halves, or normed only); an
// instance of its own, as the other layouts' look-ups in its loop cost it 2 us of 42.
template <typename T, int D, bool kInter, bool kHalves>
__global__ void __launch_bounds__(kThreads, 5) fa_append4_kernel(const Append4Args a, int hpb, const DevStatus st) {
  using R = Record<D>;
  __shared__ Pairs pairs;
  __shared__ uint4 ring[kSlots][2][kThreads];
  constexpr int kLanes = D / 16, kTokens = kThreads / kLanes;
  launch_dependents();
  wait_for_previous();
  const int lt = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  const long long t = (long long)blockIdx.x * kTokens + lt;
  // What is not turned: both vectors of one group, and neighbouring lanes' next to one
  // another (with a lane's own two so, 7357 tokens took 1.5 us more).
  const Chunk plain{64 * (c >> 2) + 8 * (c & 3), 64 * (c >> 2) + 8 * (c & 3) + 32, false};
  const Chunk ck = kHalves ? Chunk{8 * c, D / 2 + 8 * c, a.r.rot != 0} : a.r.rot ? chunk_of<kInter>(c, a.r.rot) : plain;
  const int Hkv = a.kv.Hkv, h0 = (gridDim.y - 1 - blockIdx.y) * hpb, h1 = min(h0 + hpb, a.Hq + 2 * Hkv);
  auto copy = [&](int h, int slot) {
    if (t < a.T && h < h1) {
      const bool v = h >= a.Hq + Hkv;
      const T* x = h < a.Hq ? static_cast<const T*>(a.q.p) + t * a.q.sn + h * a.q.sh
                   : !v     ? static_cast<const T*>(a.k.p) + t * a.k.sn + (h - a.Hq) * a.k.sh
                            : static_cast<const T*>(a.v.p) + t * a.v.sn + (h - a.Hq - Hkv) * a.v.sh;
      copy16(&ring[slot][0][threadIdx.x], x + (v ? plain.e0 : ck.e0));
      copy16(&ring[slot][1][threadIdx.x], x + (v ? plain.e1 : ck.e1));
    }
    copies_end();
  };
#pragma unroll
  for (int s = 0; s < kSlots; ++s) copy(h0 + s, s);
  load_pairs<kThreads>(a.r, pairs, st);
  if (a.cu && blockIdx.y == 0) check_offsets<kThreads>(a, st);
  __syncthreads();
  int page = 0, place = 0;
  const bool live = t < a.T && place_token(a, (int)t, st, page, place);
  float cs[8] = {}, sn[8] = {};
  // K's vectors: halves of the turned elements, or neighbours.
  const bool own = D == 64 || kInter || (!kHalves && (a.r.rot == 0 || a.r.rot == 64));
  uint8_t* at = static_cast<uint8_t*>(a.kv.k) + page * a.kv.s_page + (place >> 4) * (long long)R::kBytes;
  place &= 15;
  int slot = 0, h = h0;
#pragma unroll 1
  for (int part = 0; part < 3; ++part) {                  // q, k, v
    const int first = part == 0 ? 0 : part == 1 ? a.Hq : a.Hq + Hkv, end = min(h1, part == 0 ? a.Hq : first + Hkv);
    if (h >= end) continue;
    const Chunk my = part == 2 ? plain : ck;
    const bool normed = a.n.on && part < 2;
    // Each part's own, so that rows don't depend on the heads and tokens of their block.
    if (part < 2 && live && ck.turned) {
      if (part) load_fine_angles(a.r, pairs, a.r.pos + t, c, cs, sn);
      else load_angles(a.r, pairs, a.r.pos + t, c, cs, sn);
    }
    float wa[8] = {}, wb[8] = {};
    if (normed) {
      load_weights<T>(part ? a.n.wk : a.n.wq, a.n.fp32, my.e0, wa);
      load_weights<T>(part ? a.n.wk : a.n.wq, a.n.fp32, my.e1, wb);
    }
    // Where the next head's row goes.
    T* y = part == 0 ? static_cast<T*>(a.q_out.p) + t * a.q_out.sn + h * a.q_out.sh : nullptr;
    uint8_t* rec = at + (h - first) * a.kv.s_head;
    const int ca = part == 1 ? R::k_word(place, my.e0 / 8) : R::v_half(place, my.e0 / 8, 0);
    const int cb = part == 1 ? R::k_word(place, my.e1 / 8) : R::v_half(place, my.e1 / 8, 0);
    // Who has the vectors of plain_sum_of_squares.
    const int2 pa = place_of(c, a.r), pb = place_of(kLanes + c, a.r);
    const int row = threadIdx.x - c;
#pragma unroll 1
    for (; h < end; ++h) {
      copies_wait<kSlots - 1>();
      uint4 va = make_uint4(0, 0, 0, 0), vb = va;
      if (live) {
        va = ring[slot][0][threadIdx.x];
        vb = ring[slot][1][threadIdx.x];
      }
      if (part < 2 && (normed || a.r.rot)) {
        float xa[8], xb[8];
        up8<T>(va, xa);
        up8<T>(vb, xb);
        if (normed) {
          float s;
          if (part == 0) {
            s = sum_over(sum_of_squares(xa, xb), kLanes);
          } else if constexpr (kHalves) {
            s = plain_sum_of_squares<D>(xa, xb, c);
          } else {
            float ya[8], yb[8];
            __syncwarp();                          // every lane's copies have landed
            up8<T>(ring[slot][pa.y][row + pa.x], ya);
            up8<T>(ring[slot][pb.y][row + pb.x], yb);
            s = plain_sum_of_squares<D>(ya, yb, c);
            __syncwarp();                          // before the next copies
          }
          const float r = rsqrtf(s * (1.f / D) + a.n.eps);
          scale8(xa, r, wa);
          scale8(xb, r, wb);
        }
        if (my.turned && part == 1) plain_turn8<kInter>(xa, xb, cs, sn);
        else if (my.turned) turn8<kInter>(xa, xb, cs, sn);
        va = down8<T>(xa);
        vb = down8<T>(xb);
      }
      copy(h + kSlots, slot);
      slot = slot + 1 == kSlots ? 0 : slot + 1;
      if (part == 0) {
        if (live) {
          __stcs(reinterpret_cast<uint4*>(y + my.e0), va);
          __stcs(reinterpret_cast<uint4*>(y + my.e1), vb);
        }
        y += a.q_out.sh;
      } else {
        if (part == 1) {
          store_row<T, D, true>(va, vb, my, own, rec + ca, rec + cb, rec + R::kKp + place * R::kPar, c, live);
        } else {
          store_row<T, D, false>(va, vb, my, true, rec + ca, rec + cb, rec + R::kVp + place * R::kPar, c, live);
        }
        rec += a.kv.s_head;
      }
    }
  }
}

// c / 8 of the codes in place 0 of a word's halves, as fp16 by one product of the
// subnormal c 2^-18; place 1 after a shift by 4, places 2 and 3 with bytes swapped.
__device__ __forceinline__ float2 codes8(uint32_t w) {
  uint32_t h;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h) : "r"(w & 0x03c003c0u), "r"(0x78007800u));       // 2^15
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float2 codes8(uint32_t w, int place) {
  if (place & 2) w = __byte_perm(w, w, 0x2301);
  return codes8(place & 1 ? w << 4 : w);
}

// The last N keys of each sequence.  A warp a record of 16 keys, all its loads first:
// K by words, a lane eight elements of a row; V by the 16 bytes that a lane has of a
// group, eight elements of four rows.  grid: x over records, y over (sequence, kv head).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) fa_read4_kernel(const Read4Args a, const DevStatus st) {
  using R = Record<D>;
  constexpr int kG = D / 64, kWords = D / 8, kRows = 32 / kWords;      // rows of K a warp reads at once
  launch_dependents();
  wait_for_previous();
  const int lane = threadIdx.x % 32, w = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  for (long long bh = blockIdx.y; bh < (long long)a.B * a.kv.Hkv; bh += gridDim.y) {
    const int b = (int)(bh / a.kv.Hkv), h = (int)(bh - (long long)b * a.kv.Hkv);
    int len = a.seq_lens[b];
    if (len < 0 || len > (long long)a.table.cols * a.kv.page_size) {
      if (lane == 0) record_error(st, kErrBadIndex, kSiteReadLen);
      len = 0;
    }
    const int from = max(len - a.N, 0);            // first key that is read
    T* ko = static_cast<T*>(a.k.p) + b * a.k.sb + h * a.k.sh;
    T* vo = static_cast<T*>(a.v.p) + b * a.v.sb + h * a.v.sh;
    // Rows in front of the sequence.
    const int zeros = min(a.N - len, 16 * w + 16);
    for (int n = 16 * w + lane / kWords; n < zeros; n += 32 / kWords) {
      const int e = lane % kWords * 8;
      *reinterpret_cast<uint4*>(ko + n * a.k.sn + e) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(vo + n * a.v.sn + e) = make_uint4(0, 0, 0, 0);
    }
    const int key0 = (from & ~15) + 16 * w;
    if (key0 >= len) continue;
    const int col = key0 / a.kv.page_size, slot0 = key0 - col * a.kv.page_size, page = a.table.pages[b * a.table.stride + col];
    if (page < 0 || page >= a.kv.num_pages) {
      if (lane == 0) record_error(st, kErrBadIndex, kSiteReadPage);
      continue;
    }
    const uint8_t* rec = static_cast<const uint8_t*>(a.kv.k) + page * a.kv.s_page + h * a.kv.s_head +
                         (slot0 >> 4) * (long long)R::kBytes;
    const int row = lane / kWords, i = lane % kWords, r = lane >> 2, c = lane & 3;
    uint32_t kw[16 / kRows], kp[16 / kRows], vp[4][kG];
    uint4 vw[kG];
#pragma unroll
    for (int u = 0; u < 16 / kRows; ++u) {
      const int s = u * kRows + row;
      kw[u] = *reinterpret_cast<const uint32_t*>(rec + R::k_word(s, i));
      kp[u] = *reinterpret_cast<const uint32_t*>(rec + R::kKp + s * R::kPar + i / 8 * 4);
    }
#pragma unroll
    for (int k = 0; k < kG; ++k) {
      vw[k] = *reinterpret_cast<const uint4*>(rec + R::kV + k * 512 + lane * 16);
#pragma unroll
      for (int u = 0; u < 4; ++u) vp[u][k] = *reinterpret_cast<const uint32_t*>(rec + R::kVp + (c + 4 * u) * R::kPar + k * 4);
    }
    ko += (long long)(a.N - len) * a.k.sn;         // row of key 0
    vo += (long long)(a.N - len) * a.v.sn;
#pragma unroll
    for (int u = 0; u < 16 / kRows; ++u) {
      const int key = key0 + u * kRows + row;
      const float2 p = Pair2<T>::up(kp[u]);
      uint32_t y[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float2 x = codes8(kw[u], n);
        y[n] = Pair2<T>::down(fmaf(x.x, 8.f * p.x, p.y), fmaf(x.y, 8.f * p.x, p.y));
      }
      if (key >= from && key < len) __stcs(reinterpret_cast<uint4*>(ko + key * a.k.sn + 8 * i), make_uint4(y[0], y[1], y[2], y[3]));
    }
#pragma unroll
    for (int k = 0; k < kG; ++k)
#pragma unroll
      for (int g = 0; g < 2; ++g) {                // slots c and c + 4, then c + 8 and c + 12
        const uint32_t words[2] = {g ? vw[k].z : vw[k].x, g ? vw[k].w : vw[k].y};
        const float2 p0 = Pair2<T>::up(vp[2 * g][k]), p1 = Pair2<T>::up(vp[2 * g + 1][k]);
        float x0[8], x1[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float2 x = codes8(words[n / 4], n % 4);
          x0[n] = fmaf(x.x, 8.f * p0.x, p0.y);
          x1[n] = fmaf(x.y, 8.f * p1.x, p1.y);
        }
        const int key = key0 + c + 8 * g, e = 64 * k + 8 * r;
        if (key >= from && key < len) __stcs(reinterpret_cast<uint4*>(vo + key * a.v.sn + e), down8<T>(x0));
        if (key + 4 >= from && key + 4 < len) __stcs(reinterpret_cast<uint4*>(vo + (key + 4) * a.v.sn + e), down8<T>(x1));
      }
  }
}

// Somewhat more blocks than run at a time, five an SM, but not many, since each forms its
// tokens' angles anew; a head a block only where they all run at once.  us alone, outputs
// of twelve calls in turn, by 5 | 7 | 10 | 15 blocks an SM: 7357 tokens of 48
// heads 40.2 | 36.9 | 40.1 | 39.0, 8192 43.5 | 41.1 | 41.0 | 43.5, 2048 17.7 | 16.8 | 17.8
// | 19.6; 512 tokens: one head a block 10.3, two 8.1.
int heads_per_block(long long token_blocks, int heads, int num_sms) {
  const long long want = 7LL * num_sms;
  const long long splits = std::min<long long>((want + token_blocks - 1) / token_blocks, heads);
  const int hpb = (int)((heads + splits - 1) / splits);
  return hpb == 1 && token_blocks * heads > 5LL * num_sms ? 2 : hpb;
}

template <typename T, int D>
cudaError_t launch_append(const Append4Args& a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  constexpr int kTokens = kThreads / (D / 16);
  const long long blocks = ((long long)a.T + kTokens - 1) / kTokens;
  const int heads = a.Hq + 2 * a.kv.Hkv, hpb = heads_per_block(blocks, heads, num_sms);
  const dim3 grid((unsigned)blocks, (unsigned)((heads + hpb - 1) / hpb));
  const bool halves = a.r.rot == D || (a.r.rot == 0 && a.n.on);
  auto k = a.r.interleaved ? fa_append4_kernel<T, D, true, false>
           : halves        ? fa_append4_kernel<T, D, false, true>
                           : fa_append4_kernel<T, D, false, false>;
  return launch_after(k, grid, kThreads, 0, 1, stream, a, hpb, st);
}

template <typename T, int D>
cudaError_t launch_read(const Read4Args& a, const DevStatus& st, cudaStream_t stream) {
  const long long records = (a.N + 15LL) / 16 + 1;       // that N keys may lie in
  const dim3 grid((unsigned)((records + kThreads / 32 - 1) / (kThreads / 32)), (unsigned)min((long long)a.B * a.kv.Hkv, 65535LL));
  return launch_after(fa_read4_kernel<T, D>, grid, kThreads, 0, 1, stream, a, st);
}

template <typename T, int D>
cudaError_t configure() {
  cudaError_t e = preload_kernel(fa_append4_kernel<T, D, false, true>);
  if (e == cudaSuccess) e = preload_kernel(fa_append4_kernel<T, D, false, false>);
  if (e == cudaSuccess) e = preload_kernel(fa_append4_kernel<T, D, true, false>);
  if (e == cudaSuccess) e = preload_kernel(fa_read4_kernel<T, D>);
  return e;
}

}  // namespace

cudaError_t configure_append4_kernels() {
  cudaError_t e = configure<__nv_bfloat16, 64>();
  if (e == cudaSuccess) e = configure<__nv_bfloat16, 128>();
  if (e == cudaSuccess) e = configure<__half, 64>();
  if (e == cudaSuccess) e = configure<__half, 128>();
  return e;
}

cudaError_t launch_append4(int dtype, const Append4Args& a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  if (dtype == 0)
    return a.kv.d == 64 ? launch_append<__nv_bfloat16, 64>(a, st, num_sms, stream)
                        : launch_append<__nv_bfloat16, 128>(a, st, num_sms, stream);
  return a.kv.d == 64 ? launch_append<__half, 64>(a, st, num_sms, stream) : launch_append<__half, 128>(a, st, num_sms, stream);
}

cudaError_t launch_read4(int dtype, const Read4Args& a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  if (dtype == 0)
    return a.kv.d == 64 ? launch_read<__nv_bfloat16, 64>(a, st, stream) : launch_read<__nv_bfloat16, 128>(a, st, stream);
  return a.kv.d == 64 ? launch_read<__half, 64>(a, st, stream) : launch_read<__half, 128>(a, st, stream);
}

}  // namespace fa
