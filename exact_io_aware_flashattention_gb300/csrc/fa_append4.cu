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
// Bound by HBM: 16-bit rows in, 0.5625 bytes an element out (in and out
// exchanged when reading back).
#include "fa_paged4.h"
#include "fa_rotary.cuh"
#include "sm103a.cuh"

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
    for (int e = 0; e < 8; ++e) x[e] = quotient(__fsub_rn(x[e], g.z), g.s, g.inv);
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

// grid: x over groups of kThreads / (D/16) tokens, y over groups of hpb heads of q,
// then k, then v.  The first rows are on their way while the slot is looked up and
// the angles are formed.
constexpr int kSlots = 3;
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 5) fa_append4_kernel(const Append4Args a, int hpb, const DevStatus st) {
  using R = Record<D>;
  __shared__ Pairs pairs;
  __shared__ uint4 ring[kSlots][2][kThreads];
  constexpr int kLanes = D / 16, kTokens = kThreads / kLanes;
  launch_dependents();
  wait_for_previous();
  const int lt = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  const long long t = (long long)blockIdx.x * kTokens + lt;
  const Chunk ck = chunk_of<kInter>(c, a.r.rot);
  const Chunk plain{16 * c, 16 * c + 8, false};
  const int Hkv = a.kv.Hkv, h0 = blockIdx.y * hpb, h1 = min(h0 + hpb, a.Hq + 2 * Hkv);
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
  if (live && ck.turned && h0 < a.Hq + Hkv) load_fine_angles(a.r, pairs, a.r.pos + t, c, cs, sn);
  // K's vectors: halves of the turned elements, or neighbours.
  const bool own = D == 64 || kInter || a.r.rot == 0 || a.r.rot == 64;
  uint8_t* at = static_cast<uint8_t*>(a.kv.k) + page * a.kv.s_page + (place >> 4) * (long long)R::kBytes;
  place &= 15;
  int slot = 0, h = h0;
#pragma unroll 1
  for (int part = 0; part < 3; ++part) {                  // q, k, v
    const int first = part == 0 ? 0 : part == 1 ? a.Hq : a.Hq + Hkv, end = min(h1, part == 0 ? a.Hq : first + Hkv);
    if (h >= end) continue;
    const Chunk my = part == 2 ? plain : ck;
    const bool normed = a.n.on && part < 2;
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
          const float r = rsqrtf(sum_over(sum_of_squares(xa, xb), kLanes) * (1.f / D) + a.n.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            xa[i] = xa[i] * r * wa[i];
            xb[i] = xb[i] * r * wb[i];
          }
        }
        if (my.turned) turn8<kInter>(xa, xb, cs, sn);
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

// The last N keys of each sequence: a thread a word of eight elements of K and V;
// grid: x over (key, word), y over (sequence, kv head).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) fa_read4_kernel(const Read4Args a, const DevStatus st) {
  launch_dependents();
  wait_for_previous();
  constexpr int kWords = D / 8;
  const int i = threadIdx.x % kWords, n = blockIdx.x * (kThreads / kWords) + threadIdx.x / kWords;
  if (n >= a.N) return;
  for (long long bh = blockIdx.y; bh < (long long)a.B * a.kv.Hkv; bh += gridDim.y) {
    const int b = (int)(bh / a.kv.Hkv), h = (int)(bh - (long long)b * a.kv.Hkv), len = a.seq_lens[b];
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (len < 0 || len > (long long)a.table.cols * a.kv.page_size) {
      record_error(st, kErrBadIndex, kSiteReadLen);
    } else if (const int j = len - a.N + n; j >= 0) {
      const int col = j / a.kv.page_size, slot = j - col * a.kv.page_size, page = a.table.pages[b * a.table.stride + col];
      if (page < 0 || page >= a.kv.num_pages) {
        record_error(st, kErrBadIndex, kSiteReadPage);
      } else {
        const uint8_t* rec = static_cast<const uint8_t*>(a.kv.k) + page * a.kv.s_page + h * a.kv.s_head +
                             (slot >> 4) * (long long)Record<D>::kBytes;
        const int s = slot & 15, g = i / 8;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t h0 = kv ? *reinterpret_cast<const uint16_t*>(rec + Record<D>::v_half(s, i, 0))
                                 : *reinterpret_cast<const uint32_t*>(rec + Record<D>::k_word(s, i));
          const uint32_t h1 = kv ? *reinterpret_cast<const uint16_t*>(rec + Record<D>::v_half(s, i, 1)) : h0 >> 16;
          const float2 p = Pair2<T>::up(
              reinterpret_cast<const uint32_t*>(rec + (kv ? Record<D>::kVp : Record<D>::kKp) + s * Record<D>::kPar)[g]);
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = p.y + p.x * (float)(kv ? code_at(e < 4 ? h0 : h1, e % 4) : code_at(e % 2 ? h1 : h0, e / 2));
          (kv ? v : k) = down8<T>(x);
        }
      }
    }
    *reinterpret_cast<uint4*>(static_cast<T*>(a.k.p) + b * a.k.sb + h * a.k.sh + n * a.k.sn + 8 * i) = k;
    *reinterpret_cast<uint4*>(static_cast<T*>(a.v.p) + b * a.v.sb + h * a.v.sh + n * a.v.sn + 8 * i) = v;
  }
}

int heads_per_block(long long token_blocks, int heads, int num_sms) {
  const long long want = 16LL * num_sms;
  long long splits = (want + token_blocks - 1) / token_blocks;
  if (splits > heads) splits = heads;
  if (splits < 1) splits = 1;
  return (int)((heads + splits - 1) / splits);
}

template <typename T, int D>
cudaError_t launch_append(const Append4Args& a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  constexpr int kTokens = kThreads / (D / 16);
  const long long blocks = ((long long)a.T + kTokens - 1) / kTokens;
  const int heads = a.Hq + 2 * a.kv.Hkv, hpb = heads_per_block(blocks, heads, num_sms);
  const dim3 grid((unsigned)blocks, (unsigned)((heads + hpb - 1) / hpb));
  return launch_after(a.r.interleaved ? fa_append4_kernel<T, D, true> : fa_append4_kernel<T, D, false>, grid, kThreads, 0, 1,
                      stream, a, hpb, st);
}

template <typename T, int D>
cudaError_t launch_read(const Read4Args& a, const DevStatus& st, cudaStream_t stream) {
  constexpr int kKeys = kThreads / (D / 8);
  const dim3 grid((unsigned)((a.N + kKeys - 1) / kKeys), (unsigned)min((long long)a.B * a.kv.Hkv, 65535LL));
  return launch_after(fa_read4_kernel<T, D>, grid, kThreads, 0, 1, stream, a, st);
}

template <typename T, int D>
cudaError_t configure() {
  cudaError_t e = preload_kernel(fa_append4_kernel<T, D, false>);
  if (e == cudaSuccess) e = preload_kernel(fa_append4_kernel<T, D, true>);
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
