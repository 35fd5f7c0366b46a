// What the kernels that turn rows share: a block's pairs of the rotation, a
// token's cosines and sines, the part of a row that a thread owns, and where a
// new token goes in a paged cache.
#pragma once

#include <cuda_fp16.h>

#include "fa_angle.h"
#include "fa_paged.h"
#include "sm103a.cuh"

namespace fa {

namespace {

template <typename T>
struct Pair2;
template <>
struct Pair2<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ float2 up(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t down(float lo, float hi) { return cvt_bf16x2(lo, hi); }
};
template <>
struct Pair2<__half> {
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ float2 up(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t down(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// inv_freq / (2 pi) modulo 1, in units of 2^-64 turns.  inv_freq = M 2^(e-63)
// with M its mantissa in the top bits of a word, 1 / (2 pi) = C 2^-66, so the
// result is the 128-bit product M C shifted by e - 65.
__device__ __forceinline__ uint64_t turns64(double w) {
  const uint64_t bits = (uint64_t)__double_as_longlong(w);
  const int ex = (int)((bits >> 52) & 0x7ff);
  if (ex == 0 || ex == 0x7ff) return 0;                     // zero (or not a finite frequency)
  const uint64_t M = (1ull << 63) | ((bits & 0xfffffffffffffull) << 11);
  const uint64_t C = 0xA2F9836E4E44152Aull;                 // 2^66 / (2 pi)
  const uint64_t hi = __umul64hi(M, C), lo = M * C;
  const int s = ex - 1023 - 1;                              // hi:lo shifted left by s, the upper word
  uint64_t F;
  if (s >= 64) F = 0;
  else if (s > 0) F = (hi << s) | (lo >> (64 - s));
  else F = s > -64 ? hi >> -s : 0;
  return (bits >> 63) ? 0 - F : F;
}

// What a block keeps of the rotation: each pair's F and axis.
struct Pairs {
  uint64_t turns[128];
  int axis[128];
};
template <int kThreads>
__device__ __forceinline__ void load_pairs(const RotaryArgs& r, Pairs& p, const DevStatus& st) {
  for (int i = threadIdx.x; i < r.rot / 2; i += kThreads) {
    int ax = r.axes[i];
    if (ax < 0 || ax >= r.n_axes) {
      record_error(st, kErrBadIndex, kSiteAxis);
      ax = 0;
    }
    p.axis[i] = ax;
    p.turns[i] = turns64(r.inv_freq[i]);
  }
}

// Cosines and sines of the pairs 8c .. 8c+7 of the token whose positions
// start at pos.
__device__ __forceinline__ void load_angles(const RotaryArgs& r, const Pairs& p, const int* pos, int c, float (&cs)[8],
                                            float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t phase = (uint64_t)(int64_t)pos[p.axis[c * 8 + i] * r.pos_axis] * p.turns[c * 8 + i];
    const float angle = (float)(int32_t)(uint32_t)(phase >> 32) * 1.4629180792671596e-9f;   // 2 pi / 2^32
    cs[i] = __cosf(angle);
    sn[i] = __sinf(r.inverse ? -angle : angle);
  }
}

// Eight pairs: elements of a at i, of b at i (halves) or adjacent (interleaved).
template <typename T, bool kInter>
__device__ __forceinline__ void turn8(uint4& va, uint4& vb, const float (&cs)[8], const float (&sn)[8]) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&va);
  uint32_t* b = reinterpret_cast<uint32_t*>(&vb);
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = i < 4 ? a[i] : b[i - 4];
      const float2 x = Pair2<T>::up(w);
      w = Pair2<T>::down(x.x * cs[i] - x.y * sn[i], x.y * cs[i] + x.x * sn[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = Pair2<T>::up(a[i]), y = Pair2<T>::up(b[i]);
      a[i] = Pair2<T>::down(x.x * cs[2 * i] - y.x * sn[2 * i], x.y * cs[2 * i + 1] - y.y * sn[2 * i + 1]);
      b[i] = Pair2<T>::down(y.x * cs[2 * i] + x.x * sn[2 * i], y.y * cs[2 * i + 1] + x.y * sn[2 * i + 1]);
    }
  }
}

// What one thread does to a row: the two 16-byte vectors it owns, turned or
// moved unchanged.  A row has rot/16 turned chunks and then (d - rot)/16 chunks
// that pass through.
struct Chunk {
  int e0, e1;      // first elements of the two vectors
  bool turned;
};
template <bool kInter>
__device__ __forceinline__ Chunk chunk_of(int c, int rot) {
  Chunk k;
  k.turned = c < rot / 16;
  if (k.turned && !kInter) {
    k.e0 = 8 * c;
    k.e1 = rot / 2 + 8 * c;
  } else {
    k.e0 = 16 * c;
    k.e1 = 16 * c + 8;
  }
  return k;
}

// The same values in fp32: eight of a and eight of b.
template <typename T>
__device__ __forceinline__ void up8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = Pair2<T>::up(w[i]);
    x[2 * i] = y.x;
    x[2 * i + 1] = y.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 down8(const float (&x)[8]) {
  return make_uint4(Pair2<T>::down(x[0], x[1]), Pair2<T>::down(x[2], x[3]), Pair2<T>::down(x[4], x[5]),
                    Pair2<T>::down(x[6], x[7]));
}
// Two fp32 operations in one instruction, each rounded as its own.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 y;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(y))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(y))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(y))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return y;
}
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }

template <bool kInter>
__device__ __forceinline__ void turn8(float (&a)[8], float (&b)[8], const float (&cs)[8], const float (&sn)[8]) {
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& x = i < 4 ? a[2 * i] : b[2 * i - 8];
      float& y = i < 4 ? a[2 * i + 1] : b[2 * i - 7];
      const float t = x * cs[i] - y * sn[i];
      y = y * cs[i] + x * sn[i];
      x = t;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 x = make_float2(a[i], a[i + 1]), y = make_float2(b[i], b[i + 1]);
      const float2 c = make_float2(cs[i], cs[i + 1]), s = make_float2(sn[i], sn[i + 1]), z = mul2(y, s);
      const float2 u = fma2(x, c, make_float2(-z.x, -z.y)), v = fma2(x, s, mul2(y, c));
      a[i] = u.x, a[i + 1] = u.y;
      b[i] = v.x, b[i + 1] = v.y;
    }
  }
}

// A row's eight and eight elements of a thread as weights: fp32, T, or ones.
template <typename T>
__device__ __forceinline__ void load_weights(const void* w, int fp32, int e, float (&x)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 1.f;
  } else if (fp32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<const float*>(w)[e + i];
  } else {
    up8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(w) + e), x);
  }
}
__device__ __forceinline__ float sum_over(float x, int lanes) {
  for (int d = 1; d < lanes; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
__device__ __forceinline__ float sum_of_squares(const float (&a)[8], const float (&b)[8]) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 x = make_float2(a[i], a[i + 1]), y = make_float2(b[i], b[i + 1]);
    s = fma2(x, x, fma2(y, y, s));
  }
  return s.x + s.y;
}

// x r w.
__device__ __forceinline__ void scale8(float (&x)[8], float r, const float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 y = mul2(mul2(make_float2(x[i], x[i + 1]), two(r)), make_float2(w[i], w[i + 1]));
    x[i] = y.x;
    x[i + 1] = y.y;
  }
}

// Cosine and sine of phase 2^-64 turns, off by 2^-29.5 at most before they are rounded to fp32.
__device__ __forceinline__ void fine_angle(uint64_t phase, float& cs, float& sn) {
  const FixedAngle a = fixed_angle(phase);
  const float c = (float)a.cos31 * 0x1p-31f, s = (float)a.sin32 * (a.negative ? -0x1p-32f : 0x1p-32f);
  cs = a.quarter & 1 ? s : c;
  sn = a.quarter & 1 ? c : s;
  if (a.quarter == 1 || a.quarter == 2) cs = -cs;
  if (a.quarter & 2) sn = -sn;
}
// Those of the pairs 8c .. 8c+7.
__device__ __forceinline__ void load_fine_angles(const RotaryArgs& r, const Pairs& p, const int* pos, int c, float (&cs)[8],
                                                 float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    fine_angle((uint64_t)(int64_t)pos[p.axis[c * 8 + i] * r.pos_axis] * p.turns[c * 8 + i], cs[i], sn[i]);
    if (r.inverse) sn[i] = -sn[i];
  }
}

// Asynchronous copies of a thread's own vectors into its own places of a ring in
// shared memory, some rows deep: what a row needs is on its way while others are
// worked on, without registers, and nobody else waits for it.
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Offsets of new tokens run from 0 and upwards, to T at most.  The first blocks
// look at all of them: a pair out of order may leave every token with a
// sequence, but not with its own.
template <int kThreads, typename Args>
__device__ __forceinline__ void check_offsets(const Args& a, const DevStatus& st) {
  for (long long b = (long long)blockIdx.x * kThreads + threadIdx.x; b < a.B; b += (long long)gridDim.x * kThreads) {
    const int from = a.cu[b], to = a.cu[b + 1];
    if (from < 0 || to < from || to > a.T || (b == 0 && from != 0)) record_error(st, kErrBadIndex, kSiteAppend);
  }
}

// Where token t goes: sequence, index in it, page and slot.  Returns false for
// a token that is not stored: padding (past the last sequence, or a sequence
// of length 0 in the one-token form), or an index out of range, which is
// recorded here or by check_offsets.  A token that is stored lies in its
// sequence's range, and that in [0, T), so it is one of the sequence's last and
// falls on no older key.
template <typename Args>
__device__ __forceinline__ bool place_token(const Args& a, int t, const DevStatus& st, int& page, int& slot) {
  int b = t, back = 1;
  if (a.cu) {
    if (t >= a.cu[a.B]) return false;
    int lo = 0, hi = a.B;                  // last b with cu[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= t) lo = mid; else hi = mid;
    }
    b = lo;
    const int from = a.cu[b], to = a.cu[b + 1];
    if (from < 0 || from > t || to > a.T) return false;
    back = to - t;
  } else if (a.seq_lens[b] == 0) {
    return false;
  }
  const long long i = (long long)a.seq_lens[b] - back;
  if (back < 1 || i < 0 || i >= (long long)a.table.cols * a.kv.page_size) {
    record_error(st, kErrBadIndex, kSiteAppend);
    return false;
  }
  const int col = (int)i / a.kv.page_size;
  page = a.table.pages[b * a.table.stride + col];
  slot = (int)i - col * a.kv.page_size;
  if (page < 0 || page >= a.kv.num_pages) {
    record_error(st, kErrBadIndex, kSiteAppend);
    return false;
  }
  return true;
}

}  // namespace

}  // namespace fa
