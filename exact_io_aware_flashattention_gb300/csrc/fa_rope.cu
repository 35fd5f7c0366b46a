// Rotary positions with several axes, and the append of new tokens to a paged
// key / value cache with the same rotation fused in.
//
// Pair i of a row (elements i and i + rot/2, or 2i and 2i + 1 when
// interleaved) turns by angle = pos[axis_i] * inv_freq_i:
//   (x, y) -> (x cos - y sin, y cos + x sin);
// the gradient turns by -angle (the rotation is orthogonal).
//
// The angle.  pos * inv_freq reaches 1e6 radians and more, where an fp32
// product leaves no digits, and fp64 arithmetic is slow here.  Only the angle
// modulo one turn matters, so inv_freq becomes F = inv_freq / (2 pi) * 2^64
// as a 64-bit integer (from the double's mantissa and exponent, integer
// arithmetic only) and the phase is pos * F modulo 2^64: the wrap-around of
// the integer product is the reduction, exact for every int32 position.  The
// phase's top 32 bits, as a signed angle in [-pi, pi], go to __sinf and __cosf,
// which are within 2^-21.4 and 2^-21.2 there; with the roundings of the angle
// (3 2^-24 of it) a sine or cosine is off by less than 1e-6, 1/500 of the
// rounding of an fp16 result.  A block turns the frequencies into F once, in
// shared memory.
//
// Bound by HBM: every element is read once and written once.  A thread owns
// one token and eight pairs (two 16-byte vectors of a row): its eight
// cosines and sines are formed once and used for all the heads of its block.
// Loads and stores are marked as streaming: nothing is read twice.  The first
// heads' rows are requested before the angles are formed and, in the append,
// the slot is looked up (gradient 52.6 -> 51.9 us, prompt 31.4 -> 30.9).
//
// Measured (calls in a row on three sets of tensors), of the 6.79 TB/s copy
// rate: q and k of 4 x (16 + 16) heads x 2048 tokens, d = 128, 134 MB: 23.5 us,
// 84 %; the gradient for 2 x (32 + 8) x 8192, 336 MB: 51.9 us, 95 %; appending
// 7357 prompt tokens (32 q heads turned, 8 k and 8 v heads stored), 181 MB:
// 30.9 us, 86 % (90 registers leave 20 warps an SM); one token for each of 64
// sequences: 3.7 us, of which the launch is most.
#include "fa_paged.h"
#include "sm103a.cuh"

#include <cuda_fp16.h>

namespace fa {

namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;   // heads whose loads are in flight per thread

template <typename T>
struct Pair2;
template <>
struct Pair2<__nv_bfloat16> {
  static __device__ __forceinline__ float2 up(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t down(float lo, float hi) { return cvt_bf16x2(lo, hi); }
};
template <>
struct Pair2<__half> {
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

// The next heads of [h, h1) of one token, in + h * in_sh.
struct Batch {
  uint4 a[kUnroll], b[kUnroll];
};
template <typename T>
__device__ __forceinline__ void load_heads(const T* in, long long in_sh, int h, int h1, const Chunk& ck, Batch& x) {
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (h + u < h1) {
      x.a[u] = __ldcs(reinterpret_cast<const uint4*>(in + (h + u) * in_sh + ck.e0));
      x.b[u] = __ldcs(reinterpret_cast<const uint4*>(in + (h + u) * in_sh + ck.e1));
    }
}
// Heads [h0, h1) of one token: in + h * in_sh -> out + h * out_sh; the first
// of them are in x already if `loaded`.
template <typename T, bool kInter>
__device__ __forceinline__ void do_heads(const T* in, long long in_sh, T* out, long long out_sh, int h0, int h1,
                                         const Chunk& ck, bool turned, const float (&cs)[8], const float (&sn)[8], Batch& x,
                                         bool loaded) {
  for (int h = h0; h < h1; h += kUnroll) {
    if (!loaded) load_heads(in, in_sh, h, h1, ck, x);
    loaded = false;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u < h1) {
        if (turned) turn8<T, kInter>(x.a[u], x.b[u], cs, sn);
        __stcs(reinterpret_cast<uint4*>(out + (h + u) * out_sh + ck.e0), x.a[u]);
        __stcs(reinterpret_cast<uint4*>(out + (h + u) * out_sh + ck.e1), x.b[u]);
      }
  }
}

// grid: x over groups of kThreads / (d/16) tokens, y over groups of hpb heads of q
// and then k.
template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads) fa_rope_kernel(const RopeArgs a, int hpb, const DevStatus st) {
  __shared__ Pairs pairs;
  launch_dependents();
  wait_for_previous();
  const int nch = a.d / 16, tpb = kThreads / nch;
  const int lt = threadIdx.x / nch, c = threadIdx.x - lt * nch;
  const long long t = (long long)blockIdx.x * tpb + lt;
  const bool live = lt < tpb && t < (long long)a.B * a.N;
  const int b = live ? (int)(t / a.N) : 0, n = live ? (int)(t - (long long)b * a.N) : 0;
  const Chunk ck = chunk_of<kInter>(c, a.r.rot);
  const int h0 = blockIdx.y * hpb, h1 = min(h0 + hpb, a.Hq + a.Hk);
  const T* q = static_cast<const T*>(a.q.p) + b * a.q.sb + n * a.q.sn;
  const T* k = static_cast<const T*>(a.k.p) + b * a.k.sb + n * a.k.sn;
  // The first rows are on their way while the angles are formed.
  Batch x;
  if (live) {
    if (h0 < a.Hq) load_heads(q, a.q.sh, h0, min(h1, a.Hq), ck, x);
    else load_heads(k, a.k.sh, h0 - a.Hq, h1 - a.Hq, ck, x);
  }
  load_pairs(a.r, pairs, st);
  __syncthreads();
  if (!live) return;
  float cs[8] = {}, sn[8] = {};
  if (ck.turned) load_angles(a.r, pairs, a.r.pos + b * a.r.pos_batch + n, c, cs, sn);
  if (h0 < a.Hq)
    do_heads<T, kInter>(q, a.q.sh, static_cast<T*>(a.q_out.p) + b * a.q_out.sb + n * a.q_out.sn, a.q_out.sh, h0, min(h1, a.Hq),
                        ck, ck.turned, cs, sn, x, true);
  if (h1 > a.Hq)
    do_heads<T, kInter>(k, a.k.sh, static_cast<T*>(a.k_out.p) + b * a.k_out.sb + n * a.k_out.sn, a.k_out.sh,
                        max(h0 - a.Hq, 0), h1 - a.Hq, ck, ck.turned, cs, sn, x, h0 >= a.Hq);
}

// Offsets of new tokens run from 0 and upwards, to T at most.  The first blocks
// look at all of them: a pair out of order may leave every token with a
// sequence, but not with its own.
__device__ __forceinline__ void check_offsets(const AppendArgs& a, const DevStatus& st) {
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
__device__ __forceinline__ bool place_token(const AppendArgs& a, int t, const DevStatus& st, int& page, int& slot) {
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

// As fa_rope_kernel over tokens, with the heads of q, then k, then v; k and v
// rows go to their slot of the cache, whose accumulated weight starts at 0.
template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads) fa_append_kernel(const AppendArgs a, int hpb, const DevStatus st) {
  __shared__ Pairs pairs;
  launch_dependents();
  wait_for_previous();
  const int nch = a.kv.d / 16, tpb = kThreads / nch;
  const int lt = threadIdx.x / nch, c = threadIdx.x - lt * nch;
  const long long t = (long long)blockIdx.x * tpb + lt;
  const bool live = lt < tpb && t < a.T;
  const int Hkv = a.kv.Hkv;
  const int h0 = blockIdx.y * hpb, h1 = min(h0 + hpb, a.Hq + 2 * Hkv);
  const int k0 = max(h0 - a.Hq, 0), k1 = min(h1 - a.Hq, Hkv), v0 = max(h0 - a.Hq - Hkv, 0), v1 = h1 - a.Hq - Hkv;
  const Chunk ck = chunk_of<kInter>(c, a.r.rot);
  const T* q = static_cast<const T*>(a.q.p) + t * a.q.sn;
  const T* k = static_cast<const T*>(a.k.p) + t * a.k.sn;
  const T* v = static_cast<const T*>(a.v.p) + t * a.v.sn;
  // The first rows are on their way while the slot is looked up and the angles
  // are formed.
  Batch x;
  const int first = h0 < a.Hq ? 0 : k0 < k1 ? 1 : 2;
  if (live) {
    if (first == 0) load_heads(q, a.q.sh, h0, min(h1, a.Hq), ck, x);
    else if (first == 1) load_heads(k, a.k.sh, k0, k1, ck, x);
    else load_heads(v, a.v.sh, v0, v1, ck, x);
  }
  load_pairs(a.r, pairs, st);
  if (a.cu && blockIdx.y == 0) check_offsets(a, st);
  __syncthreads();
  int page, slot;
  if (!live || !place_token(a, (int)t, st, page, slot)) return;
  float cs[8] = {}, sn[8] = {};
  if (ck.turned && h0 < a.Hq + Hkv) load_angles(a.r, pairs, a.r.pos + t, c, cs, sn);
  const long long at = page * a.kv.s_page + slot * a.kv.s_slot;
  if (first == 0)
    do_heads<T, kInter>(q, a.q.sh, static_cast<T*>(a.q_out.p) + t * a.q_out.sn, a.q_out.sh, h0, min(h1, a.Hq), ck, ck.turned,
                        cs, sn, x, true);
  if (k0 < k1) {
    do_heads<T, kInter>(k, a.k.sh, static_cast<T*>(a.kv.k) + at, a.kv.s_head, k0, k1, ck, ck.turned, cs, sn, x, first == 1);
    if (a.scores)
      for (int h = k0 + c; h < k1; h += nch) a.scores[((long long)page * Hkv + h) * a.kv.page_size + slot] = 0.f;
  }
  if (v0 < v1)
    do_heads<T, kInter>(v, a.v.sh, static_cast<T*>(a.kv.v) + at, a.kv.s_head, v0, v1, ck, false, cs, sn, x, first == 2);
}

// Heads per block: as many as still leave 16 blocks of 128 threads an SM, so
// that the angles are formed for several heads at once and the last wave is
// short.  (8 an SM: the gradient above 54.5 instead of 52.6 us; 24: the prompt
// 33.7 instead of 31.4.  Equal parts of one line of (token, head) rows per
// resident block spilled and took up to twice as long.)
int heads_per_block(long long token_blocks, int heads, int num_sms) {
  const long long want = 16LL * num_sms;
  long long splits = (want + token_blocks - 1) / token_blocks;
  const long long most = (heads + kUnroll - 1) / kUnroll;
  if (splits > most) splits = most;
  if (splits < 1) splits = 1;
  return (int)((heads + splits - 1) / splits);
}

}  // namespace

cudaError_t configure_rope_kernels() {
  cudaError_t e = preload_kernel(fa_rope_kernel<__nv_bfloat16, false>);
  if (e == cudaSuccess) e = preload_kernel(fa_rope_kernel<__nv_bfloat16, true>);
  if (e == cudaSuccess) e = preload_kernel(fa_rope_kernel<__half, false>);
  if (e == cudaSuccess) e = preload_kernel(fa_rope_kernel<__half, true>);
  if (e == cudaSuccess) e = preload_kernel(fa_append_kernel<__nv_bfloat16, false>);
  if (e == cudaSuccess) e = preload_kernel(fa_append_kernel<__nv_bfloat16, true>);
  if (e == cudaSuccess) e = preload_kernel(fa_append_kernel<__half, false>);
  if (e == cudaSuccess) e = preload_kernel(fa_append_kernel<__half, true>);
  return e;
}

cudaError_t launch_rope(int dtype, const RopeArgs& a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  const int tpb = kThreads / (a.d / 16);
  const long long blocks = ((long long)a.B * a.N + tpb - 1) / tpb;
  const int heads = a.Hq + a.Hk, hpb = heads_per_block(blocks, heads, num_sms);
  const dim3 grid((unsigned)blocks, (unsigned)((heads + hpb - 1) / hpb));
  if (dtype == 0) {
    if (a.r.interleaved) return launch_after(fa_rope_kernel<__nv_bfloat16, true>, grid, kThreads, 0, 1, stream, a, hpb, st);
    return launch_after(fa_rope_kernel<__nv_bfloat16, false>, grid, kThreads, 0, 1, stream, a, hpb, st);
  }
  if (a.r.interleaved) return launch_after(fa_rope_kernel<__half, true>, grid, kThreads, 0, 1, stream, a, hpb, st);
  return launch_after(fa_rope_kernel<__half, false>, grid, kThreads, 0, 1, stream, a, hpb, st);
}

cudaError_t launch_append(int dtype, const AppendArgs& a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  const int tpb = kThreads / (a.kv.d / 16);
  const long long blocks = ((long long)a.T + tpb - 1) / tpb;
  const int heads = a.Hq + 2 * a.kv.Hkv, hpb = heads_per_block(blocks, heads, num_sms);
  const dim3 grid((unsigned)blocks, (unsigned)((heads + hpb - 1) / hpb));
  if (dtype == 0) {
    if (a.r.interleaved) return launch_after(fa_append_kernel<__nv_bfloat16, true>, grid, kThreads, 0, 1, stream, a, hpb, st);
    return launch_after(fa_append_kernel<__nv_bfloat16, false>, grid, kThreads, 0, 1, stream, a, hpb, st);
  }
  if (a.r.interleaved) return launch_after(fa_append_kernel<__half, true>, grid, kThreads, 0, 1, stream, a, hpb, st);
  return launch_after(fa_append_kernel<__half, false>, grid, kThreads, 0, 1, stream, a, hpb, st);
}

}  // namespace fa
