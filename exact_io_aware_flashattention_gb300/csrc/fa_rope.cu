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
#include "fa_rotary.cuh"
#include "sm103a.cuh"

namespace fa {

namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;   // heads whose loads are in flight per thread

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
  load_pairs<kThreads>(a.r, pairs, st);
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
  load_pairs<kThreads>(a.r, pairs, st);
  if (a.cu && blockIdx.y == 0) check_offsets<kThreads>(a, st);
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
