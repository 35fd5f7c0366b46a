// Attention of one new token per sequence over a paged key / value cache.
//
//   o_h = sum_j p_h(j) v_j,  p_h(j) = exp(scale q_h . k_j - lse_h),
//   lse_h = ln sum_j exp(scale q_h . k_j)
// over the visible keys j of [max(0, len - window), len); with scores, each
// visible key's accumulated weight grows by sum over the group's heads of
// p_h(j).
#include "fa_internal.h"
#include "sm103a.cuh"

#include <cuda_fp16.h>

namespace fa {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// One block per (sequence, query head); each warp takes every eighth key with
// a running max and sum, the warps are joined at the end.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) fa_paged_decode_kernel(const DecodeArgs a, const DevStatus st) {
  constexpr int E = D / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = h / (a.Hq / a.kv.Hkv);
  int len = a.seq_lens[b];
  if (len < 0 || len > (long long)a.table.cols * a.kv.page_size) {
    if (threadIdx.x == 0) record_error(st, kErrBadIndex, kSiteDecodeLen);
    len = 0;
  }
  const int first = a.window > 0 && len > a.window ? len - a.window : 0;
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e)
    q[e] = to_f(static_cast<const T*>(a.q)[b * a.q_sb + h * a.q_sh + lane * E + e]) * a.scale_log2;
  auto row = [&](int j) -> long long {
    const int page = a.table.pages[b * a.table.stride + j / a.kv.page_size];
    if (page < 0 || page >= a.kv.num_pages) {
      record_error(st, kErrBadIndex, kSiteDecodePage);
      return -1;
    }
    return page * a.kv.s_page + g * a.kv.s_head + (long long)(j % a.kv.page_size) * a.kv.s_slot;
  };
  auto dot = [&](long long at) {
    const T* k = static_cast<const T*>(a.kv.k) + at + lane * E;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(q[e], to_f(k[e]), s);
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    return s;
  };
  for (int j = first + warp; j < len; j += kWarps) {
    const long long at = row(j);
    if (at < 0) continue;
    const float s = dot(at), mn = fmaxf(m, s), mu = mn == -INFINITY ? 0.f : mn;
    const float al = exp2f(m - mu), p = exp2f(s - mu);
    const T* v = static_cast<const T*>(a.kv.v) + at + lane * E;
    l = l * al + p;
    for (int e = 0; e < E; ++e) o[e] = o[e] * al + p * to_f(v[e]);
    m = mn;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  const float Mu = M == -INFINITY ? 0.f : M;
  for (int w = 0; w < kWarps; ++w) L += sl[w] * exp2f(sm[w] - Mu);
  const float inv = len > first ? 1.f / L : 0.f;
  for (int e = threadIdx.x; e < D; e += blockDim.x) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += so[w][e] * exp2f(sm[w] - Mu);
    static_cast<T*>(a.o)[((long long)b * a.Hq + h) * D + e] = (T)(len > first ? x * inv : 0.f);
  }
  const float lse2 = M + log2f(L);
  if (threadIdx.x == 0) a.lse[(long long)b * a.Hq + h] = len > first ? lse2 * 0.69314718055994530942f : -INFINITY;
}

// The visible keys' weights, summed over the group's heads in order: one block
// per (sequence, kv head), one warp per key, so each entry is added to once.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) fa_paged_scores_kernel(const DecodeArgs a) {
  constexpr int E = D / 32;
  const int b = blockIdx.x / a.kv.Hkv, g = blockIdx.x % a.kv.Hkv, G = a.Hq / a.kv.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = a.seq_lens[b];
  if (len < 0 || len > (long long)a.table.cols * a.kv.page_size) return;
  const int first = a.window > 0 && len > a.window ? len - a.window : 0;
  for (int j = first + warp; j < len; j += kWarps) {
    const int page = a.table.pages[b * a.table.stride + j / a.kv.page_size], slot = j % a.kv.page_size;
    if (page < 0 || page >= a.kv.num_pages) continue;
    const T* k = static_cast<const T*>(a.kv.k) + page * a.kv.s_page + g * a.kv.s_head + slot * a.kv.s_slot + lane * E;
    float w = 0.f;
    for (int h = g * G; h < (g + 1) * G; ++h) {
      const T* q = static_cast<const T*>(a.q) + b * a.q_sb + h * a.q_sh + lane * E;
      float s = 0.f;
      for (int e = 0; e < E; ++e) s = fmaf(to_f(q[e]) * a.scale_log2, to_f(k[e]), s);
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      w += exp2f(s - a.lse[(long long)b * a.Hq + h] * 1.4426950408889634f);
    }
    if (lane == 0) atomicAdd(&a.scores[((long long)page * a.kv.Hkv + g) * a.kv.page_size + slot], w);
  }
}

template <typename T, int D>
void launch(const DecodeArgs& a, const DevStatus& st, cudaStream_t stream) {
  fa_paged_decode_kernel<T, D><<<a.B * a.Hq, kWarps * 32, 0, stream>>>(a, st);
  if (a.scores) fa_paged_scores_kernel<T, D><<<a.B * a.kv.Hkv, kWarps * 32, 0, stream>>>(a);
}

}  // namespace

cudaError_t launch_paged_decode(int dtype, const DecodeArgs& a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  if (dtype == 0) {
    if (a.kv.d == 64) launch<__nv_bfloat16, 64>(a, st, stream);
    else launch<__nv_bfloat16, 128>(a, st, stream);
  } else {
    if (a.kv.d == 64) launch<__half, 64>(a, st, stream);
    else launch<__half, 128>(a, st, stream);
  }
  return cudaGetLastError();
}

}  // namespace fa
