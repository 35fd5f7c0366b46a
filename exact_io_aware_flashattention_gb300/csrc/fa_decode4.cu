// Attention of one new token per sequence over the paged cache held in 4 bits:
//   o_h = sum_j p_h(j) v_j,  p_h(j) = exp(scale q_h . k_j - lse_h),
// where k_j and v_j are the values z + s c that the cached codes stand for.
//
// One block per (sequence, query head), a warp every fourth key, each with its
// own running maximum and sum; lane l owns D/32 elements.
#include "fa_paged4.h"
#include "fa_rotary.cuh"
#include "sm103a.cuh"

namespace fa {

namespace {

template <typename T, int D>
__global__ void __launch_bounds__(128) fa_decode4_kernel(const DecodeArgs a, const DevStatus st) {
  constexpr int kE = D / 32;
  __shared__ float so[4][D], sm[4], sl[4];
  launch_dependents();
  wait_for_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.Hq, h = blockIdx.x - b * a.Hq, g = h / (a.Hq / a.kv.Hkv);
  int len = a.seq_lens[b];
  if (len < 0 || len > (long long)a.table.cols * a.kv.page_size) {
    if (threadIdx.x == 0) record_error(st, kErrBadIndex, kSiteDecode4Len);
    len = 0;
  }
  const int first = a.window > 0 && len > a.window ? len - a.window : 0;
  float q[kE], o[kE] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < kE; ++e)
    q[e] = (float)(static_cast<const T*>(a.q) + b * a.q_sb + h * a.q_sh)[lane * kE + e];
  const int word = lane * kE / 8, group = lane * kE / 64, e0 = lane * kE % 8;
  for (int j = first + warp; j < len; j += 4) {
    const int col = j / a.kv.page_size, slot = j - col * a.kv.page_size, page = a.table.pages[b * a.table.stride + col];
    if (page < 0 || page >= a.kv.num_pages) {
      if (lane == 0) record_error(st, kErrBadIndex, kSiteDecode4Page);
      continue;
    }
    const uint8_t* rec = static_cast<const uint8_t*>(a.kv.k) + page * a.kv.s_page + g * a.kv.s_head +
                         (slot >> 4) * (long long)Record<D>::kBytes;
    float x[2][kE];
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + (kv ? Record<D>::kV : 0) + Record<D>::word(slot & 15, word));
      const float2 p = Pair2<T>::up(reinterpret_cast<const uint32_t*>(rec + (kv ? Record<D>::kVp : Record<D>::kKp) +
                                                                      (slot & 15) * Record<D>::kPar)[group]);
      for (int e = 0; e < kE; ++e) x[kv][e] = p.y + p.x * (float)((w >> (16 * (e & 1) + 4 * ((e0 + e) >> 1))) & 15u);
    }
    float s = 0.f;
    for (int e = 0; e < kE; ++e) s = fmaf(q[e], x[0][e], s);
    s = sum_over(s, 32) * a.scale_log2;
    const float n = fmaxf(m, s), f = m == -INFINITY ? 0.f : ex2(m - n), p = ex2(s - n);
    m = n;
    l = l * f + p;
    for (int e = 0; e < kE; ++e) o[e] = o[e] * f + p * x[1][e];
  }
  for (int e = 0; e < kE; ++e) so[warp][lane * kE + e] = o[e];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float L = 0.f, f[4];
  for (int i = 0; i < 4; ++i) {
    f[i] = sm[i] == -INFINITY ? 0.f : ex2(sm[i] - M);
    L += f[i] * sl[i];
  }
  const long long row = (long long)b * a.Hq + h;
  for (int d = threadIdx.x * 2; d < D; d += 256) {
    float y[2];
    for (int e = 0; e < 2; ++e) {
      y[e] = 0.f;
      for (int i = 0; i < 4; ++i) y[e] += f[i] * so[i][d + e];
      y[e] = len > 0 ? y[e] / L : 0.f;
    }
    *reinterpret_cast<uint32_t*>(static_cast<T*>(a.o) + row * D + d) = Pair2<T>::down(y[0], y[1]);
  }
  if (threadIdx.x == 0) a.lse[row] = len > 0 ? (M + log2f(L)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace

cudaError_t configure_decode4_kernels() {
  cudaError_t e = preload_kernel(fa_decode4_kernel<__nv_bfloat16, 64>);
  if (e == cudaSuccess) e = preload_kernel(fa_decode4_kernel<__nv_bfloat16, 128>);
  if (e == cudaSuccess) e = preload_kernel(fa_decode4_kernel<__half, 64>);
  if (e == cudaSuccess) e = preload_kernel(fa_decode4_kernel<__half, 128>);
  return e;
}

cudaError_t launch_decode4(int dtype, const DecodeArgs& a, const DevStatus& st, int parts, cudaStream_t stream) {
  auto k = dtype == 0 ? (a.kv.d == 64 ? fa_decode4_kernel<__nv_bfloat16, 64> : fa_decode4_kernel<__nv_bfloat16, 128>)
                      : (a.kv.d == 64 ? fa_decode4_kernel<__half, 64> : fa_decode4_kernel<__half, 128>);
  return launch_after(k, a.B * a.Hq, 128, 0, 1, stream, a, st);
}

}  // namespace fa
