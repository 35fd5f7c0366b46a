// Norm of each head's rows of q and k with the rotary positions in the same
// pass, and its gradient.
//
// Row x of d elements, weights w [d], R the rotation of pairs (fa_rope.cu):
//   r = (mean x^2 + eps)^-1/2,   y = R (x r w);
// with g = R^T dy (the turn by the opposite angles),
//   dw = sum over rows of g x r,   dx = r (g w - x r mean(g w x r)).
// The gradient needs nothing of the forward but x: r is formed again.
//
// Bound by HBM: the forward reads and writes each element once, the gradient
// reads dy and x and writes dx.  A thread owns one token and eight pairs (two
// 16-byte vectors of a row), as in fa_rope.cu; the row's sums go over its
// lanes, d / 16 rounded up to a power of two.
#include "fa_paged4.h"
#include "fa_rotary.cuh"
#include "sm103a.cuh"

namespace fa {

namespace {

constexpr int kThreads = 128;

// Lanes of a row, and this thread's token of the block's and chunk of the row.
struct Lanes {
  int per_row, tpb, lt, c;
  __device__ __forceinline__ explicit Lanes(int d) {
    per_row = 1;
    while (per_row < d / 16) per_row *= 2;
    tpb = kThreads / per_row;
    lt = threadIdx.x / per_row;
    c = threadIdx.x % per_row;
  }
};
__host__ __device__ inline int tokens_per_block(int d) {
  int p = 1;
  while (p < d / 16) p *= 2;
  return kThreads / p;
}

template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads) fa_qk_norm_kernel(const NormRopeArgs a, int hpb, const DevStatus st) {
  __shared__ Pairs pairs;
  launch_dependents();
  wait_for_previous();
  load_pairs<kThreads>(a.r, pairs, st);
  __syncthreads();
  const Lanes ln(a.d);
  const long long t = (long long)blockIdx.x * ln.tpb + ln.lt;
  const bool live = ln.c < a.d / 16 && t < (long long)a.B * a.N;
  const int b = live ? (int)(t / a.N) : 0, n = live ? (int)(t - (long long)b * a.N) : 0;
  const Chunk ck = chunk_of<kInter>(live ? ln.c : 0, a.r.rot);
  float cs[8] = {}, sn[8] = {};
  if (ck.turned) load_fine_angles(a.r, pairs, a.r.pos + b * a.r.pos_batch + n, live ? ln.c : 0, cs, sn);
  const int h0 = blockIdx.y * hpb, h1 = min(h0 + hpb, a.Hq + a.Hk);
  const float inv_d = 1.f / a.d;
  for (int part = 0; part < 2; ++part) {
    const RowView &in = part ? a.k : a.q, &out = part ? a.k_out : a.q_out;
    const int from = part ? max(h0 - a.Hq, 0) : h0, to = part ? h1 - a.Hq : min(h1, a.Hq);
    if (from >= to) continue;
    const T* x = static_cast<const T*>(in.p) + b * in.sb + n * in.sn;
    T* y = static_cast<T*>(out.p) + b * out.sb + n * out.sn;
    float wa[8], wb[8];
    load_weights<T>(part ? a.n.wk : a.n.wq, a.n.fp32, ck.e0, wa);
    load_weights<T>(part ? a.n.wk : a.n.wq, a.n.fp32, ck.e1, wb);
    for (int h = from; h < to; ++h) {
      uint4 va = make_uint4(0, 0, 0, 0), vb = va;
      if (live) {
        va = *reinterpret_cast<const uint4*>(x + h * in.sh + ck.e0);
        vb = *reinterpret_cast<const uint4*>(x + h * in.sh + ck.e1);
      }
      float xa[8], xb[8];
      up8<T>(va, xa);
      up8<T>(vb, xb);
      const float r = rsqrtf(sum_over(sum_of_squares(xa, xb), ln.per_row) * inv_d + a.n.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xa[i] = xa[i] * r * wa[i];
        xb[i] = xb[i] * r * wb[i];
      }
      if (ck.turned) turn8<kInter>(xa, xb, cs, sn);
      if (live) {
        *reinterpret_cast<uint4*>(y + h * out.sh + ck.e0) = down8<T>(xa);
        *reinterpret_cast<uint4*>(y + h * out.sh + ck.e1) = down8<T>(xb);
      }
    }
  }
}

// The blocks of q and then those of k, each block its share of the (tokens, heads)
// items of its part; what it adds up of dw goes to its row of a.part.
template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads) fa_qk_norm_bwd_kernel(const NormRopeBwdArgs a, int hpb, const DevStatus st) {
  __shared__ Pairs pairs;
  __shared__ float sums[kThreads][17];
  launch_dependents();
  wait_for_previous();
  load_pairs<kThreads>(a.r, pairs, st);
  __syncthreads();
  const Lanes ln(a.d);
  const int part = blockIdx.x >= a.blocks[0], block = blockIdx.x - (part ? a.blocks[0] : 0), H = a.H[part];
  const RowView &dy = a.dy[part], &xv = a.x[part], &dx = a.dx[part];
  const int splits = (H + hpb - 1) / hpb;
  const long long tokens = (long long)a.B * a.N, items = (tokens + ln.tpb - 1) / ln.tpb * splits;
  const bool in_row = ln.c < a.d / 16;
  const Chunk ck = chunk_of<kInter>(in_row ? ln.c : 0, a.r.rot);
  const void* w = part ? a.n.wk : a.n.wq;
  float wa[8], wb[8], da[8] = {}, db[8] = {};
  load_weights<T>(w, a.n.fp32, ck.e0, wa);
  load_weights<T>(w, a.n.fp32, ck.e1, wb);
  const float inv_d = 1.f / a.d;
  for (long long it = block; it < items; it += a.blocks[part]) {
    const long long tb = it / splits, t = tb * ln.tpb + ln.lt;
    const int h0 = (int)(it - tb * splits) * hpb, h1 = min(h0 + hpb, H);
    const bool live = in_row && t < tokens;
    const int b = live ? (int)(t / a.N) : 0, n = live ? (int)(t - (long long)b * a.N) : 0;
    float cs[8] = {}, sn[8] = {};
    if (ck.turned) load_fine_angles(a.r, pairs, a.r.pos + b * a.r.pos_batch + n, in_row ? ln.c : 0, cs, sn);
    const T* x = static_cast<const T*>(xv.p) + b * xv.sb + n * xv.sn;
    const T* g = static_cast<const T*>(dy.p) + b * dy.sb + n * dy.sn;
    T* y = static_cast<T*>(dx.p) + b * dx.sb + n * dx.sn;
    for (int h = h0; h < h1; ++h) {
      uint4 v[4] = {};
      if (live) {
        v[0] = *reinterpret_cast<const uint4*>(x + h * xv.sh + ck.e0);
        v[1] = *reinterpret_cast<const uint4*>(x + h * xv.sh + ck.e1);
        v[2] = *reinterpret_cast<const uint4*>(g + h * dy.sh + ck.e0);
        v[3] = *reinterpret_cast<const uint4*>(g + h * dy.sh + ck.e1);
      }
      float xa[8], xb[8], ga[8], gb[8];
      up8<T>(v[0], xa);
      up8<T>(v[1], xb);
      up8<T>(v[2], ga);
      up8<T>(v[3], gb);
      if (ck.turned) turn8<kInter>(ga, gb, cs, sn);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) dot = fmaf(ga[i] * wa[i], xa[i], fmaf(gb[i] * wb[i], xb[i], dot));
      const float r = rsqrtf(sum_over(sum_of_squares(xa, xb), ln.per_row) * inv_d + a.n.eps);
      const float m = sum_over(dot, ln.per_row) * r * inv_d;        // mean of g w x r
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float ya = xa[i] * r, yb = xb[i] * r;
        da[i] = fmaf(ga[i], ya, da[i]);
        db[i] = fmaf(gb[i], yb, db[i]);
        xa[i] = r * (ga[i] * wa[i] - ya * m);
        xb[i] = r * (gb[i] * wb[i] - yb * m);
      }
      if (live) {
        *reinterpret_cast<uint4*>(y + h * dx.sh + ck.e0) = down8<T>(xa);
        *reinterpret_cast<uint4*>(y + h * dx.sh + ck.e1) = down8<T>(xb);
      }
    }
  }
  if (!a.dw[part]) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sums[threadIdx.x][i] = da[i];
    sums[threadIdx.x][8 + i] = db[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.d; i += kThreads) {
    // The chunk and place of element i.
    int c, j;
    if (!kInter && i < a.r.rot) {
      const int half = a.r.rot / 2, e = i % half;
      c = e / 8;
      j = e % 8 + (i >= half ? 8 : 0);
    } else {
      c = i / 16;
      j = i % 16;
    }
    float s = 0.f;
    for (int t = 0; t < ln.tpb; ++t) s += sums[t * ln.per_row + c][j];
    a.part[(long long)blockIdx.x * a.d + i] = s;
  }
}

// dw from the blocks' sums, in a fixed order: a warp an element of q's or k's.
__global__ void __launch_bounds__(kThreads) fa_qk_norm_dw_kernel(const NormRopeBwdArgs a) {
  launch_dependents();
  wait_for_previous();
  const int i = blockIdx.x * (kThreads / 32) + threadIdx.x / 32, part = blockIdx.y, lane = threadIdx.x % 32;
  if (i >= a.d || !a.dw[part]) return;
  const float* p = a.part + (long long)(part ? a.blocks[0] : 0) * a.d + i;
  float s = 0.f;
  for (int b = lane; b < a.blocks[part]; b += 32) s += p[(long long)b * a.d];
  s = sum_over(s, 32);
  if (lane == 0) a.dw[part][i] = s;
}

int heads_per_block(long long token_blocks, int heads, int num_sms) {
  const long long want = 16LL * num_sms;
  long long splits = (want + token_blocks - 1) / token_blocks;
  if (splits > heads) splits = heads;
  if (splits < 1) splits = 1;
  return (int)((heads + splits - 1) / splits);
}

}  // namespace

cudaError_t configure_norm_kernels() {
  cudaError_t e = preload_kernel(fa_qk_norm_dw_kernel);
  for (auto k : {fa_qk_norm_kernel<__nv_bfloat16, false>, fa_qk_norm_kernel<__nv_bfloat16, true>,
                 fa_qk_norm_kernel<__half, false>, fa_qk_norm_kernel<__half, true>})
    if (e == cudaSuccess) e = preload_kernel(k);
  for (auto k : {fa_qk_norm_bwd_kernel<__nv_bfloat16, false>, fa_qk_norm_bwd_kernel<__nv_bfloat16, true>,
                 fa_qk_norm_bwd_kernel<__half, false>, fa_qk_norm_bwd_kernel<__half, true>})
    if (e == cudaSuccess) e = preload_kernel(k);
  return e;
}

cudaError_t launch_norm_rope(int dtype, const NormRopeArgs& a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  const int tpb = tokens_per_block(a.d), heads = a.Hq + a.Hk;
  const long long blocks = ((long long)a.B * a.N + tpb - 1) / tpb;
  const int hpb = heads_per_block(blocks, heads, num_sms);
  const dim3 grid((unsigned)blocks, (unsigned)((heads + hpb - 1) / hpb));
  auto k = dtype == 0 ? (a.r.interleaved ? fa_qk_norm_kernel<__nv_bfloat16, true> : fa_qk_norm_kernel<__nv_bfloat16, false>)
                      : (a.r.interleaved ? fa_qk_norm_kernel<__half, true> : fa_qk_norm_kernel<__half, false>);
  return launch_after(k, grid, kThreads, 0, 1, stream, a, hpb, st);
}

cudaError_t launch_norm_rope_bwd(int dtype, NormRopeBwdArgs a, const DevStatus& st, int num_sms, cudaStream_t stream) {
  const int tpb = tokens_per_block(a.d), hpb = 4;
  const long long token_blocks = ((long long)a.B * a.N + tpb - 1) / tpb;
  const int most = min(4 * num_sms, kNormBwdMaxBlocks), heads = a.H[0] + a.H[1];
  long long items[2];
  for (int i = 0; i < 2; ++i) items[i] = token_blocks * ((a.H[i] + hpb - 1) / hpb);
  if (items[0] + items[1] <= most) {
    for (int i = 0; i < 2; ++i) a.blocks[i] = (int)items[i];
  } else {
    a.blocks[1] = a.H[1] ? max(1, (int)((long long)most * a.H[1] / heads)) : 0;
    a.blocks[0] = max(1, most - a.blocks[1]);
  }
  auto k = dtype == 0
               ? (a.r.interleaved ? fa_qk_norm_bwd_kernel<__nv_bfloat16, true> : fa_qk_norm_bwd_kernel<__nv_bfloat16, false>)
               : (a.r.interleaved ? fa_qk_norm_bwd_kernel<__half, true> : fa_qk_norm_bwd_kernel<__half, false>);
  cudaError_t e = launch_after(k, a.blocks[0] + a.blocks[1], kThreads, 0, 1, stream, a, hpb, st);
  if (e == cudaSuccess && (a.dw[0] || a.dw[1]))
    e = launch_after(fa_qk_norm_dw_kernel, dim3((a.d + 3) / 4, a.H[1] ? 2 : 1), kThreads, 0, 1, stream, a);
  return e;
}

}  // namespace fa
