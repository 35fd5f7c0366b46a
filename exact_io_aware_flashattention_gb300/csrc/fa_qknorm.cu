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
// lanes, d / 16 rounded up to a power of two.  Vectors are copied to shared memory
// three rows ahead (four in the gradient, 32 KB a block, three blocks an SM at 152
// registers), since loads into registers kept too few bytes on their way: the
// forward 31.2 -> 24.9 us, the gradient 210 -> 87.  4 x 2048 tokens of 32 heads, d = 128,
// bf16, 134 MB: 25.0 us, 5.4 TB/s; the gradient of 2 x 8192 tokens of 40 heads, 503 MB,
// 84.6 us, 5.9 TB/s (outputs of twelve calls in turn, so that all of it is written back).
// Small calls are the latency of a load, the angles and a store, 3.3 us (8 + 2 heads of
// 513 tokens, d = 64), and of the gradient's second kernel, 6.1.
#include "fa_paged4.h"
#include "fa_rotary.cuh"
#include "sm103a.cuh"

#include <algorithm>
#include <climits>

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

constexpr int kSlots = 3, kSlotsBwd = 4;
constexpr int kBwdBlocks = 3;                      // of the backward kernel an SM

// grid: x over groups of tpb tokens, y over groups of hpb heads of q and then k.
// The first rows are on their way while the angles are formed.
template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads, 7) fa_qk_norm_kernel(const NormRopeArgs a, int hpb, const DevStatus st) {
  __shared__ Pairs pairs;
  __shared__ uint4 ring[kSlots][2][kThreads];
  launch_dependents();
  wait_for_previous();
  const Lanes ln(a.d);
  const long long t = (long long)blockIdx.x * ln.tpb + ln.lt;
  const bool live = ln.c < a.d / 16 && t < (long long)a.B * a.N;
  const int b = live ? (int)(t / a.N) : 0, n = live ? (int)(t - (long long)b * a.N) : 0;
  const Chunk ck = chunk_of<kInter>(live ? ln.c : 0, a.r.rot);
  const int h0 = blockIdx.y * hpb, h1 = min(h0 + hpb, a.Hq + a.Hk);
  const T* q = static_cast<const T*>(a.q.p) + b * a.q.sb + n * a.q.sn;
  const T* k = static_cast<const T*>(a.k.p) + b * a.k.sb + n * a.k.sn;
  auto copy = [&](int h, int slot) {
    if (live && h < h1) {
      const T* x = h < a.Hq ? q + h * a.q.sh : k + (h - a.Hq) * a.k.sh;
      copy16(&ring[slot][0][threadIdx.x], x + ck.e0);
      copy16(&ring[slot][1][threadIdx.x], x + ck.e1);
    }
    copies_end();
  };
#pragma unroll
  for (int s = 0; s < kSlots; ++s) copy(h0 + s, s);
  load_pairs<kThreads>(a.r, pairs, st);
  __syncthreads();
  float cs[8] = {}, sn[8] = {};
  if (ck.turned) load_angles(a.r, pairs, a.r.pos + b * a.r.pos_batch + n, live ? ln.c : 0, cs, sn);
  const float inv_d = 1.f / a.d;
  int slot = 0, h = h0;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int end = part ? h1 : min(h1, a.Hq);
    if (h >= end) continue;
    const RowView& out = part ? a.k_out : a.q_out;
    T* y = static_cast<T*>(out.p) + b * out.sb + n * out.sn + (h - (part ? a.Hq : 0)) * out.sh;
    float wa[8], wb[8];
    load_weights<T>(part ? a.n.wk : a.n.wq, a.n.fp32, ck.e0, wa);
    load_weights<T>(part ? a.n.wk : a.n.wq, a.n.fp32, ck.e1, wb);
#pragma unroll 1
    for (; h < end; ++h, y += out.sh) {
      copies_wait<kSlots - 1>();
      uint4 va = make_uint4(0, 0, 0, 0), vb = va;
      if (live) {
        va = ring[slot][0][threadIdx.x];
        vb = ring[slot][1][threadIdx.x];
      }
      float xa[8], xb[8];
      up8<T>(va, xa);
      up8<T>(vb, xb);
      const float r = rsqrtf(sum_over(sum_of_squares(xa, xb), ln.per_row) * inv_d + a.n.eps);
      copy(h + kSlots, slot);
      slot = slot + 1 == kSlots ? 0 : slot + 1;
      scale8(xa, r, wa);
      scale8(xb, r, wb);
      if (ck.turned) turn8<kInter>(xa, xb, cs, sn);
      if (live) {
        __stcs(reinterpret_cast<uint4*>(y + ck.e0), down8<T>(xa));
        __stcs(reinterpret_cast<uint4*>(y + ck.e1), down8<T>(xb));
      }
    }
  }
}

// The blocks of q and then those of k.  A block has a run of at most hpb heads of its
// part and every so many groups of tpb tokens; what it adds up of dw goes to its
// row of a.part.
template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) fa_qk_norm_bwd_kernel(const NormRopeBwdArgs a, int hpb, const DevStatus st) {
  __shared__ Pairs pairs;
  __shared__ uint4 ring[kSlotsBwd][4][kThreads];
  launch_dependents();
  wait_for_previous();
  load_pairs<kThreads>(a.r, pairs, st);
  __syncthreads();
  const Lanes ln(a.d);
  const int part = blockIdx.x >= a.blocks[0], block = blockIdx.x - (part ? a.blocks[0] : 0), H = a.H[part];
  const RowView &dy = a.dy[part], &xv = a.x[part], &dx = a.dx[part];
  const int splits = (H + hpb - 1) / hpb, h0 = block % splits * hpb, heads = min(hpb, H - h0);
  // (The launcher gives each part a multiple of its splits in blocks.)
  const int step = a.blocks[part] / splits * ln.tpb;
  const long long tokens = (long long)a.B * a.N;
  const bool in_row = ln.c < a.d / 16;
  const Chunk ck = chunk_of<kInter>(in_row ? ln.c : 0, a.r.rot);
  const void* w = part ? a.n.wk : a.n.wq;
  float wa[8], wb[8], da[8] = {}, db[8] = {};
  load_weights<T>(w, a.n.fp32, ck.e0, wa);
  load_weights<T>(w, a.n.fp32, ck.e1, wb);
  const float inv_d = 1.f / a.d;

  // t0: the block's first token of a group.  A thread's rows are copied kSlotsBwd
  // heads ahead of the work, into the next group where the heads end.
  const long long first = (long long)(block / splits) * ln.tpb;
  long long to_t0 = first;
  int to_h = 0;
  const T *px = nullptr, *pg = nullptr;
  auto aim = [&]() {
    const long long t = to_t0 + ln.lt;
    px = nullptr;
    if (in_row && t < tokens) {
      const int b = (int)(t / a.N), n = (int)(t - (long long)b * a.N);
      px = static_cast<const T*>(xv.p) + b * xv.sb + n * xv.sn + h0 * xv.sh;
      pg = static_cast<const T*>(dy.p) + b * dy.sb + n * dy.sn + h0 * dy.sh;
    }
  };
  auto copy = [&](int slot) {
    if (px) {
      copy16(&ring[slot][0][threadIdx.x], px + ck.e0);
      copy16(&ring[slot][1][threadIdx.x], px + ck.e1);
      copy16(&ring[slot][2][threadIdx.x], pg + ck.e0);
      copy16(&ring[slot][3][threadIdx.x], pg + ck.e1);
      px += xv.sh;
      pg += dy.sh;
    }
    copies_end();
    if (++to_h == heads) {
      to_h = 0;
      to_t0 += step;
      aim();
    }
  };
  aim();
#pragma unroll
  for (int s = 0; s < kSlotsBwd; ++s) copy(s);
  int slot = 0;
#pragma unroll 1
  for (long long t0 = first; t0 < tokens; t0 += step) {
    const long long t = t0 + ln.lt;
    const bool live = in_row && t < tokens;
    const int b = live ? (int)(t / a.N) : 0, n = live ? (int)(t - (long long)b * a.N) : 0;
    float cs[8] = {}, sn[8] = {};
    if (ck.turned) load_angles(a.r, pairs, a.r.pos + b * a.r.pos_batch + n, in_row ? ln.c : 0, cs, sn);
    T* y = static_cast<T*>(dx.p) + b * dx.sb + n * dx.sn + h0 * dx.sh;
#pragma unroll 1
    for (int h = 0; h < heads; ++h, y += dx.sh) {
      copies_wait<kSlotsBwd - 1>();
      uint4 v[4] = {};
      if (live) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ring[slot][i][threadIdx.x];
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
      copy(slot);
      slot = slot + 1 == kSlotsBwd ? 0 : slot + 1;
      if (live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float ya = xa[i] * r, yb = xb[i] * r;
          da[i] = fmaf(ga[i], ya, da[i]);
          db[i] = fmaf(gb[i], yb, db[i]);
          xa[i] = r * (ga[i] * wa[i] - ya * m);
          xb[i] = r * (gb[i] * wb[i] - yb * m);
        }
        __stcs(reinterpret_cast<uint4*>(y + ck.e0), down8<T>(xa));
        __stcs(reinterpret_cast<uint4*>(y + ck.e1), down8<T>(xb));
      }
    }
  }
  if (!a.dw[part]) return;
  copies_wait<0>();
  __syncthreads();
  float(*sums)[17] = reinterpret_cast<float(*)[17]>(ring);
  static_assert(sizeof(ring) >= sizeof(float[kThreads][17]), "room for the sums");
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
  float s = 0.f, lost = 0.f;                       // (Kahan's sum: fp64 adds took 3-6 us more)
#pragma unroll 4
  for (int b = lane; b < a.blocks[part]; b += 32) {
    const float x = __fsub_rn(p[(long long)b * a.d], lost), y = __fadd_rn(s, x);
    lost = __fsub_rn(__fsub_rn(y, s), x);
    s = y;
  }
  for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane == 0) a.dw[part][i] = s;
}

// Heads per block of the forward, which share their angles: as few blocks as run at a
// time, seven an SM, so that small calls have no second wave; but eight heads at most, as
// at the end SMs wait for one block's time at most, and a block of fewer heads is shorter
// (of six, it forms its angles too often); and a head a block only where that is no more than five an SM.  us a call, outputs
// of twelve calls in turn, d = 128: by 7 | 10 blocks an SM 1024 tokens of 40 heads 6.9 | 8.4,
// 2048 of 40 10.7 | 12.1, 4096 of 40 18.9 | 18.1 (the worst), 8192 of 40 29.7 | 29.8; with
// 6 | 8 | 11 | all heads a block 4 x 2048 of 32 heads 25.1 | 25.0 | 26.0 | 26.0, 32768 of 40
// heads 103.5 | 100.8 | 101.6 | 111.1; 512 of 40 heads with one | two 7.9 | 5.5.
int heads_per_block(long long token_blocks, int heads, int num_sms) {
  const long long want = 7LL * num_sms;
  const long long splits = std::min<long long>(std::max<long long>((want + token_blocks - 1) / token_blocks, (heads + 7) / 8), heads);
  const int hpb = (int)((heads + splits - 1) / splits);
  return hpb == 1 && token_blocks * heads > 5LL * num_sms ? 2 : hpb;
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
  const int tpb = tokens_per_block(a.d);
  const long long token_blocks = ((long long)a.B * a.N + tpb - 1) / tpb;
  const int most = min(kBwdBlocks * num_sms, kNormBwdMaxBlocks);
  // Heads of a block, which share their angles: what takes the busiest block least, a
  // group of tokens counted as its heads and two more for the angles (2048 tokens of 32 +
  // 8 heads: one head a block 32 us, four 20).
  int hpb = 1;
  long long least = LLONG_MAX;
  for (int n = 1; n <= 8; ++n) {
    int splits[2], blocks[2] = {};
    long long cost[2], all = 0, time = 0;
    for (int i = 0; i < 2; ++i) {
      splits[i] = (a.H[i] + n - 1) / n;
      cost[i] = min(n, a.H[i]) + 2;
      all += splits[i] * cost[i];
    }
    for (int i = 0; i < 2; ++i) {
      // The part's share of the blocks by its cost, a multiple of its splits, no more
      // than it has groups for and at least one a split.
      if (splits[i] == 0) continue;
      const long long share = max(1LL, min(most * cost[i] / all, token_blocks));
      blocks[i] = (int)(splits[i] * share);
      time = max(time, (token_blocks + share - 1) / share * cost[i]);
    }
    if (n < 8 && blocks[0] + blocks[1] > most) continue;               // more than run at a time
    if (time < least) {
      least = time;
      hpb = n;
      a.blocks[0] = blocks[0];
      a.blocks[1] = blocks[1];
    }
  }
  if (a.blocks[0] + a.blocks[1] > kNormBwdMaxBlocks) {
    // More heads than eight for each of these: a block for all heads of a part.
    hpb = max(a.H[0], a.H[1]);
    for (int i = 0; i < 2; ++i) a.blocks[i] = a.H[i] ? (int)min(token_blocks, (long long)max(1, most / 2)) : 0;
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
