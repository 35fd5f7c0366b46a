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

// NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T>
__device__ __forceinline__ float round_to(float x) {
  return Pair2<T>::up(Pair2<T>::down(x, 0.f)).x;
}

// Codes of eight elements, in the two halves of K's word or in V's two halves.
template <bool kKeys>
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], float s, float z) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = __float2int_rn(__fdiv_rn(__fsub_rn(x[e], z), s));
    w |= place_code((uint32_t)min(max(c, 0), 15), kKeys ? e / 2 : e % 4) << 16 * (kKeys ? e % 2 : e / 4);
  }
  return s == 0.f ? 0u : w;
}
template <int D, bool kKeys>
__device__ __forceinline__ void store_codes(uint8_t* rec, int slot, int i, uint32_t w) {
  if constexpr (kKeys) {
    *reinterpret_cast<uint32_t*>(rec + Record<D>::k_word(slot, i)) = w;
  } else {
    *reinterpret_cast<uint16_t*>(rec + Record<D>::v_half(slot, i, 0)) = (uint16_t)w;
    *reinterpret_cast<uint16_t*>(rec + Record<D>::v_half(slot, i, 1)) = (uint16_t)(w >> 16);
  }
}

// One row of K or V, 16 elements a thread, into its record.  All lanes of a row
// take part.
template <typename T, int D, bool kKeys>
__device__ __forceinline__ void store_row(const float (&xa)[8], const float (&xb)[8], const Chunk& ck, uint8_t* rec, int slot, int c,
                                          bool live) {
  constexpr int kGroups = D / 64;
  const int ga = ck.e0 / 64, gb = ck.e1 / 64;
  float lo[kGroups], hi[kGroups];
  float la = xa[0], ha = xa[0], lb = xb[0], hb = xb[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    la = min_nan(la, xa[i]);
    ha = max_nan(ha, xa[i]);
    lb = min_nan(lb, xb[i]);
    hb = max_nan(hb, xb[i]);
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    lo[g] = min_nan(g == ga ? la : INFINITY, g == gb ? lb : INFINITY);
    hi[g] = max_nan(g == ga ? ha : -INFINITY, g == gb ? hb : -INFINITY);
#pragma unroll
    for (int d = 1; d < D / 16; d <<= 1) {
      lo[g] = min_nan(lo[g], __shfl_xor_sync(0xffffffffu, lo[g], d));
      hi[g] = max_nan(hi[g], __shfl_xor_sync(0xffffffffu, hi[g], d));
    }
  }
  float s[kGroups];
  uint32_t p[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    s[g] = round_to<T>(__fdiv_rn(__fsub_rn(hi[g], lo[g]), 15.f));
    p[g] = Pair2<T>::down(s[g], lo[g]);
  }
  if (!live) return;
  const float sa = kGroups == 1 || ga == 0 ? s[0] : s[kGroups - 1], za = kGroups == 1 || ga == 0 ? lo[0] : lo[kGroups - 1];
  const float sb = kGroups == 1 || gb == 0 ? s[0] : s[kGroups - 1], zb = kGroups == 1 || gb == 0 ? lo[0] : lo[kGroups - 1];
  store_codes<D, kKeys>(rec, slot, ck.e0 / 8, encode8<kKeys>(xa, sa, za));
  store_codes<D, kKeys>(rec, slot, ck.e1 / 8, encode8<kKeys>(xb, sb, zb));
  if (c == 0) {
    uint8_t* par = rec + (kKeys ? Record<D>::kKp : Record<D>::kVp);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) reinterpret_cast<uint32_t*>(par + slot * Record<D>::kPar)[g] = p[g];
  }
}

// grid: x over groups of kThreads / (D/16) tokens, y over groups of hpb heads of q,
// then k, then v.
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads) fa_append4_kernel(const Append4Args a, int hpb, const DevStatus st) {
  __shared__ Pairs pairs;
  constexpr int kLanes = D / 16, kTokens = kThreads / kLanes;
  launch_dependents();
  wait_for_previous();
  load_pairs<kThreads>(a.r, pairs, st);
  if (a.cu && blockIdx.y == 0) check_offsets<kThreads>(a, st);
  __syncthreads();
  const int lt = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  const long long t = (long long)blockIdx.x * kTokens + lt;
  int page = 0, slot = 0;
  const bool live = t < a.T && place_token(a, (int)t, st, page, slot);
  const long long tt = live ? t : 0;
  const Chunk ck = chunk_of<kInter>(c, a.r.rot);
  const Chunk plain{16 * c, 16 * c + 8, false};
  const int Hkv = a.kv.Hkv, h0 = blockIdx.y * hpb, h1 = min(h0 + hpb, a.Hq + 2 * Hkv);
  float cs[8] = {}, sn[8] = {};
  if (live && ck.turned && h0 < a.Hq + Hkv) load_fine_angles(a.r, pairs, a.r.pos + t, c, cs, sn);
  uint8_t* at = static_cast<uint8_t*>(a.kv.k) + page * a.kv.s_page + (slot >> 4) * (long long)Record<D>::kBytes;
  const int first[4] = {0, a.Hq, a.Hq + Hkv, a.Hq + 2 * Hkv};
  for (int part = 0; part < 3; ++part) {                  // q, k, v
    const int from = max(h0 - first[part], 0), to = min(h1, first[part + 1]) - first[part];
    if (from >= to) continue;
    const RowView& in = part == 0 ? a.q : part == 1 ? a.k : a.v;
    const Chunk& my = part == 2 ? plain : ck;
    const T* x = static_cast<const T*>(in.p) + tt * in.sn;
    const bool normed = a.n.on && part < 2;
    float wa[8] = {}, wb[8] = {};
    if (normed) {
      load_weights<T>(part ? a.n.wk : a.n.wq, a.n.fp32, my.e0, wa);
      load_weights<T>(part ? a.n.wk : a.n.wq, a.n.fp32, my.e1, wb);
    }
    for (int h = from; h < to; ++h) {
      uint4 va = make_uint4(0, 0, 0, 0), vb = va;
      if (live) {
        va = *reinterpret_cast<const uint4*>(x + h * in.sh + my.e0);
        vb = *reinterpret_cast<const uint4*>(x + h * in.sh + my.e1);
      }
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
      if (part == 0) {
        T* y = static_cast<T*>(a.q_out.p) + tt * a.q_out.sn + h * a.q_out.sh;
        if (live) {
          *reinterpret_cast<uint4*>(y + my.e0) = va;
          *reinterpret_cast<uint4*>(y + my.e1) = vb;
        }
      } else {
        up8<T>(va, xa);
        up8<T>(vb, xb);
        uint8_t* rec = at + h * a.kv.s_head;
        if (part == 1) store_row<T, D, true>(xa, xb, my, rec, slot & 15, c, live);
        else store_row<T, D, false>(xa, xb, my, rec, slot & 15, c, live);
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
