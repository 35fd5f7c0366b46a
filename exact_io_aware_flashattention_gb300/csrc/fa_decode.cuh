// What the kernels that decode over a paged cache share, whatever the cache
// holds: a CTA's way through the line of tiles, and the joining of units that
// were cut over CTAs.
//
// Traits of a kernel: the tensors' type T, the head dimension D, the keys of a tile
// kKeys, the threads of a CTA that join in a cluster kJoinThreads, two fp32
// values rounded to T and packed by pack(lo, hi), and kShift: weights and sums
// are those of 2^(score - max + kShift).
#pragma once

#include "fa_paged.h"
#include "sm103a.cuh"

namespace fa {

namespace {

// Fragments of eight rows of a matrix of 16-bit values as those of its columns.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Visible keys [first, len) of a sequence, as tiles [tile0, tile0 + n) of kKeys.
struct Span {
  int len, first, tile0, n;
};
template <int kKeys>
__device__ __forceinline__ Span span_of_len(const DecodeArgs& a, int len) {
  Span s;
  s.len = len;
  if (s.len < 0 || s.len > (long long)a.table.cols * a.kv.page_size) s.len = -1;   // recorded by the caller
  s.first = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
  s.tile0 = s.first / kKeys;
  s.n = s.len > 0 ? (s.len - 1) / kKeys - s.tile0 + 1 : 0;
  return s;
}
template <int kKeys>
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b) {
  return span_of_len<kKeys>(a, a.seq_lens[b]);
}

// The line of `total` tiles is cut into min(total, CTAs) parts: none is empty.
// Start of part i, and the part a tile belongs to.
__device__ __forceinline__ long long part_start(long long total, int i, int parts) { return total * i / parts; }
__device__ __forceinline__ int part_of(long long tile, long long total, int parts) {
  return (int)(((tile + 1) * parts - 1) / total);
}

// A CTA's way through its part: unit (b, column), tile within the unit.
template <int kKeys>
struct Walk {
  int b, col, tile;
  Span s;
  long long left;      // tiles of the part from here on
  // On to the unit after this one.
  __device__ __forceinline__ void next_unit(const DecodeArgs& a, int cols) {
    tile = 0;
    if (++col < cols) return;
    col = 0;
    do {
      if (++b >= a.B) {
        left = 0;
        return;
      }
      s = span_of<kKeys>(a, b);
    } while (s.n == 0);
  }
  __device__ __forceinline__ void next(const DecodeArgs& a, int cols) {
    --left;
    if (++tile == s.n && left > 0) next_unit(a, cols);
  }
};

// Sequences without visible keys: O = 0, LSE = -inf.  One warp of each CTA
// takes every gridDim.x-th sequence.
template <typename Tr>
__device__ __forceinline__ void fill_empty(const DecodeArgs& a) {
  constexpr int D = Tr::D;
  const int lane = threadIdx.x & 31;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (span_of<Tr::kKeys>(a, b).n > 0) continue;
    uint4* o = reinterpret_cast<uint4*>(static_cast<typename Tr::T*>(a.o) + (long long)b * a.Hq * D);
    for (int i = lane; i < a.Hq * (D / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
    for (int i = lane; i < a.Hq; i += 32) a.lse[(long long)b * a.Hq + i] = -INFINITY;
  }
}

// A unit whose tiles a cluster shared: each CTA left its share's O [16][D] and
// (max, sum) [16] in its shared memory.  The threads of all CTAs take two
// elements of a head each.
template <int D>
constexpr uint32_t kClusterMl = 16u * D * 4u;
template <typename Tr>
__device__ __forceinline__ void join_cluster(const DecodeArgs& a, const uint8_t* smem, const Walk<Tr::kKeys>& w, int rank, int h0,
                                             int h1) {
  constexpr int D = Tr::D, kThreads = Tr::kJoinThreads;
  for (int i = rank * kThreads + threadIdx.x; i < (h1 - h0) * (D / 2); i += a.cluster * kThreads) {
    const int hh = i / (D / 2), d = i % (D / 2) * 2;
    float2 y[kMaxCluster], x[kMaxCluster];         // all loads in flight before the first is used
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      const int from = r < a.cluster ? r : rank;
      y[r] = ld_cluster2(reinterpret_cast<const float2*>(smem + kClusterMl<D>) + hh, from);
      x[r] = ld_cluster2(reinterpret_cast<const float2*>(smem + (hh * D + d) * 4), from);
    }
    float m = -INFINITY, l = 0.f;
    float2 o = make_float2(0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) m = fmaxf(m, y[r].x);
    const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < a.cluster) {
        const float f = ex2(y[r].x - mu);
        l = fmaf(f, y[r].y, l);
        o.x = fmaf(f, x[r].x, o.x);
        o.y = fmaf(f, x[r].y, o.y);
      }
    const long long row = (long long)w.b * a.Hq + h0 + hh;
    const bool none = w.s.n == 0;                  // no visible keys
    const float inv = none ? 0.f : 1.f / l;
    *reinterpret_cast<uint32_t*>(static_cast<typename Tr::T*>(a.o) + row * D + d) = Tr::pack(o.x * inv, o.y * inv);
    if (d == 0) a.lse[row] = none ? -INFINITY : (m + (log2f(l) - Tr::kShift)) * 0.69314718055994530942f;
  }
}

// Where part i left head hh of a unit whose first part is i0: in the part's
// last unit if that is where the unit starts, else in its first.
__device__ __forceinline__ long long left_at(int i, int i0, int hh) {
  return ((long long)i * 2 + (i == i0 ? 1 : 0)) * 16 + hh;
}

// Joins the units that were cut:
//   O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i, m = max_i m_i.
// Only the boundaries between two parts cut units, whatever the batch:
// unit_heads / 4 blocks for each boundary.  The blocks of a unit's boundaries
// share its heads: a warp per head where there are fewer blocks than heads
// (units over few parts), else a block per head, or up to D / 32 blocks per
// head, each with a slice of D.
// Parts are taken 16 bytes of O a thread, as many at a time as the block has
// threads for its slice; the order of the sums depends on the sizes alone.
template <typename Tr>
__device__ __forceinline__ void write_row(const DecodeArgs& a, long long row, int d0, const float4& o, float m, float l) {
  constexpr int D = Tr::D;
  const float inv = 1.f / l;
  *reinterpret_cast<uint2*>(static_cast<typename Tr::T*>(a.o) + row * D + d0) =
      make_uint2(Tr::pack(o.x * inv, o.y * inv), Tr::pack(o.z * inv, o.w * inv));
  if (d0 == 0) {
    const float lse2 = m + (log2f(l) - Tr::kShift);
    a.lse[row] = lse2 * 0.69314718055994530942f;
    if (a.lse2) a.lse2[row] = lse2;
  }
}
__device__ __forceinline__ void add_scaled(float4& o, float f, const float4& v) {
  o.x = fmaf(f, v.x, o.x);
  o.y = fmaf(f, v.y, o.y);
  o.z = fmaf(f, v.z, o.z);
  o.w = fmaf(f, v.w, o.w);
}
template <typename Tr>
__device__ __forceinline__ void join(const DecodeArgs& a) {
  constexpr int D = Tr::D;
  __shared__ float sf[kDecodeMaxParts], sm[4], sl[4];
  __shared__ float4 so[128];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Y = a.unit_heads / 4, i = 1 + blockIdx.x / Y;
  const DecodePart d = a.parts[i];
  if (d.left == 0 || d.tile == 0) return;    // no such part, or it starts with a unit
  const int G = a.Hq / a.kv.Hkv, per = a.unit_heads, chunks = (G + per - 1) / per;
  const int g = d.col / chunks, hc = d.col - g * chunks, heads = min(per, G - hc * per);
  const int i0 = d.i0, n = d.i1 - i0 + 1, blocks = (n - 1) * Y, z = (i - i0 - 1) * Y + blockIdx.x % Y;
  const long long row0 = (long long)d.b * a.Hq + g * G + hc * per;
  if (blocks < heads) {
    // A warp per head, D / 4 lanes: few parts.
    const int hh = z * 4 + warp;
    if (hh >= heads) return;
    float m = -INFINITY, l = 0.f;
    for (int x = lane; x < n; x += 32) m = fmaxf(m, a.part_ml[left_at(i0 + x, i0, hh)].x);
    for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    const float mu = m == -INFINITY ? 0.f : m;
    if (lane >= D / 4) return;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = 0; x < n; ++x) {
      const long long at = left_at(i0 + x, i0, hh);
      const float2 y = a.part_ml[at];
      const float f = ex2(y.x - mu);
      l = fmaf(f, y.y, l);
      add_scaled(o, f, *reinterpret_cast<const float4*>(a.part + at * D + lane * 4));
    }
    write_row<Tr>(a, row0 + hh, lane * 4, o, m, l);
    return;
  }
  int slices = D / 32;
  while (slices > 1 && slices * heads > blocks) slices /= 2;
  if (z >= heads * slices) return;
  const int hh = z / slices, lanes = D / 4 / slices, groups = 128 / lanes;
  const int d0 = (z - hh * slices) * (D / slices) + tid % lanes * 4, group = tid / lanes;
  // Scale and sum of every part.
  float2 y[(kDecodeMaxParts + 127) / 128];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int u = 0; u < (kDecodeMaxParts + 127) / 128; ++u) {
    const int x = u * 128 + tid;
    y[u] = x < n ? a.part_ml[left_at(i0 + x, i0, hh)] : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, y[u].x);
  }
  for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  if (lane == 0) sm[warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int u = 0; u < (kDecodeMaxParts + 127) / 128; ++u) {
    const int x = u * 128 + tid;
    const float f = ex2(y[u].x - mu);
    if (x < n) sf[x] = f;
    l = fmaf(f, y[u].y, l);
  }
  for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  if (lane == 0) sl[warp] = l;
  __syncthreads();
  l = (sl[0] + sl[1]) + (sl[2] + sl[3]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int x = group; x < n; x += groups)
    add_scaled(o, sf[x], *reinterpret_cast<const float4*>(a.part + left_at(i0 + x, i0, hh) * D + d0));
  so[tid] = o;
  __syncthreads();
  if (group > 0) return;
  for (int k = 1; k < groups; ++k) add_scaled(o, 1.f, so[k * lanes + tid]);
  write_row<Tr>(a, row0 + hh, d0, o, m, l);
}

}  // namespace

}  // namespace fa
