// Internal launcher interface of the normed rotary positions (fa_qknorm.cu) and
// of the cache held in 4 bits (fa_append4.cu, fa_decode4.cu), between the C-ABI
// layer (fa_api.cu) and the kernels.  Nothing here is exported.
#pragma once

#include "fa_paged.h"

namespace fa {

enum : int { kSiteReadLen = 50, kSiteReadPage = 51, kSiteDecode4Len = 52, kSiteDecode4Page = 53 };

// Norm of each head's rows: x (mean x^2 + eps)^-1/2 w.
struct NormArgs {
  const void* wq;            // [d] each, fp32 or the call's type; NULL: ones
  const void* wk;
  int fp32;
  int on;                    // 0: no norm
  float eps;
};

struct NormRopeArgs {
  RowView q, q_out, k, k_out;
  int B, Hq, Hk, N, d;
  RotaryArgs r;              // rot = 0: nothing is turned
  NormArgs n;
};

struct NormRopeBwdArgs {
  RowView dy[2], x[2], dx[2];   // q, k
  int H[2];
  int B, N, d;
  RotaryArgs r;              // inverse
  NormArgs n;
  float* dw[2];              // [d], NULL: not wanted
  float* part;               // [blocks][d], the blocks of q and then those of k
  int blocks[2];
};

// Blocks of the backward kernel at most (its workspace has a row for each).
constexpr int kNormBwdMaxBlocks = 2048;

cudaError_t launch_norm_rope(int dtype, const NormRopeArgs& a, const DevStatus& st, int num_sms, cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(int dtype, NormRopeBwdArgs a, const DevStatus& st, int num_sms, cudaStream_t stream);

// The 4-bit cache.  16 slots of a page and kv head form a record of 18 d bytes:
// K codes [16][d/2], V codes, as many bytes, (s, z) of K and of V, [16][d/64] pairs
// of the call's type each.  A page's records follow one another.
//   Codes lie in 16-bit halves of four, place n at bits 9-6, 5-2, and these two with
// the half's bytes swapped (so bits 1, 0, 15, 14 and 13-10), and two halves in a
// word are a pair of operands of a matrix product, which one mask makes fp16
// numbers of: of K neighbouring elements of d, of V two keys.
//   K: a row's word i holds elements 8 i .. 8 i + 7, element e in place e / 2 of
// half e % 2.  At d = 128 word i of both groups stand side by side, at 8-byte chunk i
// ^ 4 ((slot / 2) % 2): lanes that read 16 bytes of eight rows each then meet all
// banks of shared memory alike.
//   V: group by group, 16 bytes for each lane of a warp.  Lane 4 r + c has the
// elements 8 r .. 8 r + 7 of the slots c, c + 4, c + 8 and c + 12: four words, of
// the slots (c, c + 4) and then (c + 8, c + 12) the elements 8 r .. 8 r + 3 and then
// the other four, the first slot in the lower half.
template <int D>
struct Record {
  static constexpr int kRow = D / 2;                 // bytes of a row's codes
  static constexpr int kV = 16 * kRow, kKp = 32 * kRow, kPar = D / 64 * 4, kVp = kKp + 16 * kPar;
  static constexpr int kBytes = kVp + 16 * kPar;
  static_assert(kBytes == 18 * D, "record");
  // Byte of word i of a slot's row of K.
  static __host__ __device__ constexpr int k_word(int slot, int i) {
    return slot * kRow + (D == 128 ? (((i & 7) ^ ((slot & 2) << 1)) << 3) + ((i >> 3) << 2) : i << 2);
  }
  // Byte of the half that holds elements 8 i + 4 h .. 8 i + 4 h + 3 of a slot's row of V.
  static __host__ __device__ constexpr int v_half(int slot, int i, int h) {
    return kV + (i >> 3) * 512 + ((i & 7) * 4 + (slot & 3)) * 16 + (slot >> 3) * 8 + h * 4 + ((slot >> 2) & 1) * 2;
  }
};

struct Append4Args {
  RowView q, q_out, k, v;    // tokens as N (sb unused); q.p NULL: no q
  PagedKv kv;                // k: the records; strides in bytes
  PageTable table;
  const int* seq_lens;
  const int* cu;             // [B + 1] or NULL
  int B, T, Hq;
  RotaryArgs r;              // rot = 0: nothing is turned
  NormArgs n;
};

struct Read4Args {
  PagedKv kv;
  PageTable table;
  const int* seq_lens;
  RowView k, v;
  int B, N;
};

// Keys of a tile of the decode kernel, by equal parts of the line of tiles (two records
// a warp, whose products take turns) and by clusters (one, as their units are short); and
// the CTAs that an SM holds, by the heads of a unit.
constexpr int kDecode4TileKeys = 256, kDecode4ClusterKeys = 128;
constexpr int decode4_ctas_per_sm(int unit_heads) { return unit_heads == 8 ? 2 : 1; }

cudaError_t launch_append4(int dtype, const Append4Args& a, const DevStatus& st, int num_sms, cudaStream_t stream);
cudaError_t launch_read4(int dtype, const Read4Args& a, const DevStatus& st, int num_sms, cudaStream_t stream);
cudaError_t launch_decode4(int dtype, const DecodeArgs& a, const DevStatus& st, int parts, cudaStream_t stream);

cudaError_t configure_norm_kernels();
cudaError_t configure_append4_kernels();
cudaError_t configure_decode4_kernels();

inline cudaError_t configure_paged4_kernels() {
  cudaError_t e = configure_norm_kernels();
  if (e == cudaSuccess) e = configure_append4_kernels();
  if (e == cudaSuccess) e = configure_decode4_kernels();
  return e;
}

}  // namespace fa
