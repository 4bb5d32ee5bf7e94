// Internal interface of the projection with adapters (linear.cu, linear_narrow.cu, linear_wide.cu).
#pragma once

#include "kernels.h"

namespace mlk {

constexpr int kMaxStackedRanks = 4096;   // columns of the stacked adapters: 64 blocks of 64
constexpr int kAdapterBlock = 64;
constexpr int kFloatPieces = 3;          // bf16 pieces that carry a float32 (8 significant bits each)
constexpr int kMarkWords = 8;            // 16-bit words of a row's marks, 8 slots each

// Where each slot sits among the stacked adapter columns, and its factor; a slot that adds
// nothing (rank 0, factor 0) has hi = lo.
struct LinearSlots {
  int S;
  uint16_t lo[kMaxSlots], hi[kMaxSlots];   // columns [lo, hi)
  float scal[kMaxSlots];
};

struct LinearParams {
  CUtensorMap tmap_w;    // weights [N, K]
  CUtensorMap tmap_x;    // [T, K]
  CUtensorMap tmap_xs;   // (narrow) the same with the shrink's token tile
  CUtensorMap tmap_a;    // the stacked A [Rs, K]
  CUtensorMap tmap_b;    // the stacked B [N, Rs]
  CUtensorMap tmap_u;    // the shrunk rows [T, pieces * Rs]
  CUtensorMap tmap_y;    // (wide tiles, y_vec) [T, N], boxes of 32 tokens x 128 bytes
  int T, N, K;
  int Rs;                // stacked columns, a multiple of 64 (0: no adapters)
  // bf16 pieces of u: one for a bf16 y, whose own rounding (2^-9) hides that of the adapters' part (T 64, N 5120,
  // K 2048, ranks 8 to 64: 0.00167 off in the 2-norm, 0.00166 with a float32 u), kFloatPieces for a float32 y
  int pieces;
  int token_tiles;
  int shrink_slices;     // (wide) pairs that share a shrink tile's K, 1 to kLinearMaxSlices
  int shrink_spread;     // (wide) shrink tiles that go round all pairs, the first ones
  float* part;           // (wide, slices) their part sums, 1024 bytes per tile and column
  int k_slices;          // (wide) pairs that share a product tile's K: 1 or 2
  int shrink_tokens;     // (narrow) tokens of a shrink tile, a divisor of the token tile
  const int32_t* slot_idx;
  const float* bias;     // [N] or null
  void* y;               // [T, ldy] bf16 or float32
  __nv_bfloat16* u;      // [T, pieces * Rs]
  long long ldy;
  int y_f32;
  int y_vec;             // rows of y start on 4-value boundaries (vector stores); wide tiles: on
                         // 16-byte boundaries (TMA stores)
  int2* flags;           // per token tile: {shrink parts done, product parts past them}, and after
                         // these (slices) {part sums written, unused}; zero between calls
  uint32_t* status;      // written by the first CTA
  const unsigned long long* sick;   // slots with weights that are not finite (linear_nonfinite.cuh)
  LinearSlots slots;
  // From here on what few calls read.
  const uint16_t* marks;   // of row n: marks + n * mark_stride; slot s: bit s % 8 of word s / 8
  int mark_stride;
  const __nv_bfloat16* b;  // the stacked B, in which a marked slot's values of that row are classes
  int accs, acc_steps;     // (narrow, cluster) accumulators in TMEM of a CTA's K, and 64-wide blocks of each
};
constexpr int kLinearFlags = 8192;   // token tiles of a call with adapters
constexpr int kLinearMaxSlices = 8;

// One 128-row x bn-token tile per cluster of `split` CTAs, which share the tile's K; split is at
// most the number of 64-wide K blocks.  Maps' boxes: {64, 128} of w, a, b, {64, bn} of
// x and u, {64, shrink_tokens} of xs.
constexpr int kLinearMaxSplit = 8;
constexpr int kLinearTmem = 256;     // TMEM columns of a CTA at most: two share an SM's 512
inline __host__ __device__ unsigned linear_tmem_columns(int accs, int columns) {   // a power of two from 32
  unsigned n = 32;
  while (n < static_cast<unsigned>(accs * columns)) n *= 2;
  return n;
}
cudaError_t linear_narrow_setup();   // once per device
cudaError_t launch_linear_narrow(const LinearParams& p, int bn, int split, cudaStream_t stream);

// The same tiles (bn 16 or 32) with at most 128 stacked columns, each cluster shrinking for
// itself.  Maps' boxes: {64, 128} of w and b, {64, 64} of a, {64, bn} of x.
cudaError_t linear_cluster_setup();
cudaError_t launch_linear_cluster(const LinearParams& p, int bn, int split, cudaStream_t stream);

// What the choice of tiles goes by of a device: its SMs, and the pairs of SMs that run at one time in
// clusters of two pairs (which stay within a GPC, so not every SM finds a place in one).
struct LinearMachine {
  int sms, pairs_by_two;
  int pairs(int k_slices) const { return k_slices == 1 || pairs_by_two > sms / 2 ? sms / 2 : pairs_by_two; }
};

// Tiles of 256 tokens x bn (128, 192 or 256; float32 y: 128) weight rows on CTA pairs.  Maps' boxes: {64, 128}
// of x and u, {64, bn / 2} of w and b, {64, linear_shrink_cols(Rs, bn) / 2} of a.
cudaError_t linear_wide_setup(int* pairs_by_two);
cudaError_t launch_linear_wide(const LinearParams& p, int bn, const LinearMachine& m, cudaStream_t stream);
inline __host__ __device__ int linear_shrink_cols(int Rs, int bn) { return Rs < bn ? Rs : bn; }   // per shrink tile

struct LinearPackParams {
  const __nv_bfloat16 *A, *B;   // [S, R, K], [S, N, R]
  __nv_bfloat16 *Ap, *Bp;       // [Rs, K], [N, Rs]
  unsigned long long* sick;     // (as in LinearParams; zero before the kernel)
  uint16_t* marks;
  int mark_stride;
  int S, N, K, R, Rs;
  uint16_t lo[kMaxSlots + 1];   // first column of each slot, lo[S] = the end of the last
  uint16_t ranks[kMaxSlots];
};
cudaError_t launch_linear_pack(const LinearPackParams& p, cudaStream_t stream);

}  // namespace mlk
