// Internal interface of the projection with adapters (linear.cu, linear_narrow.cu, linear_wide.cu).
#pragma once

#include "kernels.h"

namespace mlk {

constexpr int kMaxStackedRanks = 4096;   // columns of the stacked adapters: 64 blocks of 64
constexpr int kAdapterBlock = 64;
constexpr int kFloatPieces = 3;          // bf16 pieces that carry a float32 (8 significant bits each)

// Where each slot sits among the stacked adapter columns, and its factor; a slot that adds
// nothing (rank 0, factor 0) has hi = lo.
struct LinearSlots {
  int S;
  uint16_t lo[kMaxSlots], hi[kMaxSlots];   // columns [lo, hi)
  float scal[kMaxSlots];
};

struct LinearParams {
  CUtensorMap tmap_w;    // [rows, K] box {64, 128}: weights, or the stacked A of the shrink
  CUtensorMap tmap_x;    // [T, K] box {64, token tile}
  CUtensorMap tmap_b;    // [N, Rs] box {64, 128}: the stacked B
  CUtensorMap tmap_u;    // [T, pieces * Rs] box {64, token tile}: the shrunk rows
  CUtensorMap tmap_y;    // (wide tiles, y_vec) [T, N] box {64, 32}
  int T, N, K;           // N: rows of tmap_w that count
  int Rs;                // stacked columns, a multiple of 64 (0: no adapters)
  int pieces;            // 1, or kFloatPieces bf16 pieces of a float32 u
  int window;            // (shrink) tokens whose slots decide which stacked rows are needed
  const int32_t* slot_idx;
  const float* bias;     // [N] or null
  void* y;               // [T, ldy] bf16 or float32; the shrink writes u [T, pieces * Rs] bf16
  long long ldy;
  int y_f32;
  int y_vec;             // rows of y start on 4-value boundaries (vector stores); wide tiles: on
                         // 16-byte boundaries (TMA stores)
  int token_tiles;
  int check_slots;       // this launch writes the status word (first CTA)
  uint32_t* status;
  LinearSlots slots;
};

enum { kLinOut = 0, kLinShrink = 1 };

// One 128-row x bn-token tile per cluster of `split` CTAs, which share the tile's K; split is at
// most the number of 64-wide K blocks.
constexpr int kLinearMaxSplit = 8;
cudaError_t linear_narrow_setup();   // once per device
cudaError_t launch_linear_narrow(const LinearParams& p, int mode, int bn, int split, cudaStream_t stream, bool pdl);

// Tiles of 256 tokens x bn (128 or 256) weight rows on CTA pairs, bf16 y; the maps' boxes are
// {64, 128} tokens and {64, bn / 2} weight rows.
cudaError_t linear_wide_setup();
cudaError_t launch_linear_wide(const LinearParams& p, int bn, int sms, cudaStream_t stream, bool pdl);

struct LinearPackParams {
  const __nv_bfloat16 *A, *B;   // [S, R, K], [S, N, R]
  __nv_bfloat16 *Ap, *Bp;       // [Rs, K], [N, Rs]
  int S, N, K, R, Rs;
  uint16_t lo[kMaxSlots + 1];   // first column of each slot, lo[S] = the end of the last
  uint16_t ranks[kMaxSlots];
};
cudaError_t launch_linear_pack(const LinearPackParams& p, cudaStream_t stream);

}  // namespace mlk
