// Host side of moe_lora_linear: argument checks, the layout of stacked adapters and of the
// workspace, tensor maps, the choice of tiles and the launches.
#include "linear.h"
#include "host.h"

#include <algorithm>
#include <cstring>

using namespace mlk;

namespace {

// Stacked columns: every slot's rank rounded up to 8 (16-byte pieces of a row), the end to a
// whole 64-column block.  lo[s] is slot s's first column, lo[S] the end.
int stacked_ranks(const int32_t* h_ranks, int S, int* lo) {
  int c = 0;
  for (int s = 0; s < S; ++s) {
    lo[s] = c;
    c += (h_ranks[s] + 7) / 8 * 8;
  }
  lo[S] = c;
  return (c + kAdapterBlock - 1) / kAdapterBlock * kAdapterBlock;
}

moe_lora_status check_ranks(int S, const int32_t* h_ranks, int most) {
  if (S < 0 || S > kMaxSlots || (S > 0 && h_ranks == nullptr)) return MOE_LORA_ERR_INVALID_ARG;
  for (int s = 0; s < S; ++s)
    if (h_ranks[s] < 0 || h_ranks[s] > most) return MOE_LORA_ERR_INVALID_ARG;
  int lo[kMaxSlots + 1];
  return stacked_ranks(h_ranks, S, lo) <= kMaxStackedRanks ? MOE_LORA_OK : MOE_LORA_ERR_UNSUPPORTED;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Stacked adapters: As [Rs, K], Bs [N, Rs], and the marks of weights that are not finite
// (linear_pack_kernel): a word of 64 slots, and 8 words of 16 bits per row.  Where the last slot's columns leave
// some of their 64-column block, these lie there: the word at the start of a row of As that is no
// slot's (u of its column is masked), the marks in columns of Bs that are no slot's (bf16 values below
// 2^-125, times u = 0).  Otherwise behind Bs.
struct Stack {
  size_t b, sick, marks;   // byte offsets
  int mark_stride;
  size_t bytes;
};
Stack stack_of(int Rs, int used, int N, int K) {
  const size_t a = align256(static_cast<size_t>(Rs) * K * 2), b = align256(static_cast<size_t>(Rs) * N * 2);
  if (used < Rs) return {a, static_cast<size_t>(used) * K * 2, a + static_cast<size_t>(used) * 2, Rs, a + b};
  const size_t marks = align256(static_cast<size_t>(N) * kMarkWords * 2);
  return {a, a + b + marks, a + b, kMarkWords, Rs > 0 ? a + b + marks + 256 : 0};
}

// A shrink cut into slices (deal_shrink): up to 128 stacked columns; with at most one product tile per
// pair up to 8 slices of each shrink tile and 80 in all, with more 3 of each of up to 106 (T 27136).
constexpr int kMaxSlicedRanks = 128, kMaxSliced = 80, kDealtSlices = 3, kDealtTiles = 106;

// Bytes of u, and of the slices' part sums behind it.
size_t u_bytes(int T, int Rs) { return align256(static_cast<size_t>(T) * Rs * kFloatPieces * 2); }
size_t part_bytes(int T, int Rs, int slices) {
  return slices == 1 ? 0 : static_cast<size_t>((T + 255) / 256) * slices * Rs * 1024;
}
// The most part sums of any call on up to T tokens with up to Rs stacked columns, so that what one size
// of call needs is enough for every smaller one.
size_t most_part_bytes(int T, int Rs) {
  const long long tt = T <= 128 ? 0 : std::min<long long>(T / 256 + (T % 256 != 0), kDealtTiles);
  const long long tiles = std::max(std::min<long long>(kMaxSliced, kLinearMaxSlices * tt), kDealtSlices * tt);
  return static_cast<size_t>(tiles) * std::min(Rs, kMaxSlicedRanks) * 1024;
}

bool tile_map(const moe_lora_handle* h, CUtensorMap* m, const void* base, long long rows, long long cols,
              long long stride, int box_rows, bool f32 = false) {   // boxes of 128 bytes x box_rows
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * (f32 ? 4 : 2)};
  const cuuint32_t box[2] = {f32 ? 32u : 64u, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return h->encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

enum Kernel { kNarrow, kWide, kCluster };
struct Tiles {
  Kernel kernel;    // kWide: CTA pairs, 256 tokens x `rows` weight rows
  int tokens;       // token tile
  int rows;         // weight rows of a tile
  int split;        // CTAs (kWide: pairs) that share a tile's K
  int accs, acc_steps;   // (kNarrow, kCluster) a CTA's accumulators and the K blocks of each
};
// The tensor cores truncate as they accumulate, which adds up over a long K: an accumulator of a
// float32 result takes at most 1024 of it (on narrow tiles past K 131072, where TMEM has no room for more than
// 16 accumulators of 16 columns on each of 8 CTAs, a 128th of K).  A bf16 result takes one accumulator.
constexpr int kAccSteps = 16;
void set_accumulators(Tiles& c, int nk, bool f32) {
  const int steps = (nk + c.split - 1) / c.split, room = kLinearTmem / c.tokens;
  c.accs = f32 ? (steps + kAccSteps - 1) / kAccSteps : 1;
  if (c.kernel == kNarrow && c.tokens == 16) c.accs = std::min(c.accs, room);
  c.acc_steps = std::max(kAccSteps, (steps + c.accs - 1) / c.accs);
}
bool fits_tmem(const Tiles& c) { return (c.kernel == kCluster ? 2 * c.accs + 1 : c.accs) * c.tokens <= kLinearTmem; }

// Microseconds of a call on each kernel: models fitted to measured calls in a row (T 1 to 2048, N 384
// to 16384, K 2048 and 7168, adapters of 16 to 512 stacked ranks), good to a microsecond or so and
// meant to rank the choices.
//
// Copies of a step (a 64-wide K block of a tile): an SM's shared memory takes in `one` GB/s with one
// CTA there, 115 with two.  The weights come from HBM, and from L2 again for further token tiles;
// how fast goes by the weight stages in flight on an SM (16 KB each, `stages` per CTA).
double copies_us(long long ctas, int split, double kb_step, int steps, double one, double weight_mb, int stages,
                 double wave, int sms) {
  const double mb = kb_step * steps * 1e-3;
  // CTAs that are resident together: clusters stay within a GPC and leave some of its SMs' places
  const int room = 2 * sms - (split == 8 ? sms / 4 : split == 4 ? sms / 9 : 0);
  const long long waves = (ctas + room - 1) / room;
  const double us = ctas <= sms ? mb / (one * 1e-3)
                                : static_cast<double>(waves) * 2.0 * mb / 0.115 + wave * static_cast<double>(waves - 1);
  const double hbm = ctas > sms || stages >= 6 ? 6.3 : stages == 5 ? 5.8 : stages == 4 ? 5.3 : 4.6;   // MB/us
  return std::max(us, weight_mb / hbm);
}
double weight_mb(int T, int N, int K, int bn) { return 2e-6 * N * K * (T > bn ? 1.2 : 1.0); }
// Small shrink tiles are done sooner, but each reads the stacked A again: 16 tokens at T 64 take
// 1.1 us off (13.4 -> 12.3, N 5120, K 2048) and add 1.9 at T 256 (12.3 -> 14.1, N 2048).
int shrink_tokens(int T, int bn) { return std::min(bn, T <= 64 ? 16 : T <= 128 ? 32 : 64); }
// Narrow tiles: set-up, first bytes and epilogue; the sum over a cluster (clusters of 8 do not pack
// two CTAs to every SM); with adapters what of the shrink and its way back the copies do not hide.
double narrow_us(int T, int N, int K, int Rs, int bn, int split, int sms) {
  const int steps = ((K + 63) / 64 + split - 1) / split;
  const int st = shrink_tokens(T, bn);
  const long long shrinks = static_cast<long long>((Rs + 127) / 128) * ((T + st - 1) / st);
  const long long ctas = (static_cast<long long>((N + 127) / 128) * ((T + bn - 1) / bn) + shrinks) * split;
  const double copy = copies_us(ctas, split, 16.0 + bn / 8.0, steps, 75.0, weight_mb(T, N, K, bn),
                                bn == 16 ? 6 : bn == 32 ? 5 : bn == 64 ? 4 : 3,
                                3.5 + (split == 8 ? 4.0 : 0.0) + (Rs > 0 ? 4.0 : 0.0), sms);
  double us = 2.7 + copy + bn / 128.0 * (split > 1 ? 1.2 : 0.6) + (split > 1 ? 0.4 : 0.0);
  if (split == 8 && bn > 16 && (ctas > 128 || bn == 128)) us += bn == 128 ? 2.5 : 0.85;
  if (Rs > 0)
    us += bn == 16 ? std::min(3.9, std::max(split == 8 ? 1.4 : 1.8, 5.3 - 0.4 * copy)) : bn == 128 ? 7.0 : 4.4 - 0.1 * copy;
  return us;
}
// Each cluster shrinking for itself: As beside W in every step, the exchange in the cluster.
double cluster_us(int T, int N, int K, int Rs, int bn, int split, int sms) {
  const int steps = ((K + 63) / 64 + split - 1) / split;
  const long long ctas = static_cast<long long>((N + 127) / 128) * ((T + bn - 1) / bn) * split;
  const double copy = copies_us(ctas, split, 16.0 + (Rs + 63) / 64 * 8.0 + bn / 8.0, steps, 87.0,
                                weight_mb(T, N, K, bn), Rs <= 64 && bn == 16 ? 4 : 3, 3.5 + (split == 8 ? 4.0 : 0.0), sms);
  return 4.4 + copy + (bn == 32 ? 0.9 : 0.0);
}
// How a shrink is cut and dealt out (wide tiles): the slices of a shrink tile's K, how many of all
// slices go round every pair instead of the spare ones, and the K blocks of the busiest pair.
//
// A K block of a shrink tile takes as long as one of a product tile (measured), so
// whole shrink tiles are in the way: with at most one product tile per pair they take as long as those
// that wait for them, and several in a row far longer (T 2450, N 1560, K 3632, 56 ranks: 40.3 us, 21.7
// without adapters, 27.4 in slices); with more they leave a few pairs a tile behind the others.
struct Shrink {
  int slices;
  long long spread, busiest;
};
Shrink deal_shrink(int T, int N, int K, int Rs, int rows, int split, const LinearMachine& m) {
  const long long tt = (T + 255) / 256, prods = tt * ((N + rows - 1) / rows) * split, nk = (K + 63) / 64;
  const long long cols = std::min(Rs, rows), tiles = Rs > 0 ? tt * ((Rs + cols - 1) / cols) : 0;
  const long long room = m.pairs(split), waves = (prods + room - 1) / room;
  if (tiles == 0) return {1, 0, waves * (nk / split)};
  const long long most =   // four K blocks or more each
      Rs > kMaxSlicedRanks ? 1 : std::min<long long>(kLinearMaxSlices, nk / 4);
  if (prods <= room) {   // one to a pair: those without a product tile, where they come to two or more a tile
    const long long idle = room - prods, over = std::min<long long>(kMaxSliced, idle >= 2 * tiles ? idle : room);
    const long long slices = std::min(most, over / tiles);
    if (slices > 1) {
      const bool all = idle < 2 * tiles;
      return {static_cast<int>(slices), all ? slices * tiles : 0, nk / split + (all ? (nk + slices - 1) / slices : 0)};
    }
  }
  // (as the kernel deals: pairs with a product tile less than others are spare)
  auto deal = [&](long long slices) -> Shrink {
    const long long n = tiles * slices, pairs = std::min(room, prods + n), left = prods % pairs;
    const long long spare = pairs - left, own = prods / pairs * (nk / split), block = (nk + slices - 1) / slices;
    const long long fill = spare * (slices == 1 && 2 * cols <= rows ? 2 : slices);
    // (a pair may hold no three slices of one shrink tile: linear_wide.cu's join_slice)
    const long long spread = slices > spare ? n : std::max(0LL, n - fill);
    const long long each = (spread + pairs - 1) / pairs, more = (n - spread + spare - 1) / spare;
    const long long cost = block + (slices > 1 ? 12 : 0);
    return {static_cast<int>(slices), spread,
            std::max(own + (each + more) * cost, left ? own + nk / split + each * cost : 0)};
  };
  // Writing and joining a slice holds up its pair for about 12 K blocks, more with more slices, so these
  // pay with a long K only: T 8192, N 4096, K 7168, 128 ranks: 280.5, 275.4, 269.3 and 284.8 us in 1 to 4
  // slices; N 4096, K 2048, 48 ranks: 88.0, 98.7, 91.9 and 91.6.
  Shrink best = deal(1);
  for (long long slices = 2; slices <= (tt > kDealtTiles ? 1 : std::min<long long>(most, kDealtSlices)); ++slices) {
    const Shrink s = deal(slices);
    if (s.busiest < best.busiest) best = s;
  }
  return best;
}

// Pairs: a pair walks whole tiles of 256 tokens x `rows`; a 64-deep K step takes 0.30 us at 256 rows
// (the tensor cores' rate), 0.285 at 192 and 0.28 at 128 (24 KB an SM; at 256 rows 32 KB take 0.30, so it is
// not the copies' rate: what it waits for was not found), so the smaller ones pay only where they bring no
// further wave: T 3066, N 1551, K 6624: 66.6 / 62.9 / 87.6 us.
// Two pairs with half of a tile's K each (split 2) exchange their part sums through shared memory,
// about 4 us, and have less of a main loop to hide the shrink under: T 512, N 4096, K 7168, rank 16:
// 26.5 us, one pair per tile 35.9; T 512, N 2048, K 2048: 14.8 and 13.4.  (Four pairs, clusters of 8,
// came out slower everywhere.)
double wide_us(int T, int N, int K, int Rs, int rows, int split, const LinearMachine& m) {
  const long long nk = (K + 63) / 64;
  const Shrink s = deal_shrink(T, N, K, Rs, rows, split, m);
  const double steps = static_cast<double>(nk) / split;
  if (split == 2) {   // fits K 2048 to 7168
    const double us = rows == 256 ? 9.2 + 0.26 * steps : 8.0 + 0.235 * steps;
    return Rs == 0 ? us : us + 1.5 + std::max(0.0, 0.2 * static_cast<double>(nk) / s.slices + 5.0 - 0.25 * steps);
  }
  const double us = 3.5 + (rows == 256 ? 0.3 : rows == 192 ? 0.285 : 0.28) * static_cast<double>(s.busiest);
  return Rs == 0 ? us : us + (s.slices == 1 ? 3.5 : std::max(1.0, 6.0 - 0.16 * steps));
}

Tiles pick_tiles(int T, int N, int K, bool f32, int Rs, const LinearMachine& m) {
  const int nk = (K + 63) / 64;
  Tiles best = {};
  double us = 1e30;
  auto offer = [&](double t, Tiles c) {
    if (c.kernel != kWide) {
      set_accumulators(c, nk, f32);
      if (!fits_tmem(c)) return;
    }
    if (t < us) {
      us = t;
      best = c;
    }
  };
  for (int bn = 16; bn <= 128; bn *= 2) {
    if (bn > 16 && bn / 2 >= T) break;
    for (int split = 1; split <= kLinearMaxSplit && split <= nk; split *= 2) {
      // a float32 result's accumulators lie in one CTA each as far as a cluster goes
      if (f32 && nk > 16 * split && split < kLinearMaxSplit && 2 * split <= nk) continue;
      offer(narrow_us(T, N, K, Rs, bn, split, m.sms), {kNarrow, bn, 128, split});
      if (Rs > 0 && Rs <= 128 && bn <= 32)
        offer(cluster_us(T, N, K, Rs, bn, split, m.sms), {kCluster, bn, 128, split});
    }
  }
  if (T > 128)
    for (int rows = f32 ? 128 : 256; rows >= 128; rows -= 64) {
      const long long tiles = static_cast<long long>((T + 255) / 256) * ((N + rows - 1) / rows);
      for (int split = 1; split <= 2; ++split)
        if (split == 1 || (rows != 192 && nk >= 16 && 2 * tiles <= m.pairs(2)))
          offer(wide_us(T, N, K, Rs, rows, split, m), {kWide, 256, rows, split});
    }
  return best;
}

}  // namespace

extern "C" {

moe_lora_status moe_lora_linear_adapters_size(int S, int N, int K, const int32_t* h_ranks, size_t* bytes) {
  if (bytes == nullptr || S < 1 || N < 1 || K < 8 || K % 8 != 0) return MOE_LORA_ERR_INVALID_ARG;
  if (N > kMaxExtent || K > kMaxExtent) return MOE_LORA_ERR_UNSUPPORTED;
  const moe_lora_status st = check_ranks(S, h_ranks, kMaxRank);
  if (st != MOE_LORA_OK) return st;
  int lo[kMaxSlots + 1];
  const int Rs = stacked_ranks(h_ranks, S, lo);
  *bytes = stack_of(Rs, lo[S], N, K).bytes;
  return MOE_LORA_OK;
}

moe_lora_status moe_lora_linear_pack_adapters(moe_lora_handle* h, const moe_lora_bf16* A, const moe_lora_bf16* B,
                                              int S, int N, int K, int R, const int32_t* h_ranks, void* adapters,
                                              moe_lora_stream stream) {
  if (h == nullptr || R < 0 || R > kMaxRank) return MOE_LORA_ERR_INVALID_ARG;
  size_t bytes = 0;
  moe_lora_status st = moe_lora_linear_adapters_size(S, N, K, h_ranks, &bytes);
  if (st != MOE_LORA_OK) return st;
  st = check_ranks(S, h_ranks, R);
  if (st != MOE_LORA_OK) return st;
  if (bytes == 0) return MOE_LORA_OK;   // every rank is 0
  if (A == nullptr || B == nullptr || adapters == nullptr || !aligned16(A) || !aligned2(B) || !aligned16(adapters))
    return MOE_LORA_ERR_INVALID_ARG;
  LinearPackParams p;
  int lo[kMaxSlots + 1];
  p.Rs = stacked_ranks(h_ranks, S, lo);
  for (int s = 0; s <= S; ++s) p.lo[s] = static_cast<uint16_t>(lo[s]);
  for (int s = 0; s < S; ++s) p.ranks[s] = static_cast<uint16_t>(h_ranks[s]);
  p.A = reinterpret_cast<const __nv_bfloat16*>(A);
  p.B = reinterpret_cast<const __nv_bfloat16*>(B);
  uint8_t* at = static_cast<uint8_t*>(adapters);
  const Stack k = stack_of(p.Rs, lo[S], N, K);
  p.Ap = reinterpret_cast<__nv_bfloat16*>(at);
  p.Bp = reinterpret_cast<__nv_bfloat16*>(at + k.b);
  p.sick = reinterpret_cast<unsigned long long*>(at + k.sick);
  p.marks = reinterpret_cast<uint16_t*>(at + k.marks);
  p.mark_stride = k.mark_stride;
  p.S = S;
  p.N = N;
  p.K = K;
  p.R = R;
  if (static_cast<long long>(p.Rs) * (K / 8) > 128LL * 0x7fffffff)   // 2^30 blocks for As, 2^28 for Bs at most
    return MOE_LORA_ERR_INVALID_ARG;
  ML_ON_DEVICE(h);
  ML_LAUNCH(h, launch_linear_pack(p, stream), "linear pack launch");
  return MOE_LORA_OK;
}

moe_lora_status moe_lora_linear_workspace_size(int T, int S, const int32_t* h_ranks, size_t* bytes) {
  if (bytes == nullptr || T < 0) return MOE_LORA_ERR_INVALID_ARG;
  if (T > kMaxExtent) return MOE_LORA_ERR_UNSUPPORTED;
  const moe_lora_status st = check_ranks(S, h_ranks, kMaxRank);
  if (st != MOE_LORA_OK) return st;
  int lo[kMaxSlots + 1];
  const int Rs = stacked_ranks(h_ranks, S, lo);
  *bytes = 256 + u_bytes(T, Rs) + most_part_bytes(T, Rs);
  return MOE_LORA_OK;
}

moe_lora_status moe_lora_linear(moe_lora_handle* h, const moe_lora_linear_args* a, void* workspace,
                                size_t workspace_bytes, moe_lora_stream stream) {
  if (h == nullptr || a == nullptr) return MOE_LORA_ERR_INVALID_ARG;
  if (a->T < 0 || a->N < 1 || a->K < 8 || a->K % 8 != 0) return MOE_LORA_ERR_INVALID_ARG;
  if (a->T > kMaxExtent || a->N > kMaxExtent || a->K > kMaxExtent) return MOE_LORA_ERR_UNSUPPORTED;
  moe_lora_status st = check_ranks(a->S, a->h_ranks, kMaxRank);
  if (st != MOE_LORA_OK) return st;
  if (a->S > 0) {
    if (a->h_scalings == nullptr) return MOE_LORA_ERR_INVALID_ARG;
    for (int s = 0; s < a->S; ++s)
      if (a->h_scalings[s] != a->h_scalings[s]) return MOE_LORA_ERR_INVALID_ARG;   // NaN
  }
  const long long kMaxStride = 1LL << 38;   // a tensor map's row pitch is below 2^40 bytes
  if (a->T > 1 && (a->x_stride < a->K || a->x_stride % 8 != 0 || a->x_stride > kMaxStride || a->y_stride < a->N))
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->N > 1 && (a->w_stride < a->K || a->w_stride % 8 != 0 || a->w_stride > kMaxStride))
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->T == 0) return MOE_LORA_OK;
  if (a->x == nullptr || a->w == nullptr || a->y == nullptr || workspace == nullptr) return MOE_LORA_ERR_INVALID_ARG;
  if (!aligned16(a->x) || !aligned16(a->w) || !aligned4(a->bias) || !(a->y_f32 ? aligned4(a->y) : aligned2(a->y)) ||
      !aligned16(workspace))
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->S > 0 && (a->slot_idx == nullptr || !aligned4(a->slot_idx))) return MOE_LORA_ERR_INVALID_ARG;

  LinearParams p;
  std::memset(&p, 0, sizeof(p));
  int lo[kMaxSlots + 1];
  const int Rs = stacked_ranks(a->h_ranks, a->S, lo);
  p.slots.S = a->S;
  bool active = false;   // some slot adds something
  for (int s = 0; s < a->S; ++s) {
    p.slots.lo[s] = p.slots.hi[s] = static_cast<uint16_t>(lo[s]);
    p.slots.scal[s] = a->h_scalings[s];
    if (a->h_scalings[s] != 0.0f && a->h_ranks[s] > 0) {
      p.slots.hi[s] = static_cast<uint16_t>(lo[s] + a->h_ranks[s]);
      active = true;
    }
  }
  const size_t need = 256 + (active ? u_bytes(a->T, Rs) : 0);   // and the part sums of a sliced shrink
  if (workspace_bytes < need) return MOE_LORA_ERR_WORKSPACE_TOO_SMALL;
  if (active && (a->adapters == nullptr || !aligned16(a->adapters))) return MOE_LORA_ERR_INVALID_ARG;
  ML_ON_DEVICE(h);
  if (!h->linear_ready) {
    ML_CUDA(linear_narrow_setup(), "linear setup");
    ML_CUDA(linear_wide_setup(&h->linear_pairs_by_two), "linear setup");
    ML_CUDA(linear_cluster_setup(), "linear setup");
    h->linear_ready = true;
  }

  const LinearMachine m = {h->num_sms, h->linear_pairs_by_two};
  const Tiles c = pick_tiles(a->T, a->N, a->K, a->y_f32 != 0, active ? Rs : 0, m);
  p.T = a->T;
  p.K = a->K;
  p.slot_idx = active ? a->slot_idx : nullptr;
  p.status = static_cast<uint32_t*>(workspace);
  p.pieces = a->y_f32 ? kFloatPieces : 1;
  p.accs = c.accs;
  p.acc_steps = c.acc_steps;
  p.shrink_slices = p.k_slices = 1;
  if (c.kernel == kWide) p.k_slices = c.split;
  const long long x_stride = a->T > 1 ? a->x_stride : a->K, w_stride = a->N > 1 ? a->w_stride : a->K;
  const bool wide = c.kernel == kWide;
  const int x_box = wide ? 128 : c.tokens, w_box = wide ? c.rows / 2 : 128;
  const int a_box = wide ? linear_shrink_cols(Rs, c.rows) / 2 : c.kernel == kCluster ? 64 : 128;
  bool ok = tile_map(h, &p.tmap_x, a->x, a->T, a->K, x_stride, x_box) &&
            tile_map(h, &p.tmap_w, a->w, a->N, a->K, w_stride, w_box);
  p.token_tiles = (a->T + c.tokens - 1) / c.tokens;
  if (active) {
    if (p.token_tiles > kLinearFlags) return MOE_LORA_ERR_UNSUPPORTED;
    const uint8_t* Ap = static_cast<const uint8_t*>(a->adapters);
    const Stack k = stack_of(Rs, lo[a->S], a->N, a->K);
    const uint8_t* Bp = Ap + k.b;
    p.b = reinterpret_cast<const __nv_bfloat16*>(Bp);
    p.sick = reinterpret_cast<const unsigned long long*>(Ap + k.sick);
    p.marks = reinterpret_cast<const uint16_t*>(Ap + k.marks);
    p.mark_stride = k.mark_stride;
    p.Rs = Rs;
    p.u = reinterpret_cast<__nv_bfloat16*>(static_cast<uint8_t*>(workspace) + 256);
    p.flags = h->linear_flags;
    if (wide) {
      const Shrink s = deal_shrink(a->T, a->N, a->K, Rs, c.rows, c.split, m);
      p.shrink_slices = s.slices;
      p.shrink_spread = static_cast<int>(s.spread);
      if (workspace_bytes < need + part_bytes(a->T, Rs, s.slices)) return MOE_LORA_ERR_WORKSPACE_TOO_SMALL;
    }
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256 + u_bytes(a->T, Rs));
    const long long ldu = static_cast<long long>(p.pieces) * Rs;
    p.shrink_tokens = shrink_tokens(a->T, c.tokens);
    if (c.kernel == kNarrow) ok = ok && tile_map(h, &p.tmap_xs, a->x, a->T, a->K, x_stride, p.shrink_tokens);
    ok = ok && tile_map(h, &p.tmap_a, Ap, Rs, a->K, a->K, a_box) &&
         tile_map(h, &p.tmap_b, Bp, a->N, Rs, Rs, w_box) && tile_map(h, &p.tmap_u, p.u, a->T, ldu, ldu, x_box);
  }
  p.N = a->N;
  p.bias = a->bias;
  p.y = a->y;
  p.ldy = a->T > 1 ? a->y_stride : a->N;
  p.y_f32 = a->y_f32 != 0;
  if (wide) {
    // TMA stores write whole 16-byte pieces, also the one that the last column lies in: only where
    // rows and the last column end on such pieces is nothing else written
    const int piece = p.y_f32 ? 4 : 8;
    p.y_vec = p.ldy % piece == 0 && a->N % piece == 0 && aligned16(a->y) && p.ldy < kMaxStride;
    if (p.y_vec) ok = ok && tile_map(h, &p.tmap_y, a->y, a->T, a->N, p.ldy, 32, p.y_f32 != 0);
    if (!ok) return MOE_LORA_ERR_INVALID_ARG;
    ML_LAUNCH(h, launch_linear_wide(p, c.rows, m, stream), "linear launch");
  } else {
    p.y_vec = p.ldy % 4 == 0 && (reinterpret_cast<uintptr_t>(a->y) & (p.y_f32 ? 15u : 7u)) == 0;
    if (!ok) return MOE_LORA_ERR_INVALID_ARG;
    ML_LAUNCH(h,
              c.kernel == kCluster ? launch_linear_cluster(p, c.tokens, c.split, stream)
                                   : launch_linear_narrow(p, c.tokens, c.split, stream),
              "linear launch");
  }
  return MOE_LORA_OK;
}

// For tests, on the host alone (not part of the interface): the kernel (0 narrow, 1 wide, 2 cluster), token
// tile, weight rows, split, accumulators and shrink slices that a call takes on such a device.
void mlk_linear_choice(int T, int N, int K, int y_f32, int Rs, int sms, int pairs_by_two, int32_t* out) {
  const LinearMachine m = {sms, pairs_by_two};
  const Tiles c = pick_tiles(T, N, K, y_f32 != 0, Rs, m);
  const int32_t v[6] = {c.kernel, c.tokens, c.rows, c.split, c.accs,
                        c.kernel == kWide ? deal_shrink(T, N, K, Rs, c.rows, c.split, m).slices : 1};
  std::copy(v, v + 6, out);
}

}  // extern "C"
