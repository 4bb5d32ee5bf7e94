// Projection with per-token adapters, tiles of 128 weight rows x BN tokens (moe_lora_linear):
//
//   y[t, n] = sum_k W[n, k] x[t, k] + sum_c Bs[n, c] u[t, c] (+ bias[n])
//   u[t, c] = scaling[s] sum_k As[c, k] x[t, k]  where column c belongs to the token's slot s,
//             and 0 elsewhere
//
// with every slot's A rows and B columns stacked side by side (As [Rs, K], Bs [N, Rs]), so
// adapters of any ranks and number are one more K range of the same product.  The shrink (u)
// is the same tile with As in the place of W, fewer tokens (so that it is done sooner: its result is
// waited for), and an epilogue that scales, masks and rounds; its tiles are the grid's first, so
// one launch does all.
//
// The weights are the MMA's M = 128 operand and the tokens its N = BN, so a batch of one token
// still streams whole weight rows.  A cluster of CTAs shares a tile: each takes a part of K
// into its own TMEM accumulator, parks the float32 part sums in its shared memory, and the
// cluster adds them through distributed shared memory in rank order (a fixed order, so results
// do not vary from run to run), each CTA writing its share of the tile.  For a float32 result a part of
// more than 1024 of K goes to several accumulators: the tensor cores truncate as they accumulate.  That keeps enough
// CTAs streaming when N alone gives few tiles, in one launch and without global partial sums.
//
// The product's tiles stream W and x at once and wait for u (a flag per token tile) only in front
// of the adapter blocks, which come last.  64-column blocks of the stack in which no token of the
// tile has its adapter are skipped.  The last of a token tile's product CTAs to pass the flag
// sets it back, so the flags are zero again when the kernel ends.  Blocks start in index order,
// so the tiles waited for are running before those that wait; every wait is bounded all the same.
//
// What bounds it is latency, not bandwidth: start, first copies, a few K steps, the shrink's flag, the
// adapter blocks, the sum over the cluster, each a memory round trip or two.  T 64, N 5120, K 2048,
// 120 ranks (64-token tiles, K over 4 CTAs): 12.2 us, 8.0 without adapters, 3.5 for its 24 MB at
// 6.8 TB/s; tensor pipe 5%, DRAM 18% busy.  T 128, N 384, K 7168, float32 (32-token tiles, K over 8
// CTAs): 7.4 us for 7.5 MB.
//
// Warp 0: TMA producer; warp 1: MMA issuer; warps 2-5: slots of the tile's tokens, epilogue.
// Every wait is bounded; a timeout raises the CTA's abort flag, is recorded in the status
// word, and every role still walks through the cluster barriers to the end.
#include "common.cuh"
#include "linear.h"
#include "linear_nonfinite.cuh"

namespace mlk {

namespace {

constexpr int kThreads = 192;
constexpr int kABytes = 128 * 128;
constexpr int kSmemBudget = 112 * 1024;   // two CTAs per SM
constexpr int kMaxSplit = kLinearMaxSplit;
constexpr int kBatch = 3;                 // quads of the tile that a thread sums at a time

__host__ __device__ constexpr int stage_bytes(int bn) { return kABytes + bn * 128; }
__host__ __device__ constexpr int stages_of(int bn) { return (kSmemBudget - 2048) / stage_bytes(bn); }
constexpr int smem_bytes(int bn) { return 1024 + stages_of(bn) * stage_bytes(bn) + 256 + 12 * bn; }

// LONG: a CTA's part of K takes several accumulators (kernels of their own, also in linear_cluster.cu: the
// arithmetic for them costs short calls 0.1 to 0.3 us; T 1, N 2048, K 2048, rank 16: 6.0 and 6.2 us).
template <int BN, bool LONG>
__global__ void __launch_bounds__(kThreads, 2) linear_narrow_kernel(const __grid_constant__ LinearParams p) {
  constexpr int kStages = stages_of(BN);
  constexpr uint32_t STAGE = stage_bytes(BN);
  static_assert(kStages * static_cast<int>(STAGE) >= BN * 128 * 4, "the part sums fit the stage buffers");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * STAGE);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* mask_bar = tfull + 1;
  uint64_t* drain = mask_bar + 1;
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(drain + 1);   // [2] adapter blocks present in the tile
  uint32_t* tmem_slot = mask_s + 2;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* lo_s = reinterpret_cast<int*>(tmem_slot + 2);   // (shrink) [BN] a token's columns of the stack
  int* hi_s = lo_s + BN;                               // and its factor
  float* sc_s = reinterpret_cast<float*>(hi_s + BN);

  const uint32_t tmem_cols = linear_tmem_columns(LONG ? p.accs : 1, BN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = static_cast<int>(cluster_nctas()), rank = static_cast<int>(cluster_ctarank());
  const int index = static_cast<int>(blockIdx.x) / C;
  const int a_tiles = (p.Rs + 127) / 128;   // row tiles of the stacked A
  const int shrink_parts = p.Rs > 0 ? (p.T + p.shrink_tokens - 1) / p.shrink_tokens : 0;
  const bool shrink = index < a_tiles * shrink_parts;
  const int tile = shrink ? index : index - a_tiles * shrink_parts;
  const int across = shrink ? shrink_parts : p.token_tiles;
  const int nt = tile / across, part_t = tile - nt * across;
  const int bn = shrink ? p.shrink_tokens : BN;   // tokens of the tile
  const int row0 = nt * 128, t0 = part_t * bn;
  const int qt = t0 / BN;                         // the product's token tile
  const int N = shrink ? p.Rs : p.N;
  const int nk = (p.K + 63) >> 6;
  const int k_lo = static_cast<int>(static_cast<long long>(nk) * rank / C);
  const int k_hi = static_cast<int>(static_cast<long long>(nk) * (rank + 1) / C);
  const bool lora = !shrink && p.Rs > 0;
  int* ready = reinterpret_cast<int*>(p.flags + qt);
  // shrink CTAs of this token tile
  const int ready_target =
      lora ? a_tiles * C * ((min(BN, p.T - t0) + p.shrink_tokens - 1) / p.shrink_tokens) : 0;

  // the 64-column blocks of the stack that slot sl's adapter lies in
  auto blocks_of = [&](int sl) -> uint64_t {
    if (sl < 0 || sl >= p.slots.S || p.slots.hi[sl] <= p.slots.lo[sl]) return 0ull;
    const int b0 = p.slots.lo[sl] >> 6, b1 = (p.slots.hi[sl] - 1) >> 6;
    return (~0ull >> (63 - b1)) & (~0ull << b0);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(mask_bar, 128);
    mbar_init(drain, 1);
    mask_s[0] = mask_s[1] = 0u;
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(shrink ? &p.tmap_a : &p.tmap_w);
    tma_prefetch_desc(shrink ? &p.tmap_xs : &p.tmap_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // Up to here nothing of the call's data was touched: it may still be in the making by the kernel
  // before, whose end comes next; then the kernel after this one may start as far.
  pdl_wait();
  pdl_trigger();
  const unsigned long long sick = lora ? __ldcg(p.sick) : 0;   // slots with weights that are not finite

  if (shrink && p.Rs > 128 && index > 0) {
    // a stack of several row tiles: leave out those that no token of the product's tile needs (the
    // others' blocks are read for all of its tokens; the whole cluster decides alike; the first tile
    // stays, it writes the status word)
    uint64_t m = 0;
    for (int j = qt * BN + threadIdx.x; j < (qt + 1) * BN && j < p.T; j += kThreads) m |= blocks_of(p.slot_idx[j]);
    if (!__syncthreads_or(((m >> (row0 >> 6)) & 3ull) != 0)) {
      if (threadIdx.x == 0) red_release_add(ready, 1);
      if (warp == 1) tmem_dealloc(tmem_base, tmem_cols);
      return;
    }
  }

  if (warp == 0) {   // ------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
      int stage = 0, ok = 1;
      uint32_t phase = 0, issued = 0, parity = 0;
      auto issue = [&](const CUtensorMap* wm, int kw, const CUtensorMap* xm, int kx) -> bool {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, kWhereLinear)) return false;
        uint8_t* a = smem + stage * STAGE;
        mbar_arrive_expect_tx(&full[stage], kABytes + bn * 128);
        tma_load_2d(a, wm, &full[stage], kw, row0, p.token_tiles == 1 ? pol_w : pol_x);
        tma_load_2d(a + kABytes, xm, &full[stage], kx, t0, pol_x);
        issued |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        return true;
      };
      const CUtensorMap* wmap = shrink ? &p.tmap_a : &p.tmap_w;
      const CUtensorMap* xmap = shrink ? &p.tmap_xs : &p.tmap_x;
      for (int kb = k_lo; ok && kb < k_hi; ++kb) ok = issue(wmap, kb * 64, xmap, kb * 64);
      if (ok && lora) {
        ok = mbar_wait(mask_bar, 0, abort_flag, p.status, kWhereLinear);
        const uint64_t mask = mask_s[0] | (static_cast<uint64_t>(mask_s[1]) << 32);
        if (ok && mask) {
          ok = wait_flag_geq(ready, ready_target, abort_flag, p.status, kWhereLinear);   // u is written,
          fence_proxy_async_global();                                                   // read next by TMA
          int i = 0;
          for (int piece = 0; piece < p.pieces; ++piece)
            for (uint64_t m = mask; ok && m; m &= m - 1, ++i)
              if (i % C == C - 1 - rank) {
                const int c = (__ffsll(static_cast<long long>(m)) - 1) * 64;
                ok = issue(&p.tmap_b, c, &p.tmap_u, piece * p.Rs + c);
              }
        }
        // past the flag: the last of the token tile's product CTAs sets it back
        if (ok && atomicAdd(ready + 1, 1) == (p.N + 127) / 128 * C - 1 &&
            wait_flag_geq(ready, ready_target, abort_flag, p.status, kWhereLinear)) {
          atomicExch(ready, 0);
          atomicExch(ready + 1, 0);
        }
      }
      if (!ok)
        for (int s = 0; s < kStages; ++s)
          if ((issued >> s) & 1u) mbar_wait_drain(&full[s], (parity >> s) & 1u);
    }
  } else if (warp == 1) {   // ------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(128, bn);
      int stage = 0, ok = 1, first = 1, left = p.acc_steps;
      uint32_t phase = 0, d = tmem_base;
      auto consume = [&]() -> bool {
        if (!mbar_wait(&full[stage], phase, abort_flag, p.status, kWhereLinear)) return false;
        tc_fence_after();
        const uint32_t a = smem_u32(smem + stage * STAGE);
        const uint64_t ad = sw128_kmajor_desc(a), bd = sw128_kmajor_desc(a + kABytes);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          umma_bf16(d, ad + 2 * kk, bd + 2 * kk, idesc, first ? 0u : 1u);
          first = 0;
        }
        umma_commit(&empty[stage]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        return true;
      };
      for (int kb = k_lo; ok && kb < k_hi; ++kb) {
        if (LONG && left-- == 0) {   // the next accumulator
          d += BN;
          first = 1;
          left = p.acc_steps - 1;
        }
        ok = consume();
      }
      if (ok && lora) {
        ok = mbar_wait(mask_bar, 0, abort_flag, p.status, kWhereLinear);
        const int n = __popc(mask_s[0]) + __popc(mask_s[1]);
        for (int i = 0; ok && i < p.pieces * n; ++i)
          if (i % C == C - 1 - rank) ok = consume();
      }
      if (ok) {
        umma_commit(tfull);
      } else {   // let what was issued finish before TMEM is released
        umma_commit(drain);
        mbar_wait_drain(drain, 0);
      }
    }
  } else {   // ---------------------------------------------- slots, then TMEM -> shared memory
    const int et = threadIdx.x - 64;
    if (lora) {
      uint64_t m = 0;
      for (int j = et; j < BN && t0 + j < p.T; j += 128) m |= blocks_of(p.slot_idx[t0 + j]);
      if (static_cast<uint32_t>(m)) atomicOr(&mask_s[0], static_cast<uint32_t>(m));
      if (static_cast<uint32_t>(m >> 32)) atomicOr(&mask_s[1], static_cast<uint32_t>(m >> 32));
      mbar_arrive(mask_bar);
    }
    if (shrink && et < bn) {
      const int sl = t0 + et < p.T ? p.slot_idx[t0 + et] : -1;
      const bool has = sl >= 0 && sl < p.slots.S;
      lo_s[et] = has ? p.slots.lo[sl] : 0;
      hi_s[et] = has ? p.slots.hi[sl] : 0;
      sc_s[et] = has ? p.slots.scal[sl] : 0.0f;
    }
    if (blockIdx.x == 0) {   // the only writer of the status word before a timeout
      int bad = 0;
      if (p.slot_idx != nullptr)
#pragma unroll 8
        for (int t = et; t < p.T; t += 128) {
          const int sl = p.slot_idx[t];
          bad |= sl < -1 || sl >= p.slots.S;
        }
      const bool any = any_of_128(bad);
      if (et == 0) *p.status = any ? (kDevBadSlot | (kWhereLinear << 8)) : 0u;
    }
    const int quarter = warp & 3;
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    float* part = reinterpret_cast<float*>(smem) + quarter * 32 + lane;   // [BN][128]
    const int accs = LONG ? (k_hi - k_lo - 1) / p.acc_steps + 1 : 1;   // of this CTA
    if (mbar_wait_sleep(tfull, 0, abort_flag, p.status, kWhereLinear)) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < bn && t0 + c < p.T; c += 16) {   // warp-uniform bound
        uint32_t v[16];
        __syncwarp();   // tcgen05.ld is .aligned
        tmem_ld_x16(taddr + c, v);
        tmem_ld_wait();
#pragma unroll 1
        for (int a = 1; a < accs; ++a) {   // accumulators in order
          uint32_t w[16];
          __syncwarp();
          tmem_ld_x16(taddr + a * BN + c, w);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[j]));
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * 128] = __uint_as_float(v[j]);
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols);
  }

  // this CTA's share of the tile: quads of 4 rows of a token, part sums added in rank order
  const int nvalid = min(bn, p.T - t0);
  const int quads = nvalid * 32;
  const int q_lo = static_cast<int>(static_cast<long long>(quads) * rank / C);
  const int q_hi = static_cast<int>(static_cast<long long>(quads) * (rank + 1) / C);
  const uint32_t part0 = smem_u32(smem);
  for (int q0 = q_lo + static_cast<int>(threadIdx.x); q0 < q_hi; q0 += kBatch * kThreads) {
   float4 v[kBatch][kMaxSplit], bias[kBatch];
#pragma unroll
   for (int i = 0; i < kBatch; ++i) {   // all loads of a batch in flight together
    const int q = q0 + i * kThreads, n = row0 + (q & 31) * 4;
    bias[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (q >= q_hi || n >= N) continue;
    if (!shrink && p.bias != nullptr) {
      bias[i].x = __ldg(p.bias + n);
      if (n + 1 < N) bias[i].y = __ldg(p.bias + n + 1);
      if (n + 2 < N) bias[i].z = __ldg(p.bias + n + 2);
      if (n + 3 < N) bias[i].w = __ldg(p.bias + n + 3);
    }
#pragma unroll
    for (int c = 0; c < kMaxSplit; ++c)
      if (c < C) v[i][c] = ld_cluster_f4(part0 + static_cast<uint32_t>(q) * 16u, c);
   }
#pragma unroll
   for (int i = 0; i < kBatch; ++i) {
    const int q = q0 + i * kThreads;
    const int j = q >> 5, t = t0 + j, n = row0 + (q & 31) * 4;
    if (q >= q_hi || n >= N) continue;
    float f[4] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w};
#pragma unroll
    for (int c = 1; c < kMaxSplit; ++c)
      if (c < C) {
        f[0] += v[i][c].x;
        f[1] += v[i][c].y;
        f[2] += v[i][c].z;
        f[3] += v[i][c].w;
      }
    if (shrink) {
      const int lo = lo_s[j], hi = hi_s[j];
      const float sc = sc_s[j];
      __nv_bfloat16* u = p.u + static_cast<long long>(t) * p.pieces * p.Rs + n;
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = (n + e >= lo && n + e < hi) ? sc * f[e] : 0.0f;
      if (p.pieces == 1) {
        *reinterpret_cast<uint2*>(u) = pack4(f);
      } else {   // the float32 as a sum of bf16 pieces
        for (int piece = 0; piece < p.pieces; ++piece) *reinterpret_cast<uint2*>(u + piece * p.Rs) = take_leading4(f);
      }
    } else {
      f[0] += bias[i].x;
      f[1] += bias[i].y;
      f[2] += bias[i].z;
      f[3] += bias[i].w;
      const long long at = static_cast<long long>(t) * p.ldy + n;
      if (p.y_vec && n + 4 <= p.N) {
        if (p.y_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = make_float4(f[0], f[1], f[2], f[3]);
        else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + at) = pack4(f);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) {
            if (p.y_f32) static_cast<float*>(p.y)[at + e] = f[e];
            else static_cast<__nv_bfloat16*>(p.y)[at + e] = f2bf(f[e]);
          }
      }
    }
   }
  }
  if (shrink) {   // this CTA's part of u is written: read next by other CTAs' TMA copies
    fence_proxy_async_global();
    __syncthreads();   // the release below covers every thread's writes before this barrier
    if (threadIdx.x == 0) red_release_add(ready, 1);
  }
  if (C > 1) {   // no CTA leaves while others read its part sums
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  if (sick != 0)   // (0 in shrink tiles); after all that others wait for
    for (int q = q_lo + static_cast<int>(threadIdx.x); q < q_hi; q += kThreads)
      add_nonfinite(p, sick, t0 + (q >> 5), row0 + (q & 31) * 4, 4);
}

// Stacked copies of the adapters: As [Rs, K] (blocks up to a_blocks) and Bs [N, Rs] (a warp per row).
// Ranks past a slot's own are never read; columns of no slot are zero.
//
// A product takes whole blocks of Bs's columns, with u = 0 in those of other slots: fine while these are
// finite, but 0 x inf is NaN.  So Bs holds finite values alone: where a row of a slot has one that is not,
// the slot's values of that row are stored as classes (0 for 0, +-1 for finite, +-2 for +-inf, 3 for NaN),
// the row is marked for that slot, and the epilogue adds what they stand for to the slot's own tokens
// (linear_nonfinite.cuh).
__global__ void __launch_bounds__(256) linear_pack_kernel(const __grid_constant__ LinearPackParams p, unsigned a_blocks) {
  if (blockIdx.x < a_blocks) {   // 8 values of a row of As
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int per = p.K >> 3;
    if (i >= static_cast<long long>(p.Rs) * per) return;
    const int c = static_cast<int>(i / per), k = static_cast<int>(i - static_cast<long long>(c) * per) * 8;
    int s = 0, hi = p.S;   // the slot whose columns hold c (p.S: past the last): first s with lo[s + 1] > c
    while (s < hi) {
      const int mid = (s + hi) >> 1;
      if (p.lo[mid + 1] > c) hi = mid; else s = mid + 1;
    }
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (s < p.S && c - p.lo[s] < p.ranks[s])
      v = *reinterpret_cast<const uint4*>(p.A + (static_cast<long long>(s) * p.R + c - p.lo[s]) * p.K + k);
    uint4* at = reinterpret_cast<uint4*>(p.Ap + static_cast<long long>(c) * p.K + k);
    if (static_cast<void*>(at) != static_cast<void*>(p.sick)) *at = v;
    return;
  }
  const int lane = threadIdx.x & 31;
  const long long n = static_cast<long long>(blockIdx.x - a_blocks) * 8 + (threadIdx.x >> 5);
  if (n >= p.N) return;   // whole warps
  uint16_t* row = reinterpret_cast<uint16_t*>(p.Bp) + n * p.Rs;
  unsigned long long mark = 0;
  for (int s = 0; s < p.S; ++s) {
    const int ranks = p.ranks[s], width = p.lo[s + 1] - p.lo[s];
    const uint16_t* from = reinterpret_cast<const uint16_t*>(p.B) + (static_cast<long long>(s) * p.N + n) * p.R;
    uint16_t v[kMaxRank / 32];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kMaxRank / 32; ++i) {
      const int c = i * 32 + lane;
      v[i] = c < ranks ? from[c] : 0;
      bad |= (v[i] & 0x7f80u) == 0x7f80u;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad) mark |= 1ull << s;
#pragma unroll
    for (int i = 0; i < kMaxRank / 32; ++i) {
      const int c = i * 32 + lane;
      if (bad && (v[i] & 0x7fffu) != 0) {
        const uint16_t sign = v[i] & 0x8000u, size = v[i] & 0x7fffu;
        v[i] = size > 0x7f80u ? 0x4040 : size == 0x7f80u ? sign | 0x4000 : sign | 0x3f80;   // 3, +-2, +-1
      }
      if (c < width) row[p.lo[s] + c] = v[i];
    }
  }
  for (int c = p.lo[p.S] + lane; c < p.Rs; c += 32) row[c] = 0;
  __syncwarp();
  if (lane < kMarkWords) p.marks[n * p.mark_stride + lane] = static_cast<uint16_t>((mark >> (8 * lane)) & 0xffu);
  if (lane == 0 && mark != 0) atomicOr(p.sick, mark);
}

}  // namespace

cudaError_t linear_narrow_setup() {
  cudaError_t err;
#define ML_SETUP(BN, LONG)                                                                                  \
  err = cudaFuncSetAttribute(linear_narrow_kernel<BN, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize,    \
                             smem_bytes(BN));                                                                \
  if (err != cudaSuccess) return err;
#define ML_SETUPS(BN) ML_SETUP(BN, false) ML_SETUP(BN, true)
  ML_SETUPS(16)
  ML_SETUPS(32)
  ML_SETUPS(64)
  ML_SETUPS(128)
#undef ML_SETUPS
#undef ML_SETUP
  return cudaSuccess;
}

cudaError_t launch_linear_narrow(const LinearParams& p, int bn, int split, cudaStream_t stream) {
  const long long tiles =
      static_cast<long long>((p.N + 127) / 128) * p.token_tiles +
      (p.Rs > 0 ? static_cast<long long>((p.Rs + 127) / 128) * ((p.T + p.shrink_tokens - 1) / p.shrink_tokens) : 0);
  if (tiles * split > 0x7fffffffLL || p.accs < 1 || p.accs * bn > kLinearTmem) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(tiles * split)), block(kThreads);
#define ML_LINEAR(BN)                                                                                               \
  return p.accs > 1 ? launch_kc(linear_narrow_kernel<BN, true>, grid, block, smem_bytes(BN), stream, true, split, p) \
                    : launch_kc(linear_narrow_kernel<BN, false>, grid, block, smem_bytes(BN), stream, true, split, p)
  switch (bn) {
    case 16: ML_LINEAR(16);
    case 32: ML_LINEAR(32);
    case 64: ML_LINEAR(64);
    case 128: ML_LINEAR(128);
    default: return cudaErrorInvalidValue;
  }
#undef ML_LINEAR
}

cudaError_t launch_linear_pack(const LinearPackParams& p, cudaStream_t stream) {
  const cudaError_t err = cudaMemsetAsync(p.sick, 0, sizeof(uint4), stream);   // the piece that the kernel leaves out
  if (err != cudaSuccess) return err;
  const unsigned a = static_cast<unsigned>((static_cast<long long>(p.Rs) * (p.K / 8) + 255) / 256);
  const unsigned b = static_cast<unsigned>((static_cast<long long>(p.N) + 7) / 8);
  return launch_k(linear_pack_kernel, dim3(a + b), dim3(256), 0, stream, false, p, a);
}

}  // namespace mlk
