// The projection of linear_narrow.cu for long batches: tiles of 256 tokens x BN weight rows on CTA
// pairs.
//
// Here the tokens are the MMA's M operand: a pair (cluster of two CTAs on one TPC) computes
// 256 tokens x BN columns with cta_group::2 MMAs, each CTA loading its 128 token rows and BN / 2
// of the weight rows, so a 64-deep K step of a 256 x 256 tile costs an SM 32 KB of shared memory
// traffic for 128 x 256 x 64 products.  Accumulators are double-buffered in TMEM, so a tile's
// epilogue runs under the next tile's main loop.  The adapter blocks (u against the stacked B)
// are further K steps at the end of a tile's main loop, those that no token of the tile needs
// left out.  The shrink's tiles (256 tokens x up to BN rows of the stacked A) come before a pair's
// product tiles and go first to the pairs that have one product tile less than others; a product
// tile waits for its token tile's flag only in front of its adapter blocks, by
// when the shrink tiles, which every pair runs before any product tile, are long done.  The grid
// is resident as a whole (a pair per TPC), and the last product tile of a token tile sets the flag
// back.
//
// The shrink is cut along K into slices: a pair writes its slices' part sums, waits for the token tile's
// others, and adds up its share of the columns in the slices' order.  With at most one product tile per
// pair that is one slice to a pair, and all of it runs under the product tiles' main loops: T 777,
// N 1536, K 2048, 48 ranks: 15.2 us with whole shrink tiles, 13.6 in slices, 12.5 without adapters;
// T 2450, N 1560, K 3632, 56 ranks: 40.3, 27.4 and 21.7 (there every pair has a product tile as well).
// With more, and a long K, slices fill up the pairs that have a product tile less than others and what
// is left over is spread evenly (T 8192, N 4096, K 7168, 128 ranks: 280.5 us whole, 269.3 in three).
//
// With so few tiles that two pairs are there for each, a cluster of two pairs shares a tile, half of
// its K each: the part sums (float32, over the stages, which are free by then) are exchanged through
// distributed shared memory, and each pair stores half of the columns.  T 512, N 4096, K 7168, rank 16:
// 35.9 us with a pair per tile, 26.5 with two; through L2 instead of shared memory it was 29.4.
//
// Persistent pairs walk the tiles in groups of 8 token tiles, token tile fastest, so the pairs
// running at one time share weight and token tiles in L2.
//
// Epilogue: a thread holds a token's columns; a warp parks 32 tokens x 64 columns in shared
// memory (16-byte pieces, exclusive-or swizzled as the TMA store expects) and one lane stores the
// box, or, where y's rows do not start on 16-byte boundaries, the warp stores it row by row.
//
// A float32 result (F32, BN = 128) is summed in parts: the tensor cores truncate as they accumulate,
// which adds up over a long K, so after every 1024 of K the epilogue takes the accumulator into
// registers (a token's 128 columns per thread) while the MMAs go on in the other one.
//
// Long batches are bound by the tensor cores: T 8192, N 4096, K 7168, 128 ranks of which 64 to 128 at
// work in a tile: 268 to 274 us from a graph of a few calls, 1.79 PFLOP/s of bf16 (95% of a burst of plain
// library products); without adapters 248 to 255, the rate of these.  In a row for seconds, at the power limit,
// 317 and 289.
//
// Warp 0: TMA producer; warp 1: MMA issuer (even CTA); warps 2-5: epilogue; warp 6: a tile or two
// ahead of them, which adapter blocks a tile needs, and the wait for its u (in the producer itself
// these loads and the flag's atomics cost 2 us a tile, 24 us at T 8192, K 2048, N 4096).  Waits are
// bounded as everywhere: a timeout is recorded, raises the CTA's abort flag, and the roles leave.
#include "common.cuh"
#include "linear.h"
#include "linear_nonfinite.cuh"

namespace mlk {

namespace {

constexpr int kThreads = 224;
constexpr int kABytes = 128 * 128;
constexpr int kBoxBytes = 32 * 128;            // a warp's store box: 32 tokens x 64 columns
constexpr int kYBytes = 4 * 2 * kBoxBytes;     // two per epilogue warp
constexpr int kTokenGroup = 8;
constexpr int kPartSteps = 16;                 // (F32) 64-wide K blocks of an accumulator
constexpr uint64_t kPeerDrainNs = 100000;      // 100 us for an aborted odd CTA's copies to land

__host__ __device__ constexpr int stage_bytes(int bn) { return kABytes + bn / 2 * 128; }
__host__ __device__ constexpr int stages_of(int bn) { return bn == 256 ? 6 : bn == 192 ? 6 : 8; }
__host__ __device__ constexpr int smem_bytes(int bn) { return 1024 + stages_of(bn) * stage_bytes(bn) + kYBytes + 256; }

MLDEV void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

// SLICED: a shrink's or a product's K may be in slices (in long batches, where neither is, the
// arithmetic for them costs 0.8%: T 8192, N 4096, K 7168 282.3 and 284.5 us).
template <int BN, bool F32, bool SLICED>
__global__ void __launch_bounds__(kThreads, 1) linear_wide_kernel(const __grid_constant__ LinearParams p) {
  static_assert(!F32 || BN == 128, "a thread's columns fit its registers");
  constexpr int kStages = stages_of(BN);
  constexpr uint32_t STAGE = stage_bytes(BN);
  constexpr uint32_t TMEM_COLS = BN == 128 ? 256u : 512u;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* ybuf = smem + kStages * STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(ybuf + kYBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;   // [2]
  uint64_t* tempty = tfull + 2;        // [2]
  uint64_t* mfull = tempty + 2;        // [2] the tile's block mask is there
  uint64_t* mempty = mfull + 2;        // [2] ... and read
  uint64_t* drain = mempty + 2;
  volatile uint64_t* mask_s = drain + 1;   // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint64_t* parts_bar = drain + 4;   // [4] (ks 2) the part sums of an epilogue warp and its like are written

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // A cluster is the ks pairs that share a product tile's K: one, or two with half of it each.  This CTA's place in its
  // pair, and the rank of the pair's even CTA.
  const uint32_t crank = cluster_ctarank() & 1u, even = cluster_ctarank() & ~1u;
  const bool leader = crank == 0;
  const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1;
  const int NT = (p.N + BN - 1) / BN, TT = p.token_tiles;
  const int nk = (p.K + 63) >> 6;
  const bool lora = p.Rs > 0;
  const int sh_cols = linear_shrink_cols(p.Rs, BN);            // stacked rows of a shrink tile
  const int sh_parts = lora ? (p.Rs + sh_cols - 1) / sh_cols : 0;
  const int kparts = SLICED ? p.shrink_slices : 1;             // shrink tiles that share a K
  const int nshrink = sh_parts * TT * kparts;
  const int ks = SLICED ? p.k_slices : 1;                      // pairs that share a product tile's K
  const int nprod = NT * TT * ks;

  // This pair's tiles, in order: shrink tiles (numbers below nshrink), then product tiles.  Of the
  // nprod product tiles the last pairs get one more than the first `spare` ones.  The first
  // p.shrink_spread shrink tiles go round all pairs, the others round the spare ones.
  const int vpair = pairs - 1 - pair;
  const int spare = pairs - nprod % pairs;   // pairs with nprod / pairs tiles
  const int spread = p.shrink_spread;
  const int n_spread = spread > pair ? (spread - pair + pairs - 1) / pairs : 0;
  const int n_spare = pair < spare && nshrink - spread > pair ? (nshrink - spread - pair + spare - 1) / spare : 0;
  const int n_shrink = n_spread + n_spare;
  const int n_tiles = n_shrink + (nprod > vpair ? (nprod - vpair + pairs - 1) / pairs : 0);
  auto tile_at = [&](int i) -> int {
    if (i < n_spread) return pair + i * pairs;
    if (i < n_shrink) return spread + pair + (i - n_spread) * spare;
    return nshrink + vpair + (i - n_shrink) * pairs;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&tfull[0], 1);
    mbar_init(&tfull[1], 1);
    mbar_init(&tempty[0], 8);   // the pair's epilogue warps
    mbar_init(&tempty[1], 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&mfull[i], 1);
      mbar_init(&mempty[i], leader ? 2 : 1);   // the producer and, in the even CTA, the MMA issuer
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&parts_bar[i], static_cast<uint32_t>(ks));
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmap_w);
    tma_prefetch_desc(&p.tmap_x);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_arrive();   // the peer's barriers are initialised before any remote use
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // Nothing of the call's data is touched before the kernel in front has ended; then the kernel
  // after this one may start as far.
  pdl_wait();
  pdl_trigger();

  // a shrink tile's nt: its part of the stack; its K blocks are those from first_k(tile) to last_k(tile)
  auto decode = [&](int tile, int& tt, int& nt) {
    if (tile < nshrink) {
      const int g = tile / kparts;
      tt = g / sh_parts;
      nt = g - tt * sh_parts;
      return;
    }
    tile = (tile - nshrink) / ks;
    const int g = tile / (kTokenGroup * NT), r = tile - g * kTokenGroup * NT;
    const int size = min(kTokenGroup, TT - g * kTokenGroup);
    nt = r / size;
    tt = g * kTokenGroup + r - nt * size;
  };
  auto first_k = [&](int tile) -> int {
    return tile < nshrink ? tile % kparts * nk / kparts : (tile - nshrink) % ks * nk / ks;
  };
  auto last_k = [&](int tile) -> int {
    return tile < nshrink ? (tile % kparts + 1) * nk / kparts : ((tile - nshrink) % ks + 1) * nk / ks;
  };
  auto adds = [&](int tile) -> bool {   // the slice of a product tile that takes the adapter blocks: the last
    return lora && tile >= nshrink && (tile - nshrink) % ks == ks - 1;
  };
  // the block mask of the i-th product tile of this pair, handed over by warp 6
  auto take_mask = [&](int i, uint64_t& mask) -> bool {
    if (!mbar_wait(&mfull[i & 1], (i >> 1) & 1, abort_flag, p.status, kWhereLinear)) return false;
    mask = mask_s[i & 1];
    mbar_arrive(&mempty[i & 1]);
    return true;
  };

  if (warp == 0) {   // ------------------------------------------------ TMA producer
    const uint64_t pol = l2_policy_evict_last();
    int stage = 0, ok = 1;
    uint32_t phase = 0, issued = 0, parity = 0;
    auto issue = [&](const CUtensorMap* xm, int kx, int t, const CUtensorMap* wm, int kw, int n,
                     uint32_t bytes) -> bool {
      if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, kWhereLinear)) return false;
      uint8_t* a = smem + stage * STAGE;
      if (leader) mbar_arrive_expect_tx(&full[stage], 2 * bytes);
      const uint32_t bar = cluster_addr(&full[stage], even);
      tma_load_2d_pair(a, xm, bar, kx, t, pol);
      tma_load_2d_pair(a + kABytes, wm, bar, kw, n, pol);
      issued |= 1u << stage;
      parity = (parity & ~(1u << stage)) | (phase << stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
      return true;
    };
    int nmask = 0;
    if (lane == 0)
      for (int i = 0; ok && i < n_tiles; ++i) {
        const int tile = tile_at(i);
        int tt, nt;
        decode(tile, tt, nt);
        const int t = tt * 256 + static_cast<int>(crank) * 128;
        if (tile < nshrink) {
          const int half = sh_cols / 2, k1 = last_k(tile);
          for (int kb = first_k(tile); ok && kb < k1; ++kb)
            ok = issue(&p.tmap_x, kb * 64, t, &p.tmap_a, kb * 64, nt * sh_cols + static_cast<int>(crank) * half,
                       kABytes + half * 128);
          continue;
        }
        const int n = nt * BN + static_cast<int>(crank) * (BN / 2);
        const int k1 = last_k(tile);
        for (int kb = first_k(tile); ok && kb < k1; ++kb)
          ok = issue(&p.tmap_x, kb * 64, t, &p.tmap_w, kb * 64, n, STAGE);
        if (ok && adds(tile)) {
          uint64_t mask = 0;
          ok = take_mask(nmask++, mask);
          for (int piece = 0; piece < (F32 ? kFloatPieces : 1); ++piece)
            for (uint64_t m = mask; ok && m; m &= m - 1) {
              const int c = (__ffsll(static_cast<long long>(m)) - 1) * 64;
              ok = issue(&p.tmap_u, piece * p.Rs + c, t, &p.tmap_b, c, n, STAGE);
            }
        }
      }
    if (lane == 0 && !ok) {   // let every issued copy land before the CTA exits
      if (leader) {
        for (int s = 0; s < kStages; ++s)
          if ((issued >> s) & 1u) mbar_wait_drain(&full[s], (parity >> s) & 1u);
      } else {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kPeerDrainNs) {
        }
      }
    }
  } else if (warp == 1) {   // ------------------------------------------ MMA issuer (even CTA)
    if (leader) {
      int stage = 0, ok = 1, acc = 0;
      uint32_t phase = 0, aphase = 0;
      auto consume = [&](uint32_t d, uint32_t idesc, bool first) -> bool {
        if (!mbar_wait(&full[stage], phase, abort_flag, p.status, kWhereLinear)) return false;
        tc_fence_after();
        const uint32_t a = smem_u32(smem + stage * STAGE);
        const uint64_t ad = sw128_kmajor_desc(a), bd = sw128_kmajor_desc(a + kABytes);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_bf16_pair(d, ad + 2 * kk, bd + 2 * kk, idesc, (first && kk == 0) ? 0u : 1u);
        umma_commit_pair_mc(&empty[stage], static_cast<uint16_t>(0x3u << even));
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        return true;
      };
      int nmask = 0;
      if (lane == 0)
        for (int i = 0; ok && i < n_tiles; ++i) {
          const bool shrink = i < n_shrink;
          const uint32_t idesc = idesc_bf16_f32(256, shrink ? sh_cols : BN);
          uint32_t d = 0;
          auto begin = [&]() -> bool {   // the accumulator, once its last use has been read out
            if (!mbar_wait(&tempty[acc], aphase ^ 1u, abort_flag, p.status, kWhereLinear)) return false;
            tc_fence_after();
            d = tmem_base + static_cast<uint32_t>(acc * BN);
            return true;
          };
          auto finish = [&]() {
            umma_commit_pair_mc(&tfull[acc], static_cast<uint16_t>(0x3u << even));
            if (++acc == 2) {
              acc = 0;
              aphase ^= 1u;
            }
          };
          const int tile = tile_at(i), steps_k = last_k(tile) - first_k(tile);
          ok = begin();
          for (int kb = 0; ok && kb < steps_k; ++kb) {
            bool first = kb == 0;
            if (F32 && kb > 0 && kb % kPartSteps == 0) {
              finish();
              ok = begin();
              first = true;
            }
            ok = ok && consume(d, idesc, first);
          }
          if (ok && adds(tile)) {
            uint64_t mask = 0;
            ok = take_mask(nmask++, mask);
            const int steps = __popcll(mask) * (F32 ? kFloatPieces : 1);
            for (int j = 0; ok && j < steps; ++j) ok = consume(d, idesc, false);
          }
          if (ok) finish();
        }
      if (!ok && lane == 0) {   // let what was issued finish before TMEM is released
        umma_commit_pair(drain);
        mbar_wait_drain(drain, 0);
      }
    }
  } else if (warp == 6) {   // ---------------------------- adapter blocks and flags, tiles ahead
    if (lora) {
      int ok = 1;
      for (int i = 0; i < n_tiles - n_shrink; ++i) {
        if (!adds(tile_at(n_shrink + i))) continue;   // (slices: the pair's only product tile)
        int tt, nt;
        decode(tile_at(n_shrink + i), tt, nt);
        int sl[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = tt * 256 + j * 32 + lane;
          sl[j] = t < p.T ? __ldg(p.slot_idx + t) : -1;
        }
        uint64_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (sl[j] >= 0 && sl[j] < p.slots.S && p.slots.hi[sl[j]] > p.slots.lo[sl[j]]) {
            const int b0 = p.slots.lo[sl[j]] >> 6, b1 = (p.slots.hi[sl[j]] - 1) >> 6;
            m |= (~0ull >> (63 - b1)) & (~0ull << b0);
          }
        const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(m));
        const uint32_t hi = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(m >> 32));
        m = lo | (static_cast<uint64_t>(hi) << 32);
        if (lane == 0) {
          int* ready = reinterpret_cast<int*>(p.flags + tt);
          const int target = 8 * sh_parts * kparts;   // the pair's epilogue warps, for every shrink tile
          if (m) {   // u is written, by st.global, and read next by TMA
            ok = wait_flag_geq(ready, target, abort_flag, p.status, kWhereLinear);
            fence_proxy_async_global();
          }
          ok = ok && mbar_wait_sleep(&mempty[i & 1], ((i >> 1) & 1) ^ 1, abort_flag, p.status, kWhereLinear);
          if (ok) {
            mask_s[i & 1] = m;
            mbar_arrive(&mfull[i & 1]);
            // past the flag: the last of the token tile's product CTAs sets it back
            if (atomicAdd(ready + 1, 1) == 2 * NT - 1 &&
                wait_flag_geq(ready, target, abort_flag, p.status, kWhereLinear)) {
              atomicExch(ready, 0);
              atomicExch(ready + 1, 0);
              if (kparts > 1) atomicExch(reinterpret_cast<int*>(p.flags + TT + tt), 0);   // all are past it, too
            }
          }
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      }
    }
  } else {   // ------------------------------------------------------------ epilogue
    if (blockIdx.x == 0) {   // the only writer of the status word before a timeout
      const int et = static_cast<int>(threadIdx.x) - 64;
      int bad = 0;
      if (p.slot_idx != nullptr)
#pragma unroll 8
        for (int t = et; t < p.T; t += 128) {
          const int sl = p.slot_idx[t];
          bad |= sl < -1 || sl >= p.slots.S;
        }
      if (any_of_128(bad) && et == 0) *p.status = kDevBadSlot | (kWhereLinear << 8);
      else if (et == 0) *p.status = 0u;
    }
    const unsigned long long sick = lora ? __ldcg(p.sick) : 0;   // slots with weights that are not finite
    const int quarter = warp & 3;
    uint8_t* box0 = ybuf + (warp - 2) * 2 * kBoxBytes;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y);
    int acc = 0, nbox = 0;
    uint32_t aphase = 0;
    auto release = [&]() {   // the accumulator has been read out
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&tempty[acc], even));
      if (++acc == 2) {
        acc = 0;
        aphase ^= 1u;
      }
    };
    // Columns c to c + 4 of u for this lane's token, scaled, where they are its slot's, and 0 elsewhere
    auto store_u4 = [&](int t, int c, const float4& sum, int lo, int hi, float sc) {
      const float f[4] = {sum.x, sum.y, sum.z, sum.w};
      float g[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = (c + j >= lo && c + j < hi) ? sc * f[j] : 0.0f;
      __nv_bfloat16* u = p.u + static_cast<long long>(t) * (F32 ? kFloatPieces : 1) * p.Rs + c;
#pragma unroll
      for (int piece = 0; piece < (F32 ? kFloatPieces : 1); ++piece)
        *reinterpret_cast<uint2*>(u + piece * p.Rs) = F32 ? take_leading4(g) : pack4(g);
    };
    // A slice's part sums, [column / 4][token][4] (a warp's stores are 512 bytes in a row).
    auto slice_at = [&](int tile, int quad) -> float4* {
      return reinterpret_cast<float4*>(p.part) + (static_cast<long long>(tile) * (sh_cols / 4) + quad) * 256 +
             static_cast<int>(crank) * 128 + quarter * 32 + lane;
    };
    auto slice_written = [&](int tt) {
      __syncwarp();   // the release covers every lane's writes before this
      if (lane == 0) red_release_add(reinterpret_cast<int*>(p.flags + TT + tt), 1);
    };
    // Once every slice of the token tile has written its part sums, each adds up its share of the
    // columns, in the slices' order.  A pair writes its next slice before it waits for one.  No pairs
    // wait for one another: a pair's slices are in the order of token tiles, at most two of them of
    // one, so of all token tiles waited for the first one's slices are never behind another wait.
    auto join_slice = [&](int tile) -> bool {
      int tt, nt;
      decode(tile, tt, nt);
      const int t = tt * 256 + static_cast<int>(crank) * 128 + quarter * 32 + lane;
      const int sl = t < p.T ? p.slot_idx[t] : -1;
      const bool has = sl >= 0 && sl < p.slots.S;
      const int lo = has ? p.slots.lo[sl] : 0, hi = has ? p.slots.hi[sl] : 0;
      const float sc = has ? p.slots.scal[sl] : 0.0f;
      int ok = 1;
      if (lane == 0)
        ok = wait_flag_geq(reinterpret_cast<int*>(p.flags + TT + tt), 8 * sh_parts * kparts, abort_flag, p.status,
                           kWhereLinear);
      if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
      __syncwarp();   // lane 0's acquire comes before every lane's loads (a shuffle orders no memory)
      const int slice = tile % kparts, first = tile - slice, quads = sh_cols / 4;
#pragma unroll 4
      for (int q = slice * quads / kparts; q < (slice + 1) * quads / kparts; ++q) {
        float4 v[kLinearMaxSlices];
#pragma unroll
        for (int i = 0; i < kLinearMaxSlices; ++i)
          v[i] = i < kparts ? __ldcg(slice_at(first + i, q)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 1; i < kLinearMaxSlices; ++i)
          if (i < kparts) v[0].x += v[i].x, v[0].y += v[i].y, v[0].z += v[i].z, v[0].w += v[i].w;
        if (t < p.T) store_u4(t, nt * sh_cols + 4 * q, v[0], lo, hi, sc);
      }
      fence_proxy_async_global();   // read next by other CTAs' TMA copies
      __syncwarp();
      if (lane == 0) red_release_add(reinterpret_cast<int*>(p.flags + tt), 1);
      return true;
    };
    // Halves of a product tile's K: every warp writes its part sums over the stages (all MMAs are done),
    // [column / 4][token][4], tells the same warp of the other half, waits for that one, and stores its
    // half of the columns.  The first half is the cluster's second pair's (tiles go out from the last
    // pair on).
    auto part_at = [&](int quad) -> uint32_t {
      return static_cast<uint32_t>((quad * 128 + quarter * 32 + lane) * 16);
    };
    auto all_parts = [&]() -> bool {
      __syncwarp();   // the release covers every lane's writes before this
      if (lane < ks) mbar_arrive_cluster(cluster_addr(&parts_bar[quarter], 2 * lane + crank));
      if (!mbar_wait_sleep(&parts_bar[quarter], 0, abort_flag, p.status, kWhereLinear)) return false;
      fence_cluster();
      return true;
    };
    auto sum_parts = [&](int quad, auto& sum) {   // columns from 4 quad on; all loads in flight together
      constexpr int Q = sizeof(sum) / 16;
      const uint32_t a_at = cluster_addr(smem, 2 + crank), b_at = cluster_addr(smem, crank);
      float4 a[Q], b[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        a[q] = ld_cluster_f4(a_at + part_at(quad + q));
        b[q] = ld_cluster_f4(b_at + part_at(quad + q));
      }
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        sum[4 * q] = a[q].x + b[q].x;
        sum[4 * q + 1] = a[q].y + b[q].y;
        sum[4 * q + 2] = a[q].z + b[q].z;
        sum[4 * q + 3] = a[q].w + b[q].w;
      }
    };
    auto epilogue_f32 = [&](int tile, int tt, int nt, int t_warp) -> bool {
      float f[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) f[j] = 0.0f;
      const int parts = (last_k(tile) - first_k(tile) + kPartSteps - 1) / kPartSteps;
      for (int part = 0; part < parts; ++part) {
        if (!mbar_wait_sleep(&tfull[acc], aphase, abort_flag, p.status, kWhereLinear)) return false;
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * BN);
#pragma unroll
        for (int c = 0; c < 128; c += 32) {   // (a shrink tile of 64 columns: the others are not used)
          uint32_t v[32];
          __syncwarp();
          tmem_ld_x32(taddr + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) f[c + j] += __uint_as_float(v[j]);
        }
        release();
      }
      const int t = t_warp + lane;
      if (tile < nshrink && kparts > 1) {
#pragma unroll
        for (int c = 0; c < 128; c += 4)
          if (c < sh_cols) *slice_at(tile, c / 4) = make_float4(f[c], f[c + 1], f[c + 2], f[c + 3]);
        slice_written(tt);
        return true;
      }
      if (tile < nshrink) {   // u of a token's own columns in bf16 pieces, 0 in the others
        const int sl = t < p.T ? p.slot_idx[t] : -1;
        const bool has = sl >= 0 && sl < p.slots.S;
        const int lo = has ? p.slots.lo[sl] : 0, hi = has ? p.slots.hi[sl] : 0;
        const float sc = has ? p.slots.scal[sl] : 0.0f;
        __nv_bfloat16* u = p.u + static_cast<long long>(t) * kFloatPieces * p.Rs;
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
          const int col = nt * sh_cols + c;
          if (c >= sh_cols || col >= p.Rs || t >= p.T) continue;
          float g[2][4];
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j >> 2][j & 3] = (col + j >= lo && col + j < hi) ? sc * f[c + j] : 0.0f;
#pragma unroll
          for (int piece = 0; piece < kFloatPieces; ++piece) {
            const uint2 v0 = take_leading4(g[0]), v1 = take_leading4(g[1]);
            *reinterpret_cast<uint4*>(u + piece * p.Rs + col) = make_uint4(v0.x, v0.y, v1.x, v1.y);
          }
        }
        fence_proxy_async_global();   // read next by other CTAs' TMA copies
        __syncwarp();                 // the release below covers every lane's writes before this
        if (lane == 0) red_release_add(reinterpret_cast<int*>(p.flags + tt), 1);
        return true;
      }
      float* y32 = static_cast<float*>(p.y);
      if (t_warp >= p.T) return true;   // (for this warp of every slice)
      const int prod = tile - nshrink;
      int c_lo = 0, c_hi = 128;
      if (ks > 1) {
#pragma unroll
        for (int c = 0; c < 128; c += 4)
          *reinterpret_cast<float4*>(smem + part_at(c / 4)) = make_float4(f[c], f[c + 1], f[c + 2], f[c + 3]);
        if (!all_parts()) return false;
        c_lo = prod % ks * (128 / ks);
        c_hi = c_lo + 128 / ks;
      }
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        const int n = nt * BN + c;
        if (n >= p.N || c < c_lo || c >= c_hi) continue;   // warp-uniform
        if (ks > 1) {
          float sum[32];
          sum_parts(c / 4, sum);
#pragma unroll
          for (int j = 0; j < 32; ++j) f[c + j] = sum[j];
        }
        if (p.bias != nullptr) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (n + j < p.N) f[c + j] += __ldg(p.bias + n + j);
        }
        uint8_t* box = box0 + (nbox & 1) * kBoxBytes;
        ++nbox;
        if (lane == 0) bulk_wait_read_1();   // the store that last read this box is done
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
              make_float4(f[c + 4 * j], f[c + 4 * j + 1], f[c + 4 * j + 2], f[c + 4 * j + 3]);
        if (sick != 0) add_nonfinite_to_box<true>(p, sick, box, t, n);
        if (p.y_vec) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&p.tmap_y, box, n, t_warp);
            bulk_commit();
          }
        } else {   // a column per lane, a row at a time
          __syncwarp();
          const int rows = min(32, p.T - t_warp);
          const bool in = n + lane < p.N;
          float* row = y32 + static_cast<long long>(t_warp) * p.ldy + n + lane;
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += 8) {   // eight rows' values at a time
            float one[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
              one[r] = *reinterpret_cast<const float*>(box + (r0 + r) * 128 + (((lane >> 2) ^ r) << 4) + (lane & 3) * 4);
#pragma unroll
            for (int r = 0; r < 8; ++r)
              if (in && r0 + r < rows) row[(r0 + r) * p.ldy] = one[r];
          }
        }
      }
      return true;
    };
    // After slice i of this pair is written: join the one before, and the last one, too.
    auto join_behind = [&](int i) -> bool {
      if (i >= n_shrink) return true;
      if (i > 0 && !join_slice(tile_at(i - 1))) return false;
      return i < n_shrink - 1 || join_slice(tile_at(i));
    };
    for (int i = 0; i < n_tiles; ++i) {
      const int tile = tile_at(i);
      int tt, nt;
      decode(tile, tt, nt);
      const int t_warp = tt * 256 + static_cast<int>(crank) * 128 + quarter * 32;
      if constexpr (F32) {
        if (!epilogue_f32(tile, tt, nt, t_warp)) break;
        if (kparts > 1 && !join_behind(i)) break;
        continue;
      }
      if (!mbar_wait_sleep(&tfull[acc], aphase, abort_flag, p.status, kWhereLinear)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * BN);
      if (tile < nshrink && kparts > 1) {
#pragma unroll 1
        for (int c = 0; c < sh_cols; c += 32) {
          uint32_t v[32];
          __syncwarp();
          tmem_ld_x32(taddr + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *slice_at(tile, (c + j) / 4) = make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]),
                                                       __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
        }
        release();
        slice_written(tt);
        if (!join_behind(i)) break;
        continue;
      }
      if (tile < nshrink) {   // u of a token's own columns, 0 in the others
        const int t = t_warp + lane;
        const int sl = t < p.T ? p.slot_idx[t] : -1;
        const bool has = sl >= 0 && sl < p.slots.S;
        const int lo = has ? p.slots.lo[sl] : 0, hi = has ? p.slots.hi[sl] : 0;
        const float sc = has ? p.slots.scal[sl] : 0.0f;
        __nv_bfloat16* u = p.u + static_cast<long long>(t) * p.Rs;
#pragma unroll 1
        for (int c = 0; c < sh_cols && nt * sh_cols + c < p.Rs; c += 32) {
          uint32_t v[32];
          __syncwarp();
          tmem_ld_x32(taddr + c, v);
          tmem_ld_wait();
          if (t < p.T) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              float f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int col = nt * sh_cols + c + j + i;
                f[i] = (col >= lo && col < hi) ? sc * __uint_as_float(v[j + i]) : 0.0f;
              }
              *reinterpret_cast<uint4*>(u + nt * sh_cols + c + j) = pack8(f);
            }
          }
        }
        fence_proxy_async_global();   // read next by other CTAs' TMA copies
        __syncwarp();                 // the release below covers every lane's writes before this
        if (lane == 0) red_release_add(reinterpret_cast<int*>(p.flags + tt), 1);
        release();
        continue;
      }
      const int prod = tile - nshrink;
      int c_lo = 0, c_hi = BN;
      if (ks > 1 && t_warp < p.T) {   // (the same for this warp of every slice)
#pragma unroll 1
        for (int c = 0; c < BN; c += 32) {
          uint32_t v[32];
          __syncwarp();
          tmem_ld_x32(taddr + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(smem + part_at((c + j) / 4)) =
                make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), __uint_as_float(v[j + 2]),
                            __uint_as_float(v[j + 3]));
        }
        if (!all_parts()) break;
        c_lo = prod % ks * (BN / ks);
        c_hi = c_lo + BN / ks;
      }
#pragma unroll 1
      for (int c = c_lo; c < c_hi; c += 64) {
        const int n = nt * BN + c;
        if (n >= p.N || t_warp >= p.T) break;   // warp-uniform
        uint32_t v[64];
        __syncwarp();
        if (ks > 1) {
          float sum[64];
          sum_parts(c / 4, sum);
#pragma unroll
          for (int j = 0; j < 64; ++j) v[j] = __float_as_uint(sum[j]);
        } else {
          tmem_ld_x32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(v));
          tmem_ld_x32(taddr + c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
          tmem_ld_wait();
        }
        if (p.bias != nullptr) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (n + j < p.N) v[j] = __float_as_uint(__uint_as_float(v[j]) + __ldg(p.bias + n + j));
        }
        uint8_t* box = box0 + (nbox & 1) * kBoxBytes;
        ++nbox;
        if (lane == 0) bulk_wait_read_1();   // the store that last read this box is done
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * j + i]);
          *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) = pack8(f);
        }
        if (sick != 0) add_nonfinite_to_box<false>(p, sick, box, t_warp + lane, n);
        if (p.y_vec) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&p.tmap_y, box, n, t_warp);
            bulk_commit();
          }
        } else {   // two columns per lane, a row at a time
          __syncwarp();
          const int rows = min(32, p.T - t_warp);
          const bool in0 = n + 2 * lane < p.N, in1 = n + 2 * lane + 1 < p.N;
          __nv_bfloat16* row = y + static_cast<long long>(t_warp) * p.ldy + n + 2 * lane;
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += 8) {   // eight rows' values at a time
            uint32_t two[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
              two[r] = *reinterpret_cast<const uint32_t*>(box + (r0 + r) * 128 + (((lane >> 2) ^ r) << 4) + (lane & 3) * 4);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              __nv_bfloat16* at = row + (r0 + r) * p.ldy;
              if (in0 && r0 + r < rows) at[0] = __ushort_as_bfloat16(static_cast<unsigned short>(two[r] & 0xffffu));
              if (in1 && r0 + r < rows) at[1] = __ushort_as_bfloat16(static_cast<unsigned short>(two[r] >> 16));
            }
          }
        }
      }
      release();
    }
    bulk_wait_all();   // the stores have read their boxes and landed
  }

  tc_fence_before();
  __syncwarp();
  cluster_arrive();   // neither CTA leaves while the pair's MMAs may touch its memory
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

}  // namespace

cudaError_t linear_wide_setup(int* pairs_by_two) {
  cudaError_t err;
#define ML_SETUP(BN, F32, SLICED)                                                                              \
  err = cudaFuncSetAttribute(linear_wide_kernel<BN, F32, SLICED>, cudaFuncAttributeMaxDynamicSharedMemorySize, \
                             smem_bytes(BN));                                                                  \
  if (err != cudaSuccess) return err;
#define ML_SETUPS(BN, F32) ML_SETUP(BN, F32, false) ML_SETUP(BN, F32, true)
  ML_SETUPS(256, false)
  ML_SETUPS(192, false)
  ML_SETUPS(128, false)
  ML_SETUPS(128, true)
#undef ML_SETUPS
#undef ML_SETUP
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(256);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 4;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  err = cudaOccupancyMaxActiveClusters(&n, linear_wide_kernel<256, false, true>, &cfg);
  *pairs_by_two = 2 * n;
  return err;
}

cudaError_t launch_linear_wide(const LinearParams& p, int bn, const LinearMachine& m, cudaStream_t stream) {
  const int cols = linear_shrink_cols(p.Rs, bn);
  const long long shrinks = cols ? (p.Rs + cols - 1) / cols * p.shrink_slices : 0;
  const long long tiles = ((p.N + bn - 1) / bn * p.k_slices + shrinks) * p.token_tiles;
  const int room = m.pairs(p.k_slices);
  if (p.shrink_slices > 1 && 2 * p.token_tiles > kLinearFlags) return cudaErrorInvalidValue;
  // halves of a product store whole boxes of columns each, and are their pairs' only product tiles
  const int ks = p.k_slices;
  if (ks != 1 && (ks != 2 || bn == 192 || static_cast<long long>((p.N + bn - 1) / bn) * p.token_tiles * 2 > room))
    return cudaErrorInvalidValue;
  const int pairs = static_cast<int>(tiles < room ? (tiles + ks - 1) / ks * ks : room);
  const dim3 grid(2 * pairs), block(kThreads);
#define ML_LINEAR(BN, F32)                                                                                        \
  return sliced ? launch_kc(linear_wide_kernel<BN, F32, true>, grid, block, smem_bytes(BN), stream, true, 2 * ks, p) \
                : launch_kc(linear_wide_kernel<BN, F32, false>, grid, block, smem_bytes(BN), stream, true, 2, p)
  const bool sliced = ks > 1 || p.shrink_slices > 1;
  if (p.y_f32) ML_LINEAR(128, true);
  switch (bn) {
    case 256: ML_LINEAR(256, false);
    case 192: ML_LINEAR(192, false);
    case 128: ML_LINEAR(128, false);
    default: return cudaErrorInvalidValue;
  }
#undef ML_LINEAR
}

}  // namespace mlk
