// The projection of linear_narrow.cu for long batches with a bf16 result: tiles of 256 tokens x
// BN weight rows on CTA pairs.
//
// Here the tokens are the MMA's M operand: a pair (cluster of two CTAs on one TPC) computes
// 256 tokens x BN columns with cta_group::2 MMAs, each CTA loading its 128 token rows and BN / 2
// of the weight rows, so a 64-deep K step of a 256 x 256 tile costs an SM 32 KB of shared memory
// traffic for 128 x 256 x 64 products.  Accumulators are double-buffered in TMEM, so a tile's
// epilogue runs under the next tile's main loop.  The adapter blocks (u against the stacked B)
// are further K steps at the end of a tile's main loop, those that no token of the tile needs
// left out; the first tile waits there for the shrink kernel, beside which this grid starts.
//
// Persistent pairs walk the tiles in groups of 8 token tiles, token tile fastest, so the pairs
// running at one time share weight and token tiles in L2.
//
// Epilogue: a thread holds a token's columns; a warp parks 32 tokens x 64 columns in shared
// memory (16-byte pieces, exclusive-or swizzled as the TMA store expects) and one lane stores the
// box, or, where y's rows do not start on 16-byte boundaries, the warp stores it row by row.
//
// Warp 0: TMA producer; warp 1: MMA issuer (even CTA); warps 2-5: epilogue.  Waits are bounded as
// everywhere: a timeout is recorded, raises the CTA's abort flag, and the roles leave.
#include "common.cuh"
#include "linear.h"

namespace mlk {

namespace {

constexpr int kThreads = 192;
constexpr int kABytes = 128 * 128;
constexpr int kBoxBytes = 32 * 128;            // a warp's store box: 32 tokens x 64 columns
constexpr int kYBytes = 4 * 2 * kBoxBytes;     // two per epilogue warp
constexpr int kTokenGroup = 8;
constexpr uint64_t kPeerDrainNs = 100000;      // 100 us for an aborted odd CTA's copies to land

__host__ __device__ constexpr int stage_bytes(int bn) { return kABytes + bn / 2 * 128; }
__host__ __device__ constexpr int stages_of(int bn) { return bn == 256 ? 6 : 8; }
__host__ __device__ constexpr int smem_bytes(int bn) { return 1024 + stages_of(bn) * stage_bytes(bn) + kYBytes + 256; }

template <int BN>
__global__ void __launch_bounds__(kThreads, 1) linear_wide_kernel(const __grid_constant__ LinearParams p) {
  constexpr int kStages = stages_of(BN);
  constexpr uint32_t STAGE = stage_bytes(BN);
  constexpr uint32_t TMEM_COLS = 2 * BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* ybuf = smem + kStages * STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(ybuf + kYBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;   // [2]
  uint64_t* tempty = tfull + 2;        // [2]
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const bool leader = crank == 0;
  const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1;
  const int NT = (p.N + BN - 1) / BN, TT = p.token_tiles, total = NT * TT;
  const int nk = (p.K + 63) >> 6;
  const bool lora = p.Rs > 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&tfull[0], 1);
    mbar_init(&tfull[1], 1);
    mbar_init(&tempty[0], 8);   // the pair's epilogue warps
    mbar_init(&tempty[1], 8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (p.check_slots && blockIdx.x == 0) *p.status = 0u;   // no adapters: nothing to check
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

  auto decode = [&](int tile, int& tt, int& nt) {
    const int g = tile / (kTokenGroup * NT), r = tile - g * kTokenGroup * NT;
    const int size = min(kTokenGroup, TT - g * kTokenGroup);
    nt = r / size;
    tt = g * kTokenGroup + r - nt * size;
  };
  // (whole warp) the 64-column blocks that some token of tile tt has its adapter in
  auto blocks_of_tile = [&](int tt) -> uint64_t {
    uint64_t m = 0;
    int sl[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = tt * 256 + i * 32 + lane;
      sl[i] = t < p.T ? __ldg(p.slot_idx + t) : -1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (sl[i] >= 0 && sl[i] < p.slots.S && p.slots.hi[sl[i]] > p.slots.lo[sl[i]]) {
        const int b0 = p.slots.lo[sl[i]] >> 6, b1 = (p.slots.hi[sl[i]] - 1) >> 6;
        m |= (~0ull >> (63 - b1)) & (~0ull << b0);
      }
    const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(m));
    const uint32_t hi = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(m >> 32));
    return lo | (static_cast<uint64_t>(hi) << 32);
  };

  if (warp == 0) {   // ------------------------------------------------ TMA producer
    const uint64_t pol = l2_policy_evict_last();
    int stage = 0, ok = 1;
    uint32_t phase = 0, issued = 0, parity = 0;
    bool waited = false;
    auto issue = [&](const CUtensorMap* xm, int kx, int t, const CUtensorMap* wm, int kw, int n) -> bool {
      if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, kWhereLinear)) return false;
      uint8_t* a = smem + stage * STAGE;
      if (leader) mbar_arrive_expect_tx(&full[stage], 2 * STAGE);
      const uint32_t bar = cluster_addr(&full[stage], 0);
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
    for (int tile = pair; tile < total; tile += pairs) {
      int tt, nt;
      decode(tile, tt, nt);
      const uint64_t mask = lora ? blocks_of_tile(tt) : 0ull;
      if (lane == 0) {
        const int t = tt * 256 + static_cast<int>(crank) * 128, n = nt * BN + static_cast<int>(crank) * (BN / 2);
        for (int kb = 0; ok && kb < nk; ++kb) ok = issue(&p.tmap_x, kb * 64, t, &p.tmap_w, kb * 64, n);
        if (ok && mask && !waited) {
          pdl_wait();   // u is written
          waited = true;
        }
        for (uint64_t m = mask; ok && m; m &= m - 1) {
          const int c = (__ffsll(static_cast<long long>(m)) - 1) * 64;
          ok = issue(&p.tmap_u, c, t, &p.tmap_b, c, n);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
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
      constexpr uint32_t idesc = idesc_bf16_f32(256, BN);
      int stage = 0, ok = 1, acc = 0;
      uint32_t phase = 0, aphase = 0;
      for (int tile = pair; tile < total; tile += pairs) {
        int tt, nt;
        decode(tile, tt, nt);
        const uint64_t mask = lora ? blocks_of_tile(tt) : 0ull;
        if (lane == 0) {
          const int steps = nk + __popcll(mask);
          ok = mbar_wait(&tempty[acc], aphase ^ 1u, abort_flag, p.status, kWhereLinear);
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
          for (int i = 0; ok && i < steps; ++i) {
            ok = mbar_wait(&full[stage], phase, abort_flag, p.status, kWhereLinear);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = smem_u32(smem + stage * STAGE);
            const uint64_t ad = sw128_kmajor_desc(a), bd = sw128_kmajor_desc(a + kABytes);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_bf16_pair(d, ad + 2 * kk, bd + 2 * kk, idesc, (i | kk) ? 1u : 0u);
            umma_commit_pair_mc(&empty[stage], 0x3);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) umma_commit_pair_mc(&tfull[acc], 0x3);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (++acc == 2) {
          acc = 0;
          aphase ^= 1u;
        }
      }
      if (!ok && lane == 0) {   // let what was issued finish before TMEM is released
        umma_commit_pair(drain);
        mbar_wait_drain(drain, 0);
      }
    }
  } else {   // ------------------------------------------------------------ epilogue
    if (lora) pdl_wait();   // nothing of this grid is written before the shrink has ended
    const int quarter = warp & 3;
    uint8_t* box0 = ybuf + (warp - 2) * 2 * kBoxBytes;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y);
    int acc = 0, nbox = 0;
    uint32_t aphase = 0;
    for (int tile = pair; tile < total; tile += pairs) {
      int tt, nt;
      decode(tile, tt, nt);
      const int t_warp = tt * 256 + static_cast<int>(crank) * 128 + quarter * 32;
      if (!mbar_wait_sleep(&tfull[acc], aphase, abort_flag, p.status, kWhereLinear)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * BN);
#pragma unroll 1
      for (int c = 0; c < BN; c += 64) {
        const int n = nt * BN + c;
        if (n >= p.N || t_warp >= p.T) break;   // warp-uniform
        uint32_t v[64];
        __syncwarp();
        tmem_ld_x32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(v));
        tmem_ld_x32(taddr + c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
        tmem_ld_wait();
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
          for (int r = 0; r < rows; ++r) {
            const uint32_t two = *reinterpret_cast<const uint32_t*>(box + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
            __nv_bfloat16* row = y + static_cast<long long>(t_warp + r) * p.ldy + n + 2 * lane;
            if (n + 2 * lane < p.N) row[0] = __ushort_as_bfloat16(static_cast<unsigned short>(two & 0xffffu));
            if (n + 2 * lane + 1 < p.N) row[1] = __ushort_as_bfloat16(static_cast<unsigned short>(two >> 16));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&tempty[acc], 0));
      if (++acc == 2) {
        acc = 0;
        aphase ^= 1u;
      }
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

cudaError_t linear_wide_setup() {
  cudaError_t err = cudaFuncSetAttribute(linear_wide_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes(256));
  if (err != cudaSuccess) return err;
  return cudaFuncSetAttribute(linear_wide_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(128));
}

cudaError_t launch_linear_wide(const LinearParams& p, int bn, int sms, cudaStream_t stream, bool pdl) {
  const long long tiles = static_cast<long long>((p.N + bn - 1) / bn) * p.token_tiles;
  if (tiles > 0x3fffffffLL || (bn != 128 && bn != 256)) return cudaErrorInvalidValue;
  const int pairs = static_cast<int>(tiles < sms / 2 ? tiles : sms / 2);
  const dim3 grid(2 * pairs), block(kThreads);
  if (bn == 256) return launch_kc(linear_wide_kernel<256>, grid, block, smem_bytes(256), stream, pdl, 2, p);
  return launch_kc(linear_wide_kernel<128>, grid, block, smem_bytes(128), stream, pdl, 2, p);
}

}  // namespace mlk
