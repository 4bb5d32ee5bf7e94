// The projection with adapters of linear_narrow.cu for decode batches whose stacked ranks fit one
// 128-row tile: every cluster shrinks for itself.
//
// A tile is again 128 weight rows x BN tokens whose K a cluster of CTAs shares.  Each K step also
// brings the same 64 columns of the stacked A (the 64-row blocks that a token of the tile needs)
// and a second accumulator takes As x beside W x.  Both part sums are exchanged through
// distributed shared memory behind one cluster barrier; each CTA then sums its share of the
// tokens, scales and masks u, rounds it to bf16 pieces straight into an MMA operand, and the stacked
// B (copied during the exchange) takes it to the delta in TMEM.  Against the flag of the narrow
// kernel (u through global memory from other clusters) this reads the stacked A once per row tile,
// from L2, and saves that round trip: T 1, N 2048, K 2048, rank 16 (K over 8 CTAs) takes 6.0 us, 7.9 on
// the narrow kernel, 4.3 there without adapters; T 16, N 4096, K 7168: 13.7, 14.7 and 12.4 (8.7 for
// its 59 MB at 6.8 TB/s).  Past 32 tokens a tile the narrow kernel is ahead (T 64, N 5120, K 2048:
// 11.6 us against 14.6 here).
//
// Warp 0: TMA producer (and the tile's slots); warp 1: MMA issuer; warps 2-5: epilogue.
#include "common.cuh"
#include "linear.h"
#include "linear_nonfinite.cuh"

namespace mlk {

namespace {

constexpr int kThreads = 192;
constexpr int kTile = 128 * 128;          // 128 rows x 64 columns of bf16
constexpr int kMaxSplit = kLinearMaxSplit;

// nb: 64-row blocks of the stacked A, 1 or 2.  Two CTAs share an SM.
__host__ __device__ constexpr int stage_bytes(int bn, int nb) { return kTile + nb * kTile / 2 + bn * 128; }
__host__ __device__ constexpr int stages_of(int bn, int nb) { return nb == 1 && bn == 16 ? 4 : 3; }
// The MMA over As reads 128 rows whatever nb is: past a stage's A lie its tokens and the next stage,
// past the last stage's what is left of 128 rows, allocated here (its sums are never read).
__host__ __device__ constexpr int tail_bytes(int bn, int nb) {
  const int rest = 2 * kTile - stage_bytes(bn, nb), own = bn * 12 + 256;
  return rest > own ? rest : own;
}
__host__ __device__ constexpr int smem_bytes(int bn, int nb) {
  return 1024 + stages_of(bn, nb) * stage_bytes(bn, nb) + tail_bytes(bn, nb);
}

// Sums of two neighbouring tokens' values over the C CTAs of the cluster, in rank order; all loads
// go out before the first is used.
template <int C>
MLDEV float2 cluster_sum2(uint32_t at) {
  float u[C], v[C];
#pragma unroll
  for (int r = 0; r < C; ++r) {
    u[r] = ld_cluster_f(at, r);
    v[r] = ld_cluster_f(at + 512, r);
  }
  float2 s = make_float2(u[0], v[0]);
#pragma unroll
  for (int r = 1; r < C; ++r) {
    s.x += u[r];
    s.y += v[r];
  }
  return s;
}

// LONG: as in linear_narrow.cu.
template <int BN, int NB, bool LONG>
__global__ void __launch_bounds__(kThreads, 2) linear_cluster_kernel(const __grid_constant__ LinearParams p) {
  constexpr int kStages = stages_of(BN, NB);
  constexpr uint32_t STAGE = stage_bytes(BN, NB);
  constexpr uint32_t X_AT = kTile + NB * kTile / 2;          // the tokens' part of a stage
  // after the main loop the stages hold part sums [BN][128] of W x and As x, u as an operand
  // [pieces][NB][BN rows x 128 B], and the stacked B's tile (NB blocks of 64 columns)
  constexpr uint32_t PART = BN * 128 * 4;
  constexpr uint32_t U_AT = 2 * PART, B_AT = U_AT + kFloatPieces * NB * BN * 128;
  static_assert(B_AT % 1024 == 0 && B_AT + NB * kTile <= kStages * STAGE, "they fit the stages");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* b_s = smem + B_AT;
  uint8_t* u_s = smem + U_AT;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * STAGE);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* mask_bar = tfull + 1;
  uint64_t* bfull = mask_bar + 1;
  uint64_t* dfull = bfull + 1;
  uint64_t* drain = dfull + 1;
  volatile uint32_t* mask_s = reinterpret_cast<volatile uint32_t*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1) + 1;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* lo_s = reinterpret_cast<int*>(tmem_slot + 2);         // [BN] a token's columns of the stack and
  int* hi_s = lo_s + BN;                                     // its factor
  float* sc_s = reinterpret_cast<float*>(hi_s + BN);

  // TMEM: the accumulators of W x, those of As x, the delta
  const uint32_t kaccs = LONG ? p.accs : 1, as_at = kaccs * BN, delta_at = 2 * as_at;
  const uint32_t tmem_cols = linear_tmem_columns(2 * kaccs + 1, BN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = static_cast<int>(cluster_nctas()), rank = static_cast<int>(cluster_ctarank());
  const int tile = static_cast<int>(blockIdx.x) / C;
  const int nt = tile / p.token_tiles, qt = tile - nt * p.token_tiles;
  const int row0 = nt * 128, t0 = qt * BN;
  const int nvalid = min(BN, p.T - t0);
  // this CTA's tokens of the tile: [j_lo, j_hi)
  const int j_lo = nvalid * rank / C, j_hi = nvalid * (rank + 1) / C, count = j_hi - j_lo;
  const int nk = (p.K + 63) >> 6;
  const int k_lo = static_cast<int>(static_cast<long long>(nk) * rank / C);
  const int k_hi = static_cast<int>(static_cast<long long>(nk) * (rank + 1) / C);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 2);   // W and x; the blocks of A
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(mask_bar, 1);
    mbar_init(bfull, 1);
    mbar_init(dfull, 1);
    mbar_init(drain, 1);
    *mask_s = 0u;
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmap_w);
    tma_prefetch_desc(&p.tmap_x);
    tma_prefetch_desc(&p.tmap_a);
    tma_prefetch_desc(&p.tmap_b);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();   // the kernel in front may have made the call's data
  pdl_trigger();
  unsigned long long sick = 0;   // (epilogue) slots with weights that are not finite

  if (warp == 0) {   // ------------------------------------------------ TMA producer
    const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
    const int ahead = min(kStages, k_hi - k_lo);
    auto load_w = [&](int s, int kb) {
      uint8_t* a = smem + s * STAGE;
      mbar_arrive_expect_tx(&full[s], kTile + BN * 128);
      tma_load_2d(a, &p.tmap_w, &full[s], kb * 64, row0, p.token_tiles == 1 ? pol_w : pol_x);
      tma_load_2d(a + X_AT, &p.tmap_x, &full[s], kb * 64, t0, pol_x);
    };
    if (lane == 0)   // the first stages go out before the slots are known
      for (int s = 0; s < ahead; ++s) load_w(s, k_lo + s);
    __syncwarp();
    unsigned m = 0;   // 64-row blocks of the stack (NB at most) that a token needs
#pragma unroll
    for (int j = lane; j < BN; j += 32) {
      const int sl = j < nvalid ? p.slot_idx[t0 + j] : -1;
      if (sl >= 0 && sl < p.slots.S && p.slots.hi[sl] > p.slots.lo[sl])
        m |= (1u << (p.slots.lo[sl] >> 6)) | (1u << ((p.slots.hi[sl] - 1) >> 6));
    }
    const unsigned mask = __reduce_or_sync(0xffffffffu, m);
    if (lane == 0) {
      *mask_s = mask;
      mbar_arrive(mask_bar);
      auto load_a = [&](int s, int kb) {
        uint8_t* a = smem + s * STAGE + kTile;
        if (mask == 0) {
          mbar_arrive(&full[s]);
          return;
        }
        mbar_arrive_expect_tx(&full[s], __popc(mask) * (kTile / 2));
        for (int b = 0; b < NB; ++b)
          if ((mask >> b) & 1u) tma_load_2d(a + b * (kTile / 2), &p.tmap_a, &full[s], kb * 64, b * 64, pol_x);
      };
      for (int s = 0; s < ahead; ++s) load_a(s, k_lo + s);
      int stage = 0, ok = 1;
      uint32_t phase = 1;   // the second use of each stage on
      if (ahead < kStages) stage = ahead;
      for (int kb = k_lo + ahead; ok && kb < k_hi; ++kb) {
        ok = mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, kWhereLinear);
        if (!ok) break;
        load_w(stage, kb);
        load_a(stage, kb);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {   // let every issued copy land: each stage's last use
        const int n = k_hi - k_lo;
        for (int s = 0; s < kStages && s < n; ++s) {
          mbar_wait_drain(&full[s], 0);
          mbar_wait_drain(&full[s], 1);
        }
      }
    }
  } else if (warp == 1) {   // ------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, BN);
      int stage = 0, left = p.acc_steps;
      bool first = true;
      uint32_t phase = 0, d = tmem_base;
      int ok = mbar_wait(mask_bar, 0, abort_flag, p.status, kWhereLinear);
      const bool shrink = *mask_s != 0u;
      for (int kb = k_lo; ok && kb < k_hi; ++kb) {
        ok = mbar_wait(&full[stage], phase, abort_flag, p.status, kWhereLinear);
        if (!ok) break;
        if (LONG && left-- == 0) {   // the next accumulators
          d += BN;
          first = true;
          left = p.acc_steps - 1;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(smem + stage * STAGE);
        const uint64_t wd = sw128_kmajor_desc(a), ad = sw128_kmajor_desc(a + kTile), xd = sw128_kmajor_desc(a + X_AT);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16(d, wd + 2 * kk, xd + 2 * kk, idesc, ((LONG ? !first : kb > k_lo) || kk > 0) ? 1u : 0u);
        if (shrink) {   // rows of blocks that were not copied give sums that nothing reads
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(d + as_at, ad + 2 * kk, xd + 2 * kk, idesc, ((LONG ? !first : kb > k_lo) || kk > 0) ? 1u : 0u);
        }
        first = false;
        umma_commit(&empty[stage]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
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
    sick = __ldcg(p.sick);
    if (et < BN) {
      const int sl = et < nvalid ? p.slot_idx[t0 + et] : -1;
      const bool has = sl >= 0 && sl < p.slots.S;
      lo_s[et] = has ? p.slots.lo[sl] : 0;
      hi_s[et] = has ? p.slots.hi[sl] : 0;
      sc_s[et] = has ? p.slots.scal[sl] : 0.0f;
    }
    if (blockIdx.x == 0) {   // the only writer of the status word before a timeout
      int bad = 0;
#pragma unroll 4
      for (int t = et; t < p.T; t += 128) {
        const int sl = p.slot_idx[t];
        bad |= sl < -1 || sl >= p.slots.S;
      }
      const bool any = any_of_128(bad);
      if (et == 0) *p.status = any ? (kDevBadSlot | (kWhereLinear << 8)) : 0u;
    }
    const int quarter = warp & 3;
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    float* part = reinterpret_cast<float*>(smem) + quarter * 32 + lane;   // W x, then As x: [BN][128]
    if (mbar_wait(mask_bar, 0, abort_flag, p.status, kWhereLinear) &&
        mbar_wait_sleep(tfull, 0, abort_flag, p.status, kWhereLinear)) {
      const unsigned mask = *mask_s;
      const bool shrink = mask != 0u;
      const int accs = LONG ? (k_hi - k_lo - 1) / p.acc_steps + 1 : 1;   // of this CTA
      tc_fence_after();
      // The MMAs are past the stages: B's tile comes in, where tokens of this CTA will use it (a copy
      // that nothing waits for must not outlive the CTA).
      if (shrink && count > 0 && threadIdx.x == 64) {
        mbar_arrive_expect_tx(bfull, __popc(mask) * kTile);
        const uint64_t pol = l2_policy_evict_last();
        for (int b = 0; b < NB; ++b)
          if ((mask >> b) & 1u) tma_load_2d(b_s + b * kTile, &p.tmap_b, bfull, b * 64, row0, pol);
      }
#pragma unroll 1
      for (int c = 0; c < BN && t0 + c < p.T; c += 16) {   // warp-uniform bound
        uint32_t v[16], w[16];
        __syncwarp();   // tcgen05.ld is .aligned
        tmem_ld_x16(taddr + c, v);
        if (shrink) tmem_ld_x16(taddr + as_at + c, w);   // (rows past NB * 64: never read)
        tmem_ld_wait();
#pragma unroll 1
        for (int a = 1; a < accs; ++a) {   // accumulators in order
          uint32_t x[16], y[16];
          __syncwarp();
          tmem_ld_x16(taddr + a * BN + c, x);
          if (shrink) tmem_ld_x16(taddr + as_at + a * BN + c, y);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(x[j]));
          if (shrink) {
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) + __uint_as_float(y[j]));
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * 128] = __uint_as_float(v[j]);
        if (shrink) {
#pragma unroll
          for (int j = 0; j < 16; ++j) part[(BN + c + j) * 128] = __uint_as_float(w[j]);
        }
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();

  const unsigned mask = *mask_s;
  const uint32_t part0 = smem_u32(smem);
  if (count > 0 && mask != 0u) {   // u of these tokens, as rows of an MMA operand
    for (int i = threadIdx.x; i < count * 16 * NB; i += kThreads) {
      const int j = i / (16 * NB), c = (i & (16 * NB - 1)) * 4, b = c >> 6;
      if (!((mask >> b) & 1u)) continue;
      const int lo = lo_s[j_lo + j], hi = hi_s[j_lo + j];
      const float sc = sc_s[j_lo + j];
      float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (c + 4 > lo && c < hi) {
        float4 v[kMaxSplit];
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r)
          if (r < C) v[r] = ld_cluster_f4(part0 + PART + static_cast<uint32_t>(((j_lo + j) * 128 + c) * 4), r);
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r)
          if (r < C) {
            f[0] += v[r].x;
            f[1] += v[r].y;
            f[2] += v[r].z;
            f[3] += v[r].w;
          }
#pragma unroll
        for (int q = 0; q < 4; ++q) f[q] = (c + q >= lo && c + q < hi) ? sc * f[q] : 0.0f;
      }
      uint8_t* at = u_s + b * BN * 128 + j * 128 + ((((c & 63) >> 3) ^ (j & 7)) << 4) + (c & 7) * 2;
      if (p.pieces == 1) {
        *reinterpret_cast<uint2*>(at) = pack4(f);
      } else {   // a float32 as a sum of bf16 pieces
        for (int piece = 0; piece < p.pieces; ++piece)
          *reinterpret_cast<uint2*>(at + piece * NB * BN * 128) = take_leading4(f);
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (warp == 1 && lane == 0) {
      if (mbar_wait(bfull, 0, abort_flag, p.status, kWhereLinear)) {
        const uint32_t idesc = idesc_bf16_f32(128, (count + 15) / 16 * 16);
        int first = 1;
        for (int piece = 0; piece < p.pieces; ++piece)
          for (int b = 0; b < NB; ++b) {
            if (!((mask >> b) & 1u)) continue;
            const uint64_t bd = sw128_kmajor_desc(smem_u32(b_s + b * kTile));
            const uint64_t ud = sw128_kmajor_desc(smem_u32(u_s + (piece * NB + b) * BN * 128));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              umma_bf16(tmem_base + delta_at, bd + 2 * kk, ud + 2 * kk, idesc, first ? 0u : 1u);
              first = 0;
            }
          }
        umma_commit(dfull);
        mbar_wait_drain(dfull, 0);   // also where the epilogue has given up: nothing is freed under the MMAs
      } else {
        mbar_wait_drain(bfull, 0);   // given up: B's tile may be on its way, and lands before the CTA leaves
      }
    }
  }
  if (count > 0 && warp >= 2) {   // a thread per weight row: sums in rank order, delta, bias
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane, n = row0 + row;
    const float bias = (p.bias != nullptr && n < p.N) ? __ldg(p.bias + n) : 0.0f;
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + delta_at;
    bool waited = mask == 0u;
#pragma unroll 1
    for (int c = 0; c < count; c += 8) {   // warp-uniform bound
      float f[8];
      const uint32_t at = part0 + static_cast<uint32_t>(((j_lo + c) * 128 + row) * 4);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        if (c + j >= count) break;   // (the second token of a pair may lie past the share: not used)
        const float2 s = C == 8   ? cluster_sum2<8>(at + j * 512)
                         : C == 4 ? cluster_sum2<4>(at + j * 512)
                         : C == 2 ? cluster_sum2<2>(at + j * 512)
                                  : cluster_sum2<1>(at + j * 512);
        f[j] = s.x;
        f[j + 1] = s.y;
      }
      if (mask != 0u) {
        if (!waited && !mbar_wait_sleep(dfull, 0, abort_flag, p.status, kWhereLinear)) break;
        waited = true;
        tc_fence_after();
        uint32_t d[8];
        __syncwarp();
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]), "=r"(d[7])
                     : "r"(taddr + c));
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += __uint_as_float(d[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (c + j < count && n < p.N) {
          const long long at = static_cast<long long>(t0 + j_lo + c + j) * p.ldy + n;
          if (p.y_f32) static_cast<float*>(p.y)[at] = f[j] + bias;
          else static_cast<__nv_bfloat16*>(p.y)[at] = f2bf(f[j] + bias);
        }
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_arrive();   // no CTA leaves while others read its part sums
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols);
  }
  if (sick != 0 && mask != 0u)
    add_nonfinite_of_operand<BN, NB>(p, sick, u_s, t0 + j_lo, count, row0 + (warp & 3) * 32 + lane);
}

}  // namespace

cudaError_t linear_cluster_setup() {
  cudaError_t err;
#define ML_SETUP(BN, NB, LONG)                                                                                    \
  err = cudaFuncSetAttribute(linear_cluster_kernel<BN, NB, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize,    \
                             smem_bytes(BN, NB));                                                                 \
  if (err != cudaSuccess) return err;
#define ML_SETUPS(BN, NB) ML_SETUP(BN, NB, false) ML_SETUP(BN, NB, true)
  ML_SETUPS(16, 1)
  ML_SETUPS(16, 2)
  ML_SETUPS(32, 1)
  ML_SETUPS(32, 2)
#undef ML_SETUPS
#undef ML_SETUP
  return cudaSuccess;
}

cudaError_t launch_linear_cluster(const LinearParams& p, int bn, int split, cudaStream_t stream) {
  const long long tiles = static_cast<long long>((p.N + 127) / 128) * p.token_tiles;
  if (p.Rs < 1 || p.Rs > 128 || (bn != 16 && bn != 32) || tiles * split > 0x7fffffffLL || p.accs < 1 ||
      (2 * p.accs + 1) * bn > kLinearTmem)
    return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(tiles * split)), block(kThreads);
#define ML_LINEAR(BN, NB)                                                                                             \
  return p.accs > 1                                                                                                   \
             ? launch_kc(linear_cluster_kernel<BN, NB, true>, grid, block, smem_bytes(BN, NB), stream, true, split, p) \
             : launch_kc(linear_cluster_kernel<BN, NB, false>, grid, block, smem_bytes(BN, NB), stream, true, split, p)
  if (p.Rs <= 64) {
    if (bn == 16) ML_LINEAR(16, 1);
    ML_LINEAR(32, 1);
  }
  if (bn == 16) ML_LINEAR(16, 2);
  ML_LINEAR(32, 2);
#undef ML_LINEAR
}

}  // namespace mlk
