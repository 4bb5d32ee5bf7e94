// Attention of few rows a key head (decoding, short drafts): up to 16 query rows of a request and key head
// against its pages, and the sum of the pieces of items that were cut.
//
// What bounds it is memory: 8 query heads on a key head of 128 do 16 operations a byte of the cache.  So the
// cache is streamed by TMA (a box a page, 128-byte swizzle) through a ring of 32 KB stages, 64 keys and their
// values each, two blocks an SM; the products are small enough for mma.sync, whose fragments keep a
// warp's 16 keys x 16 rows in registers from the scores to the weights, and whose idle tile rows cost
// nothing that is scarce here.  Each warp has a quarter of every stage and a softmax of its own; the four are
// added at the end of the item's part.  Weights go into the second product as two bf16 pieces.
#include "attention.h"
#include "host.h"

namespace mlk {
namespace {

constexpr int kRows = kFewRows, kKeys = kFewKeys;
constexpr int kConsumers = 4, kThreads = 32 * (kConsumers + 1);
using Sched = Schedule<kRows, kKeys, kFewOver>;
using Place = Walk<kRows, kKeys, kFewOver>;

__host__ __device__ constexpr int stage_bytes(int dp) { return 2 * kKeys * dp * 2; }   // keys, then values
__host__ __device__ constexpr int stages_of(int dp) { return dp == 64 ? 6 : 3; }
// the ring, the block's sum of its warps' results, and the rest
constexpr int smem_bytes(int dp) { return stages_of(dp) * stage_bytes(dp) + kRows * dp * 4 + 1024; }

MLDEV void ldsm4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
MLDEV void ldsm4_t(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
MLDEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
MLDEV uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
MLDEV void consumer_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

template <int DP>
__global__ void __launch_bounds__(kThreads, kFewPerSm) attention_rows_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int kStages = stages_of(DP), STAGE = stage_bytes(DP), HALVES = DP / 64;
  constexpr int kHalf = kKeys * 128;   // 64 values of every key of a stage
  extern __shared__ __align__(1024) uint8_t smem[];
  float* sum_s = reinterpret_cast<float*>(smem + kStages * STAGE);   // [kRows][DP]
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ float m_s[kConsumers][kRows], l_s[kConsumers][kRows];
  __shared__ ScheduleSmem sched_s;
  __shared__ long long sums_s[kThreads];
  __shared__ uint32_t error_s;
  __shared__ int abort_s;
  volatile int* abort_flag = &abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = static_cast<int>(blockIdx.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kConsumers);
    }
    error_s = 0;
    abort_s = 0;
    fence_mbar_init();
  }
  if (warp == kConsumers && lane == 0) {
    tma_prefetch_desc(&p.tmap_k);
    tma_prefetch_desc(&p.tmap_v);
  }
  __syncthreads();
  // With shared keys the kernel in front is their launch, whose results are not needed here; what came before
  // it is done, since it has waited for that.
  if (p.prefix_splits == 0) pdl_wait();
  pdl_trigger();

  Sched s;
  Place w;
  make_schedule<kRows, kKeys, kFewOver>(p, cta, s, w, sched_s, sums_s);
  if (threadIdx.x == 0 && s.bad) record_status(&error_s, kDevBadSlot, kWhereAttention);

  if (warp == kConsumers) {   // ------------------------------------------------ producer
    const uint64_t policy = l2_policy_evict_first();
    const int box_log2 = min(p.page_log2, 6), box = 1 << box_log2, boxes = kKeys >> box_log2;   // boxes of a unit
    int stage = 0, ok = 1;
    uint32_t phase = 0, issued = 0, parity = 0;
    for (; ok && more<kRows, kKeys, kFewOver>(s, w, p); w.next(p)) {
      const Part x = part_of<kRows, kKeys, kFewOver>(p, s, w, cta);
      const int sees = Sched::seen_by(p, w.r, w.i);
      const int32_t* table = p.tables + w.b * p.table_stride;
      // A lane a box; its page is looked up a unit ahead of its use.
      auto page_at = [&](int j) -> int {
        const int key = p.shared + j * kKeys + (lane << box_log2);
        return lane < boxes && j < x.hi && key < sees ? table[key >> p.page_log2] : -1;
      };
      int ahead = x.lo < x.hi ? page_at(x.lo) : -1;
      for (int j = x.lo; j < x.hi; ++j) {
        const int key = p.shared + j * kKeys + (lane << box_log2);
        const bool mine = lane < boxes && key < sees;
        int page = ahead;
        ahead = page_at(j + 1);
        if (mine && (page < 0 || page >= p.num_pages)) {   // read as zeros: outside the map
          record_status(&error_s, kDevBadSlot, kWhereAttention);
          page = -1;
        }
        const int n = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) {
          ok = wait_soon(&empty[stage], phase ^ 1u, abort_flag, &error_s);
          if (ok) mbar_arrive_expect_tx(&full[stage], n * 2 * box * HALVES * 128);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (mine) {
          uint8_t* at = smem + stage * STAGE + lane * box * 128;
          const int token = key & (p.page - 1);
#pragma unroll
          for (int half = 0; half < HALVES; ++half) {
            tma_load_page(at + half * kHalf, &p.tmap_k, &full[stage], half * 64, token, w.kh, page, policy);
            tma_load_page(at + (HALVES + half) * kHalf, &p.tmap_v, &full[stage], half * 64, token, w.kh, page, policy);
          }
        }
        issued |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0)
      for (int t = 0; t < kStages; ++t)
        if ((issued >> t) & 1u) mbar_wait_drain(&full[t], (parity >> t) & 1u);
    __syncwarp();
  } else {   // ------------------------------------------------------------------ consumers
    const int ra = lane >> 2, rb = ra + 8, pair = (lane & 3) * 2;
    int stage = 0, ok = 1;
    uint32_t phase = 0;
    bool started = false;   // an item whose rest is other blocks'
    for (; ok && more<kRows, kKeys, kFewOver>(s, w, p); w.next(p)) {
      const Part x = part_of<kRows, kKeys, kFewOver>(p, s, w, cta);
      if (x.lo >= x.hi) continue;
      const int row0 = w.i * kRows;
      const int rows = min(kRows, w.r.n * p.G - row0);
      const int sees = Sched::seen_by(p, w.r, w.i);
      const bool upper = rows > 8;   // the fragments' rows 8 to 15 are in use
      int lim_a = 0, lim_b = 0;      // keys that this lane's two rows see
      uint32_t qf[DP / 16][4];
      {
        const __nv_bfloat16 *qa = nullptr, *qb = nullptr;
        if (ra < rows) {
          const int t = (row0 + ra) / p.G;
          qa = p.q + (w.r.q0 + t) * p.q_t + (w.kh * p.G + (row0 + ra) % p.G) * p.q_h;
          lim_a = max(w.r.kv - w.r.n + t + 1, 0);
        }
        if (rb < rows) {
          const int t = (row0 + rb) / p.G;
          qb = p.q + (w.r.q0 + t) * p.q_t + (w.kh * p.G + (row0 + rb) % p.G) * p.q_h;
          lim_b = max(w.r.kv - w.r.n + t + 1, 0);
        }
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
          const int c = ks * 16 + pair;
          auto at = [&](const __nv_bfloat16* q, int d) {
            return q != nullptr && d < p.D ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
          };
          qf[ks][0] = at(qa, c);
          qf[ks][1] = at(qb, c);
          qf[ks][2] = at(qa, c + 8);
          qf[ks][3] = at(qb, c + 8);
        }
      }
      const int all_see = max(w.r.kv - w.r.n + row0 / p.G + 1, 0);   // keys that every row of the item sees
      float o[DP / 8][4];
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
      float ma = -INFINITY, mb = -INFINITY, la = 0.0f, lb = 0.0f;
      for (int j = x.lo; j < x.hi; ++j) {
        ok = wait_soon(&full[stage], phase, abort_flag, &error_s);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int k0 = p.shared + j * kKeys + warp * 16;   // this warp's keys of the unit
        if (k0 < sees) {
          const uint32_t kb = smem_u32(smem) + stage * STAGE + warp * 16 * 128;
          const uint32_t vb = kb + HALVES * kHalf;
          const int t8 = lane & 7;
          bool wrote = false;
          if (k0 + 16 > sees) {   // values that no row sees may be anything, and 0 times it would stay
            wrote = true;
            for (int c = lane; c < 16 * 8 * HALVES; c += 32) {
              const int t = (c >> 3) & 15;
              if (k0 + t >= sees)
                *reinterpret_cast<uint4*>(smem + stage * STAGE + (HALVES + (c >> 7)) * kHalf + (warp * 16 + t) * 128 +
                                          (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
          }
          float sc[2][4] = {};
          // matrices of a ldmatrix: keys 0-7 and 8-15, each with 8 dims and the next 8
          const uint32_t krow = kb + ((lane >> 4) * 8 + t8) * 128;
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks) {
            uint32_t f[4];
            ldsm4(krow + (ks >> 2) * kHalf + (((((ks & 3) << 1) + ((lane >> 3) & 1)) ^ t8) << 4), f);
            mma16816(sc[0], qf[ks], f[0], f[1]);
            mma16816(sc[1], qf[ks], f[2], f[3]);
          }
          const bool cut = k0 + 16 > all_see;
          float xa = ma, xb = mb;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sc[n][e] *= p.scale_log2;
              if (cut && k0 + n * 8 + pair + (e & 1) >= (e < 2 ? lim_a : lim_b)) sc[n][e] = -INFINITY;
            }
            xa = fmaxf(xa, fmaxf(sc[n][0], sc[n][1]));
            xb = fmaxf(xb, fmaxf(sc[n][2], sc[n][3]));
          }
          xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
          xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
          xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2));
          xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2));
          const float refa = reference_of(xa), refb = reference_of(xb);
          if (__any_sync(0xffffffffu, xa > ma || xb > mb)) {
            const float fa = exp2_approx(ma - refa), fb = exp2_approx(mb - refb);
            la *= fa;
            lb *= fb;
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
              o[n][0] *= fa;
              o[n][1] *= fa;
              o[n][2] *= fb;
              o[n][3] *= fb;
            }
            ma = xa;
            mb = xb;
          }
          uint32_t hi[4], lo[4];   // weights as the second product's operand, in two bf16 pieces
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float w0 = exp2_approx(sc[n][0] - refa), w1 = exp2_approx(sc[n][1] - refa);
            float w2 = exp2_approx(sc[n][2] - refb), w3 = exp2_approx(sc[n][3] - refb);
            la += w0 + w1;
            lb += w2 + w3;
            hi[2 * n] = pack2(w0, w1);
            hi[2 * n + 1] = pack2(w2, w3);
            const __nv_bfloat162 ha = *reinterpret_cast<__nv_bfloat162*>(&hi[2 * n]);
            const __nv_bfloat162 hb = *reinterpret_cast<__nv_bfloat162*>(&hi[2 * n + 1]);
            lo[2 * n] = pack2(w0 - __low2float(ha), w1 - __high2float(ha));
            lo[2 * n + 1] = pack2(w2 - __low2float(hb), w3 - __high2float(hb));
          }
          // matrices: keys 0-7 and 8-15 of 8 dims, then of the next 8
          const uint32_t vrow = vb + (((lane >> 3) & 1) * 8 + t8) * 128;
#pragma unroll
          for (int n2 = 0; n2 < DP / 16; ++n2) {
            uint32_t f[4];
            ldsm4_t(vrow + (n2 >> 2) * kHalf + (((((n2 & 3) << 1) + (lane >> 4)) ^ t8) << 4), f);
            mma16816(o[2 * n2], hi, f[0], f[1]);
            mma16816(o[2 * n2 + 1], hi, f[2], f[3]);
            mma16816(o[2 * n2], lo, f[0], f[1]);
            mma16816(o[2 * n2 + 1], lo, f[2], f[3]);
          }
          if (wrote) fence_proxy_async_smem();   // before the stage is filled again by TMA
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // ---- the four warps' results together
      la += __shfl_xor_sync(0xffffffffu, la, 1);
      lb += __shfl_xor_sync(0xffffffffu, lb, 1);
      la += __shfl_xor_sync(0xffffffffu, la, 2);
      lb += __shfl_xor_sync(0xffffffffu, lb, 2);
      if ((lane & 3) == 0) {
        m_s[warp][ra] = ma;
        m_s[warp][rb] = mb;
        l_s[warp][ra] = la;
        l_s[warp][rb] = lb;
      }
      ok = !any_of_128(!ok);   // a barrier; a wait that ran out ends the work of all four
      if (!ok) break;
      float Ma = -INFINITY, Mb = -INFINITY;
#pragma unroll
      for (int v = 0; v < kConsumers; ++v) {
        Ma = fmaxf(Ma, m_s[v][ra]);
        Mb = fmaxf(Mb, m_s[v][rb]);
      }
      const float fa = exp2_approx(ma - reference_of(Ma)), fb = exp2_approx(mb - reference_of(Mb));
#pragma unroll
      for (int v = 0; v < kConsumers; ++v) {   // one warp after another: a fixed order
        if (warp == v) {
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            float2* a = reinterpret_cast<float2*>(sum_s + ra * DP + n * 8 + pair);
            float2 t = v == 0 ? make_float2(0.0f, 0.0f) : *a;
            *a = make_float2(t.x + o[n][0] * fa, t.y + o[n][1] * fa);
            if (upper) {
              float2* c = reinterpret_cast<float2*>(sum_s + rb * DP + n * 8 + pair);
              t = v == 0 ? make_float2(0.0f, 0.0f) : *c;
              *c = make_float2(t.x + o[n][2] * fb, t.y + o[n][3] * fb);
            }
          }
        }
        consumer_sync();
      }
      // ---- eight values of a row a thread
      for (int c = threadIdx.x; c < rows * (DP / 8); c += 32 * kConsumers) {
        const int r = c / (DP / 8), d = (c % (DP / 8)) * 8;
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int v = 0; v < kConsumers; ++v) m = fmaxf(m, m_s[v][r]);
#pragma unroll
        for (int v = 0; v < kConsumers; ++v) l += l_s[v][r] * exp2_approx(m_s[v][r] - reference_of(m));
        float val[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) val[i] = sum_s[r * DP + d + i];
        const long long token = w.r.q0 + (row0 + r) / p.G;
        const int head = w.kh * p.G + (row0 + r) % p.G;
        if (x.all && p.prefix_splits == 0) {
          write_row8(p, token, head, d, m, l, val);
        } else {
          const long long at = x.all ? part_row(p, token, head) : static_cast<long long>(x.slot) * p.item_rows + r;
          float4* to = reinterpret_cast<float4*>((x.all ? p.part_o : p.piece_o) + at * DP + d);
          to[0] = make_float4(val[0], val[1], val[2], val[3]);
          to[1] = make_float4(val[4], val[5], val[6], val[7]);
          if (d == 0) (x.all ? p.part_ml : p.piece_ml)[at] = make_float2(m, l);
        }
      }
      if (!x.all && x.lo == 0 && threadIdx.x == 0) {
        p.records[cta] = record_of<kRows, kKeys, kFewOver>(p, s, w, x, cta);
        started = true;
      }
    }
    if (!started && threadIdx.x == 0 && p.records != nullptr) p.records[cta].pieces = 0;
  }
  if (p.prefix_splits > 0) pdl_wait();   // not to end before the launch in front, which the next one reads from
  __syncthreads();
  if (threadIdx.x == 0) finish_status(p, error_s, p.records == nullptr && p.prefix_splits == 0);
}

}  // namespace

cudaError_t prepare_attention_rows() {
  cudaError_t e = cudaFuncSetAttribute(attention_rows_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(64));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attention_rows_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(128));
  return e;
}

cudaError_t launch_attention_rows(const AttentionParams& p, int dp, cudaStream_t stream) {
  const dim3 grid(p.plan.ctas), block(kThreads);
  return dp == 64 ? launch_k(attention_rows_kernel<64>, grid, block, smem_bytes(64), stream, true, p)
                  : launch_k(attention_rows_kernel<128>, grid, block, smem_bytes(128), stream, true, p);
}

}  // namespace mlk
