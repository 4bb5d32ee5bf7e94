// Attention of few rows a key head (decoding, short drafts): up to 16 query rows of a request and key head
// against its pages, and the sum of the pieces of items that were cut.
//
// What bounds it is memory: 8 query heads on a key head of 128 do 16 operations a byte of the cache.  So the
// cache is streamed by TMA (a box a page, 128-byte swizzle) through a ring of 32 KB stages, 64 keys and their
// values each, two blocks an SM.  The products run on mma.sync with the keys, then the values' dimensions, as its 16
// rows and up to 8 query rows as its 8 columns, so that nothing is padded:
//
//   S^T [16 keys, 8 rows] = K Q^T,   O^T [16 dimensions, 8 rows] += V^T P^T
//
// (with query rows on the 16-row side there were twice as many MMAs, 48 for a warp's 16 keys, and these, at
// about 32 cycles each, and not the memory were what decoding waited for).  P^T goes from the first product's layout to
// the second's by transposing 8 x 8 matrices between lanes.  Each warp has a quarter of every stage and a softmax of
// its own, relative to the maxima of its first 16 keys (attention.h, kHeadroom, says why that is enough); the four are
// added at the end of the item's part.  Weights go into the second product as two bf16 pieces (16 bits), which costs no
// time, since the tensor cores are 13% busy.
//
// Measured, 32 query heads on 4 key heads of 128: 64 requests on 200 to 5000 keys, 374 MB, 62.5 to 63.7 us, 5.9 TB/s (88% of a
// plain copy's rate); 256 on 1000 keys 89; one on 700 keys 6.7 and the join's 2, a chain of dependent latencies: lengths,
// table, keys, products, the sum of the warps, and the fetch of code that no call before has left in the caches.
// Items of 8 rows for up to 8 rows, else of 16 (NT): 16 requests of 8 rows on 2000 keys 16.4 us, in items of 16 19.7, and 256 on
// 100 keys 21.5 and 27.1; 24 requests of 28 rows on 1000 to 9000 keys in items of 16 74, of 32, whose queries do not fit into
// registers, 99 (on tiles 54).  (With items of 16 and heads of 128 a thread spills 76 bytes; no other instance does.)
#include "attention.h"
#include "host.h"

namespace mlk {
namespace {

constexpr int kKeys = kFewKeys;
constexpr int kConsumers = 4, kThreads = 32 * (kConsumers + 1);

__host__ __device__ constexpr int stage_bytes(int dp) { return 2 * kKeys * dp * 2; }   // keys, then values
__host__ __device__ constexpr int stages_of(int dp) { return dp == 64 ? 6 : 3; }
// the ring, and 8 rows of three warps' results
constexpr int smem_bytes(int dp) { return stages_of(dp) * stage_bytes(dp) + 3 * 8 * (dp + 4) * 4; }

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
MLDEV uint32_t transposed(uint32_t x) {   // an 8 x 8 matrix of 16-bit values, two a lane
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
MLDEV uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
MLDEV void consumer_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

// NT: groups of 8 query rows of an item.
template <int DP, int NT>
__global__ void __launch_bounds__(kThreads, kFewPerSm) attention_rows_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int kRows = 8 * NT;
  using Sched = Schedule<kRows, kKeys, kFewOver>;
  using Place = Walk<kRows, kKeys, kFewOver>;
  constexpr int kStages = stages_of(DP), STAGE = stage_bytes(DP), HALVES = DP / 64;
  // A stage holds the unit's boxes one after another, each 64 values of its keys (rows of 128 bytes), then the
  // other 64: keys, then values.
  constexpr int kKeyBytes = DP * 2, kValues = kKeys * kKeyBytes;
  const int box_log2 = min(p.page_log2, 6), box = 1 << box_log2, half_bytes = box * 128;
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kSum = DP + 4;   // (rows two apart on other banks)
  float* sum_s = reinterpret_cast<float*>(smem + kStages * STAGE);   // [3][8][kSum]
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ float m_s[kConsumers][kRows], l_s[kConsumers][kRows];
  __shared__ ScheduleSmem sched_s;
  __shared__ int sums_s[kThreads];
  __shared__ uint32_t error_s;
  __shared__ int abort_s;
  __shared__ unsigned odd_s, done_s;   // rows whose result is not finite, and those that are written already
  volatile int* abort_flag = &abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = static_cast<int>(blockIdx.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kConsumers);
    }
    error_s = 0;
    abort_s = 0;
    odd_s = done_s = 0;
    fence_mbar_init();
  }
  if (warp == kConsumers && lane == 0) {
    tma_prefetch_desc(&p.tmap_k);
    tma_prefetch_desc(&p.tmap_v);
  }
  __syncthreads();
  // Where the kernel in front is another of this call, what came before that one is done, since it has waited for it.
  if (!p.follows) pdl_wait();
  pdl_trigger();

  Sched s;
  Place w;
  make_schedule<kRows, kKeys, kFewOver>(p, cta, s, w, sched_s, sums_s);
  if (threadIdx.x == 0 && s.bad) record_status(&error_s, kDevBadSlot, kWhereAttention);

  if (warp == kConsumers) {   // ------------------------------------------------ producer
    const uint64_t policy = l2_policy_evict_first();
    const int boxes = kKeys >> box_log2;   // of a unit
    int stage = 0, ok = 1;
    uint32_t phase = 0, issued = 0, parity = 0;
    for (; ok && more<kRows, kKeys, kFewOver>(s, w, p); w.next(p, s.end)) {
      const Part x = part_of<kRows, kKeys, kFewOver>(p, s, w, cta);
      if (x.lo >= x.hi) continue;
      const int sees = Sched::seen_by(p, w.r, w.i);
      const int32_t* table = p.tables + w.b * p.table_stride;
      // A lane holds the page of one of 32 boxes in a row, and of one of the next 32.
      const int first = (p.shared + x.lo * kKeys) >> box_log2, count = (min(sees, p.shared + x.hi * kKeys) + box - 1) >> box_log2;
      const int per_page = p.page_log2 - box_log2;
      auto page_at = [&](int b) { return b < count ? table[b >> per_page] : -1; };
      int base = first, here = page_at(base + lane), ahead = page_at(base + 32 + lane);
      for (int j = x.lo; j < x.hi; ++j) {
        const int b0 = (p.shared + j * kKeys) >> box_log2;   // the unit's first box
        if (b0 - base >= 32) {   // (32 is a multiple of a unit's boxes)
          base += 32;
          here = ahead;
          ahead = page_at(base + 32 + lane);
        }
        const int which = lane & (boxes - 1), key = (b0 + which) << box_log2;   // lanes for the keys' boxes, then the values'
        const bool mine = lane < 2 * boxes && key < sees;
        int page = __shfl_sync(0xffffffffu, here, (b0 - base + which) & 31);
        if (mine && (page < 0 || page >= p.num_pages)) {   // read as zeros: outside the map
          record_status(&error_s, kDevBadSlot, kWhereAttention);
          page = -1;
        }
        const int n = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) {
          ok = wait_soon(&empty[stage], phase ^ 1u, abort_flag, &error_s);
          if (ok) mbar_arrive_expect_tx(&full[stage], n * box * kKeyBytes);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (mine) {
          const bool values = lane >= boxes;
          uint8_t* at = smem + stage * STAGE + (values ? kValues : 0) + which * box * kKeyBytes;
          const CUtensorMap* map = values ? &p.tmap_v : &p.tmap_k;
          const int token = key & (p.page - 1);
          if (HALVES == 2 && p.both_halves) {
            tma_load_page2(at, map, &full[stage], token, w.kh, page, policy);
          } else {
#pragma unroll
            for (int half = 0; half < HALVES; ++half)
              tma_load_page(at + half * half_bytes, map, &full[stage], half * 64, token, w.kh, page, policy);
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
    const int quad = lane >> 2, pair = (lane & 3) * 2;   // a fragment's row and first of two columns
    const int t8 = lane & 7;
    // the warp's 16 keys of a unit: within their box, and further on in the unit
    const int first_key = (warp * 16 >> box_log2) * box * kKeyBytes + (warp * 16 & (box - 1)) * 128;
    int stage = 0, ok = 1;
    uint32_t phase = 0;
    bool started = false;   // an item whose rest is other blocks'
    for (; ok && more<kRows, kKeys, kFewOver>(s, w, p); w.next(p, s.end)) {
      const Part x = part_of<kRows, kKeys, kFewOver>(p, s, w, cta);
      if (x.lo >= x.hi) continue;
      const int row0 = w.i * kRows;
      const int rows = min(kRows, w.r.n * p.G - row0);
      const int sees = Sched::seen_by(p, w.r, w.i);
      uint32_t qf[NT][DP / 16][2];   // Q^T: dimensions pair, pair + 1 (and 8 on) of row quad
      int limit[NT][2];              // keys that rows pair and pair + 1 see
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int row = row0 + t * 8 + quad, token = token_of(p, row);
        const __nv_bfloat16* q =
            t * 8 + quad < rows ? p.q + (w.r.q0 + token) * p.q_t + (w.kh * p.G + row - token * p.G) * p.q_h : nullptr;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d = ks * 16 + e * 8 + pair;
            qf[t][ks][e] = q != nullptr && d < p.D ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = t * 8 + pair + e;
          limit[t][e] = r < rows ? max(w.r.kv - w.r.n + token_of(p, row0 + r) + 1, 0) : 0;
        }
      }
      const int all_see = max(w.r.kv - w.r.n + token_of(p, row0) + 1, 0);   // keys that every row of the item sees
      float o[NT][DP / 16][4];
      float ref[NT][2], l[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.0f;
        // (columns that are no row, or see none of this warp's keys, have the reference 0 and weights of 0)
        ref[t][0] = limit[t][0] > p.shared + x.lo * kKeys + warp * 16 ? -INFINITY : 0.0f;
        ref[t][1] = limit[t][1] > p.shared + x.lo * kKeys + warp * 16 ? -INFINITY : 0.0f;
        l[t][0] = l[t][1] = 0.0f;
      }
      for (int j = x.lo; j < x.hi; ++j) {
        ok = wait_soon(&full[stage], phase, abort_flag, &error_s);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int k0 = p.shared + j * kKeys + warp * 16;   // this warp's keys of the unit
        if (k0 < sees) {
          const uint32_t kb = smem_u32(smem) + stage * STAGE + first_key, vb = kb + kValues;
          const bool tail = k0 + 16 > sees;
          if (tail) {   // values that no row sees may be anything, and 0 times it would stay
            for (int c = lane; c < 16 * 8 * HALVES; c += 32) {
              const int t = (c >> 3) & 15;
              if (k0 + t >= sees)
                *reinterpret_cast<uint4*>(smem + stage * STAGE + kValues + first_key + (c >> 7) * half_bytes + t * 128 +
                                          (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
          }
          // ---- S^T: two sums of every second step, so that an MMA waits for one before the last
          float sc[NT][2][4] = {};
          const uint32_t krow = kb + (((lane >> 3) & 1) * 8 + t8) * 128;   // keys 0-7, 8-15; then 8 dimensions on
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks) {
            uint32_t f[4];
            ldsm4(krow + (ks >> 2) * half_bytes + (((((ks & 3) << 1) + (lane >> 4)) ^ t8) << 4), f);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816(sc[t][ks & 1], f, qf[t][ks][0], qf[t][ks][1]);
          }
          const bool cut = k0 + 16 > all_see;
          uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float v[4];   // keys quad, quad + 8 (e >> 1) of rows pair, pair + 1 (e & 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[e] = (sc[t][0][e] + sc[t][1][e]) * p.scale_log2;
              if (cut && k0 + quad + (e >> 1) * 8 >= limit[t][e & 1]) v[e] = -INFINITY;
            }
            float wt[4];
            for (int tries = 0;; ++tries) {
#pragma unroll
              for (int e = 0; e < 4; ++e) wt[e] = exp2_approx(v[e] - reference_of(ref[t][e & 1]));
              const bool renew = ref[t][0] == -INFINITY || ref[t][1] == -INFINITY || !(wt[0] + wt[1] + wt[2] + wt[3] <= kMostWeight);
              if (tries > 0 || !__any_sync(0xffffffffu, renew)) break;
              // first, and rarely later: the maxima over the warp's keys give the references
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float top = fmaxf(v[e], v[e + 2]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                top += kHeadroom;
                if (t * 8 + pair + e < rows && top > ref[t][e]) {
                  const float f = exp2_approx(ref[t][e] - top);
                  ref[t][e] = top;
                  l[t][e] *= f;
#pragma unroll
                  for (int n = 0; n < DP / 16; ++n) {
                    o[t][n][e] *= f;
                    o[t][n][e + 2] *= f;
                  }
                }
              }
            }
            l[t][0] += wt[0] + wt[2];
            l[t][1] += wt[1] + wt[3];
#pragma unroll
            for (int e = 0; e < 2; ++e) {   // two bf16 pieces, as the second product's operand
              const uint32_t h = pack2(wt[2 * e], wt[2 * e + 1]);
              const __nv_bfloat162 hb = *reinterpret_cast<const __nv_bfloat162*>(&h);
              hi[t][e] = transposed(h);
              lo[t][e] = transposed(pack2(wt[2 * e] - __low2float(hb), wt[2 * e + 1] - __high2float(hb)));
            }
          }
          // ---- O^T: dimensions 0-7 and 8-15 of keys 0-7, then of keys 8-15
          const uint32_t vrow = vb + ((lane >> 4) * 8 + t8) * 128;
#pragma unroll
          for (int n = 0; n < DP / 16; ++n) {
            uint32_t f[4];
            ldsm4_t(vrow + (n >> 2) * half_bytes + (((((n & 3) << 1) + ((lane >> 3) & 1)) ^ t8) << 4), f);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma16816(o[t][n], f, hi[t][0], hi[t][1]);
              mma16816(o[t][n], f, lo[t][0], lo[t][1]);
            }
          }
          if (tail) fence_proxy_async_smem();   // before the stage is filled again by TMA
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // ---- the four warps' results together
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], off);
          if (quad == 0) {
            m_s[warp][t * 8 + pair + e] = ref[t][e];
            l_s[warp][t * 8 + pair + e] = l[t][e];
          }
        }
      ok = !any_of_128(!ok);   // a barrier; a wait that ran out ends the work of all four
      if (!ok) break;
#pragma unroll
      for (int t = 0; t < NT; ++t) {   // 8 rows at a time
        if (t * 8 >= rows) break;
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = t * 8 + pair + e;
          float m = -INFINITY;
#pragma unroll
          for (int v = 0; v < kConsumers; ++v)
            if (l_s[v][r] != 0.0f) m = fmaxf(m, m_s[v][r]);
          f[e] = l_s[warp][r] == 0.0f ? 0.0f : exp2_approx(m_s[warp][r] - reference_of(m));
        }
        if (warp > 0) {
#pragma unroll
          for (int n = 0; n < DP / 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sum_s[((warp - 1) * 8 + pair + (e & 1)) * kSum + n * 16 + (e >> 1) * 8 + quad] = f[e & 1] == 0.0f ? 0.0f : o[t][n][e] * f[e & 1];
        }
        consumer_sync();
        if (warp == 0) {
#pragma unroll
          for (int n = 0; n < DP / 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = (pair + (e & 1)) * kSum + n * 16 + (e >> 1) * 8 + quad;
              float sum = f[e & 1] == 0.0f ? 0.0f : o[t][n][e] * f[e & 1];
#pragma unroll
              for (int v = 0; v < kConsumers - 1; ++v) sum += sum_s[v * 8 * kSum + at];
              sum_s[at] = sum;
            }
        }
        consumer_sync();
        // ---- eight values of a row a thread; rows that an unseen value has spoilt first, if any is not finite
        const int here = min(8, rows - t * 8) * (DP / 8);
        auto total = [&](int r, float& m, float& all) {
          m = -INFINITY;
          all = 0.0f;
#pragma unroll
          for (int v = 0; v < kConsumers; ++v)
            if (l_s[v][r] != 0.0f) m = fmaxf(m, m_s[v][r]);
#pragma unroll
          for (int v = 0; v < kConsumers; ++v)
            if (l_s[v][r] != 0.0f) all += l_s[v][r] * exp2_approx(m_s[v][r] - reference_of(m));
        };
        auto place = [&](int r, long long& token, int& head) {   // where the result goes, as a piece or part (index of its row)
          const int in = token_of(p, row0 + r);
          token = w.r.q0 + in;
          head = w.kh * p.G + (row0 + r) - in * p.G;
          return x.all ? part_row(p, token, head) : static_cast<long long>(x.slot) * p.item_rows + r;
        };
        const bool final = x.all && p.prefix_splits == 0;
        float* parts = x.all ? p.part_o : p.piece_o;
        if (all_see < sees) {   // some row does not see some of these keys
          for (int c = threadIdx.x; c < here; c += 32 * kConsumers) {
            const int r8 = c / (DP / 8), d = (c % (DP / 8)) * 8;
            float odd = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) odd = fmaf(sum_s[r8 * kSum + d + i], 0.0f, odd);
            if (odd != 0.0f) atomicOr(&odd_s, 1u << r8);
          }
          consumer_sync();
          const unsigned odd = odd_s;
          if (odd != 0) {
            for (int r8 = warp; r8 < 8; r8 += kConsumers) {
              if (((odd >> r8) & 1u) == 0) continue;
              const int r = t * 8 + r8;
              float m, all;
              total(r, m, all);
              if (!(all > 0.0f && all < INFINITY)) continue;
              long long token;
              int head;
              const long long at = place(r, token, head);
              if (repair_row(p, w.b, token, head, p.shared + x.lo * kKeys, min(sees, p.shared + x.hi * kKeys),
                             max(w.r.kv - w.r.n + token_of(p, row0 + r) + 1, 0), m, all, DP, p.out + token * p.o_t + head * p.o_h,
                             final ? nullptr : parts + at * DP) &&
                  lane == 0)
                atomicOr(&done_s, 1u << r8);
            }
            consumer_sync();
          }
        }
        const unsigned done = done_s;
        for (int c = threadIdx.x; c < here; c += 32 * kConsumers) {
          const int r8 = c / (DP / 8), r = t * 8 + r8, d = (c % (DP / 8)) * 8;
          float m, all;
          total(r, m, all);
          float val[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) val[i] = sum_s[r8 * kSum + d + i];
          long long token;
          int head;
          const long long at = place(r, token, head);
          if (final) {
            if (((done >> r8) & 1u) == 0) write_row8(p, token, head, d, m, all, val);
            else if (d == 0 && p.lse != nullptr) p.lse[token * p.Hq + head] = log_of_sum(m, all);
          } else {
            if (((done >> r8) & 1u) == 0) {
              float4* to = reinterpret_cast<float4*>(parts + at * DP + d);
              to[0] = make_float4(val[0], val[1], val[2], val[3]);
              to[1] = make_float4(val[4], val[5], val[6], val[7]);
            }
            if (d == 0) (x.all ? p.part_ml : p.piece_ml)[at] = make_float2(m, all);
          }
        }
        if (all_see < sees) {
          consumer_sync();
          if (threadIdx.x == 0) odd_s = done_s = 0;
        }
        consumer_sync();
      }
      if (!x.all && x.lo == 0 && threadIdx.x == 0) {
        p.records[cta] = record_of<kRows, kKeys, kFewOver>(p, s, w, x, cta);
        started = true;
      }
    }
    if (!started && threadIdx.x == 0 && p.records != nullptr) p.records[cta].pieces = 0;
  }
  if (p.follows) pdl_wait();   // not to end before it: what comes next reads its results, too
  __syncthreads();
  if (threadIdx.x == 0) finish_status(p, error_s, p.alone);
}

}  // namespace

cudaError_t prepare_attention_rows() {
  for (auto* k : {attention_rows_kernel<64, 1>, attention_rows_kernel<64, 2>}) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(64));
    if (e != cudaSuccess) return e;
  }
  for (auto* k : {attention_rows_kernel<128, 1>, attention_rows_kernel<128, 2>}) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(128));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_attention_rows(const AttentionParams& p, int dp, bool eight, cudaStream_t stream) {
  const dim3 grid(p.plan.ctas), block(kThreads);
  if (dp == 64)
    return eight ? launch_k(attention_rows_kernel<64, 1>, grid, block, smem_bytes(64), stream, true, p)
                 : launch_k(attention_rows_kernel<64, 2>, grid, block, smem_bytes(64), stream, true, p);
  return eight ? launch_k(attention_rows_kernel<128, 1>, grid, block, smem_bytes(128), stream, true, p)
               : launch_k(attention_rows_kernel<128, 2>, grid, block, smem_bytes(128), stream, true, p);
}

}  // namespace mlk
