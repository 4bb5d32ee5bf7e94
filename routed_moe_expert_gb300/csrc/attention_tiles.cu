// Attention of many rows a key head (prompts, pieces of prompts, drafts, the common prefix of a batch):
// 256 query rows against 128 keys a step, on tcgen05.
//
//   S = Q K^T                    M 128 rows, N 128 keys, both operands K-major in shared memory
//   P = 2^(scale S - reference)  by the row's thread, S read from TMEM, P written over it as bf16
//   O += P V                     P from TMEM, V [keys][values] as the MN-major operand, O stays in TMEM
//
// P is one bf16 a weight, off by up to 2^-8 of it, while their sum is of the float32 weights: 0.0023 of the result in the 2-norm
// where its own rounding is 0.0017.  A second bf16 for the rest would make three products of the two that prompts are bound by.
//
// A block takes two tiles of 128 rows, so that the tensor cores multiply for one while the threads of the
// other take exponentials, and a key is fetched once for both.  TMEM: S of both tiles (2 x 128 columns), O of both
// (2 x head size).  MMAs run in the order of issue, O_0 += P_0 V, S_0 of the next keys, then the same for
// tile 1, so S may overwrite the P that was just multiplied, and the tiles' weights are due in turn.
//
// The row's reference is 20 above the maximum of its first 128 scores, and stays (attention.h, kHeadroom).  Only when a
// unit's weights come to more than 1, at scores some 13 to 20 above the first ones, are its maximum taken and O, which
// lives in TMEM, multiplied.  So no maximum stands between a score and its weight, and O is hardly ever touched.
//
// Up to 128 rows take both tiles too: they hold the same rows and take the units of keys in turn, and their
// two results are added at the end (each thread finds its row's other half in its own TMEM lanes).
//
// What bounds it: at length the MMAs, which take about 81 cycles for a 128 x 128 x 16 instead of 64, since both operands'
// shared-memory reads are as long: 2600 cycles a unit of 256 rows and 128 keys, where the exponentials of both tiles
// (4.4 cycles a warp's) take 1130 beside them.  Measured, 32 query heads on 4 key heads of 128: a prompt of 8192 399 us, 1.38
// PFLOP/s, 72% of the library's rate (of its products alone, the cut triangle counted as what it is); 2048 52 us, 1024 23.5,
// 512 17.2, 128 12.6.  A part's own cost is about 4 units' (its queries, the first weights, the last result), and below
// about 1024 tokens this and the fetch of the kernel's code are most of the time.  (With heads of 64 a thread spills 20 bytes.)
//
// Warps 0-3 and 4-7: the rows of tiles 0 and 1, a thread a row; warp 8: TMA; warp 9: MMA issue, and zeroes for
// values behind the last key that is seen; warp 11: the block's parts of items.  Items come from the schedule in
// attention.h; with `prefix` the block's item is a part of the shared keys for 256 rows of the whole batch.
#include "attention.h"
#include "host.h"

namespace mlk {
namespace {

constexpr int kRows = kTileRows, kKeys = kTileKeys;
constexpr int kThreads = 384;
constexpr int kProducer = 8, kMma = 9, kScheduler = 11;
using Sched = Schedule<kRows, kKeys, kTileOver>;
using Place = Walk<kRows, kKeys, kTileOver>;

constexpr int kHalf = kKeys * 128;   // 64 values of 128 rows
__host__ __device__ constexpr int tile_bytes(int dp) { return dp / 64 * kHalf; }
__host__ __device__ constexpr int slots_of(int dp) { return dp == 64 ? 10 : 5; }
constexpr int smem_bytes(int dp) { return (2 + slots_of(dp)) * tile_bytes(dp); }

// D[tmem] (+)= A * B[smem], issued by the lane whose `leader` is not 0; A in shared memory (umma_ss) or in TMEM
// (umma_ts: K-major, a lane a row, two bf16 a column).  Descriptors by halves: the upper is a constant.
MLDEV void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate,
                   uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
MLDEV void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t accumulate,
                   uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// Lower half of a descriptor: the address (and, of the MN-major one, LBO above it).  Upper half: SBO 1024 bytes
// between atoms of eight rows, version 1, 128-byte swizzle.  K-major: rows of 64 values along K.  MN-major: 64
// values (128 bytes) of eight keys an atom, the next eight keys behind it, the next 64 values kHalf further (LBO).
MLDEV uint32_t desc_lo(uint32_t smem_addr) { return (smem_addr & 0x3FFFFu) >> 4; }
constexpr uint32_t kMnMajorHi = (1024 >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kKMajorHi = kMnMajorHi;
constexpr uint32_t kMnMajorB = 1u << 16;

// Two float32 operations an instruction.
MLDEV float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
MLDEV float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// 32 bytes of a thread's row: whole sectors, where the address allows (`wide`), else two pieces of 16.  (Four lanes trading
// pieces, so that a warp wrote longer runs, took twice the time of this.)
MLDEV void st_row16(unsigned long long at, const uint32_t (&x)[8], bool wide, bool first, bool second) {
  if (wide && second) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                 "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
    return;
  }
  if (first) *reinterpret_cast<uint4*>(at) = make_uint4(x[0], x[1], x[2], x[3]);
  if (second) *reinterpret_cast<uint4*>(at + 16) = make_uint4(x[4], x[5], x[6], x[7]);
}

// A part of an item as every role sees it, made by the scheduling warp.
struct Step {
  int end;             // no more parts
  int lo, most;        // units [lo, most) that some tile takes
  int hi0, hi1;        // tile k takes those below hi_k: as far as its last row sees
  int lead;            // 2: both tiles hold the same rows, tile k takes units lo + k, lo + k + 2, ...; else 1
  int rows0, rows1;    // rows of the tiles
  int sees;            // keys that the item's last row sees
  int b, kh, row0;     // request, key head, first row of the item
  int q0, n, kv;       // the request's first query row, query rows, keys
  int all, slot;       // the result is final, or a piece's slot
  int unused[3];
  MLDEV int hi(int k) const { return k == 0 ? hi0 : hi1; }
  MLDEV int rows(int k) const { return k == 0 ? rows0 : rows1; }
  MLDEV int first(int k) const { return lo + (lead == 2 ? k : 0); }
};
constexpr int kSteps = 4;

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) attention_tiles_kernel(const __grid_constant__ AttentionParams p,
                                                                      const __grid_constant__ PrefixRun prefix) {
  constexpr int kSlots = slots_of(DP), TILE = tile_bytes(DP), HALVES = DP / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + 2 * TILE;
  __shared__ uint64_t full[kSlots], empty[kSlots], s_full[2], p_ready[2], o_full[2], q_full[2], both[2], repaired[4],
      drain;
  __shared__ uint64_t step_full[kSteps], step_empty[kSteps];
  __shared__ Step steps[kSteps];
  __shared__ ScheduleSmem sched_s;
  __shared__ float2 ml_s[2][128];
  __shared__ uint32_t tmem_s, error_s;
  __shared__ int abort_s;
  volatile int* abort_flag = &abort_s;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
  const int cta = static_cast<int>(blockIdx.x);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_ready[t], 4);   // a lane a warp
      mbar_init(&o_full[t], 1);
      mbar_init(&q_full[t], 4);
      mbar_init(&both[t], 8);
    }
    for (int i = 0; i < kSteps; ++i) {
      mbar_init(&step_full[i], 1);
      mbar_init(&step_empty[i], 10);   // the other warps that work
    }
    for (int i = 0; i < 4; ++i) mbar_init(&repaired[i], 1);
    mbar_init(&drain, 1);
    error_s = 0;
    abort_s = 0;
    fence_mbar_init();
  }
  if (warp == kProducer && lane == 0) {
    tma_prefetch_desc(&p.tmap_k);
    tma_prefetch_desc(&p.tmap_v);
  }
  if (warp == kMma) {
    tmem_alloc(&tmem_s, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_s, 0);
  if (!p.follows) pdl_wait();   // (as in attention_rows.cu)
  pdl_trigger();

  Sched s;
  Place w;
  if (prefix.splits == 0) {
    make_schedule<kRows, kKeys, kTileOver>(p, cta, s, w, sched_s, reinterpret_cast<int*>(smem));
    __syncthreads();   // the scratch is the query tiles' again
    if (threadIdx.x == 0 && s.bad) record_status(&error_s, kDevBadSlot, kWhereAttention);
  }
  const int key0 = prefix.splits > 0 ? 0 : p.shared;   // first key of unit 0
  int ok = 1;
  int at_step = 0;            // of the ring of steps
  uint32_t step_phase = 0;
  auto step_here = [&]() {    // waits for the next part; the warp's lanes together
    ok = wait_soon(&step_full[at_step], step_phase, abort_flag, &error_s);
    ok = __all_sync(0xffffffffu, ok);
    return ok != 0;
  };
  auto step_read = [&]() {    // the warp has what it needs of it
    __syncwarp();
    if (lane == 0) mbar_arrive(&step_empty[at_step]);
    if (++at_step == kSteps) {
      at_step = 0;
      step_phase ^= 1u;
    }
  };

  // Registers: the block starts with 168 a thread (64512); the row threads take 200 (51200), in which a row's 128
  // scores stay, the other four warps keep 104 (13312).
  if (warp >= kProducer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == kScheduler) {   // -------------------------------------------- the block's parts
      bool first = true, started = false;
      while (ok) {
        Step t;
        t.end = 0;
        int hi, units[2];
        if (prefix.splits > 0) {   // one: a split of the shared keys for a tile of all rows
          t.end = first ? 0 : 1;
          const int item = cta / prefix.splits, split = cta - item * prefix.splits;
          t.kh = item / prefix.row_tiles;
          t.row0 = (item - t.kh * prefix.row_tiles) * kRows;
          t.b = t.q0 = 0;
          t.n = p.T;
          t.kv = t.sees = prefix.units * kKeys;
          t.lo = static_cast<int>(static_cast<long long>(prefix.units) * split / prefix.splits);
          hi = static_cast<int>(static_cast<long long>(prefix.units) * (split + 1) / prefix.splits);
          t.all = 0;
          t.slot = split;
        } else {
          if (!first) w.next(p, s.end);
          Part x;
          while (true) {
            if (!more<kRows, kKeys, kTileOver>(s, w, p)) {
              t.end = 1;
              break;
            }
            x = part_of<kRows, kKeys, kTileOver>(p, s, w, cta);
            if (x.lo < x.hi) break;
            w.next(p, s.end);
          }
          if (t.end == 0) {
            t.sees = Sched::seen_by(p, w.r, w.i);
            t.b = w.b;
            t.kh = w.kh;
            t.row0 = w.i * kRows;
            t.q0 = w.r.q0;
            t.n = w.r.n;
            t.kv = w.r.kv;
            t.lo = x.lo;
            hi = x.hi;
            t.all = x.all;
            t.slot = x.slot;
            if (!x.all && x.lo == 0) {
              if (lane == 0) p.records[cta] = record_of<kRows, kKeys, kTileOver>(p, s, w, x, cta);
              started = true;
            }
          }
        }
        first = false;
        if (t.end == 0) {
          const int left = t.n * p.G - t.row0;
          t.rows0 = min(128, left);
          t.rows1 = max(0, min(128, left - 128));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int rows = t.rows(k);
            int n = 0;
            if (rows > 0 && prefix.splits > 0) n = prefix.units;
            if (rows > 0 && prefix.splits == 0) {
              const int last = t.row0 + 128 * k + rows - 1;
              n = (max(max(t.kv - t.n + token_of(p, last) + 1, 0) - p.shared, 0) + kKeys - 1) / kKeys;
            }
            units[k] = max(t.lo, min(hi, n));
          }
          t.lead = 1;
          if (left <= 128) {
            t.lead = 2;
            t.rows1 = t.rows0;
            units[1] = units[0];
          }
          t.hi0 = units[0];
          t.hi1 = units[1];
          t.most = max(units[0], units[1]);
        }
        ok = wait_soon(&step_empty[at_step], step_phase ^ 1u, abort_flag, &error_s);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          steps[at_step] = t;
          mbar_arrive(&step_full[at_step]);
        }
        if (++at_step == kSteps) {
          at_step = 0;
          step_phase ^= 1u;
        }
        if (t.end) break;
      }
      if (prefix.splits == 0 && !started && lane == 0 && p.records != nullptr) p.records[cta].pieces = 0;
    } else if (warp == kProducer) {   // -------------------------------------- TMA
      const uint64_t policy = l2_policy_evict_last();
      const int box_log2 = min(p.page_log2, 7), box = 1 << box_log2, boxes = kKeys >> box_log2;
      int slot = 0;
      uint32_t phase = 0, issued = 0, parity = 0;
      while (ok && step_here()) {
        const Step t = steps[at_step];
        step_read();
        if (t.end) break;
        const int32_t* table = p.tables + t.b * p.table_stride;
        // A lane a box; its page is looked up a unit ahead of its use.
        auto page_at = [&](int j) -> int {
          const int key = key0 + j * kKeys + (lane << box_log2);
          return lane < boxes && j < t.most && key < t.sees ? table[key >> p.page_log2] : -1;
        };
        // The order of use: the first `lead` units' keys, then a unit's values and the keys `lead` units on.
        const int n = t.most - t.lo, lead = min(t.lead, n);
        int pages[2] = {-1, -1}, next_page = n > 0 ? page_at(t.lo) : -1;
        for (int i = 0; i < 2 * n; ++i) {
          const bool keys = i < lead || (i < 2 * n - lead && ((i - lead) & 1));
          const int u = i < lead ? i : keys ? (i - lead) / 2 + lead : i < 2 * n - lead ? (i - lead) / 2 : i - n;
          const int j = t.lo + u;
          const int key = key0 + j * kKeys + (lane << box_log2);
          const bool mine = lane < boxes && key < t.sees;
          int page;
          if (keys) {
            page = next_page;
            next_page = page_at(j + 1);
            if (mine && (page < 0 || page >= p.num_pages)) {   // read as zeros: outside the map
              record_status(&error_s, kDevBadSlot, kWhereAttention);
              page = -1;
            }
            if (u & 1) pages[1] = page;
            else pages[0] = page;
          } else {
            page = (u & 1) ? pages[1] : pages[0];
          }
          const int count = __popc(__ballot_sync(0xffffffffu, mine));
          if (lane == 0) {
            ok = wait_soon(&empty[slot], phase ^ 1u, abort_flag, &error_s);
            if (ok) mbar_arrive_expect_tx(&full[slot], count * box * HALVES * 128);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (mine) {
            uint8_t* at = ring + slot * TILE + lane * box * 128;
            const int token = key & (p.page - 1);
#pragma unroll
            for (int half = 0; half < HALVES; ++half)
              tma_load_page(at + half * kHalf, keys ? &p.tmap_k : &p.tmap_v, &full[slot], half * 64, token, t.kh, page, policy);
          }
          issued |= 1u << slot;
          parity = (parity & ~(1u << slot)) | (phase << slot);
          if (++slot == kSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && lane == 0)
        for (int i = 0; i < kSlots; ++i)
          if ((issued >> i) & 1u) mbar_wait_drain(&full[i], (parity >> i) & 1u);
      __syncwarp();
    } else if (warp == kMma) {   // ------------------------------------------ MMA issue
      // The whole warp walks along, so that descriptors stay in uniform registers; one lane issues.  The pipe holds
      // only a few MMAs ahead, so whatever has to be waited for is waited for behind MMAs just issued.
      const uint32_t s_idesc = idesc_bf16_f32(128, kKeys), o_idesc = idesc_bf16_f32(128, DP) | kMnMajorB;
      const uint32_t q_lo = desc_lo(smem_u32(smem)) | (1u << 16), ring_lo = desc_lo(smem_u32(ring));
      const uint32_t leader = lane == 0;
      int slot = 0;
      uint32_t phase = 0, q_phase = 0, p_phase = 0;
      // No vote on a wait's outcome, which would be part of every unit's time: after one that ran out the others
      // end at once, so the part's remaining steps are gone through on whatever is there.
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        wait_soon(bar, parity, abort_flag, &error_s);
        __syncwarp();
      };
      auto take_slot = [&]() {   // the next slot, filled
        const int at = slot;
        wait(&full[slot], phase);
        if (++slot == kSlots) {
          slot = 0;
          phase ^= 1u;
        }
        return at;
      };
      auto scores = [&](int k, int at) {   // S of tile k with the keys in slot `at`
        const uint32_t a = q_lo + k * (TILE >> 4), b = (ring_lo + at * (TILE >> 4)) | (1u << 16);
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
          const uint32_t step = (ks >> 2) * (kHalf >> 4) + 2 * (ks & 3);
          umma_ss(tmem + k * 128, a + step, b + step, kKMajorHi, s_idesc, ks > 0, leader);
        }
        if (leader) umma_commit(&s_full[k]);
      };
      while (step_here()) {
        const Step& in = steps[at_step];
        auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
        const int end = uniform(in.end), lo = uniform(in.lo), n = uniform(in.most) - lo, lead = uniform(in.lead);
        const int units0 = uniform(in.hi0) - lo, units1 = uniform(in.hi1) - lo, sees = uniform(in.sees);
        step_read();
        if (end) break;
        if (n == 0) continue;
        const bool tail = key0 + (lo + n) * kKeys > sees;   // the part's last unit has values behind the last key
        auto has = [&](int k, int u) { return u < (k == 0 ? units0 : units1) && (lead == 1 || (u & 1) == k); };
        for (int u = 0; u < lead && u < n; ++u) {   // the first keys
          const int at = take_slot();
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (!has(k, u)) continue;
            wait(&q_full[k], (q_phase >> k) & 1u);
            q_phase ^= 1u << k;
            tc_fence_after();
            scores(k, at);
          }
          if (leader) umma_commit(&empty[at]);
          __syncwarp();
        }
        int v_slot = take_slot(), k_slot = lead < n ? take_slot() : -1;
        for (int u = 0; u < n; ++u) {   // a unit's values, and the keys `lead` units on
          if (tail && u == n - 1) {   // zeroed, since 0 times an infinity would stay
            const int from = sees - (key0 + (lo + u) * kKeys);   // 1..127
            for (int c = lane; c < (kKeys - from) * 8; c += 32)
#pragma unroll
              for (int half = 0; half < HALVES; ++half)
                *reinterpret_cast<uint4*>(ring + v_slot * TILE + half * kHalf + from * 128 + c * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          const uint32_t b = (ring_lo + v_slot * (TILE >> 4)) | (static_cast<uint32_t>(kHalf >> 4) << 16);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (!has(k, u)) continue;
            wait(&p_ready[k], (p_phase >> k) & 1u);
            p_phase ^= 1u << k;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < kKeys / 16; ++ks)
              umma_ts(tmem + 256 + k * DP, tmem + k * 128 + ks * 8, b + ks * (2048 >> 4), kMnMajorHi, o_idesc,
                      u >= lead || ks > 0, leader);
            if (u + lead >= (k == 0 ? units0 : units1) && leader) umma_commit(&o_full[k]);
            if (has(k, u + lead)) scores(k, k_slot);
          }
          if (leader) {
            umma_commit(&empty[v_slot]);
            if (k_slot >= 0) umma_commit(&empty[k_slot]);
          }
          __syncwarp();
          if (u + 1 < n) {
            v_slot = take_slot();
            k_slot = u + 1 + lead < n ? take_slot() : -1;
          }
        }
        if (*abort_flag != 0) break;
      }
      ok = *abort_flag == 0;
      if (!ok && leader) {   // let what was issued finish before TMEM is released
        umma_commit(&drain);
        mbar_wait_drain(&drain, 0);
      }
      __syncwarp();
    }
  } else {   // ---------------------------------------------------------------- rows
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int k = warp >> 2, r = threadIdx.x & 127;   // tile, row of it
    const int wr = (warp & 3) * 32;                   // the warp's first row
    const uint32_t lanes = tmem + (static_cast<uint32_t>(wr) << 16);
    const uint32_t s_at = lanes + k * 128, o_at = lanes + 256 + k * DP;
    uint32_t s_phase = 0, o_phase = 0, both_phase = 0;   // of `both`, and above it of `repaired`
    const float scale = p.scale_log2;   // (not 0)
    const uint32_t unseen = scale < 0.0f ? 0x7f800000u : 0xff800000u;   // the score that scaled is -inf
    // Copies the part's query rows to the products' layout, a warp its own 32 of them, whole rows at a time.
    auto fetch_queries = [&](const Step& t) {
      const int row = t.row0 + (t.lead == 2 ? r : k * 128 + r);
      const int token = token_of(p, row);
      const __nv_bfloat16* from = nullptr;
      if (r < t.rows(k)) from = p.q + (t.q0 + token) * p.q_t + (t.kh * p.G + row - token * p.G) * p.q_h;
      constexpr int kLanes = DP / 8;   // a row
#pragma unroll 2
      for (int i = 0; i < 32; i += 32 / kLanes) {
        const int of = i + lane / kLanes, c = lane % kLanes, tr = wr + of;
        const __nv_bfloat16* src =
            reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(from), of));
        const bool real = src != nullptr && c * 8 < p.D;
        const uint32_t dst = smem_u32(smem) + k * TILE + (c >> 3) * kHalf + tr * 128 + (((c & 7) ^ (tr & 7)) << 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(real ? src + c * 8 : p.q), "r"(real ? 16 : 0)
                     : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto queries_there = [&]() {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      fence_proxy_async_smem();
      arrive(&q_full[k]);
    };
    bool asked = false;   // the query rows of the part at hand are on their way, or there
    while (step_here()) {
      if (steps[at_step].end) {
        step_read();
        break;
      }
      // What the units need; the rest is looked up behind them, since registers are short there.
      const int step_at = at_step;
      const int lo = steps[step_at].lo, hi = steps[step_at].hi(k), lead = steps[step_at].lead, rows = steps[step_at].rows(k);
      const int first_unit = steps[step_at].first(k);
      auto row_token = [&](int& head) {   // this thread's row: its token, and head
        const Step& t = steps[step_at];
        const int row = t.row0 + (lead == 2 ? r : k * 128 + r);   // of the request and key head
        const int token_in = token_of(p, row);
        head = t.kh * p.G + row - token_in * p.G;
        return t.q0 + token_in;
      };
      int sees = 0;
      {
        const Step& t = steps[step_at];
        int head;
        const int token = row_token(head);
        if (r < rows) {
          if (prefix.splits > 0) sees = min(max(keys_of_token(p, token), 0), t.sees);
          else sees = max(t.kv - t.n + (token - t.q0) + 1, 0);
        }
        if (!asked && first_unit < hi) {
          fetch_queries(t);
          queries_there();
        }
      }
      if (++at_step == kSteps) {
        at_step = 0;
        step_phase ^= 1u;
      }
      asked = false;
      // The next part's query rows, once the tile's last scores are there: they are what still reads these.
      auto fetch_next = [&]() {
        if (!step_here()) return;
        const Step& t = steps[at_step];
        if (t.end || t.first(k) >= t.hi(k)) return;
        fetch_queries(t);
        asked = true;
      };
      // (As in the MMA warp, a wait that ran out is looked at behind the units.)
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        wait_soon(bar, parity, abort_flag, &error_s);
        __syncwarp();
      };
      // (A row that sees nothing here asks for no reference: a whole warp looks for it, unit by unit, until it has one.)
      float ref = sees > key0 + first_unit * kKeys ? -INFINITY : 0.0f, l = 0.0f;
      if (wr >= rows) {   // no row of this warp is one: its weights may be anything
        for (int j = first_unit; j < hi; j += lead) {
          wait(&s_full[k], s_phase);
          s_phase ^= 1u;
          arrive(&p_ready[k]);
        }
      } else {
        // Units in front of `whole` are seen in full by all rows of the warp.
        const int whole = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<unsigned>(max(sees - key0, 0)))) / kKeys;
        const float2 scales = make_float2(scale, scale);
        for (int j = first_unit; j < hi; j += lead) {
          wait(&s_full[k], s_phase);
          s_phase ^= 1u;
          tc_fence_after();
          const int limit = sees - (key0 + j * kKeys);   // columns below it are seen
          float sum;
          bool renew = j == first_unit;   // the row's reference, and rarely a new one
          for (int tries = 0;; ++tries) {
            if (tries > 0 || j == first_unit) {   // (in loops: this is one unit's work, and its code waits to be fetched)
              float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
              for (int c = 0; c < kKeys; c += 32) {
                uint32_t x[32];
                tmem_ld_x32(s_at + c, x);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  tops[i & 3] = fmaxf(tops[i & 3], c + i < limit ? __uint_as_float(x[i]) * scale : -INFINITY);
              }
              const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) + kHeadroom;
              const bool grow = renew && top > ref;
              const float f = grow ? exp2_approx(ref - top) : 1.0f;
              if (grow) ref = top;
              l *= f;
              if (j >= lo + lead) {
#pragma unroll 1
                for (int c = 0; c < DP; c += 16) {
                  uint32_t o[16];
                  tmem_ld_x16(o_at + c, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tmem_st_x16(o_at + c, o);
                }
              }
            }
            uint32_t v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_x32(s_at + c * 32, v[c]);
            tmem_ld_wait();
            if (j >= whole) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) v[c][i] = c * 32 + i < limit ? v[c][i] : unseen;
            }
            const float2 off = make_float2(-reference_of(ref), -reference_of(ref));
            float2 sums[2] = {};
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                float2 x = fma2(make_float2(__uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1])), scales, off);
                x.x = exp2_approx(x.x);
                x.y = exp2_approx(x.y);
                sums[(i >> 1) & 1] = add2(sums[(i >> 1) & 1], x);
                const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
                v[c >> 1][(c & 1) * 16 + i / 2] = *reinterpret_cast<const uint32_t*>(&h);   // (read already)
              }
            sum = (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
            renew = ref == -INFINITY || !(sum <= kMostWeight);
            if (tries > 0 || !__any_sync(0xffffffffu, renew)) {
              tmem_st_x32(s_at, v[0]);   // over the scores
              tmem_st_x32(s_at + 32, v[1]);
              break;
            }
          }
          l += sum;
          tmem_st_wait();
          tc_fence_before();
          arrive(&p_ready[k]);
        }
      }
      if (l == 0.0f) ref = -INFINITY;
      fetch_next();
      if (!ok) break;
      if (asked) queries_there();
      if (first_unit < hi) {
        wait(&o_full[k], o_phase);
        o_phase ^= 1u;
        tc_fence_after();
      }
      if (*abort_flag != 0) break;
      const int hi_other = steps[step_at].hi(k ^ 1), all = steps[step_at].all, slot = steps[step_at].slot;
      const int request = steps[step_at].b, seen_here = steps[step_at].sees;
      const int tile_row = lead == 2 ? r : k * 128 + r;
      int head;
      const int token = row_token(head);
      __syncwarp();
      if (lane == 0) mbar_arrive(&step_empty[step_at]);
      // ---- with the same rows in both tiles: the other tile's maximum and sum, and half of the columns each
      const bool pair = lead == 2;
      float other = 0.0f, mine = 1.0f;   // factors of the other tile's result and this one's
      bool mine_0 = false, other_0 = false;   // nothing was seen there
      if (pair) {
        ml_s[k][r] = make_float2(ref, l);
        tc_fence_before();
        arrive(&both[0]);
        ok = wait_soon(&both[0], both_phase & 1u, abort_flag, &error_s);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float2 a = ml_s[0][r], b = ml_s[1][r];
        const float m = fmaxf(a.x, b.x), base = reference_of(m);
        const float fa = exp2_approx(a.x - base), fb = exp2_approx(b.x - base);
        ref = m;
        l = a.y * fa + b.y * fb;
        mine = k == 0 ? fa : fb;
        other = k == 0 ? fb : fa;
        mine_0 = (k == 0 ? a.y : b.y) == 0.0f;
        other_0 = (k == 0 ? b.y : a.y) == 0.0f;
      }
      const bool use_mine = first_unit < hi && !mine_0, use_other = pair && lo + (k ^ 1) < hi_other && !other_0;
      const int c_lo = pair ? k * (DP / 2) : 0;   // its columns: DP from there, or half as many
      const bool real = r < rows;
      const bool final = all && p.prefix_splits == 0;
      const bool by_token = prefix.splits > 0 || all;   // not a piece but a part of the row
      const long long at = prefix.splits > 0 ? (static_cast<long long>(slot) * p.T + token) * p.Hq + head
                           : all             ? part_row(p, token, head)
                                             : static_cast<long long>(slot) * p.item_rows + tile_row;
      float* piece_o = by_token ? p.part_o : p.piece_o;
      unsigned long long to = 0;   // the row's result
      if (real)
        to = final ? reinterpret_cast<unsigned long long>(p.out + token * p.o_t + head * p.o_h)
                   : reinterpret_cast<unsigned long long>(piece_o + at * DP);
      if (final) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        mine *= inv;
        other *= inv;
      }
      if (wr < rows) {
        const int chunks = pair ? DP / 32 : DP / 16;   // of 16 columns: little code, which has to be fetched
        const int key_hi = min(seen_here, key0 + hi * kKeys);
        // Rows that a value which they do not see has spoilt; `odd` is a sum of 0 times each of a row's results.
        auto repair = [&](float odd, int columns) {
          const bool maybe = real && odd != 0.0f && sees < key_hi;
          return __any_sync(0xffffffffu, maybe) && repair_rows(p, request, maybe, token, head, key0 + lo * kKeys, key_hi, sees, ref, l,
                                                               c_lo, columns, to, !final);
        };
        uint32_t own[16], mate[16];
        auto fetch = [&](int c) {
          __syncwarp();
          tmem_ld_x16(o_at + c_lo + c * 16, own);   // (whatever is there, if the tile had no unit)
          if (pair) tmem_ld_x16(lanes + 256 + (k ^ 1) * DP + c_lo + c * 16, mate);
        };
        auto result = [&](int i) {
          const float o = use_mine ? __uint_as_float(own[i]) * mine : 0.0f;
          return use_other ? fmaf(__uint_as_float(mate[i]), other, o) : o;
        };
        bool write = real;
        if (p.in_place && final) {   // the query row is needed for the repair, and gone afterwards
          // Rows that both tiles hold: the first tile repairs them whole, and the other one, whose columns lie over the
          // query as well, writes only behind that.
          uint32_t* left_s = reinterpret_cast<uint32_t*>(sched_s.items);   // rows of a warp that are still to be written
          if (k == 0 || !pair) {
            float odd = 0.0f;
#pragma unroll 1
            for (int c = 0; c < DP / 16; ++c) {
              fetch(c);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) odd = fmaf(result(i), 0.0f, odd);
            }
            if (repair(odd, DP)) write = false;
            if (pair) {
              const unsigned left = __ballot_sync(0xffffffffu, write);
              if (lane == 0) left_s[warp] = left;
              arrive(&repaired[warp]);
            }
          } else {
            ok = wait_soon(&repaired[warp - 4], both_phase >> 1, abort_flag, &error_s);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            write = (left_s[warp - 4] >> lane) & 1u;
            both_phase ^= 2u;
          }
        }
        float odds[4] = {};
        fetch(0);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {   // the next chunk's load is under way while one is written
          float o[16];
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            o[i] = result(i);
            odds[i & 3] = fmaf(o[i], 0.0f, odds[i & 3]);
          }
          if (c + 1 < chunks) fetch(c + 1);
          const int col = c_lo + c * 16;
          uint32_t x[8];
          if (final) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
              x[e] = l == 0.0f ? 0u : *reinterpret_cast<const uint32_t*>(&h);   // nothing is seen, or nothing weighs
            }
            if (write) st_row16(to + 2 * col, x, p.out_wide, col < p.D, col + 8 < p.D);
          } else {
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = __float_as_uint(o[i + e]);
              if (write) st_row16(to + 4 * (col + i), x, p.pieces_wide, true, true);
            }
          }
        }
        if (!(p.in_place && final)) repair((odds[0] + odds[1]) + (odds[2] + odds[3]), pair ? DP / 2 : DP);
      }
      if (real && c_lo == 0) {
        if (!final) (by_token ? p.part_ml : p.piece_ml)[at] = make_float2(ref, l);
        else if (p.lse != nullptr)
          p.lse[static_cast<long long>(token) * p.Hq + head] = log_of_sum(ref, l);
      }
      tc_fence_before();
      if (pair) {   // neither tile's next item overwrites what the other still reads
        arrive(&both[1]);
        ok = wait_soon(&both[1], both_phase & 1u, abort_flag, &error_s);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        both_phase ^= 1u;
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }

  if (p.follows) pdl_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) finish_status(p, error_s, p.alone);
}

}  // namespace

cudaError_t prepare_attention_tiles() {
  cudaError_t e = cudaFuncSetAttribute(attention_tiles_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(64));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attention_tiles_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(128));
  return e;
}

cudaError_t launch_attention_tiles(const AttentionParams& p, const PrefixRun& prefix, int blocks, int dp, cudaStream_t stream) {
  const dim3 grid(blocks), block(kThreads);
  return dp == 64 ? launch_k(attention_tiles_kernel<64>, grid, block, smem_bytes(64), stream, true, p, prefix)
                  : launch_k(attention_tiles_kernel<128>, grid, block, smem_bytes(128), stream, true, p, prefix);
}

}  // namespace mlk
