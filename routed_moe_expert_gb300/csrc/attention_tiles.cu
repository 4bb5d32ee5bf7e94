// Attention of many rows a key head (prompts, pieces of prompts, drafts, the common prefix of a batch):
// 256 query rows against 128 keys a step, on tcgen05.
//
//   S = Q K^T                    M 128 rows, N 128 keys, both operands K-major in shared memory
//   P = 2^(scale S - reference)  by the row's thread, S read from TMEM, P written over it as bf16
//   O += P V                     P from TMEM, V [keys][values] as the MN-major operand, O stays in TMEM
//
// A block takes two tiles of 128 rows, so that the tensor cores multiply for one while the threads of the
// other take exponentials, and a key is fetched once for both.  TMEM: S of both tiles (2 x 128 columns), O of both
// (2 x head size).  MMAs run in the order of issue, O_0 += P_0 V, S_0 of the next keys, then the same for
// tile 1, so S may overwrite the P that was just multiplied.
//
// The row's reference is its maximum when that was last taken over; a new maximum is taken over, and O
// multiplied, only when it is more than 2^8 times the weights' scale away: in float32 and bf16 weights
// up to 256 are as exact as weights up to 1, and O, which lives in TMEM, hardly ever has to be touched.
//
// Warps 0-3 and 4-7: the rows of tiles 0 and 1, a thread a row; warp 8: TMA; warp 9: MMA issue; warp 10: zeroes
// values behind the last key that is seen (0 times an infinity would stay).  Items come from the schedule in
// attention.h; with `prefix` the block's item is a part of the shared keys for 256 rows of the whole batch.
#include "attention.h"
#include "host.h"

namespace mlk {
namespace {

constexpr int kRows = kTileRows, kKeys = kTileKeys;
constexpr int kThreads = 352;
constexpr int kProducer = 8, kMma = 9, kCleaner = 10;
using Sched = Schedule<kRows, kKeys>;
using Place = Walk<kRows, kKeys>;

constexpr int kHalf = kKeys * 128;   // 64 values of 128 rows
__host__ __device__ constexpr int tile_bytes(int dp) { return dp / 64 * kHalf; }
__host__ __device__ constexpr int slots_of(int dp) { return dp == 64 ? 8 : 5; }
constexpr int smem_bytes(int dp) { return (2 + slots_of(dp)) * tile_bytes(dp); }

// D[tmem] (+)= A[tmem] * B[smem]: A K-major (a lane a row, two bf16 a column), B as its descriptor says.
MLDEV void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// MN-major operand with the 128-byte swizzle: 64 values (128 bytes) of 8 keys an atom of 1024 bytes, the next
// 8 keys behind it (SBO), the next 64 values kHalf further (LBO).
MLDEV uint64_t sw128_mnmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kHalf >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
constexpr uint32_t kMnMajorB = 1u << 16;

// Keys that query row `token` of the whole batch sees, -1 if it is no request's.
MLDEV int keys_of_token(const AttentionParams& p, int token) {
  int b = token;
  Request r;
  if (p.offsets != nullptr) {
    int lo = 0, n = p.B;   // the last request that starts at or before the token
    while (n > 1) {
      const int half = n >> 1;
      if (p.offsets[lo + half] <= token) lo += half;
      n -= half;
    }
    b = lo;
  }
  r = request_of(p, b);
  if (token < r.q0 || token >= r.q0 + r.n) return -1;
  return max(r.kv - r.n + (token - r.q0) + 1, 0);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) attention_tiles_kernel(const __grid_constant__ AttentionParams p,
                                                                      const __grid_constant__ PrefixRun prefix) {
  constexpr int kSlots = slots_of(DP), TILE = tile_bytes(DP), HALVES = DP / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + 2 * TILE;
  __shared__ uint64_t full[kSlots], empty[kSlots], s_full[2], p_ready[2], o_full[2], q_full[2], v_asked, v_clean, drain;
  __shared__ ScheduleSmem sched_s;
  __shared__ uint32_t tmem_s, error_s;
  __shared__ int abort_s;
  volatile int* abort_flag = &abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = static_cast<int>(blockIdx.x);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_ready[t], 128);
      mbar_init(&o_full[t], 1);
      mbar_init(&q_full[t], 128);
    }
    mbar_init(&v_asked, 1);
    mbar_init(&v_clean, 1);
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
  const uint32_t tmem = tmem_s;
  pdl_wait();
  pdl_trigger();

  Sched s;
  Place w;
  Part only;   // of a prefix run
  if (prefix.splits > 0) {
    const int item = cta / prefix.splits, split = cta - item * prefix.splits;
    w.kh = item / prefix.row_tiles;
    w.i = item - w.kh * prefix.row_tiles;
    w.b = 0;
    w.r.q0 = 0;
    w.r.n = p.T;
    w.r.kv = prefix.units * kKeys;
    w.u0 = 0;
    only.lo = static_cast<int>(static_cast<long long>(prefix.units) * split / prefix.splits);
    only.hi = static_cast<int>(static_cast<long long>(prefix.units) * (split + 1) / prefix.splits);
    only.all = false;
    only.slot = split;
  } else {
    make_schedule<kRows, kKeys>(p, cta, s, w, sched_s, reinterpret_cast<long long*>(smem));
    __syncthreads();   // the scratch is the query tiles' again
    if (threadIdx.x == 0 && s.bad) record_status(&error_s, kDevBadSlot, kWhereAttention);
  }
  // The block's parts of items, the same for every role.  A tile works up to hi[t]: as far as its last row sees.
  bool first = true;
  struct Step {
    Part x;
    int hi[2], most, rows[2], sees;
  };
  auto next_step = [&](Step& t) -> bool {
    if (prefix.splits > 0) {
      if (!first) return false;
      first = false;
      t.x = only;
      t.sees = prefix.units * kKeys;
    } else {
      if (!first) w.next(p);
      first = false;
      while (true) {
        if (!more<kRows, kKeys>(s, w, p)) return false;
        t.x = part_of<kRows, kKeys>(p, s, w, cta);
        if (t.x.lo < t.x.hi) break;
        w.next(p);
      }
      t.sees = Sched::seen_by(p, w.r, w.i);
    }
    const long long left = static_cast<long long>(w.r.n) * p.G - static_cast<long long>(w.i) * kRows;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      t.rows[k] = static_cast<int>(max(0ll, min(128ll, left - 128 * k)));
      int units = 0;
      if (t.rows[k] > 0) {
        if (prefix.splits > 0) {
          units = prefix.units;
        } else {
          const long long last = static_cast<long long>(w.i) * kRows + 128 * k + t.rows[k] - 1;
          const int sees = max(w.r.kv - w.r.n + static_cast<int>(last / p.G) + 1, 0) - p.shared;
          units = sees <= 0 ? 0 : (sees + kKeys - 1) / kKeys;
        }
      }
      t.hi[k] = max(t.x.lo, min(t.x.hi, units));
    }
    t.most = max(t.hi[0], t.hi[1]);
    return true;
  };
  const int key0 = prefix.splits > 0 ? 0 : p.shared;   // first key of unit 0
  Step t;
  int ok = 1;

  if (warp == kProducer) {   // ------------------------------------------------ TMA
    const uint64_t policy = l2_policy_evict_last();
    const int box_log2 = min(p.page_log2, 7), box = 1 << box_log2, boxes = kKeys >> box_log2;
    int slot = 0;
    uint32_t phase = 0, issued = 0, parity = 0;
    while (ok && next_step(t)) {
      const int32_t* table = p.tables + w.b * p.table_stride;
      auto page_at = [&](int j) -> int {
        const int key = key0 + j * kKeys + (lane << box_log2);
        return lane < boxes && j < t.most && key < t.sees ? table[key >> p.page_log2] : -1;
      };
      int ahead = page_at(t.x.lo);
      for (int j = t.x.lo; ok && j < t.most; ++j) {
        const int key = key0 + j * kKeys + (lane << box_log2);
        const bool mine = lane < boxes && key < t.sees;
        int page = ahead;
        ahead = page_at(j + 1);
        if (mine && (page < 0 || page >= p.num_pages)) {   // read as zeros: outside the map
          record_status(&error_s, kDevBadSlot, kWhereAttention);
          page = -1;
        }
        const int n = __popc(__ballot_sync(0xffffffffu, mine));
        const int token = key & (p.page - 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (lane == 0) {
            ok = mbar_wait(&empty[slot], phase ^ 1u, abort_flag, &error_s, kWhereAttention);
            if (ok) mbar_arrive_expect_tx(&full[slot], n * box * HALVES * 128);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (mine) {
            uint8_t* at = ring + slot * TILE + lane * box * 128;
#pragma unroll
            for (int half = 0; half < HALVES; ++half)
              tma_load_page(at + half * kHalf, kv == 0 ? &p.tmap_k : &p.tmap_v, &full[slot], half * 64, token, w.kh, page, policy);
          }
          issued |= 1u << slot;
          parity = (parity & ~(1u << slot)) | (phase << slot);
          if (++slot == kSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
    }
    if (!ok && lane == 0)
      for (int i = 0; i < kSlots; ++i)
        if ((issued >> i) & 1u) mbar_wait_drain(&full[i], (parity >> i) & 1u);
    __syncwarp();
  } else if (warp == kMma) {   // ---------------------------------------------- MMA issue
    if (lane == 0) {
      const uint32_t s_idesc = idesc_bf16_f32(128, kKeys), o_idesc = idesc_bf16_f32(128, DP) | kMnMajorB;
      const uint32_t q_at = smem_u32(smem), ring_at = smem_u32(ring);
      int slot = 0;
      uint32_t phase = 0, q_phase = 0, p_phase = 0, clean_phase = 0;
      auto wait_slot = [&]() { return mbar_wait(&full[slot], phase, abort_flag, &error_s, kWhereAttention); };
      auto advance = [&]() {
        if (++slot == kSlots) {
          slot = 0;
          phase ^= 1u;
        }
      };
      auto scores = [&](int k, uint32_t at) {   // S of tile k with the keys at `at`
        const uint64_t ad = sw128_kmajor_desc(q_at + k * TILE), bd = sw128_kmajor_desc(at);
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
          const uint32_t step = (ks >> 2) * (kHalf >> 4) + 2 * (ks & 3);
          umma_bf16(tmem + k * 128, ad + step, bd + step, s_idesc, ks > 0);
        }
        umma_commit(&s_full[k]);
      };
      while (ok && next_step(t)) {
        if (t.most == t.x.lo) continue;
        ok = wait_slot();
        if (!ok) break;
        for (int k = 0; ok && k < 2; ++k) {
          if (t.hi[k] <= t.x.lo) continue;
          ok = mbar_wait(&q_full[k], (q_phase >> k) & 1u, abort_flag, &error_s, kWhereAttention);
          q_phase ^= 1u << k;
          tc_fence_after();
          if (ok) scores(k, ring_at + slot * TILE);
        }
        if (!ok) break;
        umma_commit(&empty[slot]);
        advance();
        for (int j = t.x.lo; ok && j < t.most; ++j) {
          const int v_slot = slot;
          ok = wait_slot();
          advance();
          if (ok && key0 + (j + 1) * kKeys > t.sees) {   // values behind the last key
            mbar_arrive(&v_asked);
            ok = mbar_wait(&v_clean, clean_phase, abort_flag, &error_s, kWhereAttention);
            clean_phase ^= 1u;
          }
          const bool another = j + 1 < t.most;
          const int k_slot = slot;
          bool have_keys = false;
          for (int k = 0; ok && k < 2; ++k) {
            if (j < t.hi[k]) {
              ok = mbar_wait(&p_ready[k], (p_phase >> k) & 1u, abort_flag, &error_s, kWhereAttention);
              if (!ok) break;
              p_phase ^= 1u << k;
              tc_fence_after();
              const uint64_t bd = sw128_mnmajor_desc(ring_at + v_slot * TILE);
#pragma unroll
              for (int ks = 0; ks < kKeys / 16; ++ks)
                umma_bf16_ts(tmem + 256 + k * DP, tmem + k * 128 + ks * 8, bd + ks * (2048 >> 4), o_idesc, j > t.x.lo || ks > 0);
              if (j + 1 == t.hi[k]) umma_commit(&o_full[k]);
            }
            if (j + 1 < t.hi[k]) {
              if (!have_keys) ok = wait_slot();
              have_keys = true;
              if (ok) scores(k, ring_at + k_slot * TILE);
            }
          }
          if (!ok) break;
          umma_commit(&empty[v_slot]);
          if (another) {
            umma_commit(&empty[k_slot]);
            advance();
          }
        }
      }
      if (!ok) {   // let what was issued finish before TMEM is released
        umma_commit(&drain);
        mbar_wait_drain(&drain, 0);
      }
    }
    __syncwarp();
  } else if (warp == kCleaner) {   // ------------------------------------------ values behind the last key
    // Asked for by the MMA warp once they have landed: by itself this warp would run ahead of the ring by
    // more than a lap, where a parity says nothing.
    unsigned long long used = 0;   // ring slots of the steps before
    uint32_t asked_phase = 0;
    while (ok && next_step(t)) {
      const int n = t.most - t.x.lo;
      if (n > 0 && key0 + t.most * kKeys > t.sees) {   // the part's last unit
        const unsigned long long at = used + 2ull * n - 1;
        const int slot = static_cast<int>(at % kSlots);
        ok = mbar_wait_sleep(&v_asked, asked_phase, abort_flag, &error_s, kWhereAttention) &&
             mbar_wait(&full[slot], static_cast<uint32_t>(at / kSlots) & 1u, abort_flag, &error_s, kWhereAttention);
        asked_phase ^= 1u;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int k0 = key0 + (t.most - 1) * kKeys;
        const int from = t.sees - k0;   // 1..127
        for (int c = lane; c < (kKeys - from) * 8 * HALVES; c += 32) {
          const int row = from + (c >> 3) % (kKeys - from), half = (c >> 3) / (kKeys - from);
          *reinterpret_cast<uint4*>(ring + slot * TILE + half * kHalf + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_clean);
      }
      used += 2ull * n;
    }
  } else {   // -------------------------------------------------------------- rows
    const int k = warp >> 2, r = threadIdx.x & 127;   // tile, row of it
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_at = lanes + k * 128, o_at = lanes + 256 + k * DP;
    uint32_t s_phase = 0, o_phase = 0;
    bool started = false;
    const float sign = p.scale_log2 < 0.0f ? -1.0f : 1.0f, scale = fabsf(p.scale_log2);
    while (ok && next_step(t)) {
      const int rows = t.rows[k], lo = t.x.lo, hi = t.hi[k];
      const long long row = static_cast<long long>(w.i) * kRows + k * 128 + r;   // of the request and key head
      const int token_in = static_cast<int>(row / p.G), head = w.kh * p.G + static_cast<int>(row - static_cast<long long>(token_in) * p.G);
      const long long token = w.r.q0 + token_in;
      int sees = 0;
      if (r < rows) {
        if (prefix.splits > 0) sees = min(max(keys_of_token(p, static_cast<int>(token)), 0), t.sees);
        else sees = max(w.r.kv - w.r.n + token_in + 1, 0);
      }
      float ref = -INFINITY, l = 0.0f;
      if (hi > lo) {
        // ---- the query row, in the products' layout; a negative scale is the row's sign
        uint8_t* q_s = smem + k * TILE + r * 128;
        const __nv_bfloat16* q = p.q + token * p.q_t + head * p.q_h;
#pragma unroll
        for (int c = 0; c < DP / 8; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (r < rows && c * 8 < p.D) v = *reinterpret_cast<const uint4*>(q + c * 8);
          if (sign < 0.0f) {
            v.x ^= 0x80008000u;
            v.y ^= 0x80008000u;
            v.z ^= 0x80008000u;
            v.w ^= 0x80008000u;
          }
          *reinterpret_cast<uint4*>(q_s + (c >> 3) * kHalf + (((c & 7) ^ (r & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
        mbar_arrive(&q_full[k]);
        for (int j = lo; j < hi; ++j) {
          ok = mbar_wait(&s_full[k], s_phase, abort_flag, &error_s, kWhereAttention);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          s_phase ^= 1u;
          tc_fence_after();
          const int limit = sees - (key0 + j * kKeys);   // columns below it are seen
          const bool cut = __any_sync(0xffffffffu, limit < kKeys);
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t v[32];
            tmem_ld_x32(s_at + c, v);
            tmem_ld_wait();
            if (cut) {
#pragma unroll
              for (int i = 0; i < 32; ++i) top = fmaxf(top, c + i < limit ? __uint_as_float(v[i]) : -INFINITY);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) top = fmaxf(top, __uint_as_float(v[i]));
            }
          }
          top *= scale;   // (scale is not 0)
          const bool grow = top > ref + 8.0f;
          if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? exp2_approx(ref - top) : 1.0f;
            if (grow) ref = top;
            l *= f;
            if (j > lo) {
#pragma unroll 1
              for (int c = 0; c < DP; c += 32) {
                uint32_t v[32];
                tmem_ld_x32(o_at + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                tmem_st_x32(o_at + c, v);
              }
              tmem_st_wait();
            }
          }
          const float off = -reference_of(ref);
          float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t v[32], w2[16];
            tmem_ld_x32(s_at + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float a = __uint_as_float(v[i]), b = __uint_as_float(v[i + 1]);
              if (cut) {
                a = c + i < limit ? a : -INFINITY;
                b = c + i + 1 < limit ? b : -INFINITY;
              }
              a = exp2_approx(fmaf(a, scale, off));
              b = exp2_approx(fmaf(b, scale, off));
              sum0 += a;
              sum1 += b;
              const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
              w2[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
            }
            tmem_st_x16(s_at + c / 2, w2);   // over scores that are read already
          }
          l += sum0 + sum1;
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_ready[k]);
        }
        if (!ok) break;
        ok = mbar_wait(&o_full[k], o_phase, abort_flag, &error_s, kWhereAttention);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        o_phase ^= 1u;
        tc_fence_after();
      }
      // ---- the result, eight values at a time
      const long long at = prefix.splits > 0 ? t.x.slot * (static_cast<long long>(p.T) * p.Hq) + token * p.Hq + head
                                             : static_cast<long long>(t.x.slot) * p.item_rows + k * 128 + r;
      float* piece_o = prefix.splits > 0 ? p.prefix_o : p.piece_o;
      float2* piece_ml = prefix.splits > 0 ? p.prefix_ml : p.piece_ml;
#pragma unroll 1
      for (int c = 0; c < DP; c += 32) {
        uint32_t v[32];
        if (hi > lo) {
          __syncwarp();
          tmem_ld_x32(o_at + c, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
        if (r < rows) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __uint_as_float(v[i + e]);
            if (t.x.all) {
              float m = ref, sum = l;
              add_prefix<DP>(p, token * p.Hq + head, c + i, m, sum, o);
              write_row8(p, token, head, c + i, m, sum, o);
            } else {
              float4* to = reinterpret_cast<float4*>(piece_o + at * DP + c + i);
              to[0] = make_float4(o[0], o[1], o[2], o[3]);
              to[1] = make_float4(o[4], o[5], o[6], o[7]);
            }
          }
        }
      }
      if (!t.x.all && r < rows) piece_ml[at] = make_float2(ref, l);
      tc_fence_before();
      if (prefix.splits == 0 && !t.x.all && t.x.lo == 0 && threadIdx.x == 0) {
        p.records[cta] = record_of<kRows, kKeys>(p, s, w, t.x, cta);
        started = true;
      }
    }
    if (prefix.splits == 0 && !started && threadIdx.x == 0 && p.records != nullptr) p.records[cta].pieces = 0;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) {
    if (prefix.splits > 0) {   // the launch that follows gathers errors
      if (error_s != 0) atomicCAS(p.flags, 0, static_cast<int>(error_s));
    } else {
      finish_status(p, error_s);
    }
  }
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
