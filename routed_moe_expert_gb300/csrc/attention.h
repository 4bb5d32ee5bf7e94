// Shared by the kernels of moe_lora_attention (attention*.cu).
#pragma once

#include "common.cuh"

namespace mlk {

// Items of the kernel for few rows (attention_rows.cu) and of the tiles' (attention_tiles.cu).
constexpr int kFewRows = 16, kFewKeys = 64, kFewPerSm = 2, kFewOver = 3;
constexpr int kTileRows = 256, kTileKeys = 128, kTileOver = 4;

// How a call's work is dealt out.  Rows of a request and key head are its query rows times the G query
// heads of that key head, row r being token r / G and head r % G: a key is read once for all of them.  An
// item is up to `rows` of them (Plan::rows) with the keys that its last row sees, cut into units of
// `keys` keys.  The units of all items, one request after another, are dealt to the blocks in equal runs,
// whatever the requests' lengths (which only the device knows): a block works on the end of one item, whole
// items, and the start of another.  An item weighs some units more than it has (OVER), for what a block does at its
// start and end; a run that ends within these has none of the item.  (Tiles 4: a prompt of 8192 397 us, with 6
// 406, and with 2 451 for 419 when it was chosen; 16 prompts on up to 1500 keys 72, with 0 99, with 8 76.  Few rows 3: 64
// requests on up to 2000 keys 25.2 us, with 0 32.5, with 1 28.8, with 6 25.7.)  Where a run holds part of an item its result is a piece (unnormalised
// sums, reference, sum of weights) in the workspace, at most two a block, and the block that has the item's
// first unit leaves a record, by which the kernel that follows adds the pieces up.
//
// With `whole` (no item is long) items are not cut: a block takes those whose first unit is in its run.  `whole_units` is the
// same by the lengths themselves: where no item has more units, and there are items for a third of the blocks.
struct Plan {
  int ctas;          // blocks of the launch
  int least;         // units that a block takes at least, when that leaves blocks without work
  int whole, whole_units;
  int few;           // up to 256 requests (32 long ones): every warp plans for itself
};

struct PieceRecord {
  int pieces;        // 0: the block starts no item that was cut
  int slot;          // of the first piece; the others are the first slots of the blocks that follow
  int q0, kh;        // the request's first row, the key head
  int row0, rows;    // rows of the item
  int unused[2];
};

struct AttentionParams {
  CUtensorMap tmap_k, tmap_v;                  // {D, page, Hk, pages}, box {64, keys of a page or unit, 1, 1}
  const __nv_bfloat16 *q, *k, *v;
  const int32_t *tables, *kv_lens, *offsets;   // offsets null: row b is request b's
  __nv_bfloat16* out;
  float* lse;
  long long q_t, q_h, o_t, o_h, k_p, k_h, k_t, v_p, v_h, v_t, table_stride;
  int T, B, Hq, Hk, G, D;
  uint32_t g_inverse;                          // 2^32 / G rounded up: rows are divided by G by its product's upper half
  int num_pages, page, page_log2, width;
  int shared;                                  // keys that are read from request 0's table
  int few_rows;                                // > 0: requests of up to so many rows a key head alone, < 0: the others
  int follows;                                 // the kernel in front is one of this call whose results are not needed
  int alone;                                   // no other kernel of the call follows: it writes the status word
  int long_queries;                            // requests have many items each
  int out_wide;                                // rows of `out` start on 32-byte boundaries
  int pieces_wide;                             // the workspace does, and so pieces and parts
  int in_place;                                // `out` is q
  int both_halves;                             // the maps have both halves of a key in a box (tma_load_page2)
  float scale_log2;                            // scale * log2(e): weights are powers of two
  Plan plan;
  PieceRecord* records;                        // [ctas], null with `whole`
  int item_rows;                               // rows of a piece's slot
  float2* piece_ml;                            // [2 ctas][item_rows] reference (of scaled scores, base 2), sum
  float* piece_o;                              // [2 ctas][item_rows][DP]
  // Parts of every row by token and head where keys are shared: the launch over those makes parts 0 to
  // prefix_splits - 1, the requests' own keys the last.  [prefix_splits + 1][T * Hq]
  float2* part_ml;
  float* part_o;
  int prefix_splits;                           // 0: no keys are shared
  uint32_t* status;
  int* flags;                                  // the handle's: error gathered so far, blocks that are done
};

constexpr float kLn2 = 0.693147180559945f;

// row / G, exact while row * G < 2^32, which the host sees to.  (A division is some 20 instructions, and these kernels'
// time is partly that of fetching their code.)
MLDEV int token_of(const AttentionParams& p, int row) {
  return p.G == 1 ? row : static_cast<int>(__umulhi(static_cast<uint32_t>(row), p.g_inverse));
}

// A request's rows [q0, q0 + n) and its keys, checked: rows within [0, T), at most width * page keys.
constexpr int kBadLength = 1, kBadRows = 2;
struct Request {
  int q0, n, kv, bad;
};
MLDEV Request request_of(const AttentionParams& p, int b) {
  Request r;
  r.bad = 0;
  if (p.offsets == nullptr) {
    r.q0 = b;
    r.n = 1;
  } else {
    const int lo = p.offsets[b], hi = p.offsets[b + 1];
    if (lo < 0 || hi < lo || hi > p.T) r.bad = kBadRows;
    r.q0 = r.bad ? 0 : lo;
    r.n = r.bad ? 0 : hi - lo;
  }
  const int kv = p.kv_lens[b];
  const long long room = static_cast<long long>(p.width) * p.page;
  if (kv < 0 || kv > room) r.bad |= kBadLength;
  r.kv = static_cast<int>(min(static_cast<long long>(max(kv, 0)), room));
  return r;
}

// Keys that query row `token` of the whole batch sees, -1 if it is no request's.
MLDEV int keys_of_token(const AttentionParams& p, int token) {
  int b = token;
  Request r;
  if (p.offsets != nullptr) {
    int lo = 0, n = p.B;   // the last request that starts at or before the token
#pragma unroll 1
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

// mbar_wait in little code, and with the timer read only now and then.  Raises the abort flag when it runs out, after which
// every wait of the block ends soon.  The limit leaves time for a repair (repair_rows) over more than a million keys, at
// 6.3 us a key for 32 rows.
constexpr uint64_t kWaitRepairNs = 10000000000ull;   // 10 s
MLDEV bool wait_soon(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
  uint64_t since = 0;
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 31u) != 0) continue;
    if (*abort_flag) return false;
    const uint64_t now = globaltimer_ns();
    if (since == 0) since = now;
    if (now - since > kWaitRepairNs) {
      *abort_flag = 1;
      record_status(status, kDevTimeout, kWhereAttention);
      return false;
    }
  }
  return true;
}

MLDEV float low_half(uint32_t x) { return __uint_as_float(x << 16); }    // of two bf16
MLDEV float high_half(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

MLDEV float exp2_approx(float x) {   // 2^-22 relative; 0 for -inf
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The reference that weights are taken relative to: 0 while nothing is seen, so that they are 0 and not NaN.
MLDEV float reference_of(float m) { return m == -INFINITY ? 0.0f : m; }

// A row's reference is kHeadroom above the maximum of its first scores, and stays: weights start at 2^-20, and later scores
// that are up to 20 higher (base 2) have weights of at most 1.  When some come to more than kMostWeight, their maximum and
// kHeadroom are the new reference.  So no weight is above 1, and sum p v passes float32's end only where it does with
// a running maximum, values of 1e37 under rising scores included.  (bf16 and float32 hold the smaller weights as
// exactly; those below 2^-126 are 0, which is 2^-106 of the largest.)
constexpr float kHeadroom = 20.0f, kMostWeight = 1.0f;

// Natural logarithm of a softmax's sum from a reference and the sum l relative to it.
MLDEV float log_of_sum(float ref, float l) { return ((reference_of(ref) - kHeadroom) + log2f(l * 1048576.0f)) * kLn2; }

// ---------------------------------------------------------------- the plan, worked out by every block
template <int ROWS, int KEYS, int OVER>
struct Schedule {
  // of this launch and block (the host sees to it that all items' weight is below 2^30)
  int ctas;              // blocks that work
  int units;             // all items' weight
  int each, rest;        // units = each * ctas + rest
  int start, end;        // this block's run
  int bad;               // of all requests; with kBadRows, no block works
  int whole;             // items are not cut

  // What item i of a request weighs: its units (at least one, so that rows that see nothing are written) and OVER.
  static MLDEV int weight_of(const AttentionParams& p, const Request& r, int i) {
    const int sees = seen_by(p, r, i) - p.shared;
    return (sees <= 0 ? 1 : (sees + KEYS - 1) / KEYS) + OVER;
  }
  // Keys that the last row of item i sees.
  static MLDEV int seen_by(const AttentionParams& p, const Request& r, int i) {
    const int last = min(i * ROWS + ROWS, r.n * p.G) - 1;   // (T * Hq is below 2^31 - 256)
    return max(r.kv - r.n + token_of(p, last) + 1, 0);
  }
  static MLDEV int items_of(const AttentionParams& p, const Request& r) {
    const int rows = r.n * p.G;
    if (p.few_rows != 0 && (rows <= abs(p.few_rows)) != (p.few_rows > 0)) return 0;   // another kernel's
    return (rows + ROWS - 1) / ROWS;
  }

  // Where a block's run starts, floor(units c / ctas), and the block whose run has u.
  MLDEV int start_of(int c) const { return each * c + static_cast<int>(static_cast<uint32_t>(rest * c) / static_cast<uint32_t>(ctas)); }
  MLDEV int block_of(int u) const {
    int c = min(ctas - 1, static_cast<int>(static_cast<float>(u) * (static_cast<float>(ctas) / static_cast<float>(units))));
#pragma unroll 1
    while (c + 1 < ctas && start_of(c + 1) <= u) ++c;   // (the estimate is one off at most)
#pragma unroll 1
    while (start_of(c) > u) --c;
    return c;
  }
};

// A place in the schedule, advanced item by item; every role of a block walks through the same ones.
template <int ROWS, int KEYS, int OVER>
struct Walk {
  using S = Schedule<ROWS, KEYS, OVER>;
  int b, kh, i, items, units;   // of the request's items; weight of this item
  int u0;                       // of all items before it
  Request r;

  // The first item of request b, or of one behind it that has any (32 looked at together; a whole warp).
  MLDEV void enter(const AttentionParams& p) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    while (b < p.B) {
      const int n = b + lane < p.B ? S::items_of(p, request_of(p, b + lane)) : 0;
      const unsigned any = __ballot_sync(0xffffffffu, n > 0);
      if (any == 0) {
        b += 32;
        continue;
      }
      const int at = __ffs(any) - 1;
      b += at;
      items = __shfl_sync(0xffffffffu, n, at);
      r = request_of(p, b);
      units = S::weight_of(p, r, 0);
      break;
    }
    kh = i = 0;
  }
  MLDEV void next(const AttentionParams& p, int end) {   // (behind `end` nothing is looked up any more)
    u0 += units;
    if (u0 >= end) return;
    if (++i == items) {
      i = 0;
      if (++kh == p.Hk) {
        ++b;
        enter(p);
        return;
      }
    }
    if (items > 1) units = S::weight_of(p, r, i);
  }
};

struct ScheduleSmem {
  int sums[32], items[32], most[32];
  int found_base, found_b, found_i, found_u, found_kh;
};

// The blocks that work, and this one's run.  `most`: what the largest item weighs.
template <int ROWS, int KEYS, int OVER>
MLDEV void deal_out(const AttentionParams& p, int cta, Schedule<ROWS, KEYS, OVER>& s, int units, int items, int most) {
  s.units = units;
  s.whole = p.plan.whole || (most <= p.plan.whole_units + OVER && 3 * items >= p.plan.ctas);
  s.ctas = max(1, min(p.plan.ctas, max(units / p.plan.least, items)));
  s.each = units / s.ctas;
  s.rest = units - s.each * s.ctas;
  s.start = s.start_of(min(cta, s.ctas));
  s.end = cta < s.ctas ? s.start_of(cta + 1) : s.start;
}

// No work for any block: rows out of order may be several requests', whose weights' sum could pass 32 bits.
template <int ROWS, int KEYS, int OVER>
MLDEV void deal_nothing(Schedule<ROWS, KEYS, OVER>& s) {
  s.ctas = 1;
  s.units = s.each = s.rest = s.start = s.end = s.whole = 0;
}

// The plan of up to 256 requests (32 long ones), by every warp for itself: a lane has up to eight neighbouring ones.  (33
// requests on 2000 keys 29.5 us, with the block's threads together as in plan_many 30.9.)
template <int ROWS, int KEYS, int OVER>
MLDEV void plan_few(const AttentionParams& p, int cta, Schedule<ROWS, KEYS, OVER>& s, Walk<ROWS, KEYS, OVER>& w) {
  using S = Schedule<ROWS, KEYS, OVER>;
  const int lane = threadIdx.x & 31, of_lane = (p.B + 31) >> 5, b0 = lane * of_lane;
  w.b = p.B;
  int items = 0, mine = 0, bad = 0, most = 0;
  Request r;
  r.q0 = r.n = r.kv = 0;
#pragma unroll 4
  for (int k = 0; k < of_lane; ++k) {
    if (b0 + k >= p.B) break;
    r = request_of(p, b0 + k);
    bad |= r.bad;
    const int n = S::items_of(p, r);
    items += n;
    if (ROWS > kFewRows && n > 0) most = max(most, S::weight_of(p, r, n - 1));   // (the last item sees most)
    if (ROWS <= kFewRows || !p.long_queries)
#pragma unroll 1
      for (int i = 0; i < n; ++i) mine += S::weight_of(p, r, i);
  }
  if (ROWS > kFewRows && p.long_queries) {   // one of many items a lane: the lanes add up one after the other's
#pragma unroll 1
    for (int b = 0; b < p.B; ++b) {
      Request other;
      other.n = __shfl_sync(0xffffffffu, r.n, b);
      other.kv = __shfl_sync(0xffffffffu, r.kv, b);
      const int n = __shfl_sync(0xffffffffu, items, b);
      int part = 0;
#pragma unroll 1
      for (int i = lane; i < n; i += 32) part += S::weight_of(p, other, i);
      part = __reduce_add_sync(0xffffffffu, part);
      if (lane == b) mine = part;
    }
  }
  mine *= p.Hk;
  s.bad = static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(bad)));
  if (s.bad & kBadRows) return deal_nothing(s);
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += u;
  }
  deal_out(p, cta, s, __shfl_sync(0xffffffffu, incl, 31), __reduce_add_sync(0xffffffffu, items) * p.Hk,
           ROWS > kFewRows ? __reduce_max_sync(0xffffffffu, most) : 0x7fffffff);
  if (s.start == s.end) return;
  const int start = s.start;
  // the lane whose requests have it, then which of them
  const int l = __ffs(__ballot_sync(0xffffffffu, incl - mine <= start && start < incl)) - 1;
  int before = __shfl_sync(0xffffffffu, incl - mine, l), all = __shfl_sync(0xffffffffu, mine, l);
  w.b = l * of_lane;
  w.r = request_of(p, w.b);
  w.items = S::items_of(p, w.r);
  if (of_lane > 1) {
#pragma unroll 1
    for (;;) {
      all = 0;
#pragma unroll 1
      for (int i = 0; i < w.items; ++i) all += S::weight_of(p, w.r, i);
      all *= p.Hk;
      if (start < before + all) break;
      before += all;
      w.r = request_of(p, ++w.b);
      w.items = S::items_of(p, w.r);
    }
  }
  const int per = all / p.Hk;
  w.kh = (start - before) / per;
  int at = before + w.kh * per;
#pragma unroll 1
  for (w.i = 0;; w.i += 32) {   // 32 items at a time
    const int own = w.i + lane < w.items ? S::weight_of(p, w.r, w.i + lane) : 0;
    int to = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, to, off);
      if (lane >= off) to += u;
    }
    const unsigned found = __ballot_sync(0xffffffffu, start < at + to);
    if (found != 0) {
      const int l = __ffs(found) - 1;
      w.i += l;
      w.units = __shfl_sync(0xffffffffu, own, l);
      at += __shfl_sync(0xffffffffu, to, l) - w.units;
      break;
    }
    at += __shfl_sync(0xffffffffu, to, 31);
  }
  w.u0 = at;
}

// The plan of any requests.  All threads of the block; `sums_s` [blockDim] scratch.  (Not inlined, as the code that
// every call runs is to be short.)
template <int ROWS, int KEYS, int OVER>
__device__ __noinline__ void plan_many(const AttentionParams& p, int cta, Schedule<ROWS, KEYS, OVER>& s, Walk<ROWS, KEYS, OVER>& w,
                                       ScheduleSmem& sm, int* sums_s) {
  using S = Schedule<ROWS, KEYS, OVER>;
  const int tid = threadIdx.x, NT = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = NT >> 5;
  w.b = p.B;
  // What the requests b0 + tid of a chunk weigh, and their items.
  int most = 0;
  auto chunk = [&](int b0, int& items, int& bad) -> int {
    int sum = 0;
    items = 0;
    if (b0 + tid < p.B) {
      const Request r = request_of(p, b0 + tid);
      items = S::items_of(p, r);
      bad |= r.bad;
      if (ROWS > kFewRows && items > 0) most = max(most, S::weight_of(p, r, items - 1));
      if (ROWS <= kFewRows || !p.long_queries)
#pragma unroll 1
        for (int i = 0; i < items; ++i) sum += S::weight_of(p, r, i);
    }
    if (ROWS > kFewRows && p.long_queries) {   // a warp a request
#pragma unroll 1
      for (int k = warp; k < NT && b0 + k < p.B; k += warps) {
        const Request r = request_of(p, b0 + k);
        const int n = S::items_of(p, r);
        int part = 0;
#pragma unroll 1
        for (int i = lane; i < n; i += 32) part += S::weight_of(p, r, i);
        part = __reduce_add_sync(0xffffffffu, part);
        if (lane == 0) sums_s[k] = part;
      }
      __syncthreads();
      if (b0 + tid < p.B) sum = sums_s[tid];
      __syncthreads();
    }
    return sum * p.Hk;
  };
  int bad = 0, total = 0, mine = 0, all_items = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    int items;
    mine = chunk(b0, items, bad);
    total += mine;
    all_items += items * p.Hk;
  }
  total = __reduce_add_sync(0xffffffffu, total);
  all_items = __reduce_add_sync(0xffffffffu, all_items);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    sm.sums[warp] = total;
    sm.items[warp] = all_items;
    sm.most[warp] = most;
  }
  s.bad = (__syncthreads_or(bad & kBadRows) ? kBadRows : 0) | (__syncthreads_or(bad & kBadLength) ? kBadLength : 0);
  if (s.bad & kBadRows) return deal_nothing(s);
  deal_out(p, cta, s, __reduce_add_sync(0xffffffffu, lane < warps ? sm.sums[lane] : 0),
           __reduce_add_sync(0xffffffffu, lane < warps ? sm.items[lane] : 0),
           ROWS > kFewRows ? __reduce_max_sync(0xffffffffu, lane < warps ? sm.most[lane] : 0) : 0x7fffffff);
  if (s.start == s.end) return;
  // the request that has unit `start`
  __syncthreads();
  int base = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    if (p.B > NT) {
      int items, ignored = 0;
      mine = chunk(b0, items, ignored);
    }
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += u;
    }
    if (lane == 31) sm.sums[warp] = incl;
    __syncthreads();
    const int before = base + __reduce_add_sync(0xffffffffu, lane < warp ? sm.sums[lane] : 0);
    base += __reduce_add_sync(0xffffffffu, lane < warps ? sm.sums[lane] : 0);
    if (before + incl - mine <= s.start && s.start < before + incl) {
      sm.found_b = b0 + tid;
      sm.found_base = before + incl - mine;
    }
    __syncthreads();
    if (s.start < base) break;
  }
  // its key head and item
  w.b = sm.found_b;
  w.r = request_of(p, w.b);
  w.items = S::items_of(p, w.r);
  if (warp == 0) {
    int per = 0;
#pragma unroll 1
    for (int i = lane; i < w.items; i += 32) per += S::weight_of(p, w.r, i);
    per = __reduce_add_sync(0xffffffffu, per);
    const int kh = (s.start - sm.found_base) / per;
    int at = sm.found_base + kh * per;   // first unit of items i0..
#pragma unroll 1
    for (int i0 = 0; i0 < w.items; i0 += 32) {
      const int own = i0 + lane < w.items ? S::weight_of(p, w.r, i0 + lane) : 0;
      int incl = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += u;
      }
      if (own > 0 && at + incl - own <= s.start && s.start < at + incl) {
        sm.found_i = i0 + lane;
        sm.found_u = at + incl - own;
        sm.found_kh = kh;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  __syncthreads();
  w.i = sm.found_i;
  w.u0 = sm.found_u;
  w.kh = sm.found_kh;
  w.units = S::weight_of(p, w.r, w.i);
}

// Works out the schedule and the block's first item.  All threads of the block; `sums_s` [blockDim] scratch.
template <int ROWS, int KEYS, int OVER>
MLDEV void make_schedule(const AttentionParams& p, int cta, Schedule<ROWS, KEYS, OVER>& s, Walk<ROWS, KEYS, OVER>& w, ScheduleSmem& sm,
                         int* sums_s) {
  if (p.plan.few) {
    plan_few<ROWS, KEYS, OVER>(p, cta, s, w);
  } else {
    Schedule<ROWS, KEYS, OVER> made;   // (what a function takes by its address stays in memory)
    Walk<ROWS, KEYS, OVER> place;
    plan_many<ROWS, KEYS, OVER>(p, cta, made, place, sm, sums_s);
    s = made;
    w = place;
  }
}

// What a block does of the item that a walk is at: units [lo, hi), and where the result goes.
struct Part {
  int lo, hi;
  bool all;      // the whole item: the result is final
  int slot;      // else: the piece's slot
};
template <int ROWS, int KEYS, int OVER>
MLDEV Part part_of(const AttentionParams& p, const Schedule<ROWS, KEYS, OVER>& s, const Walk<ROWS, KEYS, OVER>& w, int cta) {
  Part x;
  if (s.whole) {
    x.lo = 0;
    x.hi = w.u0 < s.start ? 0 : w.units - OVER;   // hi 0: begun in the run of a block before
    x.all = true;
    x.slot = 0;
    return x;
  }
  x.lo = max(s.start - w.u0 - OVER, 0);
  x.hi = min(s.end - w.u0 - OVER, w.units - OVER);
  x.all = x.lo == 0 && x.hi == w.units - OVER;
  x.slot = 2 * cta + (w.u0 > s.start ? 1 : 0);
  return x;
}
template <int ROWS, int KEYS, int OVER>
MLDEV bool more(const Schedule<ROWS, KEYS, OVER>& s, const Walk<ROWS, KEYS, OVER>& w, const AttentionParams& p) {
  return w.b < p.B && w.u0 < s.end;
}
// The record of a piece that begins an item (one thread).
template <int ROWS, int KEYS, int OVER>
MLDEV PieceRecord record_of(const AttentionParams& p, const Schedule<ROWS, KEYS, OVER>& s, const Walk<ROWS, KEYS, OVER>& w, const Part& x,
                            int cta) {
  PieceRecord c;
  c.pieces = s.block_of(w.u0 + w.units - 1) - cta + 1;
  c.slot = x.slot;
  c.q0 = w.r.q0;
  c.kh = w.kh;
  c.row0 = w.i * ROWS;
  c.rows = min(ROWS, w.r.n * p.G - c.row0);
  return c;
}

// The end of a block's work (one thread): its error, if it met one, goes to the handle's flag.  Where no other
// kernel of the call follows (`last`), the last block writes the status word and leaves the flags zero; else
// the call's last kernel does (take_status).
MLDEV void finish_status(const AttentionParams& p, uint32_t error, bool last) {
  if (error != 0) atomicCAS(p.flags, 0, static_cast<int>(error));
  if (!last) return;
  __threadfence();
  if (atomicAdd(p.flags + 1, 1) == static_cast<int>(gridDim.x) - 1) {
    __threadfence();
    *p.status = static_cast<uint32_t>(atomicExch(p.flags, 0));
    atomicExch(p.flags + 1, 0);
  }
}

MLDEV void take_status(const AttentionParams& p) { *p.status = static_cast<uint32_t>(atomicExch(p.flags, 0)); }

// Where the result of a row goes when it is not final: a piece, or the last part of the row.
MLDEV long long part_row(const AttentionParams& p, long long token, int head) {
  return (static_cast<long long>(p.prefix_splits) * p.T + token) * p.Hq + head;
}

// Eight values of a finished row, and its logarithm where d is 0.
MLDEV void write_row8(const AttentionParams& p, long long token, int head, int d, float m, float l, const float (&o)[8]) {
  const float inv = 1.0f / l;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = l == 0.0f ? 0.0f : o[i] * inv;
  __nv_bfloat16* at = p.out + token * p.o_t + head * p.o_h + d;
  if (d < p.D) *reinterpret_cast<uint4*>(at) = pack8(v);   // (D is a multiple of 8)
  if (d == 0 && p.lse != nullptr) p.lse[token * p.Hq + head] = log_of_sum(m, l);
}

// Rows whose result is not finite although their weights are may have been spoilt by a value that they do not see: 0 times
// it is NaN.  A warp has up to 32 of them, a lane a row: whether it may be one, its token and head, the keys that it sees,
// its reference and sum of weights, the place of its result.  Of the keys [key_lo, key_hi) that were multiplied the last one
// is looked for of which one of the values [d_lo, d_lo + d_n) is not finite, and rows that do not see it are summed again
// on plain cores and written, as bf16 over their sum of weights, or as they are (`piece`).  Returns whether the lane's was.
//
// Rare, so it is out of the way, and called with what is at hand.  It takes as long as there are keys, 32 rows in turn at
// most: a prompt of 8192 whose last value but one is infinite 51 ms (value by value 363), one with an infinity at its 100th
// key 1.2.  The waits leave time for that (kWaitRepairNs).
__device__ __noinline__ inline bool repair_rows(const AttentionParams& p, int b, bool maybe, int token, int head, int key_lo,
                                                int key_hi, int sees, float ref, float sum, int d_lo, int d_n,
                                                unsigned long long result, bool piece) {
  const int lane = threadIdx.x & 31, per = d_n / 8, side = 32 / per, mine = lane / per, d = d_lo + lane % per * 8;
  const int kh = __shfl_sync(0xffffffffu, token_of(p, head), 0);   // (the first row is one)
  const int limit = maybe && sum > 0.0f && sum < INFINITY ? min(sees, key_hi) : key_hi;
  const int32_t* table = p.tables + b * p.table_stride;
  int last = -1;   // a lane a piece of a key's values, as many keys side by side as fit
#pragma unroll 4
  for (int j = max(key_lo, static_cast<int>(__reduce_min_sync(0xffffffffu, limit))) + mine; j < key_hi; j += side) {
    const int page = table[j >> p.page_log2];
    const bool real = page >= 0 && page < p.num_pages && d < p.D;   // (loads without a branch, several in flight)
    const uint4 x =
        *reinterpret_cast<const uint4*>(real ? p.v + page * p.v_p + kh * p.v_h + (j & (p.page - 1)) * p.v_t + d : p.v);
    bool bad = false;
    for (const uint32_t y : {x.x, x.y, x.z, x.w}) bad = bad || (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
    if (real && bad) last = j;
  }
  last = __reduce_max_sync(0xffffffffu, last);
  const unsigned all = __ballot_sync(0xffffffffu, limit <= last);
#pragma unroll 1
  for (unsigned left = all; left != 0; left &= left - 1) {
    const int of = __ffs(left) - 1;
    const __nv_bfloat16* q =
        p.q + __shfl_sync(0xffffffffu, token, of) * p.q_t + __shfl_sync(0xffffffffu, head, of) * p.q_h;
    const int end = __shfl_sync(0xffffffffu, limit, of);
    const float reference = __shfl_sync(0xffffffffu, ref, of);
    float o[8] = {};
#pragma unroll 1
    for (int j0 = key_lo; j0 < end; j0 += 32) {   // a lane a key for the scores, then a lane a piece of the values
      const int j = j0 + lane, page = j < end ? table[j >> p.page_log2] : -1;
      const __nv_bfloat16* row = nullptr;
      float w = 0.0f;
      if (page >= 0 && page < p.num_pages) {   // (the values of another page count as zeros)
        const long long place = j & (p.page - 1);
        const __nv_bfloat16* k = p.k + page * p.k_p + kh * p.k_h + place * p.k_t;
        row = p.v + page * p.v_p + kh * p.v_h + place * p.v_t;
        float dot[2] = {0.0f, 0.0f};
#pragma unroll 8
        for (int c = 0; c < p.D; c += 8) {
          const uint4 x = *reinterpret_cast<const uint4*>(k + c), y = *reinterpret_cast<const uint4*>(q + c);
          const uint32_t x4[4] = {x.x, x.y, x.z, x.w}, y4[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dot[0] = fmaf(low_half(x4[e]), low_half(y4[e]), dot[0]);
            dot[1] = fmaf(high_half(x4[e]), high_half(y4[e]), dot[1]);
          }
        }
        w = exp2_approx((dot[0] + dot[1]) * p.scale_log2 - reference);
      }
#pragma unroll 8
      for (int t0 = 0; t0 < 32; t0 += side) {
        const float wt = __shfl_sync(0xffffffffu, w, t0 + mine);
        const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), t0 + mine));
        const bool real = v != nullptr && d < p.D;
        const uint4 x = *reinterpret_cast<const uint4*>(real ? v + d : q);
        const uint32_t x4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[2 * e] += real ? wt * low_half(x4[e]) : 0.0f;
          o[2 * e + 1] += real ? wt * high_half(x4[e]) : 0.0f;
        }
      }
    }
    for (int off = per; off < 32; off <<= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += __shfl_xor_sync(0xffffffffu, o[e], off);
    const float f = 1.0f / __shfl_sync(0xffffffffu, sum, of);
    const unsigned long long to = __shfl_sync(0xffffffffu, result, of);
    if (mine == 0) {
      if (piece) {
        float4* at = reinterpret_cast<float4*>(to) + d / 4;
        at[0] = make_float4(o[0], o[1], o[2], o[3]);
        at[1] = make_float4(o[4], o[5], o[6], o[7]);
      } else if (d < p.D) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= f;
        *(reinterpret_cast<uint4*>(to) + d / 8) = pack8(o);
      }
    }
    __syncwarp();
  }
  return (all >> lane) & 1u;
}

// The same for one row of the whole warp.
__device__ __noinline__ inline bool repair_row(const AttentionParams& p, int b, int token, int head, int key_lo, int key_hi, int sees,
                                               float ref, float sum, int d_n, __nv_bfloat16* out, float* piece) {
  const unsigned long long to = piece != nullptr ? reinterpret_cast<unsigned long long>(piece) : reinterpret_cast<unsigned long long>(out);
  return __any_sync(0xffffffffu, repair_rows(p, b, (threadIdx.x & 31) == 0, token, head, key_lo, key_hi, sees, ref, sum, 0, d_n, to,
                                             piece != nullptr));
}

// Box of one page's keys (or a part of a page) from the caches' maps; x a multiple of 64.
MLDEV void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int token, int head, int page,
                         uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(token), "r"(head), "r"(page), "l"(policy)
      : "memory");
}

// Both halves of a page's keys of 128 values, one behind the other (map {64, page, 2, Hk, pages}).
MLDEV void tma_load_page2(void* dst, const CUtensorMap* map, uint64_t* bar, int token, int head, int page, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %3, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(token), "r"(head), "r"(page), "l"(policy)
      : "memory");
}

// The shared keys' part of all rows, as a launch of the tiles' kernel: for every key head, tile of 256 rows
// (token-major, as an item's) and split of the keys a block.
struct PrefixRun {
  int splits;      // 0: an ordinary run
  int row_tiles;   // of a key head
  int units;       // of 128 keys
};

// Launches (attention_rows.cu, attention_tiles.cu)
cudaError_t prepare_attention_rows();
cudaError_t launch_attention_rows(const AttentionParams& p, int dp, bool eight, cudaStream_t stream);   // items of 8 rows, or 16
cudaError_t prepare_attention_tiles();
cudaError_t launch_attention_tiles(const AttentionParams& p, const PrefixRun& prefix, int blocks, int dp, cudaStream_t stream);

}  // namespace mlk
