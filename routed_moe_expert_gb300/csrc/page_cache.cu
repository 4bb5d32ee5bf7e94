// A paged cache of keys and values: the block tables, slots and positions of a step's tokens from the
// requests' lengths (moe_lora_page_tables), and the write of their keys and values (moe_lora_cache_write).
#include "common.cuh"
#include "host.h"

#include <algorithm>

namespace mlk {
namespace {

// ---------------------------------------------------------------------------------------
// Block tables.  With held_b = ceil(cached_b / p) and more_b = ceil((cached_b + new_b) / p) - held_b, request
// b's pages start at the exclusive prefix sum of more in the free list, and its tokens at that of new.
//
// Every block takes both sums over all requests (they are a few KB), 1024 requests at a time, and then its
// share of the new pages and tokens, each of which finds its request by bisection in the block's table of
// sums: a request with a long prompt is spread like any other.  Where lengths or cursor are updated in place the blocks
// form one cluster, whose barrier stands between the last read of them and the first write.
//
// Bound by latency: lengths, sums, one dependent load (table or free list), store.  From a graph 2.6 us for one request, 3.9
// for 64 with a chunk of 449 among them, 4.6 for 511 with 15 000 tokens (6.4 when all blocks were always one cluster).
// ---------------------------------------------------------------------------------------
constexpr int kTableThreads = 1024;

struct TableParams {
  int32_t* tables;
  const int32_t *cached, *added, *free_pages, *taken;
  int32_t *kv, *offsets, *slots, *positions, *taken_out;
  long long stride;
  int B, width, page, num_free, T;
  int in_place;   // kv is cached, or taken_out is taken: the blocks are one cluster
  uint32_t* status;
};

// Exclusive prefix sums of two values over the block's threads, and their totals.
MLDEV void scan2(long long& a, int& b, long long& total_a, int& total_b, long long* wa, int* wb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long own_a = a;
  const int own_b = b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long ua = __shfl_up_sync(0xffffffffu, a, off);
    const int ub = __shfl_up_sync(0xffffffffu, b, off);
    if (lane >= off) {
      a += ua;
      b += ub;
    }
  }
  if (lane == 31) {
    wa[warp] = a;
    wb[warp] = b;
  }
  __syncthreads();
  if (warp == 0) {
    const int n = blockDim.x >> 5;
    long long va = lane < n ? wa[lane] : 0;
    int vb = lane < n ? wb[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long ua = __shfl_up_sync(0xffffffffu, va, off);
      const int ub = __shfl_up_sync(0xffffffffu, vb, off);
      if (lane >= off) {
        va += ua;
        vb += ub;
      }
    }
    wa[lane] = va;
    wb[lane] = vb;
  }
  __syncthreads();
  a += (warp > 0 ? wa[warp - 1] : 0) - own_a;
  b += (warp > 0 ? wb[warp - 1] : 0) - own_b;
  total_a = wa[31];
  total_b = wb[31];
}

// The last i < n with start[i] <= v (start[0] <= v).
template <typename V>
MLDEV int last_not_above(const V* start, int n, V v) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    if (start[lo + half] <= v) lo += half;
    n -= half;
  }
  return lo;
}

__global__ void __launch_bounds__(kTableThreads) page_tables_kernel(const __grid_constant__ TableParams p) {
  __shared__ long long tok0[kTableThreads];   // first token of a request, among the step's
  __shared__ int page0[kTableThreads];        // first of its new pages, in the free list behind the cursor
  __shared__ int cached_s[kTableThreads], held_s[kTableThreads], pages_s[kTableThreads];   // pages: held and granted
  __shared__ long long wa[32];
  __shared__ int wb[32];
  const int C = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);
  const int tid = threadIdx.x, NT = blockDim.x;
  pdl_wait();
  pdl_trigger();
  const int taken = *p.taken;
  bool bad = taken < 0 || taken > p.num_free;
  const int cursor = min(max(taken, 0), p.num_free);
  const int left = p.num_free - cursor;      // free pages
  const long long room = min(static_cast<long long>(p.width) * p.page, 0x7fffffffll);   // (lengths are 32 bits)
  long long tokens = 0;                      // of the requests before this chunk, and
  int pages = 0;                             // the pages they lack (at most left: granted)
  for (int b0 = 0; b0 == 0 || b0 < p.B; b0 += NT) {
    const int b = b0 + tid, n = min(NT, p.B - b0);
    int cached = 0, added = 0;
    if (b < p.B) {
      cached = p.cached[b];
      added = p.added[b];
      bad = bad || cached < 0 || added < 0;
      cached = max(cached, 0);
      added = max(added, 0);
    }
    if (p.in_place && C > 1) {   // the lengths are read by all blocks first
      cluster_arrive();
      cluster_wait();
    }
    const int held = static_cast<int>(min((static_cast<long long>(cached) + p.page - 1) / p.page, static_cast<long long>(p.width)));
    const long long after = static_cast<long long>(cached) + added;
    const int need = static_cast<int>(min((after + p.page - 1) / p.page, static_cast<long long>(p.width)));
    bad = bad || after > room;
    long long first_tok = added, all_tok;
    int first_page = max(need - held, 0), all_pages;
    const int lacks = first_page;
    scan2(first_tok, first_page, all_tok, all_pages, wa, wb);
    first_tok += tokens;
    // `pages` and the sum stay below 2^31: every request lacks at most `width`, and B * width is
    first_page += pages;
    const int granted = min(lacks, max(left - first_page, 0));
    bad = bad || granted < lacks;
    tok0[tid] = first_tok;
    page0[tid] = min(first_page, left);
    cached_s[tid] = cached;
    held_s[tid] = held;
    pages_s[tid] = held + granted;
    const long long kv = min(min(after, room), static_cast<long long>(held + granted) * p.page);
    if (rank == 0 && b < p.B) {
      p.kv[b] = static_cast<int>(kv);
      p.offsets[b] = static_cast<int>(min(first_tok, static_cast<long long>(p.T)));
    }
    __syncthreads();
    const int base = min(pages, left);
    tokens += all_tok;
    pages += all_pages;
    const int end = min(pages, left);
    for (int i = base + rank * NT + tid; i < end; i += C * NT) {   // the chunk's new pages
      const int r = last_not_above(page0, n, i);
      p.tables[(b0 + r) * p.stride + held_s[r] + (i - page0[r])] = p.free_pages[cursor + i];
    }
    const long long t_end = min(tokens, static_cast<long long>(p.T));
    for (long long t = tokens - all_tok + rank * NT + tid; t < t_end; t += C * NT) {   // and its tokens
      const int r = last_not_above(tok0, n, t);
      const long long pos = cached_s[r] + (t - tok0[r]);
      const long long at = pos / p.page;
      int slot = -1;
      if (at < pages_s[r]) {
        const int page = at < held_s[r] ? p.tables[(b0 + r) * p.stride + at]
                                        : p.free_pages[cursor + page0[r] + static_cast<int>(at) - held_s[r]];
        const long long s = static_cast<long long>(page) * p.page + (pos - at * p.page);
        if (page >= 0 && s <= 0x7fffffff) slot = static_cast<int>(s);
      }
      p.slots[t] = slot;
      p.positions[t] = static_cast<int>(min(pos, 0x7fffffffll));
    }
    __syncthreads();
  }
  bad = bad || tokens > p.T;
  for (long long t = tokens + rank * NT + tid; t < p.T; t += C * NT) {   // padding
    p.slots[t] = -1;
    p.positions[t] = 0;
  }
  const bool any = __syncthreads_or(bad) != 0;
  if (rank == 0 && tid == 0) {
    p.offsets[p.B] = static_cast<int>(min(tokens, static_cast<long long>(p.T)));
    *p.taken_out = cursor + min(pages, left);
    if (p.status != nullptr) *p.status = any ? kDevBadSlot | (kWherePageTables << 8) : 0u;
  }
}

// ---------------------------------------------------------------------------------------
// Cache writes: a copy of T rows of heads to scattered rows, in pieces of V values.  A thread keeps to one piece of
// a row (its head and place are worked out once) and takes tokens in turn, kFlight of them in flight: all loads,
// which do not wait for the slots, then the stores.  Bound by memory at length, by latency below: 8192 tokens of 2 x 4 heads
// of 128 6.7 us, 33.6 MB at 5.0 TB/s (10.8 us when a thread worked out head and place of every piece); one token 1.7 us.
// ---------------------------------------------------------------------------------------
constexpr int kFlight = 4;

struct WriteParams {
  const __nv_bfloat16 *k, *v;
  __nv_bfloat16 *kc, *vc;
  const int32_t* slots;
  long long k_t, k_h, v_t, v_h, kc_p, kc_h, kc_t, vc_p, vc_h, vc_t;
  int T, page, page_log2, num_slots;   // page_log2 -1: not a power of two
  int pieces;        // of a token: keys' heads, then values'
  int per_head;      // pieces of a head
  int at_once;       // tokens that a block takes side by side
  uint32_t* status;
};

template <int V>
struct Piece {
  using type = __nv_bfloat16;
};
template <>
struct Piece<8> {
  using type = uint4;
};

template <int V>
__global__ void __launch_bounds__(256) cache_write_kernel(const __grid_constant__ WriteParams p) {
  using U = typename Piece<V>::type;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == gridDim.x - 1) {   // the status word, by a block of its own
    if (p.status == nullptr || blockIdx.y > 0) return;
    int most = -1;
    for (long long t = threadIdx.x; t < p.T; t += 8 * blockDim.x) {
      int s[8];   // in flight together: at 8192 tokens this block takes less time than the copy
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = t + j * blockDim.x < p.T ? p.slots[t + j * blockDim.x] : -1;
#pragma unroll
      for (int j = 0; j < 8; ++j) most = max(most, s[j]);
    }
    const bool any = __syncthreads_or(most >= p.num_slots) != 0;
    if (threadIdx.x == 0) *p.status = any ? kDevBadSlot | (kWhereCacheWrite << 8) : 0u;
    return;
  }
  const int lane_token = p.at_once > 1 ? static_cast<int>(threadIdx.x) / p.pieces : 0;
  int piece = static_cast<int>(blockIdx.y) * blockDim.x + threadIdx.x - lane_token * p.pieces;
  if (piece >= p.pieces || lane_token >= p.at_once) return;
  const bool values = piece >= p.pieces / 2;
  if (values) piece -= p.pieces / 2;
  const int h = piece / p.per_head, d = (piece - h * p.per_head) * V;
  const __nv_bfloat16* src = (values ? p.v + h * p.v_h : p.k + h * p.k_h) + d;
  __nv_bfloat16* dst = (values ? p.vc + h * p.vc_h : p.kc + h * p.kc_h) + d;
  const long long src_t = values ? p.v_t : p.k_t, dst_p = values ? p.vc_p : p.kc_p, dst_t = values ? p.vc_t : p.kc_t;
  const long long step = static_cast<long long>(gridDim.x - 1) * p.at_once;
  for (long long t0 = static_cast<long long>(blockIdx.x) * p.at_once + lane_token; t0 < p.T; t0 += kFlight * step) {
    U val[kFlight];
    int slot[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const long long t = t0 + f * step;
      slot[f] = -1;
      if (t < p.T) {
        slot[f] = p.slots[t];
        val[f] = *reinterpret_cast<const U*>(src + t * src_t);
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (slot[f] < 0 || slot[f] >= p.num_slots) continue;
      const int page = p.page_log2 >= 0 ? slot[f] >> p.page_log2 : slot[f] / p.page;
      *reinterpret_cast<U*>(dst + page * dst_p + (slot[f] - page * p.page) * dst_t) = val[f];
    }
  }
}

}  // namespace
}  // namespace mlk

extern "C" moe_lora_status moe_lora_page_tables(moe_lora_handle* h, const moe_lora_page_tables_args* a, void* workspace,
                                                size_t workspace_bytes, moe_lora_stream stream) {
  using namespace mlk;
  if (h == nullptr || a == nullptr) return MOE_LORA_ERR_INVALID_ARG;
  if (a->B < 0 || a->T < 0 || a->T > kMaxExtent || a->table_width < 0 || a->page_size < 1 || a->num_free < 0 ||
      static_cast<long long>(a->B) * a->table_width > 0x7fffffffLL || (a->B > 1 && a->table_stride < a->table_width))
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->query_offsets == nullptr || a->taken == nullptr || a->taken_out == nullptr ||
      (a->B > 0 && (a->cached_lens == nullptr || a->new_lens == nullptr || a->kv_lens == nullptr)) ||
      (a->B > 0 && a->table_width > 0 && a->block_tables == nullptr) || (a->num_free > 0 && a->free_pages == nullptr) ||
      (a->T > 0 && (a->slot_map == nullptr || a->positions == nullptr)))
    return MOE_LORA_ERR_INVALID_ARG;
  if (workspace != nullptr && workspace_bytes < 4) return MOE_LORA_ERR_WORKSPACE_TOO_SMALL;
  for (const void* q : {static_cast<const void*>(a->block_tables), static_cast<const void*>(a->cached_lens),
                        static_cast<const void*>(a->new_lens), static_cast<const void*>(a->free_pages),
                        static_cast<const void*>(a->taken), static_cast<const void*>(a->kv_lens),
                        static_cast<const void*>(a->query_offsets), static_cast<const void*>(a->slot_map),
                        static_cast<const void*>(a->positions), static_cast<const void*>(a->taken_out),
                        static_cast<const void*>(workspace)})
    if (!aligned4(q)) return MOE_LORA_ERR_INVALID_ARG;
  TableParams p;
  p.tables = a->block_tables;
  p.cached = a->cached_lens;
  p.added = a->new_lens;
  p.free_pages = a->free_pages;
  p.taken = a->taken;
  p.kv = a->kv_lens;
  p.offsets = a->query_offsets;
  p.slots = a->slot_map;
  p.positions = a->positions;
  p.taken_out = a->taken_out;
  p.stride = a->table_stride;
  p.B = a->B;
  p.width = a->table_width;
  p.page = a->page_size;
  p.num_free = a->num_free;
  p.T = a->T;
  p.status = static_cast<uint32_t*>(workspace);
  p.in_place = a->kv_lens == a->cached_lens || a->taken_out == a->taken;
  // a block for every 1024 tokens; a cluster has eight at most
  const int ctas = std::min(p.in_place ? 8 : 64, 1 + a->T / 1024);
  const int threads = std::max(a->B, a->T) <= 128 ? 128 : kTableThreads;
  ML_ON_DEVICE(h);
  ML_LAUNCH(h, launch_kc(page_tables_kernel, dim3(ctas), dim3(threads), 0, stream, true, p.in_place ? ctas : 1, p), "page_tables launch");
  return MOE_LORA_OK;
}

extern "C" moe_lora_status moe_lora_cache_write(moe_lora_handle* h, const moe_lora_cache_write_args* a, void* workspace,
                                                size_t workspace_bytes, moe_lora_stream stream) {
  using namespace mlk;
  if (h == nullptr || a == nullptr) return MOE_LORA_ERR_INVALID_ARG;
  if (a->T < 0 || a->heads < 1 || a->heads > 65536 || a->head_dim < 1 || a->num_pages < 0 || a->page_size < 1 ||
      static_cast<long long>(a->num_pages) * a->page_size > 0x7fffffffLL)
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->head_dim > 512 || a->T > kMaxExtent) return MOE_LORA_ERR_UNSUPPORTED;
  if (workspace != nullptr && workspace_bytes < 4) return MOE_LORA_ERR_WORKSPACE_TOO_SMALL;
  if (a->T == 0) return MOE_LORA_OK;
  if (a->k == nullptr || a->v == nullptr || a->slot_map == nullptr ||
      (a->num_pages > 0 && (a->k_cache == nullptr || a->v_cache == nullptr)))
    return MOE_LORA_ERR_INVALID_ARG;
  if (!aligned2(a->k) || !aligned2(a->v) || !aligned2(a->k_cache) || !aligned2(a->v_cache) || !aligned4(a->slot_map) ||
      !aligned4(workspace))
    return MOE_LORA_ERR_INVALID_ARG;
  WriteParams p;
  p.k = reinterpret_cast<const __nv_bfloat16*>(a->k);
  p.v = reinterpret_cast<const __nv_bfloat16*>(a->v);
  p.kc = reinterpret_cast<__nv_bfloat16*>(a->k_cache);
  p.vc = reinterpret_cast<__nv_bfloat16*>(a->v_cache);
  p.slots = a->slot_map;
  p.k_t = a->k_stride_t;
  p.k_h = a->k_stride_h;
  p.v_t = a->v_stride_t;
  p.v_h = a->v_stride_h;
  p.kc_p = a->k_stride_page;
  p.kc_h = a->k_stride_head;
  p.kc_t = a->k_stride_token;
  p.vc_p = a->v_stride_page;
  p.vc_h = a->v_stride_head;
  p.vc_t = a->v_stride_token;
  p.T = a->T;
  p.page = a->page_size;
  p.page_log2 = -1;
  if ((p.page & (p.page - 1)) == 0)
    for (p.page_log2 = 0; (1 << p.page_log2) < p.page;) ++p.page_log2;
  p.num_slots = a->num_pages * a->page_size;
  p.status = static_cast<uint32_t*>(workspace);
  uintptr_t bits = static_cast<uintptr_t>(a->head_dim);
  for (const void* q : {static_cast<const void*>(p.k), static_cast<const void*>(p.v), static_cast<const void*>(p.kc),
                        static_cast<const void*>(p.vc)})
    bits |= reinterpret_cast<uintptr_t>(q) / 2;
  for (long long s : {p.k_t, p.k_h, p.v_t, p.v_h, p.kc_p, p.kc_h, p.kc_t, p.vc_p, p.vc_h, p.vc_t}) bits |= static_cast<uintptr_t>(s);
  const int V = (bits & 7) == 0 ? 8 : 1;
  p.per_head = a->head_dim / V;
  p.pieces = 2 * a->heads * p.per_head;   // (at most 2^27)
  p.at_once = p.pieces >= 256 ? 1 : 256 / p.pieces;
  const int across = (p.pieces + 255) / 256;
  if (across > 65535) return MOE_LORA_ERR_UNSUPPORTED;
  // as many blocks as the GPU holds, and threads of them with one token to copy while that is enough
  const long long groups = (static_cast<long long>(p.T) + p.at_once - 1) / p.at_once;
  const int blocks = static_cast<int>(std::min<long long>(groups, std::max(1, 8 * h->num_sms / across))) + 1;
  const dim3 grid(blocks, across);
  const int threads = p.at_once > 1 ? (p.at_once * p.pieces + 31) / 32 * 32 : std::min(256, (p.pieces + 31) / 32 * 32);
  ML_ON_DEVICE(h);
  ML_LAUNCH(h, V == 8 ? launch_k(cache_write_kernel<8>, grid, dim3(threads), 0, stream, true, p)
                      : launch_k(cache_write_kernel<1>, grid, dim3(threads), 0, stream, true, p),
            "cache_write launch");
  return MOE_LORA_OK;
}
