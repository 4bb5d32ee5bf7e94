// Causal attention to a paged cache (moe_lora_attention): the entry point, the kernel for any layout, and the
// sum of the pieces of items that were cut.
#include "attention.h"
#include "host.h"
#include "linear.h"

#include <algorithm>
#include <cmath>

namespace mlk {
namespace {

// ---------------------------------------------------------------------------------------
// Any head size, page size and alignment, on plain cores: a block per query row and head.  Its warps take
// the keys 32 at a time in turn, a lane a key, each warp with a running maximum m, sum l and result o
// (o <- o 2^(m - m') + sum p v), and the block adds the warps' results at the end.  Bound by loads from L2: every head of
// a group reads its keys again.  16 requests on 4000 keys, 32 + 4 heads of 128, pages of 48: 214 us (value by value, as
// where pieces of 16 bytes do not fit, 1245); heads of 192 358, heads of 100 639; a prompt of 512 461.
// ---------------------------------------------------------------------------------------
constexpr int kAnyWarps = 8;

// V: values of a piece, 8 where head size, addresses and strides allow.  Then a lane reads its key by pieces, and the values
// a lane a piece, as many keys side by side as fit into a warp.
template <int V>
__global__ void __launch_bounds__(32 * kAnyWarps) attention_any_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int kPasses = 512 / (32 * V);   // of a warp over a row's pieces, at most
  __shared__ __align__(16) float q_s[512];
  __shared__ float o_s[kAnyWarps][512];
  __shared__ float m_s[kAnyWarps], l_s[kAnyWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const int b = static_cast<int>(blockIdx.y), h = static_cast<int>(blockIdx.z), kh = h / p.G;
  const int pieces = p.D / V;
  int of_key = 32;   // lanes to a key's values
  while (of_key / 2 >= pieces && of_key > 1) of_key /= 2;
  const int side = 32 / of_key, mine = lane / of_key, piece0 = lane - mine * of_key;
  const Request r = request_of(p, b);
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0 && r.bad) record_status(p.status, kDevBadSlot, kWhereAttention);
  for (int i = static_cast<int>(blockIdx.x); i < r.n; i += static_cast<int>(gridDim.x)) {
    const long long row = r.q0 + i;
    for (int d = threadIdx.x; d < p.D; d += blockDim.x) q_s[d] = bf2f(p.q[row * p.q_t + h * p.q_h + d]);
    __syncthreads();
    const int sees = max(r.kv - r.n + i + 1, 0);
    const int of_shared = min(sees, p.shared);
    float m = -INFINITY, l = 0.0f;
    float o[kPasses][V];
#pragma unroll
    for (int c = 0; c < kPasses; ++c)
#pragma unroll
      for (int e = 0; e < V; ++e) o[c][e] = 0.0f;
    for (int j0 = warp * 32; j0 < sees; j0 += 32 * kAnyWarps) {
      const int j = j0 + lane;
      int page = -1;
      float s = -INFINITY;
      if (j < sees) {
        page = p.tables[(j < of_shared ? 0 : b) * p.table_stride + j / p.page];
        if (page < 0 || page >= p.num_pages) {
          record_status(p.status, kDevBadSlot, kWhereAttention);
          page = -1;
        }
        float dot = 0.0f;
        if (page >= 0) {
          const __nv_bfloat16* k = p.k + page * p.k_p + kh * p.k_h + (j % p.page) * p.k_t;
          if constexpr (V == 8) {
#pragma unroll 8
            for (int c = 0; c < pieces; ++c) {
              const uint4 x = *reinterpret_cast<const uint4*>(k + 8 * c);
              const uint32_t x4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) dot += q_s[8 * c + 2 * e] * low_half(x4[e]) + q_s[8 * c + 2 * e + 1] * high_half(x4[e]);
            }
          } else {
            for (int d = 0; d < p.D; ++d) dot += q_s[d] * bf2f(k[d]);
          }
        }
        s = dot * p.scale_log2;
      }
      float top = s;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float m2 = fmaxf(m, top), ref = m2 == -INFINITY ? 0.0f : m2;
      const float old = exp2f(m - ref), w = exp2f(s - ref);
      float sum = w;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l = l * old + sum;
      m = m2;
#pragma unroll
      for (int c = 0; c < kPasses; ++c)
#pragma unroll
        for (int e = 0; e < V; ++e) o[c][e] *= old;
      const int n = min(32, sees - j0);
      const __nv_bfloat16* row = page < 0 ? nullptr : p.v + page * p.v_p + kh * p.v_h + (j % p.page) * p.v_t;
#pragma unroll 4
      for (int t0 = 0; t0 < n; t0 += side) {
        const int t = t0 + mine;   // (below 32; the weight of a key from n on is 0, and its page none)
        const float wt = __shfl_sync(0xffffffffu, w, t);
        const __nv_bfloat16* v =
            reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), t));
        if (v == nullptr) continue;
#pragma unroll
        for (int c = 0; c < kPasses; ++c) {
          const int piece = c * 32 + piece0;
          if (piece >= pieces) break;
          if constexpr (V == 8) {
            const uint4 x = *reinterpret_cast<const uint4*>(v + 8 * piece);
            const uint32_t x4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[c][2 * e] += wt * low_half(x4[e]);
              o[c][2 * e + 1] += wt * high_half(x4[e]);
            }
          } else {
            o[c][0] += wt * bf2f(v[piece]);
          }
        }
      }
    }
    for (int off = of_key; off < 32; off <<= 1)   // keys side by side
#pragma unroll
      for (int c = 0; c < kPasses; ++c)
#pragma unroll
        for (int e = 0; e < V; ++e) o[c][e] += __shfl_xor_sync(0xffffffffu, o[c][e], off);
#pragma unroll
    for (int c = 0; c < kPasses; ++c) {
      const int piece = c * 32 + piece0;
      if (mine == 0 && piece < pieces)
#pragma unroll
        for (int e = 0; e < V; ++e) o_s[warp][piece * V + e] = o[c][e];
    }
    if (lane == 0) {
      m_s[warp] = m;
      l_s[warp] = l;
    }
    __syncthreads();
    float all_m = -INFINITY;
    for (int w = 0; w < kAnyWarps; ++w) all_m = fmaxf(all_m, m_s[w]);
    const float ref = all_m == -INFINITY ? 0.0f : all_m;
    float all_l = 0.0f;
    for (int w = 0; w < kAnyWarps; ++w) all_l += l_s[w] * exp2f(m_s[w] - ref);
    for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
      float v = 0.0f;
      for (int w = 0; w < kAnyWarps; ++w) v += o_s[w][d] * exp2f(m_s[w] - ref);
      p.out[row * p.o_t + h * p.o_h + d] = f2bf(all_l == 0.0f ? 0.0f : v / all_l);
    }
    if (threadIdx.x == 0 && p.lse != nullptr) p.lse[row * p.Hq + h] = (ref + log2f(all_l)) * 0.693147180559945f;
    __syncthreads();
  }
}


// ---------------------------------------------------------------------------------------
// Results of a row from several places together.  Sixteen teams of threads a block, DP / 8 threads a team with eight
// values each; `per_row` teams (1, 4 or 16, by the number of results) take those of a row in turn, so that the 76
// pieces of a long request are five loads deep, and are added in order.  (One team up to 8 results: one request on
// 1000 keys 9.5 us for 8.9; 16 teams from 13 on: 64 tokens on 4000 keys 31.7 us for 25.1.)  Bound by latency, and by the L2
// reads of the pieces: about 2 us behind the 6.7 of one request's 700 keys, beginning early.
// ---------------------------------------------------------------------------------------
constexpr int kTeams = 16;

__host__ __device__ __forceinline__ int teams_per_row(int results) { return results <= 4 ? 1 : results <= 24 ? 4 : 16; }

// The sum over i < n of the results at row(i) of (ml, o), for the rows that the block's teams have at hand; every
// thread of the block takes part (`active`: the team has a row).  Valid in the first team of a row.
template <int DP, typename RowOf>
MLDEV void join_results(const float2* ml, const float* part, int n, int per_row, bool active, RowOf row, float& m, float& l,
                        float (&o)[8]) {
  constexpr int kLanes = DP / 8;
  __shared__ float o_s[kTeams][DP];
  __shared__ float m_s[kTeams], l_s[kTeams];
  const int team = threadIdx.x / kLanes, d = (threadIdx.x % kLanes) * 8, member = team % per_row;
  m = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] = 0.0f;
  if (active) {
#pragma unroll 4
    for (int i = member; i < n; i += per_row) {
      const long long at = row(i);
      const float2 x = ml[at];
      const float4* src = reinterpret_cast<const float4*>(part + at * DP + d);
      const float4 a = src[0], b = src[1];   // (no branch in front of them, so that several results' loads are in flight)
      const bool none = x.y == 0.0f;         // nothing was seen there, or nothing that weighs (a NaN is not 0)
      const float top = none ? m : fmaxf(m, x.x), ref = reference_of(top);
      const float f = exp2_approx(m - ref), g = none ? 0.0f : exp2_approx(x.x - ref);
      m = top;
      l = l * f + (none ? 0.0f : x.y * g);
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = o[k] * f + (none ? 0.0f : v[k] * g);
    }
  }
  if (per_row == 1) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) o_s[team][d + k] = o[k];
  if (d == 0) {
    m_s[team] = m;
    l_s[team] = l;
  }
  __syncthreads();
  if (member == 0) {
    for (int g = 1; g < per_row; ++g) m = fmaxf(m, m_s[team + g]);
    const float ref = reference_of(m);
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = 0.0f;
    for (int g = 0; g < per_row; ++g) {
      const float f = exp2_approx(m_s[team + g] - ref);
      l += l_s[team + g] * f;
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] += o_s[team + g][d + k] * f;
    }
  }
  __syncthreads();
}

// A kernel's pieces: records by block, of which `across` blocks here take each.
struct Pieces {
  const PieceRecord* records;
  const float2* ml;
  const float* o;
  int item_rows, ctas, across;
};

// The pieces of items that were cut, of the tiles' kernel and that for few rows together: `across` blocks take a record, if
// it is one, and its rows by team.  The result is final, or with shared keys the last part of the row.
template <int DP>
__global__ void __launch_bounds__(kTeams * DP / 8) attention_join_kernel(const __grid_constant__ AttentionParams p, const Pieces first,
                                                                         const Pieces second) {
  const bool later = static_cast<int>(blockIdx.x) >= first.ctas * first.across;
  const Pieces& x = later ? second : first;
  const int at = static_cast<int>(blockIdx.x) - (later ? first.ctas * first.across : 0);
  const int share = at / x.ctas, cta = at - share * x.ctas;   // (blocks with rows come first, since most items have few)
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.alone) take_status(p);
  const PieceRecord c = x.records[cta];
  if (c.pieces == 0) return;
  const int per_row = teams_per_row(c.pieces), at_once = kTeams / per_row;
  const int team = threadIdx.x / (DP / 8), d = (threadIdx.x % (DP / 8)) * 8;
  for (int r0 = share * at_once; r0 < c.rows; r0 += x.across * at_once) {
    const int r = r0 + team / per_row;
    float m, l, o[8];
    join_results<DP>(
        x.ml, x.o, c.pieces, per_row, r < c.rows,
        [&](int i) { return static_cast<long long>(i == 0 ? c.slot : 2 * (cta + i)) * x.item_rows + r; },
        m, l, o);
    if (r >= c.rows || team % per_row != 0) continue;
    const long long token = c.q0 + token_of(p, c.row0 + r);
    const int head = c.kh * p.G + c.row0 + r - static_cast<int>(token - c.q0) * p.G;
    if (p.prefix_splits == 0) {
      write_row8(p, token, head, d, m, l, o);
    } else {
      const long long part = part_row(p, token, head);
      float4* to = reinterpret_cast<float4*>(p.part_o + part * DP + d);
      to[0] = make_float4(o[0], o[1], o[2], o[3]);
      to[1] = make_float4(o[4], o[5], o[6], o[7]);
      if (d == 0) p.part_ml[part] = make_float2(m, l);
    }
  }
}

// The parts of the rows of all requests: the shared keys' and the requests' own.
template <int DP>
__global__ void __launch_bounds__(kTeams * DP / 8) attention_fold_kernel(const __grid_constant__ AttentionParams p) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) take_status(p);
  const int per_row = teams_per_row(p.prefix_splits + 1), at_once = kTeams / per_row;
  const int team = threadIdx.x / (DP / 8), d = (threadIdx.x % (DP / 8)) * 8;
  const int rows = p.T * p.Hq;
  const int r = static_cast<int>(blockIdx.x) * at_once + team / per_row;
  const int token = r / p.Hq;
  // rows of no request are left alone (keys that all requests share make no part of them either)
  const bool real = r < rows && keys_of_token(p, token) >= 0;
  float m, l, o[8];
  join_results<DP>(
      p.part_ml, p.part_o, p.prefix_splits + 1, per_row, real,
      [&](int i) { return static_cast<long long>(i) * rows + r; }, m, l, o);
  if (real && team % per_row == 0) write_row8(p, token, r - token * p.Hq, d, m, l, o);
}

// Blocks to a record: four for few rows; of tiles a block for every 16 rows, or 8 where the items are few, and so of many
// pieces each (64 tokens on 4000 keys 26.2 us for 30.5; but 24 requests of 4 drafts 55.4 for 54.4, of blocks with nothing to do).
Pieces pieces_of(const AttentionParams& p, bool any, bool few_items) {
  const int each = few_items ? kTeams / 2 : kTeams;
  const int across = p.item_rows <= kFewRows ? std::min(4, p.item_rows) : (p.item_rows + each - 1) / each;
  return any ? Pieces{p.records, p.piece_ml, p.piece_o, p.item_rows, p.plan.ctas, across} : Pieces{nullptr, nullptr, nullptr, 0, 0, 1};
}
cudaError_t launch_join(const AttentionParams& p, const Pieces& first, const Pieces& second, int dp, cudaStream_t stream) {
  const dim3 grid(first.ctas * first.across + second.ctas * second.across), block(kTeams * dp / 8);
  return dp == 64 ? launch_k(attention_join_kernel<64>, grid, block, 0, stream, true, p, first, second)
                  : launch_k(attention_join_kernel<128>, grid, block, 0, stream, true, p, first, second);
}
cudaError_t launch_fold(const AttentionParams& p, int dp, cudaStream_t stream) {
  const int per_row = teams_per_row(p.prefix_splits + 1);
  const dim3 grid((p.T * p.Hq + kTeams / per_row - 1) / (kTeams / per_row)), block(kTeams * dp / 8);
  return dp == 64 ? launch_k(attention_fold_kernel<64>, grid, block, 0, stream, true, p)
                  : launch_k(attention_fold_kernel<128>, grid, block, 0, stream, true, p);
}

// ---------------------------------------------------------------- workspace
// The status word; records and pieces (2 slots a block) of the tiles' kernel, and of that for few rows; the parts of each
// row where keys are shared.
// Every part grows with T alone, so what is enough for T rows is enough for fewer.
constexpr int kWholeUnits = 12;   // see moe_lora_attention
constexpr long long kMostKeys = 0x80000000LL - 8192;   // of a table: the kernels round up to units and look ahead in 32 bits
constexpr int kMaxSms = 160;   // blocks are a multiple of the GPU's 152
constexpr int kPrefixSplits = 64, kPrefixBlocks = 2 * kMaxSms;
constexpr size_t round256(size_t n) { return (n + 255) / 256 * 256; }
struct Workspace {
  size_t records, ml, o, few_records, few_ml, few_o, part_ml, part_o, bytes;
};
int slot_rows(bool tiles, long long T, int G) {
  return static_cast<int>(std::min<long long>(tiles ? kTileRows : kFewRows, T * G));
}
Workspace workspace_for(int T, int Hq, int Hk, int D) {
  const int G = Hq / Hk, dp = D <= 64 ? 64 : 128;
  const size_t slots = 2 * kMaxSms * slot_rows(true, T, G), few = 2 * kFewPerSm * kMaxSms * slot_rows(false, T, G);
  // rows x (splits of the shared keys' launch and one): splits <= kPrefixBlocks / items + 1, rows <= 256 items
  const size_t rows = static_cast<size_t>(T) * Hq;
  const size_t parts = std::min<size_t>(kPrefixSplits * rows, kPrefixBlocks * kTileRows + rows) + rows;
  Workspace w;
  w.records = 256;
  w.ml = w.records + round256(sizeof(PieceRecord) * kMaxSms);
  w.o = w.ml + round256(sizeof(float2) * slots);
  w.few_records = w.o + round256(sizeof(float) * slots * dp);
  w.few_ml = w.few_records + round256(sizeof(PieceRecord) * kFewPerSm * kMaxSms);
  w.few_o = w.few_ml + round256(sizeof(float2) * few);
  w.part_ml = w.few_o + round256(sizeof(float) * few * dp);
  w.part_o = w.part_ml + round256(sizeof(float2) * parts);
  w.bytes = w.part_o + round256(sizeof(float) * parts * dp);
  return w;
}

// Splits of the shared keys: the least time by units, a part costing about three more (its query tile, its
// result) than its keys.
PrefixRun prefix_run(int T, int G, int Hk, int keys, int sms) {
  PrefixRun r;
  r.units = keys / kTileKeys;
  r.row_tiles = static_cast<int>((static_cast<long long>(T) * G + kTileRows - 1) / kTileRows);
  const long long items = static_cast<long long>(r.row_tiles) * Hk;
  r.splits = 1;
  long long best = -1;
  const long long most = std::min<long long>({r.units, kPrefixSplits, kPrefixBlocks / items + 1});
  for (int s = 1; s <= most; ++s) {
    const long long cost = (items * s + sms - 1) / sms * ((r.units + s - 1) / s + 3);
    if (best < 0 || cost < best) {
      best = cost;
      r.splits = s;
    }
  }
  return r;
}

// The caches' tensor map: 64 values of up to `keys` tokens of a page at a time, or both halves of 128 values.
// Extents of one have no stride of their own.
bool page_map(moe_lora_handle* h, CUtensorMap* m, const void* base, const AttentionParams& p, long long s_token,
              long long s_head, long long s_page, int keys, bool both) {
  const cuuint64_t any = 2ull * p.D;   // (D is a multiple of 8)
  const cuuint64_t token = p.page > 1 ? 2 * s_token : any, head = p.Hk > 1 ? 2 * s_head : any,
                   page = p.num_pages > 1 ? 2 * s_page : any;
  const cuuint64_t tokens = p.page, heads = p.Hk, pages = p.num_pages;
  const cuuint32_t rows = static_cast<cuuint32_t>(p.page < keys ? p.page : keys);
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  const cuuint64_t dims4[4] = {static_cast<cuuint64_t>(p.D), tokens, heads, pages}, strides4[3] = {token, head, page};
  const cuuint64_t dims5[5] = {64, tokens, 2, heads, pages}, strides5[4] = {token, 128, head, page};
  const cuuint32_t box4[4] = {64, rows, 1, 1}, box5[5] = {64, rows, 2, 1, 1};
  return h->encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, both ? 5 : 4, const_cast<void*>(base), both ? dims5 : dims4,
                   both ? strides5 : strides4, both ? box5 : box4, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether whole 16-byte pieces and the caches' maps can be used.
bool fast_layout(const moe_lora_attention_args* a) {
  if (a->head_dim % 8 != 0 || a->head_dim > 128 || a->page_size < 16 || (a->page_size & (a->page_size - 1)) != 0 ||
      a->num_pages < 1 || a->table_width < 1)
    return false;
  if (!aligned16(a->q) || !aligned16(a->out) || !aligned16(a->k_cache) || !aligned16(a->v_cache) || a->q_stride_t % 8 != 0 ||
      a->q_stride_h % 8 != 0 || a->out_stride_t % 8 != 0 || a->out_stride_h % 8 != 0)
    return false;
  const long long limit = 1LL << 38;   // of a map's strides, in elements
  auto fits = [&](long long s, int extent) { return extent <= 1 || (s > 0 && s < limit && s % 8 == 0); };
  return fits(a->k_stride_token, a->page_size) && fits(a->v_stride_token, a->page_size) && fits(a->k_stride_head, a->k_heads) &&
         fits(a->v_stride_head, a->k_heads) && fits(a->k_stride_page, a->num_pages) && fits(a->v_stride_page, a->num_pages);
}

}  // namespace
}  // namespace mlk

extern "C" moe_lora_status moe_lora_attention_workspace_size(int T, int q_heads, int k_heads, int head_dim, size_t* bytes) {
  if (bytes == nullptr || T < 0 || q_heads < 1 || k_heads < 1 || q_heads % k_heads != 0 || head_dim < 1)
    return MOE_LORA_ERR_INVALID_ARG;
  *bytes = mlk::workspace_for(T, q_heads, k_heads, head_dim).bytes;
  return MOE_LORA_OK;
}

extern "C" moe_lora_status moe_lora_attention(moe_lora_handle* h, const moe_lora_attention_args* a, void* workspace,
                                              size_t workspace_bytes, moe_lora_stream stream) {
  using namespace mlk;
  if (h == nullptr || a == nullptr) return MOE_LORA_ERR_INVALID_ARG;
  if (a->T < 0 || a->B < 0 || a->q_heads < 1 || a->k_heads < 1 || a->q_heads % a->k_heads != 0 || a->q_heads > 65535 ||
      a->head_dim < 1 || a->num_pages < 0 || a->page_size < 1 || a->table_width < 0 || a->max_query_len < 0 ||
      a->shared_len < 0 || (a->B > 1 && a->table_stride < a->table_width) ||
      static_cast<long long>(a->num_pages) * a->page_size > 0x7fffffffLL ||
      static_cast<long long>(a->table_width) * a->page_size > kMostKeys)
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->query_offsets == nullptr && a->T != a->B) return MOE_LORA_ERR_INVALID_ARG;
  const float scale_log2 = a->scale * 1.4426950408889634f;
  if (!(std::fabs(scale_log2) < INFINITY)) return MOE_LORA_ERR_INVALID_ARG;
  if (a->shared_len > static_cast<long long>(a->table_width) * a->page_size) return MOE_LORA_ERR_INVALID_ARG;
  if (a->head_dim > 512 || a->B > 65535 || static_cast<long long>(a->T) * a->q_heads > kMaxExtent) return MOE_LORA_ERR_UNSUPPORTED;
  if (a->T == 0 || a->B == 0) return MOE_LORA_OK;
  if (a->q == nullptr || a->out == nullptr || a->kv_lens == nullptr || (a->table_width > 0 && a->block_tables == nullptr) ||
      (a->num_pages > 0 && (a->k_cache == nullptr || a->v_cache == nullptr)))
    return MOE_LORA_ERR_INVALID_ARG;
  size_t need = 0;
  moe_lora_attention_workspace_size(a->T, a->q_heads, a->k_heads, a->head_dim, &need);
  if (workspace == nullptr || !aligned16(workspace)) return MOE_LORA_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_LORA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned2(a->q) || !aligned2(a->out) || !aligned2(a->k_cache) || !aligned2(a->v_cache) || !aligned4(a->block_tables) ||
      !aligned4(a->kv_lens) || !aligned4(a->query_offsets) || !aligned4(a->lse))
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->out == a->q && ((a->T > 1 && a->out_stride_t != a->q_stride_t) || (a->q_heads > 1 && a->out_stride_h != a->q_stride_h)))
    return MOE_LORA_ERR_INVALID_ARG;   // in place is row by row
  AttentionParams p;
  p.q = reinterpret_cast<const __nv_bfloat16*>(a->q);
  p.k = reinterpret_cast<const __nv_bfloat16*>(a->k_cache);
  p.v = reinterpret_cast<const __nv_bfloat16*>(a->v_cache);
  p.tables = a->block_tables;
  p.kv_lens = a->kv_lens;
  p.offsets = a->query_offsets;
  p.out = reinterpret_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.q_t = a->q_stride_t;
  p.q_h = a->q_stride_h;
  p.o_t = a->out_stride_t;
  p.o_h = a->out_stride_h;
  p.k_p = a->k_stride_page;
  p.k_h = a->k_stride_head;
  p.k_t = a->k_stride_token;
  p.v_p = a->v_stride_page;
  p.v_h = a->v_stride_head;
  p.v_t = a->v_stride_token;
  p.table_stride = a->table_stride;
  p.T = a->T;
  p.B = a->B;
  p.Hq = a->q_heads;
  p.Hk = a->k_heads;
  p.G = a->q_heads / a->k_heads;
  p.g_inverse = static_cast<uint32_t>(((1ull << 32) + p.G - 1) / p.G);
  p.D = a->head_dim;
  p.num_pages = a->num_pages;
  p.page = a->page_size;
  p.width = a->table_width;
  p.shared = a->shared_len;
  p.scale_log2 = scale_log2;
  p.status = static_cast<uint32_t*>(workspace);
  p.flags = reinterpret_cast<int*>(h->linear_flags + kLinearFlags);
  p.prefix_splits = 0;
  p.out_wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0 && p.o_t % 16 == 0 && p.o_h % 16 == 0;
  p.pieces_wide = (reinterpret_cast<uintptr_t>(workspace) & 31u) == 0;   // (16 are asked for)
  p.in_place = p.out == p.q;
  p.records = nullptr;
  p.piece_ml = nullptr;
  p.piece_o = nullptr;
  ML_ON_DEVICE(h);
  // what the kernels' 32-bit arithmetic holds: rows divided by G (token_of), and the weight of all items, at most
  const long long group_rows = static_cast<long long>(p.T) * p.G;
  const long long own_most = static_cast<long long>(p.width) * p.page;
  // Up to 16 rows a key head run on the kernel for few rows, more on tiles (4 drafts of 24 requests on 1000 to 9000 keys, by
  // 4, 5 and 7 query heads of 128 to each of 4 key heads: 47, 80 and 74 us on that kernel, 54 on tiles; on 1000 to 4000 keys 30, 44 and
  // 46, and 36).  A batch that may have both, by its longest request and the rows left to the others, is split by request, each
  // kernel taking its own, where the short ones have an item for every SM: 256 requests of one token on 1000 keys beside a
  // prompt of 512 107 us, 141 on tiles alone; with 32 of them 36.7 and 34.9, and 16 on 4000 keys beside a prompt of 2048 77 and 76.
  const bool tiles = static_cast<long long>(a->max_query_len) * p.G > kFewRows;
  const bool eight = (tiles ? p.G : static_cast<long long>(a->max_query_len) * p.G) <= 8;
  const int few_rows = eight ? 8 : kFewRows;
  const long long others = p.B - 1LL;
  const bool mixed = tiles && p.offsets != nullptr && p.G <= few_rows && others * p.Hk > h->num_sms &&
                     (p.T - static_cast<long long>(a->max_query_len)) * p.G <= 2 * others * few_rows;
  const long long few_items = tiles ? 2LL * p.B : group_rows / 8 + p.B;
  const bool fits = std::max<long long>(group_rows, p.Hq) * p.G < (1LL << 32) &&
                    (!tiles || (group_rows / kTileRows + p.B) * p.Hk * (own_most / kTileKeys + 1 + kTileOver) < (1LL << 30)) &&
                    ((tiles && !mixed) || few_items * p.Hk * (own_most / kFewKeys + 1 + kFewOver) < (1LL << 30));
  if (!fast_layout(a) || !fits || p.scale_log2 == 0.0f || h->num_sms > kMaxSms) {
    ML_CUDA(cudaMemsetAsync(workspace, 0, 4, stream), "attention status");
    const int across = std::max(1, std::min(a->T, 65536 / std::max(1, a->B)));
    uintptr_t bits = reinterpret_cast<uintptr_t>(p.k) / 2 | reinterpret_cast<uintptr_t>(p.v) / 2 | static_cast<uintptr_t>(p.D);
    for (long long s : {p.k_p, p.k_h, p.k_t, p.v_p, p.v_h, p.v_t}) bits |= static_cast<uintptr_t>(s);
    ML_LAUNCH(h, launch_k((bits & 7) == 0 ? attention_any_kernel<8> : attention_any_kernel<1>, dim3(across, a->B, a->q_heads),
                          dim3(32 * kAnyWarps), 0, stream, false, p),
              "attention launch");
    return MOE_LORA_OK;
  }
  if (!h->attention_ready) {
    ML_CUDA(prepare_attention_rows(), "attention shared memory");
    ML_CUDA(prepare_attention_tiles(), "attention shared memory");
    h->attention_ready = true;
  }
  const int dp = p.D <= 64 ? 64 : 128;
  p.page_log2 = 0;
  while ((1 << p.page_log2) < p.page) ++p.page_log2;
  const Workspace at = workspace_for(p.T, p.Hq, p.Hk, p.D);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(base + at.part_ml);
  p.part_o = reinterpret_cast<float*>(base + at.part_o);
  p.shared = a->B > 1 ? a->shared_len / kTileKeys * kTileKeys : 0;   // the rest is each request's own
  p.both_halves = p.D == 128;   // (fewer values would be read past)
  auto maps = [&](AttentionParams& x, int keys, bool both) {
    return page_map(h, &x.tmap_k, x.k, x, x.k_t, x.k_h, x.k_p, keys, both) &&
           page_map(h, &x.tmap_v, x.v, x, x.v_t, x.v_h, x.v_p, keys, both);
  };
  const long long own_keys = static_cast<long long>(p.width) * p.page - p.shared;   // of a request, at most
  AttentionParams few = p;
  if ((tiles || p.shared > 0) && !maps(p, kTileKeys, false)) return cuda_fail(cudaErrorInvalidValue, "attention tensor maps");
  if ((!tiles || mixed) && !maps(few, kFewKeys, p.both_halves)) return cuda_fail(cudaErrorInvalidValue, "attention tensor maps");
  auto plan_for = [&](AttentionParams& x, int ctas, bool whole, int least, int whole_units) {
    x.plan.ctas = ctas;
    x.plan.whole = whole;
    x.plan.least = least;
    x.plan.whole_units = whole_units;
    x.plan.few = p.B <= (x.long_queries ? 32 : 256);
  };
  // Items are whole, without pieces and the launch that joins them, where tables hold few keys.  On tiles: 4 units (16
  // prompts of 200 35.0 us, cut 39.0), or 12 where there are many items (a prompt of 512 17.3 us, cut 20.9, of 1500 38.6 and
  // 40.3; but 8 drafts of one request on 1000 keys 16.6, cut 13.9, and with 16 units a prompt of 2048 61.0, cut 53.3).  Few
  // rows: 8 units (64 requests of up to 300 keys 13.4 us, cut 14.8; with 16 one request of 700 keys took 13.6 us, cut 9.2).
  const long long most_items = std::max<long long>(group_rows / kTileRows, std::min(p.B, p.T)) * p.Hk;
  const bool tiles_whole = own_keys <= 4 * kTileKeys || (own_keys <= kWholeUnits * kTileKeys && 3 * most_items >= h->num_sms);
  const bool few_whole = own_keys <= 8 * kFewKeys;
  p.follows = few.follows = 0;
  p.alone = few.alone = 0;
  p.few_rows = few.few_rows = 0;
  if (p.shared > 0) {
    const PrefixRun run = prefix_run(p.T, p.G, p.Hk, p.shared, h->num_sms);
    const long long blocks = static_cast<long long>(run.row_tiles) * p.Hk * run.splits;
    if (blocks > 0x7fffffff) return MOE_LORA_ERR_UNSUPPORTED;
    p.plan = Plan{};
    ML_LAUNCH(h, launch_attention_tiles(p, run, static_cast<int>(blocks), dp, stream), "attention prefix launch");
    p.prefix_splits = few.prefix_splits = run.splits;
    p.follows = few.follows = 1;
  }
  const bool fold = p.prefix_splits > 0;
  p.item_rows = slot_rows(true, p.T, p.G);
  p.long_queries = static_cast<long long>(a->max_query_len) * p.G > 8LL * kTileRows;
  plan_for(p, h->num_sms, tiles_whole, 2, kWholeUnits);
  p.piece_ml = reinterpret_cast<float2*>(base + at.ml);
  p.piece_o = reinterpret_cast<float*>(base + at.o);
  p.records = p.plan.whole ? nullptr : reinterpret_cast<PieceRecord*>(base + at.records);
  few.item_rows = slot_rows(false, p.T, p.G);
  few.long_queries = 0;
  plan_for(few, kFewPerSm * h->num_sms, few_whole, few_whole ? 1 + kFewOver : 2, 0);
  few.piece_ml = reinterpret_cast<float2*>(base + at.few_ml);
  few.piece_o = reinterpret_cast<float*>(base + at.few_o);
  few.records = few.plan.whole ? nullptr : reinterpret_cast<PieceRecord*>(base + at.few_records);
  const bool join_tiles = tiles && !p.plan.whole, join_few = (!tiles || mixed) && !few.plan.whole;
  if (mixed) {
    few.few_rows = few_rows;
    p.few_rows = -few_rows;
  }
  if (tiles) {
    p.alone = !mixed && !join_tiles && !fold;
    ML_LAUNCH(h, launch_attention_tiles(p, PrefixRun{}, p.plan.ctas, dp, stream), "attention launch");
  }
  if (!tiles || mixed) {
    few.follows = few.follows || tiles;
    few.alone = !join_tiles && !join_few && !fold;
    ML_LAUNCH(h, launch_attention_rows(few, dp, eight, stream), "attention launch");
  }
  if (join_tiles || join_few) {
    p.alone = !fold;
    ML_LAUNCH(h, launch_join(p, pieces_of(p, join_tiles, 8 * most_items <= h->num_sms), pieces_of(few, join_few, false), dp, stream), "attention join launch");
  }
  if (fold) ML_LAUNCH(h, launch_fold(p, dp, stream), "attention fold launch");
  return MOE_LORA_OK;
}
