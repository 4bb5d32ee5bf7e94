// Causal attention to a paged cache (moe_lora_attention): the entry point and the kernel for any layout.
#include "attention.h"
#include "host.h"

#include <algorithm>
#include <cmath>

namespace mlk {
namespace {

// ---------------------------------------------------------------------------------------
// Any head size, page size and alignment, on plain cores: a block per query row and head.  Its warps take
// the keys 32 at a time in turn, a lane a key, each warp with a running maximum m, sum l and result o
// (o <- o 2^(m - m') + sum p v), and the block adds the warps' results at the end.
// ---------------------------------------------------------------------------------------
constexpr int kAnyWarps = 8;

__global__ void __launch_bounds__(32 * kAnyWarps) attention_any_kernel(const __grid_constant__ AttentionParams p) {
  __shared__ float q_s[512];
  __shared__ float o_s[kAnyWarps][512];
  __shared__ float m_s[kAnyWarps], l_s[kAnyWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const int b = static_cast<int>(blockIdx.y), h = static_cast<int>(blockIdx.z), kh = h / p.G;
  const Request r = request_of(p, b);
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0 && r.bad) record_status(p.status, kDevBadSlot, kWhereAttention);
  for (int i = static_cast<int>(blockIdx.x); i < r.n; i += static_cast<int>(gridDim.x)) {
    const long long row = r.q0 + i;
    for (int d = threadIdx.x; d < p.D; d += blockDim.x) q_s[d] = bf2f(p.q[row * p.q_t + h * p.q_h + d]);
    __syncthreads();
    const int sees = max(r.kv - r.n + i + 1, 0);
    const int of_shared = min(sees, p.shared_len);
    float m = -INFINITY, l = 0.0f;
    float o[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) o[c] = 0.0f;
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
          for (int d = 0; d < p.D; ++d) dot += q_s[d] * bf2f(k[d]);
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
      for (int c = 0; c < 16; ++c) o[c] *= old;
      const int n = min(32, sees - j0);
      for (int t = 0; t < n; ++t) {
        const float wt = __shfl_sync(0xffffffffu, w, t);
        const int pg = __shfl_sync(0xffffffffu, page, t);
        if (pg < 0) continue;
        const __nv_bfloat16* v = p.v + pg * p.v_p + kh * p.v_h + ((j0 + t) % p.page) * p.v_t;
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (c * 32 + lane < p.D) o[c] += wt * bf2f(v[c * 32 + lane]);
      }
    }
#pragma unroll
    for (int c = 0; c < 16; ++c)
      if (c * 32 + lane < p.D) o_s[warp][c * 32 + lane] = o[c];
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

}  // namespace
}  // namespace mlk

extern "C" moe_lora_status moe_lora_attention_workspace_size(int T, int q_heads, int k_heads, int head_dim, size_t* bytes) {
  if (bytes == nullptr || T < 0 || q_heads < 1 || k_heads < 1 || q_heads % k_heads != 0 || head_dim < 1)
    return MOE_LORA_ERR_INVALID_ARG;
  *bytes = 256;
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
      static_cast<long long>(a->table_width) * a->page_size > 0x7fffffffLL)
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->query_offsets == nullptr && a->T != a->B) return MOE_LORA_ERR_INVALID_ARG;
  if (!(std::fabs(a->scale) < INFINITY)) return MOE_LORA_ERR_INVALID_ARG;
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
  p.D = a->head_dim;
  p.num_pages = a->num_pages;
  p.page = a->page_size;
  p.width = a->table_width;
  p.shared_len = a->shared_len;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.status = static_cast<uint32_t*>(workspace);
  ML_ON_DEVICE(h);
  ML_CUDA(cudaMemsetAsync(workspace, 0, 4, stream), "attention status");
  const int across = std::max(1, std::min(a->T, 65536 / std::max(1, a->B)));
  ML_LAUNCH(h, launch_k(attention_any_kernel, dim3(across, a->B, a->q_heads), dim3(32 * kAnyWarps), 0, stream, false, p),
            "attention launch");
  return MOE_LORA_OK;
}
