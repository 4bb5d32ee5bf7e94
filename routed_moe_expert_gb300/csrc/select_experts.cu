// Choice of experts from the router's logits (moe_lora_select_experts), one warp per token.
//
//   s_e   = exp(z_e - max z) / sum_e exp(z_e - max z)   or   1 / (1 + exp(-z_e))
//   key_e = s_e + bias_e, and -inf where z_e is -inf or NaN (an expert ruled out)
//   a group of E / n_group neighbouring experts scores its best key, or the sum of its two
//   best; the experts outside the topk_group best groups get key -inf
//   ids   = the top_k largest keys, ties to the lower id
//   w_j   = s of id j (0 where its key is -inf) [/ sum of these] * factor
//
// Every value that decides a choice is one float32 operation sequence that no order of
// threads changes: the exponentials and divisions are IEEE float32 operations of one lane,
// and the softmax sum is taken in fixed point with steps of 2^-52 (the terms lie in [0, 1],
// so 1024 of them fit 64 bits), exact for every term of 2^-28 and more.
//
// A lane holds NQ chunks of V consecutive experts, so loads are one vector per chunk and a
// chunk lies in one group.  A pick is a warp maximum over order-preserving unsigned keys and
// a warp minimum over the ids that hold it (redux.sync), then the owning lane alone looks
// through its values again.
#include "common.cuh"
#include "host.h"
#include "kernels.h"

#include <cfloat>

namespace mlk {

struct SelectParams {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t* packed;
  long long stride;      // elements between two tokens' logits
  int T, E, k, sigmoid, n_group, topk_group, top2, renormalize, group_size;
  float factor;
};

namespace {

constexpr int kSelectMaxGroups = 32;   // a lane per group

// Unsigned integer with the order of the float keys; 0 is free for "taken".
MLDEV uint32_t ordered(float f) {
  uint32_t u = __float_as_uint(f);
  if (u == 0x80000000u) u = 0u;   // -0 and +0 are equal
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kRuledOut = 0x007fffffu;   // ordered(-inf)

MLDEV float unordered(uint32_t v) { return __uint_as_float((v & 0x80000000u) ? (v & 0x7fffffffu) : ~v); }

// A logit as it counts: NaN is a ruled-out expert, +inf the largest finite value.
MLDEV float usable(float z) { return (z != z) ? -INFINITY : fminf(z, FLT_MAX); }

template <typename TL, int V>
MLDEV void load_logits(const TL* row, int e, float (&z)[V]) {
  if constexpr (V == 4 && sizeof(TL) == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(row + e));
    z[0] = v.x;
    z[1] = v.y;
    z[2] = v.z;
    z[3] = v.w;
  } else if constexpr (V == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + e));
    z[0] = __uint_as_float(v.x << 16);
    z[1] = __uint_as_float(v.x & 0xffff0000u);
    z[2] = __uint_as_float(v.y << 16);
    z[3] = __uint_as_float(v.y & 0xffff0000u);
  } else if constexpr (sizeof(TL) == 4) {
    z[0] = row[e];
  } else {
    z[0] = bf2f(row[e]);
  }
}

// The sum over the warp of values below 2^58, through three 32-bit reductions of 26 bits.
MLDEV unsigned long long warp_sum_u58(unsigned long long v) {
  constexpr unsigned kMask = (1u << 26) - 1;
  const unsigned a = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v) & kMask);
  const unsigned b = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v >> 26) & kMask);
  const unsigned c = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v >> 52));
  return a + (static_cast<unsigned long long>(b) << 26) + (static_cast<unsigned long long>(c) << 52);
}

MLDEV float exp_above(float z, float zmax) { return z == -INFINITY ? 0.0f : expf(__fsub_rn(z, zmax)); }

template <typename TL, int NQ, int V>
__global__ void __launch_bounds__(256) select_experts_kernel(const SelectParams p) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.T) return;   // whole warps
  const TL* row = static_cast<const TL*>(p.logits) + static_cast<long long>(t) * p.stride;
  constexpr unsigned kAll = 0xffffffffu;

  float z[NQ][V];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int e = (i * 32 + lane) * V;   // V == 4: E is a multiple of 4
    if (e < p.E) {
      load_logits<TL, V>(row, e, z[i]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) z[i][v] = -INFINITY;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) z[i][v] = usable(z[i][v]);
  }

  // scores and keys
  uint32_t key[NQ][V];
  float zmax = 0.0f, total = 1.0f;
  if (!p.sigmoid) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) m = max(m, ordered(z[i][v]));
    zmax = unordered(__reduce_max_sync(kAll, m));
    unsigned long long sum = 0;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) sum += __float2ull_rz(exp_above(z[i][v], zmax) * 0x1p52f);
    total = __ull2float_rn(warp_sum_u58(sum)) * 0x1p-52f;   // 0 only when every expert is ruled out
  }
  auto score = [&](float zz) -> float {
    if (p.sigmoid) return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-zz)));
    return total > 0.0f ? __fdiv_rn(exp_above(zz, zmax), total) : 0.0f;
  };
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int e = (i * 32 + lane) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (e < p.E) {
        float f = score(z[i][v]);
        if (p.bias != nullptr) f = __fadd_rn(f, __ldg(p.bias + e + v));
        key[i][v] = (z[i][v] == -INFINITY || f != f) ? kRuledOut : ordered(f);
      } else {
        key[i][v] = 0u;
      }
    }
  }

  if (p.n_group > 1) {
    // each chunk's best two keys (a chunk lies in one group), then a warp maximum per group
    uint32_t b1[NQ], b2[NQ];
    int group[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int e = (i * 32 + lane) * V;
      group[i] = e < p.E ? e / p.group_size : -1;
      b1[i] = key[i][0];
      b2[i] = 0u;
#pragma unroll
      for (int v = 1; v < V; ++v) {
        b2[i] = max(b2[i], min(b1[i], key[i][v]));
        b1[i] = max(b1[i], key[i][v]);
      }
    }
    uint32_t mine = 0u;   // lane g: the order key of group g's score
    for (int g = 0; g < p.n_group; ++g) {
      uint32_t l1 = 0u, l2 = 0u;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        if (group[i] == g) {
          l2 = max(max(l2, b2[i]), min(l1, b1[i]));
          l1 = max(l1, b1[i]);
        }
      }
      const uint32_t m1 = __reduce_max_sync(kAll, l1);
      uint32_t score_g = m1;
      if (p.top2) {
        const unsigned owners = __ballot_sync(kAll, l1 == m1);
        const uint32_t m2 = __reduce_max_sync(kAll, lane == __ffs(owners) - 1 ? l2 : l1);
        const float f = __fadd_rn(unordered(m1), unordered(m2));
        score_g = f != f ? kRuledOut : ordered(f);
      }
      if (lane == g) mine = score_g;
    }
    unsigned stay = 0;
    for (int j = 0; j < p.topk_group; ++j) {
      const uint32_t m = __reduce_max_sync(kAll, mine);
      const int g = __ffs(__ballot_sync(kAll, mine == m)) - 1;   // the lowest group that holds it
      stay |= 1u << g;
      if (lane == g) mine = 0u;
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i)
      if (group[i] >= 0 && !((stay >> group[i]) & 1u)) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[i][v] = kRuledOut;
      }
  }

  // top_k: lane j keeps pick j
  int my_id = 0;
  uint32_t my_key = 0u;
  uint32_t best = 0u;   // this lane's largest key and the lowest id that holds it
  int best_id = 0;
  auto look = [&]() {
    best = 0u;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (key[i][v] > best) {
          best = key[i][v];
          best_id = (i * 32 + lane) * V + v;
        }
  };
  look();
  for (int j = 0; j < p.k; ++j) {
    const uint32_t m = __reduce_max_sync(kAll, best);
    const int id = __reduce_min_sync(kAll, best == m ? best_id : 0x7fffffff);
    if (lane == j) {
      my_id = id;
      my_key = m;
    }
    if (best == m && best_id == id) {   // the owner
#pragma unroll
      for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v)
          if ((i * 32 + lane) * V + v == id) key[i][v] = 0u;
      look();
    }
  }

  // weights: lane j's score again, from its logit
  float w = 0.0f;
  if (lane < p.k && my_key > kRuledOut) {
    float zz[1];
    load_logits<TL, 1>(row, my_id, zz);
    w = score(usable(zz[0]));
  }
  if (p.renormalize) {
    float sum = w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(kAll, sum, off));
    w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
  }
  w = __fmul_rn(w, p.factor);
  if (lane < p.k) {
    const long long at = static_cast<long long>(t) * p.k + lane;
    p.ids[at] = my_id;
    p.weights[at] = w;
    if (p.packed != nullptr)
      p.packed[at] = (my_id << 16) | static_cast<int>(__bfloat16_as_ushort(f2bf(w)));
  }
}

template <typename TL>
cudaError_t launch_select(const SelectParams& p, bool vec, cudaStream_t stream) {
  // one warp per block while that leaves SMs idle, then eight
  const int warps = p.T <= 1024 ? 1 : 8;
  const dim3 grid((p.T + warps - 1) / warps), block(32 * warps);
#define ML_SELECT(NQ, V) \
  return launch_k(select_experts_kernel<TL, NQ, V>, grid, block, 0, stream, false, p)
  if (vec) {
    if (p.E <= 128) ML_SELECT(1, 4);
    if (p.E <= 256) ML_SELECT(2, 4);
    if (p.E <= 384) ML_SELECT(3, 4);
    if (p.E <= 512) ML_SELECT(4, 4);
    ML_SELECT(8, 4);
  }
  if (p.E <= 256) ML_SELECT(8, 1);
  ML_SELECT(32, 1);
#undef ML_SELECT
}

}  // namespace
}  // namespace mlk

extern "C" moe_lora_status moe_lora_select_experts(moe_lora_handle* h, const moe_lora_select_args* a,
                                                   moe_lora_stream stream) {
  using namespace mlk;
  if (h == nullptr || a == nullptr) return MOE_LORA_ERR_INVALID_ARG;
  if (a->T < 0 || a->E < 1 || a->E > kMaxExperts || a->top_k < 1 || a->top_k > kMaxTopK || a->top_k > a->E)
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->scoring != MOE_LORA_SCORE_SOFTMAX && a->scoring != MOE_LORA_SCORE_SIGMOID) return MOE_LORA_ERR_INVALID_ARG;
  if (a->group_score != MOE_LORA_GROUP_MAX && a->group_score != MOE_LORA_GROUP_TOP2) return MOE_LORA_ERR_INVALID_ARG;
  if (a->n_group < 1 || a->topk_group < 1 || a->topk_group > a->n_group || a->E % a->n_group != 0)
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->n_group > kSelectMaxGroups) return MOE_LORA_ERR_UNSUPPORTED;
  const int group_size = a->E / a->n_group;
  if (a->top_k > a->topk_group * group_size) return MOE_LORA_ERR_INVALID_ARG;
  if (a->n_group > 1 && a->group_score == MOE_LORA_GROUP_TOP2 && group_size < 2) return MOE_LORA_ERR_INVALID_ARG;
  if (!(a->routed_scaling_factor == a->routed_scaling_factor)) return MOE_LORA_ERR_INVALID_ARG;
  if (a->logits_stride < a->E && a->T > 1) return MOE_LORA_ERR_INVALID_ARG;
  if (a->T == 0) return MOE_LORA_OK;
  if (a->logits == nullptr || a->topk_ids == nullptr || a->topk_weights == nullptr) return MOE_LORA_ERR_INVALID_ARG;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a->logits);
  if ((at & (a->logits_f32 ? 3u : 1u)) != 0 || !aligned4(a->bias) || !aligned4(a->topk_ids) ||
      !aligned4(a->topk_weights) || !aligned4(a->packed_topk_ids))
    return MOE_LORA_ERR_INVALID_ARG;
  SelectParams p;
  p.logits = a->logits;
  p.bias = a->bias;
  p.ids = a->topk_ids;
  p.weights = a->topk_weights;
  p.packed = a->packed_topk_ids;
  p.stride = a->logits_stride;
  p.T = a->T;
  p.E = a->E;
  p.k = a->top_k;
  p.sigmoid = a->scoring == MOE_LORA_SCORE_SIGMOID;
  p.n_group = a->n_group;
  p.topk_group = a->topk_group;
  p.top2 = a->group_score == MOE_LORA_GROUP_TOP2;
  p.renormalize = a->renormalize != 0;
  p.group_size = group_size;
  p.factor = a->routed_scaling_factor;
  // four experts per load when rows and groups divide into aligned quads
  const bool vec = a->E % 4 == 0 && group_size % 4 == 0 && a->logits_stride % 4 == 0 &&
                   (at & (a->logits_f32 ? 15u : 7u)) == 0;
  ML_LAUNCH(h, a->logits_f32 ? launch_select<float>(p, vec, stream) : launch_select<__nv_bfloat16>(p, vec, stream),
            "select_experts launch");
  return MOE_LORA_OK;
}
