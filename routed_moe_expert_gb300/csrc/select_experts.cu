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
// threads changes: exponentials and quotients are IEEE float32 results, and the softmax sum is
// taken in fixed point with steps of 2^-43, exact for every term of 2^-20 and more.
//
// A lane holds NQ chunks of V consecutive experts, so loads are one vector per chunk and, where
// groups are a power of two of chunks, a group's best is a few shuffles among neighbouring
// lanes; other groups go through shared memory, a few lanes to a group.  The choice itself: the
// top_k-th largest of the lanes' best keys is a bound below which nothing is chosen; the (few) keys on
// or above it are handed to one lane each, and every lane counts how many come before its own.
//
// Instruction issue bounds long batches: T 16384, E 256, softmax, 8 groups, top_k 6: 11.3 us, 660
// instructions a token, issue slots 79% busy (17 MB at 1.5 TB/s; 2.6 us at 6.8).  So what is computed
// is cut: a softmax without a bias is ordered by its numerators and only the last candidates are
// divided (all divided, and a maximum and a minimum over the warp per pick: 14.4 us with the sum in
// 64-bit integers, whose conversions run at the rate of double precision).  T 4095, E 384, sigmoid with
// a bias, bf16: 5.1 us.  One token: 3.2 us, latency.
#include "common.cuh"
#include "host.h"
#include "kernels.h"

#include <cfloat>
#include <climits>

namespace mlk {

struct SelectParams {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t* packed;
  long long stride;      // elements between two tokens' logits
  int bias_vec;          // bias starts on a 16-byte boundary
  int T, E, k, sigmoid, n_group, topk_group, top2, renormalize, group_size;
  int group_inv;         // ceil(2^20 / group_size): e * group_inv >> 20 = e / group_size for e < 1024
  int group_lanes;       // (any groups) lanes that look through a group
  float factor;
};

namespace {

constexpr int kSelectMaxGroups = 32;   // a lane per group

constexpr unsigned kAll = 0xffffffffu;

MLDEV float warp_max(float v) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

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

// (x0 + y, x1 + y) in one instruction, each rounded as an addition is.
MLDEV float2 add_pair(float x0, float x1, float y) {
  unsigned long long r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %3};\n\tadd.rn.f32x2 %0, a, b;\n\t}"
      : "=l"(r)
      : "f"(x0), "f"(x1), "f"(y));
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
  return f;
}

// A sum of values in [0, 1] in fixed point, with steps of 2^-43 in two parts: adding 4 rounds a value
// to steps of 2^-21, whose number is then the low bits of the result; adding 1.5 x 2^-20 does it to
// what that left out, |rest| <= 2^-22.  (A conversion to 64-bit integers would be exact, but it runs at
// the rate of double precision, a quarter of this kernel's time.)
struct FixedSum {
  uint32_t high = 0, low = 0;   // low: a signed number
  MLDEV void add(float e0, float e1) {
    const float2 h = add_pair(e0, e1, 4.0f);
    const float2 r = add_pair(h.x, h.y, -4.0f);
    const float2 l = add_pair(__fsub_rn(e0, r.x), __fsub_rn(e1, r.y), 0x1.8p-20f);
    high += __float_as_uint(h.x) + __float_as_uint(h.y) - 2 * __float_as_uint(4.0f);
    low += __float_as_uint(l.x) + __float_as_uint(l.y) - 2 * __float_as_uint(0x1.8p-20f);
  }
  // over the warp, rounded once; up to 1024 values, the largest of them 1 (or none above 0)
  MLDEV float warp_total() const {
    const unsigned long long h = __reduce_add_sync(0xffffffffu, high);
    const long long l = __reduce_add_sync(0xffffffffu, static_cast<int>(low));
    return __ull2float_rn((h << 22) + l) * 0x1p-43f;
  }
};

// 1 / d, correctly rounded, for 1 <= d < 2^100: a reciprocal within an ulp and one residual
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J.
// Res. Dev. 34, 1990).
MLDEV float reciprocal(float d) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
  return __fmaf_rn(__fmaf_rn(-d, r, 1.0f), r, r);
}

// What a token's softmax subtracts and divides by.
struct Softmax {
  float zmax, total, inverse;   // inverse: the correctly rounded reciprocal of total
  MLDEV float numerator(float z) const { return expf(__fsub_rn(z, zmax)); }
  // e / total, correctly rounded: with the correctly rounded reciprocal one residual makes
  // q = e / total exact (Markstein) while it does not underflow
  MLDEV float quotient(float e) const {
    const float q = __fmul_rn(e, inverse);
    return __fmaf_rn(__fmaf_rn(-q, total, e), inverse, q);
  }
  MLDEV float any_quotient(float e) const { return e < 0x1p-100f ? __fdiv_rn(e, total) : quotient(e); }
};

MLDEV float sigmoid_score(float z) { return __frcp_rn(__fadd_rn(1.0f, expf(-z))); }

// Keys (and their ids) on or above a bound, one per lane, for the ordered choice.
constexpr int kCandidates = 32;

// GROUPS: 0 no groups, 1 groups of 2^n chunks (shuffles), 2 any groups (shared memory, E floats a
// warp).
template <typename TL, int NQ, int V, int GROUPS>
__global__ void __launch_bounds__(256) select_experts_kernel(const SelectParams p) {
  constexpr int NV = NQ * V;
  __shared__ __align__(16) float2 cand_s[8][kCandidates];
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (t >= p.T) return;   // whole warps
  float2* cand = cand_s[threadIdx.x >> 5];
  const TL* row = static_cast<const TL*>(p.logits) + static_cast<long long>(t) * p.stride;
  auto id_of = [&](int n) -> int { return ((n / V) * 32 + lane) * V + n % V; };   // lane's n-th value

  float z[NV];   // logits; -inf: ruled out
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    float c[V];
    const int e = (i * 32 + lane) * V;   // V == 4: E is a multiple of 4
    if (e < p.E) {
      load_logits<TL, V>(row, e, c);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = -INFINITY;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) z[i * V + v] = fmaxf(c[v], -INFINITY);
  }

  // Keys; NaN, which maxima and comparisons pass over, or -inf: ruled out.  Without a bias a softmax's
  // are its numerators: dividing by the sum keeps their order (rounding can make neighbours equal).
  float key[NV];
  Softmax soft = {0.0f, 1.0f, 1.0f};
  const bool numerators = !p.sigmoid && p.bias == nullptr;
  if (!p.sigmoid) {
    float m = z[0];
#pragma unroll
    for (int n = 1; n < NV; ++n) m = fmaxf(m, z[n]);
    soft.zmax = warp_max(m);
    if (soft.zmax == INFINITY) {   // +inf counts as the largest finite value
      soft.zmax = FLT_MAX;
#pragma unroll
      for (int n = 0; n < NV; ++n) z[n] = fminf(z[n], FLT_MAX);
    }
    if (soft.zmax == -INFINITY) soft.zmax = 0.0f;   // all ruled out
    FixedSum sum;
#pragma unroll
    for (int n = 0; n < NV; n += 2) {
      const float e0 = soft.numerator(z[n]), e1 = soft.numerator(z[n + 1]);
      sum.add(e0, e1);
      key[n] = __fmaf_rn(z[n], 0.0f, e0);   // NaN where z is -inf
      key[n + 1] = __fmaf_rn(z[n + 1], 0.0f, e1);
    }
    soft.total = fmaxf(sum.warp_total(), 1.0f);   // at least 1, or all are ruled out
    soft.inverse = reciprocal(soft.total);
    if (!numerators) {
      uint32_t least = 0xffffffffu;   // bits of the smallest nonzero numerator, less 1
#pragma unroll
      for (int n = 0; n < NV; ++n) least = min(least, __float_as_uint(key[n]) - 1u);
      if (least >= __float_as_uint(0x1p-100f)) {
#pragma unroll
        for (int n = 0; n < NV; ++n) key[n] = soft.quotient(key[n]);
      } else {
#pragma unroll
        for (int n = 0; n < NV; ++n) key[n] = __fdiv_rn(key[n], soft.total);
      }
    }
  } else {
    // 1 + exp(-z) stays below 2^100 for z >= -60; with lower (finite) ones all take the division
    uint32_t low = 0xffffffffu;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      low = min(low, __float_as_uint(z[n]) - (__float_as_uint(-60.0f) + 1u));
      const float s = reciprocal(__fadd_rn(1.0f, expf(-fmaxf(z[n], -60.0f))));
      key[n] = z[n] > -INFINITY ? s : __int_as_float(0x7fffffff);
    }
    if (low < __float_as_uint(-INFINITY) - (__float_as_uint(-60.0f) + 1u)) {
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (z[n] > -INFINITY) key[n] = sigmoid_score(z[n]);
    }
  }
  if (p.bias != nullptr) {   // (a NaN bias rules out, too)
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int e = (i * 32 + lane) * V;
      if (e < p.E) {
        float b[V];
        if (V == 4 && p.bias_vec) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(p.bias + e));
          b[0] = v.x;
          b[V > 1 ? 1 : 0] = v.y;
          b[V > 1 ? 2 : 0] = v.z;
          b[V > 1 ? 3 : 0] = v.w;
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) b[v] = __ldg(p.bias + e + v);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) key[i * V + v] = __fadd_rn(key[i * V + v], b[v]);
      }
    }
  }
  // the score that a group's best key stands for
  auto scored = [&](float f) { return !numerators ? f : f >= 0.0f ? soft.any_quotient(f) : -INFINITY; };

  if constexpr (GROUPS != 0) {
    float mine = -INFINITY;   // lane g: group g's score
    if constexpr (GROUPS == 1) {
      // the best two keys of each chunk (it lies in one group), then of the group's chunks
      float b1[NQ], b2[NQ];
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        b1[i] = fmaxf(key[i * V], -INFINITY);
        b2[i] = -INFINITY;
        if (p.top2) {
#pragma unroll
          for (int v = 1; v < V; ++v) {
            const float f = fmaxf(key[i * V + v], -INFINITY);
            b2[i] = fmaxf(b2[i], fminf(b1[i], f));
            b1[i] = fmaxf(b1[i], f);
          }
        } else {
#pragma unroll
          for (int v = 1; v < V; ++v) b1[i] = fmaxf(b1[i], key[i * V + v]);
        }
      }
      const int width = p.group_size / V;   // chunks (lanes) of a group: 2^n <= 32
      for (int off = 1; off < width; off *= 2) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const float o1 = __shfl_xor_sync(kAll, b1[i], off);
          if (p.top2) {
            const float o2 = __shfl_xor_sync(kAll, b2[i], off);
            b2[i] = fmaxf(fmaxf(b2[i], o2), fminf(b1[i], o1));
          }
          b1[i] = fmaxf(b1[i], o1);
        }
      }
      const int first = lane * width;   // group g's first chunk
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const float own = p.top2 ? __fadd_rn(scored(b1[i]), scored(b2[i])) : scored(b1[i]);
        const float of = __shfl_sync(kAll, own, first & 31);
        if ((first >> 5) == i) mine = of;
      }
    } else {
      extern __shared__ __align__(16) float keys_s[];
      float* keys = keys_s + (threadIdx.x >> 5) * p.E;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int e = (i * 32 + lane) * V;
        if (e < p.E) {
          if constexpr (V == 4)
            *reinterpret_cast<float4*>(keys + e) =
                make_float4(key[i * V], key[i * V + 1], key[i * V + 2], key[i * V + 3]);
          else
            keys[e] = key[i];
        }
      }
      __syncwarp();
      const int width = p.group_lanes;   // lanes of a group: 2^n, width * n_group <= 32
      const int g = lane / width;
      float b1 = -INFINITY, b2 = -INFINITY;
      if (g < p.n_group)
        for (int e = lane & (width - 1); e < p.group_size; e += width) {
          const float f = fmaxf(keys[g * p.group_size + e], -INFINITY);
          b2 = fmaxf(b2, fminf(b1, f));
          b1 = fmaxf(b1, f);
        }
      for (int off = 1; off < width; off *= 2) {
        const float o1 = __shfl_xor_sync(kAll, b1, off), o2 = __shfl_xor_sync(kAll, b2, off);
        b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
        b1 = fmaxf(b1, o1);
      }
      mine = __shfl_sync(kAll, p.top2 ? __fadd_rn(scored(b1), scored(b2)) : scored(b1), (lane * width) & 31);
    }
    if (mine != mine) mine = -INFINITY;   // +inf (a bias) and a ruled-out second
    unsigned stay = 0;   // ties, also of groups without an expert left: the lower group
    bool taken = lane >= p.n_group;
    for (int j = 0; j < p.topk_group; ++j) {
      const float m = warp_max(taken ? -INFINITY : mine);
      const int g = __ffs(__ballot_sync(kAll, !taken && mine == m)) - 1;
      stay |= 1u << g;
      taken |= lane == g;
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      // groups of 2^n chunks: a chunk's group is its first value's
      bool stays = false;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (GROUPS == 2 || v == 0) {
          const int g = (((i * 32 + lane) * V + v) * p.group_inv) >> 20;   // e / group_size
          stays = (stay >> (g & 31)) & 1u;
        }
        if (!stays) key[i * V + v] = -INFINITY;
      }
    }
  }

  // the bound: the top_k-th largest of the lanes' best keys (equal ones taken out together, which
  // only lowers it; -inf when that leaves fewer)
  float best = key[0];
#pragma unroll
  for (int n = 1; n < NV; ++n) best = fmaxf(best, key[n]);
  float bound = -INFINITY;
  {
    float left = best;
    for (int j = 0; j < p.k; ++j) {
      bound = warp_max(left);
      if (left == bound) left = -INFINITY;
    }
  }
  // numerators a little below the bound may give the same quotient (within 2^-23 while it is no
  // subnormal number)
  if (numerators) bound = bound >= 0x1p-100f ? bound * 0x1.fffffp-1f : -INFINITY;
  // candidates: keys on or above the bound (all that is left when there is no bound), each lane's
  // after those of the lanes below it
  int count = kCandidates + 1;
  if (bound > -INFINITY) {
    int own = 0;
#pragma unroll
    for (int n = 0; n < NV; ++n) own += key[n] >= bound;
    const unsigned below = (1u << lane) - 1u;
    int at = 0;
    count = 0;
#pragma unroll
    for (int bit = 0; (1 << bit) <= NV; ++bit) {
      const unsigned who = __ballot_sync(kAll, (own >> bit) & 1);
      at += __popc(who & below) << bit;
      count += __popc(who) << bit;
    }
    if (own != 0 && count <= kCandidates) {
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (key[n] >= bound) cand[at++] = make_float2(key[n], __int_as_float(id_of(n)));
    }
  }
  int my_id = 0, chosen = 0;   // lane j keeps pick j
  float w = 0.0f;              // and its weight
  if (count <= kCandidates) {
    // count >= top_k.  A lane ranks its candidate among all: larger keys first, then lower ids; as
    // 64-bit numbers, the key's bits above the id's complement.
    __syncwarp();
    const float2 c = lane < count ? cand[lane] : make_float2(0.0f, 0.0f);
    const float s = numerators && lane < count ? soft.any_quotient(c.x) : c.x;
    const int id = __float_as_int(c.y);
    const int bits = __float_as_int(s);
    const uint32_t up = static_cast<uint32_t>(bits ^ ((bits >> 31) | INT_MIN));   // in the order of s
    const unsigned long long mine =
        lane < count ? static_cast<unsigned long long>(up) << 32 | static_cast<uint32_t>(~id) : 0ull;
    unsigned long long* order = reinterpret_cast<unsigned long long*>(cand);
    __syncwarp();
    order[lane] = mine;
    __syncwarp();
    int rank = 0;
    for (int j = 0; j < count; j += 2) {
      const ulonglong2 other = *reinterpret_cast<const ulonglong2*>(order + j);
      rank += other.x > mine;
      rank += other.y > mine;
    }
    __syncwarp();
    if (lane < count) cand[rank] = make_float2(s, c.y);
    __syncwarp();
    const float2 pick = cand[lane];
    my_id = __float_as_int(pick.y);
    w = pick.x;
    chosen = p.k;
  } else {
#pragma unroll
    for (int n = 0; n < NV; ++n) key[n] = fmaxf(scored(key[n]), -INFINITY);
    // many equal keys, or fewer lanes with an expert left than top_k: pick by pick
    int best_n = 0;
    auto look = [&]() {
      best = -INFINITY;
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (key[n] > best) {
          best = key[n];
          best_n = n;
        }
    };
    // ids of a lane ascend with n, so the first of its equal keys is its lowest id
    uint32_t gone[(NV + 31) / 32] = {};
    look();
    for (; chosen < p.k; ++chosen) {
      const float m = warp_max(best);
      if (m == -INFINITY) break;
      const int mine = id_of(0) + (best_n / V) * 32 * V + best_n % V;
      const int pick = __reduce_min_sync(kAll, best == m ? mine : 0x7fffffff);
      if (lane == chosen) {
        my_id = pick;
        w = m;
      }
      if (best == m && mine == pick) {
#pragma unroll
        for (int n = 0; n < NV; ++n)
          if (n == best_n) {
            key[n] = -INFINITY;
            gone[n / 32] |= 1u << (n % 32);
          }
        look();
      }
    }
    // the rest: the lowest ids that are ruled out, in order, with weight 0
    int next = chosen;
    for (int i = 0; i < NQ && next < p.k; ++i) {
      int mine = 0;   // this lane's ruled-out values of chunk i
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (n / V == i) mine += id_of(n) < p.E && !((gone[n / 32] >> (n % 32)) & 1u);
      int incl = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kAll, incl, off);
        if (lane >= off) incl += y;
      }
      int at = next + incl - mine;
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (n / V == i && id_of(n) < p.E && !((gone[n / 32] >> (n % 32)) & 1u)) {
          if (at < p.k) {
            const float w = __fmul_rn(0.0f, p.factor);
            const long long o = static_cast<long long>(t) * p.k + at;
            p.ids[o] = id_of(n);
            p.weights[o] = w;
            if (p.packed != nullptr)
              p.packed[o] = (id_of(n) << 16) | static_cast<int>(__bfloat16_as_ushort(f2bf(w)));
          }
          ++at;
        }
      next += __shfl_sync(kAll, incl, 31);
    }
  }

  if (lane >= chosen) w = 0.0f;
  if (p.bias != nullptr && lane < chosen) {   // the score without the bias, again from the logit
    float c[1];
    load_logits<TL, 1>(row, my_id, c);
    w = p.sigmoid ? sigmoid_score(c[0]) : soft.any_quotient(soft.numerator(fminf(c[0], FLT_MAX)));
  }
  if (p.renormalize) {
    float sum = w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(kAll, sum, off));
    w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
  }
  w = __fmul_rn(w, p.factor);
  if (lane < chosen) {
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
  const int width = p.group_size / 4;   // chunks of a group on the vector path
  const int groups = p.n_group == p.topk_group ? 0   // all of them stay
                     : vec && p.group_size % 4 == 0 && width <= 32 && (width & (width - 1)) == 0 ? 1 : 2;
#define ML_SELECT(NQ, V, G) \
  return launch_k(select_experts_kernel<TL, NQ, V, G>, grid, block, G == 2 ? warps * p.E * 4 : 0, stream, true, p)
#define ML_SELECT_G(NQ)              \
  do {                               \
    if (groups == 0) ML_SELECT(NQ, 4, 0); \
    if (groups == 1) ML_SELECT(NQ, 4, 1); \
    ML_SELECT(NQ, 4, 2);             \
  } while (0)
  if (vec) {
    if (p.E <= 128) ML_SELECT_G(1);
    if (p.E <= 256) ML_SELECT_G(2);
    if (p.E <= 384) ML_SELECT_G(3);
    if (p.E <= 512) ML_SELECT_G(4);
    ML_SELECT_G(8);
  }
#define ML_SELECT_1(NQ)              \
  do {                               \
    if (groups == 0) ML_SELECT(NQ, 1, 0); \
    ML_SELECT(NQ, 1, 2);             \
  } while (0)
  if (p.E <= 128) ML_SELECT_1(4);
  if (p.E <= 256) ML_SELECT_1(8);
  if (p.E <= 384) ML_SELECT_1(12);
  if (p.E <= 512) ML_SELECT_1(16);
  ML_SELECT_1(32);
#undef ML_SELECT_1
#undef ML_SELECT_G
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
  if (a->n_group > kSelectMaxGroups || a->T > kMaxExtent) return MOE_LORA_ERR_UNSUPPORTED;
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
  p.bias_vec = aligned16(a->bias);
  p.group_inv = ((1 << 20) + group_size - 1) / group_size;
  p.group_lanes = 32;
  while (p.group_lanes * p.n_group > 32) p.group_lanes /= 2;
  p.factor = a->routed_scaling_factor;
  // four experts per load when rows divide into aligned quads
  const bool vec = a->E % 4 == 0 && a->logits_stride % 4 == 0 &&
                   (at & (a->logits_f32 ? 15u : 7u)) == 0;
  ML_ON_DEVICE(h);
  ML_LAUNCH(h, a->logits_f32 ? launch_select<float>(p, vec, stream) : launch_select<__nv_bfloat16>(p, vec, stream),
            "select_experts launch");
  return MOE_LORA_OK;
}
