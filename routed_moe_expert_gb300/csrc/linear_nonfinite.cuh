// What adapter weights that are not finite add to the tokens of their own slot (moe_lora_linear).
//
// The stacked B holds finite values alone (linear_pack_kernel in linear_narrow.cu): in a marked row a
// slot's values are classes, 0, +-1 (finite), +-2 (infinite) and 3 (NaN).  The products with them are
// finite, and so nothing to other slots' tokens; to a token of the slot itself this file adds the sum of
// u times what the classes stand for, which is infinite or NaN as the formula's sum is, whatever its
// finite terms are.  None of it runs for adapters that are finite: a kernel reads one word, the
// slots that have any mark.
#pragma once

#include "common.cuh"
#include "linear.h"

namespace mlk {

MLDEV bool marked(const LinearParams& p, int s, int n) {
  return (__ldcg(p.marks + static_cast<long long>(n) * p.mark_stride + (s >> 3)) >> (s & 7)) & 1;
}
MLDEV bool is_sick(const LinearParams& p, unsigned long long sick, int s) {
  return s >= 0 && s < p.slots.S && p.slots.hi[s] > p.slots.lo[s] && ((sick >> s) & 1);
}
// u times the class of slot column c in row n
MLDEV float class_term(const LinearParams& p, float u, int c, int n) {
  const float k = bf2f(__ldcg(p.b + static_cast<long long>(n) * p.Rs + c)), size = fabsf(k);
  return u * (size == 3.0f ? NAN : size == 2.0f ? copysignf(INFINITY, k) : k);
}

// Row n, a token of slot s, whose u lies in global memory.
static __device__ __noinline__ float nonfinite_of_row(const LinearParams& p, int t, int s, int n) {
  const __nv_bfloat16* row = p.u + static_cast<long long>(t) * p.pieces * p.Rs;
  float sum = 0.0f;
  for (int c = p.slots.lo[s]; c < p.slots.hi[s]; ++c) {
    float u = bf2f(__ldcg(row + c));
    for (int i = 1; i < p.pieces; ++i) u += bf2f(__ldcg(row + i * p.Rs + c));
    sum += class_term(p, u, c, n);
  }
  return sum;
}
// Rows n to n + rows of token t, whose y this thread has stored.
MLDEV void add_to_y(const LinearParams& p, int t, int n, float add) {
  const long long at = static_cast<long long>(t) * p.ldy + n;
  if (p.y_f32) {
    static_cast<float*>(p.y)[at] += add;
  } else {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + at;
    *y = f2bf(bf2f(*y) + add);
  }
}
static __device__ __noinline__ void add_nonfinite(const LinearParams& p, unsigned long long sick, int t, int n, int rows) {
  const int s = p.slot_idx[t];
  if (!is_sick(p, sick, s)) return;
  for (int e = n; e < n + rows && e < p.N; ++e)
    if (marked(p, s, e)) add_to_y(p, t, e, nonfinite_of_row(p, t, s, e));
}
// A lane's 128 bytes of a store box (linear_wide.cu), the columns of its token t from n on.
template <bool F32>
static __device__ __noinline__ void add_nonfinite_to_box(const LinearParams& p, unsigned long long sick, uint8_t* box, int t, int n) {
  const int s = t < p.T ? p.slot_idx[t] : -1, lane = threadIdx.x & 31;
  if (!is_sick(p, sick, s)) return;
  for (int j = 0; j < (F32 ? 32 : 64) && n + j < p.N; ++j) {
    if (!marked(p, s, n + j)) continue;
    const float add = nonfinite_of_row(p, t, s, n + j);
    uint8_t* at = box + lane * 128 + (((F32 ? j >> 2 : j >> 3) ^ (lane & 7)) << 4) + (F32 ? (j & 3) * 4 : (j & 7) * 2);
    if constexpr (F32) {
      *reinterpret_cast<float*>(at) += add;
    } else {
      __nv_bfloat16* v = reinterpret_cast<__nv_bfloat16*>(at);
      *v = f2bf(bf2f(*v) + add);
    }
  }
}
// Row n of the tokens t0 to t0 + count, whose y this thread has stored and whose u is the operand u_s in
// shared memory (linear_cluster.cu).
template <int BN, int NB>
__device__ __noinline__ void add_nonfinite_of_operand(const LinearParams& p, unsigned long long sick, const uint8_t* u_s,
                                                      int t0, int count, int n) {
  for (int j = 0; n < p.N && j < count; ++j) {
    const int s = p.slot_idx[t0 + j];
    if (!is_sick(p, sick, s) || !marked(p, s, n)) continue;
    float sum = 0.0f;
    for (int c = p.slots.lo[s]; c < p.slots.hi[s]; ++c) {
      float u = 0.0f;
      for (int i = 0; i < p.pieces; ++i)
        u += bf2f(*reinterpret_cast<const __nv_bfloat16*>(u_s + (i * NB + (c >> 6)) * BN * 128 + j * 128 +
                                                          ((((c & 63) >> 3) ^ (j & 7)) << 4) + (c & 7) * 2));
      sum += class_term(p, u, c, n);
    }
    add_to_y(p, t0 + j, n, sum);
  }
}

}  // namespace mlk
