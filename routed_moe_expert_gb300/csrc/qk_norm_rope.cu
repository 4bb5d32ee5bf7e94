// Norm of every query and key head with the position rotation, in one pass
// (moe_lora_qk_norm_rope).  For a head x of D values with norm weights w:
//
//   n_i = x_i / sqrt(mean_j x_j^2 + eps) * w_i
//   the first R values are rotated by the token's position row of the table (R/2 cosines c,
//   then R/2 sines s), pairing (i, i + R/2), or (2i, 2i + 1) when interleaved:
//     a' = a c - b s,  b' = b c + a s
//   and the other D - R values stay n_i.
//
// All in float32 from the bf16 inputs, rounded to bf16 once at the end (the norm's result is
// not rounded before the rotation).
//
// It is bound by memory: each value is read once and written once.  L lanes hold a head, so a
// warp holds 32 / L heads of one token at a time; a lane's V-value pieces are chosen so that
// both members of every rotated pair sit in the same lane (pieces i and i + R/2 of a half-split
// rotation), so the only exchange between lanes is the sum of squares.
#include "common.cuh"
#include "host.h"
#include "kernels.h"

#include <algorithm>

namespace mlk {

struct QkParams {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *q_out, *k_out;
  const void *wq, *wk;
  const float* table;
  const void* positions;
  uint32_t* status;
  long long q_t, q_h, k_t, k_h, qo_t, qo_h, ko_t, ko_h, table_t;   // strides in elements
  int T, Hq, Hk, D, R, num_positions, w_f32, pos_i64, interleaved;
  int lanes;        // L: lanes per head, a power of two
  int heads_per_warp;   // heads one warp goes through
  int splits;       // warps per token
  float eps;
};

namespace {

// Plain loads: the output may be the input itself (every head is read before it is written).
template <int V>
MLDEV void load_bf(const __nv_bfloat16* p, float (&f)[V]) {
  if constexpr (V == 8) {
    unpack8(*reinterpret_cast<const uint4*>(p), f);
  } else if constexpr (V == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
  } else if constexpr (V == 2) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    f[0] = __uint_as_float(v << 16);
    f[1] = __uint_as_float(v & 0xffff0000u);
  } else {
    f[0] = bf2f(*p);
  }
}
template <int V>
MLDEV void store_bf(__nv_bfloat16* p, const float (&f)[V]) {
  if constexpr (V == 8) {
    *reinterpret_cast<uint4*>(p) = pack8(f);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(p) = pack4(f);
  } else if constexpr (V == 2) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0], f[1]);
  } else {
    *p = f2bf(f[0]);
  }
}
template <int V>
MLDEV void load_f32(const float* p, float (&f)[V]) {   // p is 4-byte aligned
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = __ldg(p + i);
}
template <int V>
MLDEV void load_w(const void* w, int f32, int at, float (&f)[V]) {
  if (f32) {
    load_f32<V>(static_cast<const float*>(w) + at, f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = bf2f(static_cast<const __nv_bfloat16*>(w)[at + i]);
  }
}

// A lane's unit u of a head: two V-value pieces, at a and b (b < 0: none).  Units below `rot`
// are rotated: half-split pieces u V and u V + R/2; interleaved neighbours, two pieces of R.
template <int V>
MLDEV void unit_at(const QkParams& p, int u, int& a, int& b, bool& rotated) {
  const int rot = p.R / (2 * V);   // half-split: R is a multiple of 2 V
  if (!p.interleaved) {
    rotated = u < rot;
    a = rotated ? u * V : p.R + (u - rot) * 2 * V;
    b = rotated ? a + p.R / 2 : a + V;
  } else {
    rotated = true;   // each piece by itself: rotated while it lies below R
    a = u * 2 * V;
    b = a + V;
  }
  if (a >= p.D) a = -1;
  if (b >= p.D) b = -1;
}

// V values per piece, NU units per lane.
template <int V, int NU>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const QkParams p) {
  const int lane = threadIdx.x & 31;
  const long long warp = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (blockIdx.x == gridDim.x - 1) {   // one more block than the work needs: the positions' check
    if (p.status == nullptr) return;
    __shared__ int bad_s;
    if (threadIdx.x == 0) bad_s = 0;
    __syncthreads();
    bool bad = false;
    for (int t = threadIdx.x; t < p.T; t += blockDim.x) {
      const long long pos = p.pos_i64 ? static_cast<const long long*>(p.positions)[t]
                                      : static_cast<const int32_t*>(p.positions)[t];
      bad |= pos < 0 || pos >= p.num_positions;
    }
    if (bad) bad_s = 1;
    __syncthreads();
    if (threadIdx.x == 0) *p.status = bad_s ? (kDevBadSlot | (kWhereQkPosition << 8)) : 0u;
    return;
  }
  const long long t = warp / p.splits;
  if (t >= p.T) return;   // whole warps
  const int part = static_cast<int>(warp - t * p.splits);
  const int H = p.Hq + p.Hk;
  const int sub = lane & (p.lanes - 1), per = 32 / p.lanes;
  const long long pos = p.pos_i64 ? static_cast<const long long*>(p.positions)[t]
                                  : static_cast<const int32_t*>(p.positions)[t];
  const bool turn = pos >= 0 && pos < p.num_positions;   // a bad position: no rotation, and reported
  const float* row = p.table + (turn ? pos * p.table_t : 0);

  const int h_end = min(H, (part + 1) * p.heads_per_warp);
  for (int h0 = part * p.heads_per_warp; h0 < h_end; h0 += per) {
    const int h = h0 + lane / p.lanes;
    const bool live = h < h_end;
    const bool is_q = h < p.Hq;
    const __nv_bfloat16* x = is_q ? p.q + t * p.q_t + h * p.q_h : p.k + t * p.k_t + (h - p.Hq) * p.k_h;
    float fa[NU][V], fb[NU][V];
    float ss = 0.0f;
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      int a, b;
      bool rotated;
      unit_at<V>(p, sub + n * p.lanes, a, b, rotated);
#pragma unroll
      for (int i = 0; i < V; ++i) fa[n][i] = fb[n][i] = 0.0f;
      if (live && a >= 0) load_bf<V>(x + a, fa[n]);
      if (live && b >= 0) load_bf<V>(x + b, fb[n]);
    }
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int i = 0; i < V; ++i) ss += fa[n][i] * fa[n][i] + fb[n][i] * fb[n][i];
    for (int off = p.lanes >> 1; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float scale = rsqrtf(ss / static_cast<float>(p.D) + p.eps);
    if (!live) continue;
    const void* w = is_q ? p.wq : p.wk;
    __nv_bfloat16* out = is_q ? p.q_out + t * p.qo_t + h * p.qo_h : p.k_out + t * p.ko_t + (h - p.Hq) * p.ko_h;
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      int a, b;
      bool rotated;
      unit_at<V>(p, sub + n * p.lanes, a, b, rotated);
      float wv[V];
      if (a >= 0) {
        load_w<V>(w, p.w_f32, a, wv);
#pragma unroll
        for (int i = 0; i < V; ++i) fa[n][i] *= scale * wv[i];
      }
      if (b >= 0) {
        load_w<V>(w, p.w_f32, b, wv);
#pragma unroll
        for (int i = 0; i < V; ++i) fb[n][i] *= scale * wv[i];
      }
      if (turn) {
        if (!p.interleaved) {
          if (rotated) {
            float c[V], s[V];
            load_f32<V>(row + a, c);
            load_f32<V>(row + p.R / 2 + a, s);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float u = fa[n][i], v = fb[n][i];
              fa[n][i] = u * c[i] - v * s[i];
              fb[n][i] = v * c[i] + u * s[i];
            }
          }
        } else if constexpr (V > 1) {
          auto swing = [&](float (&f)[V], int at) {
            if (at < 0 || at >= p.R) return;   // R is a multiple of V
            float c[V / 2], s[V / 2];
            load_f32<V / 2>(row + at / 2, c);
            load_f32<V / 2>(row + p.R / 2 + at / 2, s);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
              const float u = f[2 * i], v = f[2 * i + 1];
              f[2 * i] = u * c[i] - v * s[i];
              f[2 * i + 1] = v * c[i] + u * s[i];
            }
          };
          swing(fa[n], a);
          swing(fb[n], b);
        } else if (a >= 0 && a < p.R) {   // V == 1: the two pieces are the pair (R is even)
          const float c = row[a / 2], s = row[p.R / 2 + a / 2];
          const float u = fa[n][0], v = fb[n][0];
          fa[n][0] = u * c - v * s;
          fb[n][0] = v * c + u * s;
        }
      }
      if (a >= 0) store_bf<V>(out + a, fa[n]);
      if (b >= 0) store_bf<V>(out + b, fb[n]);
    }
  }
}

}  // namespace
}  // namespace mlk

extern "C" moe_lora_status moe_lora_qk_norm_rope(moe_lora_handle* h, const moe_lora_qk_args* a, void* workspace,
                                                 size_t workspace_bytes, moe_lora_stream stream) {
  using namespace mlk;
  if (h == nullptr || a == nullptr) return MOE_LORA_ERR_INVALID_ARG;
  const int H = a->q_heads + a->k_heads;
  if (a->T < 0 || a->q_heads < 0 || a->k_heads < 0 || H < 1 || H > 65536 || a->head_dim < 1 || a->rotary_dim < 0 ||
      a->rotary_dim > a->head_dim || a->rotary_dim % 2 != 0 || a->num_positions < 0)
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->head_dim > 512) return MOE_LORA_ERR_UNSUPPORTED;
  if (!(a->eps >= 0.0f)) return MOE_LORA_ERR_INVALID_ARG;
  if (a->T == 0) return MOE_LORA_OK;
  if ((a->q_heads > 0 && (a->q == nullptr || a->q_out == nullptr || a->q_weight == nullptr)) ||
      (a->k_heads > 0 && (a->k == nullptr || a->k_out == nullptr || a->k_weight == nullptr)) ||
      a->positions == nullptr || (a->rotary_dim > 0 && a->cos_sin == nullptr))
    return MOE_LORA_ERR_INVALID_ARG;
  if (workspace != nullptr && workspace_bytes < 4) return MOE_LORA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned4(workspace) || !aligned4(a->cos_sin) || !aligned4(a->positions) ||
      (a->positions_i64 && (reinterpret_cast<uintptr_t>(a->positions) & 7u) != 0) || !aligned2(a->q) ||
      !aligned2(a->k) || !aligned2(a->q_out) || !aligned2(a->k_out) || !aligned2(a->q_weight) ||
      !aligned2(a->k_weight) || (a->weight_f32 && (!aligned4(a->q_weight) || !aligned4(a->k_weight))))
    return MOE_LORA_ERR_INVALID_ARG;
  QkParams p;
  p.q = reinterpret_cast<const __nv_bfloat16*>(a->q);
  p.k = reinterpret_cast<const __nv_bfloat16*>(a->k);
  p.q_out = reinterpret_cast<__nv_bfloat16*>(a->q_out);
  p.k_out = reinterpret_cast<__nv_bfloat16*>(a->k_out);
  p.wq = a->q_weight;
  p.wk = a->k_weight;
  p.table = a->cos_sin;
  p.positions = a->positions;
  p.status = static_cast<uint32_t*>(workspace);
  p.q_t = a->q_stride_t;
  p.q_h = a->q_stride_h;
  p.k_t = a->k_stride_t;
  p.k_h = a->k_stride_h;
  p.qo_t = a->q_out_stride_t;
  p.qo_h = a->q_out_stride_h;
  p.ko_t = a->k_out_stride_t;
  p.ko_h = a->k_out_stride_h;
  p.table_t = a->cos_sin_stride;
  p.T = a->T;
  p.Hq = a->q_heads;
  p.Hk = a->k_heads;
  p.D = a->head_dim;
  p.R = a->rotary_dim;
  p.num_positions = a->num_positions;
  p.w_f32 = a->weight_f32 != 0;
  p.pos_i64 = a->positions_i64 != 0;
  p.interleaved = a->interleaved != 0;
  p.eps = a->eps;
  // the widest piece that every address and the rotation's halves allow
  uintptr_t bits = 0;   // element offsets of everything a piece can start at
  if (p.Hq > 0)
    bits |= reinterpret_cast<uintptr_t>(p.q) / 2 | reinterpret_cast<uintptr_t>(p.q_out) / 2 |
            static_cast<uintptr_t>(p.q_t) | static_cast<uintptr_t>(p.qo_t) | static_cast<uintptr_t>(p.q_h) |
            static_cast<uintptr_t>(p.qo_h);
  if (p.Hk > 0)
    bits |= reinterpret_cast<uintptr_t>(p.k) / 2 | reinterpret_cast<uintptr_t>(p.k_out) / 2 |
            static_cast<uintptr_t>(p.k_t) | static_cast<uintptr_t>(p.ko_t) | static_cast<uintptr_t>(p.k_h) |
            static_cast<uintptr_t>(p.ko_h);
  bits |= static_cast<uintptr_t>(p.D) | static_cast<uintptr_t>(p.interleaved ? p.R : p.R / 2);
  const int V = (bits & 7) == 0 ? 8 : (bits & 3) == 0 ? 4 : (bits & 1) == 0 ? 2 : 1;
  const int units = (p.D + 2 * V - 1) / (2 * V);
  p.lanes = 1;
  while (p.lanes < units && p.lanes < 32) p.lanes *= 2;
  // a warp takes a token's heads in turn; short batches spread them over more warps
  const int per = 32 / p.lanes;
  const int rounds = (H + per - 1) / per;   // warp rounds per token
  int splits = static_cast<int>(std::min<long long>(rounds, (16LL * h->num_sms + a->T - 1) / a->T));
  if (splits < 1) splits = 1;
  p.heads_per_warp = (rounds + splits - 1) / splits * per;
  p.splits = (H + p.heads_per_warp - 1) / p.heads_per_warp;
  const long long warps = static_cast<long long>(p.T) * p.splits;
  const int block = warps < 4LL * h->num_sms ? 32 : 256;
  const long long blocks = (warps * 32 + block - 1) / block + 1;   // and the positions' check
  if (blocks > 0x7fffffffLL) return MOE_LORA_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned>(blocks)), threads(block);
  cudaError_t err;
  switch (V) {
    case 8: err = launch_k(qk_norm_rope_kernel<8, 1>, grid, threads, 0, stream, false, p); break;
    case 4: err = launch_k(qk_norm_rope_kernel<4, 2>, grid, threads, 0, stream, false, p); break;
    case 2: err = launch_k(qk_norm_rope_kernel<2, 4>, grid, threads, 0, stream, false, p); break;
    default: err = launch_k(qk_norm_rope_kernel<1, 8>, grid, threads, 0, stream, false, p); break;
  }
  ML_LAUNCH(h, err, "qk_norm_rope launch");
  return MOE_LORA_OK;
}
