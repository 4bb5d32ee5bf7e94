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
// It is bound by memory: each value is read once and written once.  T 8192, 32 + 4 heads of 128:
// 28.4 us for 155 MB, 5.5 TB/s (80% of a plain copy's rate).  T 333, 24 + 8 heads of 192: 4.5 us for
// 8.3 MB, one token 2.4 us: latency.
//
// L lanes hold a head, so a warp holds 32 / L heads at a time; a lane's pieces are chosen so that both
// members of every rotated pair sit in the same lane (pieces i and i + R/2 of a half-split rotation),
// so the only exchange between lanes is the sum of squares.
//
// Where everything starts on 16-byte boundaries (qk_norm_rope_kernel) a lane's 16 values of every
// head of a token have the same weights and angles: out_i = scale (x_i C_i + x_partner S_i), with
// C = w c and S = -+ w_partner s made once per token and kind of head and kept in registers, and
// the next heads' values are loaded before the current ones are used.  Everything else (odd
// strides, offsets and sizes) goes through qk_norm_rope_any_kernel, which works its indices out
// value by value: T 8192, 32 + 4 heads of 80 with R 40 (8-byte pieces) 62 us, with R 80
// (16-byte pieces, the other kernel) 25; heads of 100 (4-byte pieces) 203, of 90 (2-byte) 359; 14 to 18 for
// their bytes.  What bounds it was not measured.
#include "common.cuh"
#include "host.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace mlk {

struct QkParams {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *q_out, *k_out;
  const void *wq, *wk;
  const float* table;
  const void* positions;
  uint32_t* status;
  long long q_t, q_h, k_t, k_h, qo_t, qo_h, ko_t, ko_h, table_t;   // strides in elements
  int T, Hq, Hk, D, R, num_positions, w_f32, pos_i64, interleaved, table_vec, w_vec;
  int lanes;        // L: lanes per head, a power of two
  int heads_per_warp, splits;   // (any alignment) heads one warp goes through, warps per token
  // (aligned) rounds in all, of a warp, of a token; heads packed across tokens, and then the steps
  unsigned rounds, run;
  int token_rounds, packed, step_t, step_h;
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

// eight weights; at is a multiple of 8
MLDEV void load_w8(const QkParams& p, const void* w, int at, float (&f)[8]) {
  if (!p.w_vec) {
    load_w<8>(w, p.w_f32, at, f);
  } else if (p.w_f32) {
    const float4* v = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 x = __ldg(v), y = __ldg(v + 1);
    f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
    f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
  } else {
    unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + at)), f);
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

// The last block, one more than the work needs: the positions' check, the only write of the status.
MLDEV void check_positions(const QkParams& p) {
  if (p.status == nullptr) return;
  __shared__ int bad_s;
  if (threadIdx.x == 0) bad_s = 0;
  __syncthreads();
  bool bad = false;
#pragma unroll 4
  for (int t = threadIdx.x; t < p.T; t += blockDim.x) {
    const long long pos = p.pos_i64 ? static_cast<const long long*>(p.positions)[t]
                                    : static_cast<const int32_t*>(p.positions)[t];
    bad |= pos < 0 || pos >= p.num_positions;
  }
  if (bad) bad_s = 1;
  __syncthreads();
  if (threadIdx.x == 0) *p.status = bad_s ? (kDevBadSlot | (kWhereQkPosition << 8)) : 0u;
}

constexpr int kAhead = 2;             // rounds whose copies are in flight (T 8192: 28.4 us; 3: 28.8, 4: 29.3)
constexpr int kRing = kAhead + 1;

MLDEV void copy16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
MLDEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MLDEV void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Two float32 operations in one instruction.
struct F2 {
  unsigned long long v;
};
MLDEV F2 pair_of(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
MLDEV float2 floats_of(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
  return r;
}
MLDEV F2 mul2(F2 x, F2 y) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(x.v), "l"(y.v));
  return r;
}
MLDEV F2 fma2(F2 x, F2 y, F2 z) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(x.v), "l"(y.v), "l"(z.v));
  return r;
}
MLDEV F2 swapped(F2 x) {
  const float2 f = floats_of(x);
  return pair_of(f.y, f.x);
}
MLDEV void unpack_pairs(const uint4& x, F2 (&f)[4]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
MLDEV uint4 pack_pairs(const F2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = floats_of(f[i]);
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

MLDEV long long position_of(const QkParams& p, int t) {
  return p.pos_i64 ? static_cast<const long long*>(p.positions)[t] : static_cast<const int32_t*>(p.positions)[t];
}

// The aligned case: a lane's 16 values of a head are two 16-byte pieces.  A round is one head per
// lane group: 32 / L heads of a token (the rest of a token's last round idle), or, with few heads
// (`packed`), any 32 / L consecutive (token, head) pairs.  Each warp takes a run of rounds.
// LANES > 0: that many lanes per head, each with both pieces (D = 16 LANES); 0: as p says.
template <bool INTERLEAVED, int LANES>
__global__ void __launch_bounds__(256, 3) qk_norm_rope_kernel(const QkParams p) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == gridDim.x - 1) {
    check_positions(p);
    return;
  }
  __shared__ uint4 ring[kRing][2][256];
  const int lane = threadIdx.x & 31;
  const unsigned warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int H = p.Hq + p.Hk;
  const int L = LANES > 0 ? LANES : p.lanes, per = 32 / L, group = lane / L, sub = lane & (L - 1);
  const unsigned g0 = min(warp * p.run, p.rounds), g1 = min(g0 + p.run, p.rounds);
  const int n = static_cast<int>(g1 - g0);   // rounds of this warp

  // this lane's pieces (has_a, has_b: they lie in the head), next to its neighbours' so that whole
  // 32-byte sectors are read and written (pieces 2 sub and 2 sub + 1: 5.15 us at T 333, 32 heads of 192)
  int a, b;
  bool turned, has_a, has_b;
  if constexpr (INTERLEAVED) {
    const int half = (p.D + 15) >> 4;
    a = sub * 8;
    b = a + half * 8;
    turned = true;   // decided piece by piece
    has_a = LANES > 0 || sub < half;
  } else {
    const int rot = p.R >> 4, half = (p.D - p.R + 15) >> 4;
    turned = sub < rot;
    a = turned ? sub * 8 : p.R + (sub - rot) * 8;
    b = a + (turned ? p.R >> 1 : half * 8);
    has_a = LANES > 0 || sub < rot + half;
  }
  has_b = LANES > 0 || (has_a && b < p.D);

  // a lane group's place: (token, head) and where the head's values are read and written
  struct At {
    int t, h;
    const __nv_bfloat16* in;
    __nv_bfloat16* out;
  };
  auto settle = [&](At& x) {
    if (x.h < p.Hq) {
      x.in = p.q + x.t * p.q_t + x.h * p.q_h;
      x.out = p.q_out + x.t * p.qo_t + x.h * p.qo_h;
    } else {
      x.in = p.k + x.t * p.k_t + (x.h - p.Hq) * p.k_h;
      x.out = p.k_out + x.t * p.ko_t + (x.h - p.Hq) * p.ko_h;
    }
  };
  const long long in_step = per * p.q_h, out_step = per * p.qo_h;
  auto next = [&](At& x) {
    if (p.packed) {
      x.t += p.step_t;
      x.h += p.step_h;
      if (x.h >= H) {
        x.h -= H;
        ++x.t;
      }
      settle(x);
    } else {
      x.h += per;
      if (x.h < p.Hq) {
        x.in += in_step;
        x.out += out_step;
      } else {
        if (x.h - group >= H) {
          x.h = group;
          ++x.t;
        }
        settle(x);
      }
    }
  };
  auto live = [&](const At& x) -> bool { return x.h < H && x.t < p.T; };
  At now;
  if (p.packed) {
    const unsigned task = g0 * per + group;
    now.t = static_cast<int>(task / H);
    now.h = static_cast<int>(task % H);
  } else {
    now.t = static_cast<int>(g0 / p.token_rounds);
    now.h = static_cast<int>(g0 % p.token_rounds) * per + group;
  }
  settle(now);
  At ahead = now;
  int fetched = 0;
  auto fetch = [&]() {   // the copies of the next round not yet on its way
    if (fetched < n && live(ahead)) {
      if (has_a) copy16(&ring[fetched % kRing][0][threadIdx.x], ahead.in + a);
      if (has_b) copy16(&ring[fetched % kRing][1][threadIdx.x], ahead.in + b);
    }
    copy_commit();
    ++fetched;
    next(ahead);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch();

  F2 ca[4], sa[4], cb[4], sb[4];   // coefficients of the own values and of the partners
  int kind = -1, token = -1;       // the heads they are for: 0 query, 1 key; of which token
  const float inv_d = 1.0f / static_cast<float>(p.D);

  for (int i = 0; i < n; ++i, next(now)) {
    fetch();
    const bool on = live(now);
    const int is_k = now.h >= p.Hq;
    if (on && (token != now.t || kind != is_k)) {
      const void* w = is_k ? p.wk : p.wq;
      kind = is_k;
      token = now.t;
      const long long pos = position_of(p, token);
      // angles of the lane's values: half-split, one per pair of pieces; interleaved, four pairs of
      // piece a, then four of piece b.  A bad position: no rotation (and reported)
      float c[8], s[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c[j] = 1.0f;
        s[j] = 0.0f;
      }
      const bool known = pos >= 0 && pos < p.num_positions;
      const bool turn_a = known && (INTERLEAVED ? a < p.R : turned), turn_b = known && (INTERLEAVED ? b < p.R : turned);
      if (known) {
        const float* row = p.table + pos * p.table_t;
        auto angles = [&](int at, float* cp, float* sp, auto count) {
          constexpr int kN = decltype(count)::value;
          if (p.table_vec) {
#pragma unroll
            for (int j = 0; j < kN; j += 4) {
              const float4 cv = __ldg(reinterpret_cast<const float4*>(row + at + j));
              const float4 sv = __ldg(reinterpret_cast<const float4*>(row + p.R / 2 + at + j));
              cp[j] = cv.x, cp[j + 1] = cv.y, cp[j + 2] = cv.z, cp[j + 3] = cv.w;
              sp[j] = sv.x, sp[j + 1] = sv.y, sp[j + 2] = sv.z, sp[j + 3] = sv.w;
            }
          } else {
#pragma unroll
            for (int j = 0; j < kN; ++j) {
              cp[j] = __ldg(row + at + j);
              sp[j] = __ldg(row + p.R / 2 + at + j);
            }
          }
        };
        if constexpr (INTERLEAVED) {
          if (turn_a) angles(a / 2, c, s, std::integral_constant<int, 4>());
          if (turn_b) angles(b / 2, c + 4, s + 4, std::integral_constant<int, 4>());
        } else if (turn_a) {
          angles(a, c, s, std::integral_constant<int, 8>());
        }
      }
      float wa[8] = {}, wb[8] = {};
      if (has_a) load_w8(p, w, a, wa);
      if (has_b) load_w8(p, w, b, wb);
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // values 2j and 2j + 1 of each piece
        const int u = 2 * j, v = u + 1;
        if constexpr (INTERLEAVED) {
          ca[j] = pair_of(wa[u] * c[j], wa[v] * c[j]);
          cb[j] = pair_of(wb[u] * c[4 + j], wb[v] * c[4 + j]);
          sa[j] = pair_of(-wa[v] * s[j], wa[u] * s[j]);
          sb[j] = pair_of(-wb[v] * s[4 + j], wb[u] * s[4 + j]);
        } else {
          ca[j] = pair_of(wa[u] * c[u], wa[v] * c[v]);
          cb[j] = pair_of(wb[u] * c[u], wb[v] * c[v]);
          sa[j] = pair_of(-wb[u] * s[u], -wb[v] * s[v]);
          sb[j] = pair_of(wa[u] * s[u], wa[v] * s[v]);
        }
        if (!turn_a) sa[j] = F2{0ull};   // (a partner's weight may be infinite)
        if (!turn_b) sb[j] = F2{0ull};
      }
    }
    copy_wait<kAhead>();
    F2 fa[4] = {}, fb[4] = {};
    if (on && has_a) unpack_pairs(ring[i % kRing][0][threadIdx.x], fa);
    if (on && has_b) unpack_pairs(ring[i % kRing][1][threadIdx.x], fb);
    F2 sq = {0ull};
#pragma unroll
    for (int j = 0; j < 4; ++j) sq = fma2(fb[j], fb[j], fma2(fa[j], fa[j], sq));
    const float2 both = floats_of(sq);
    float ss = both.x + both.y;
#pragma unroll
    for (int off = (LANES > 0 ? LANES : 32) / 2; off > 0; off >>= 1)
      if (LANES > 0 || off < L) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float scale = rsqrtf(ss * inv_d + p.eps);
    auto put = [&](bool turn_a, bool turn_b) {   // the round's values; a piece that is not turned takes nothing
      const F2 scale2 = pair_of(scale, scale);   // from its partner
      F2 oa[4], ob[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 pa = !turn_a ? F2{0ull} : INTERLEAVED ? swapped(fa[j]) : fb[j];
        const F2 pb = !turn_b ? F2{0ull} : INTERLEAVED ? swapped(fb[j]) : fa[j];
        oa[j] = mul2(scale2, fma2(pa, sa[j], mul2(fa[j], ca[j])));
        ob[j] = mul2(scale2, fma2(pb, sb[j], mul2(fb[j], cb[j])));
      }
      if (has_a) *reinterpret_cast<uint4*>(now.out + a) = pack_pairs(oa);
      if (has_b) *reinterpret_cast<uint4*>(now.out + b) = pack_pairs(ob);
    };
    // Finite partners of a piece that is not turned have coefficients of 0; in a head with an infinite
    // value (0 times it is NaN) they are left out.
    if (on && scale != 0.0f) {
      put(true, true);
    } else if (on) {
      const long long pos = position_of(p, now.t);
      const bool known = pos >= 0 && pos < p.num_positions;
      put(known && (INTERLEAVED ? a < p.R : turned), known && (INTERLEAVED ? b < p.R : turned));
    }
  }
}

// Any alignment: V values per piece, NU units per lane.
template <int V, int NU>
__global__ void __launch_bounds__(256) qk_norm_rope_any_kernel(const QkParams p) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == gridDim.x - 1) {
    check_positions(p);
    return;
  }
  const int lane = threadIdx.x & 31;
  const long long warp = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
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
  const long long heads = static_cast<long long>(a->q_heads) + a->k_heads;
  if (a->T < 0 || a->q_heads < 0 || a->k_heads < 0 || heads < 1 || heads > 65536 || a->head_dim < 1 || a->rotary_dim < 0 ||
      a->rotary_dim > a->head_dim || a->rotary_dim % 2 != 0 || a->num_positions < 0)
    return MOE_LORA_ERR_INVALID_ARG;
  if (a->head_dim > 512 || a->T > kMaxExtent) return MOE_LORA_ERR_UNSUPPORTED;
  const int H = static_cast<int>(heads);
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
  p.table_vec = p.table_t % 4 == 0 && p.R % 8 == 0 && aligned16(p.table);
  p.w_vec = (p.Hq == 0 || aligned16(p.wq)) && (p.Hk == 0 || aligned16(p.wk));
  const int per = 32 / p.lanes;
  p.token_rounds = (H + per - 1) / per;
  long long warps;
  if (V == 8) {
    // heads that would leave half of a token's rounds idle are packed, whatever their token
    p.packed = 2 * H <= p.token_rounds * per;
    p.step_t = per / H;
    p.step_h = per % H;
    const long long tasks = static_cast<long long>(a->T) * H;
    const long long rounds = p.packed ? (tasks + per - 1) / per : static_cast<long long>(a->T) * p.token_rounds;
    if (rounds * per > 0x7fffffffLL) return MOE_LORA_ERR_INVALID_ARG;
    // as many warps as the GPU holds (three blocks of eight an SM), each a run of rounds
    const long long most = 24LL * h->num_sms;
    p.rounds = static_cast<unsigned>(rounds);
    p.run = static_cast<unsigned>((rounds + most - 1) / most);
    warps = (rounds + p.run - 1) / p.run;
  } else {
    // a warp takes a token's heads in turn, short batches spread them over more warps
    int splits = static_cast<int>(std::min<long long>(p.token_rounds, (16LL * h->num_sms + a->T - 1) / a->T));
    if (splits < 1) splits = 1;
    p.heads_per_warp = (p.token_rounds + splits - 1) / splits * per;
    p.splits = (H + p.heads_per_warp - 1) / p.heads_per_warp;
    warps = static_cast<long long>(p.T) * p.splits;
  }
  const int block = warps < 4LL * h->num_sms ? 32 : 256;
  const long long blocks = (warps * 32 + block - 1) / block + 1;   // and the positions' check
  if (blocks > 0x7fffffffLL) return MOE_LORA_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned>(blocks)), threads(block);
  ML_ON_DEVICE(h);
  cudaError_t err;
  switch (V) {
    case 8:
#define ML_QK(LANES)                                                                        \
  (p.interleaved ? launch_k(qk_norm_rope_kernel<true, LANES>, grid, threads, 0, stream, true, p) \
                 : launch_k(qk_norm_rope_kernel<false, LANES>, grid, threads, 0, stream, true, p))
      if (p.D == 64) err = ML_QK(4);
      else if (p.D == 128) err = ML_QK(8);
      else if (p.D == 256) err = ML_QK(16);
      else err = ML_QK(0);
#undef ML_QK
      break;
    case 4: err = launch_k(qk_norm_rope_any_kernel<4, 2>, grid, threads, 0, stream, true, p); break;
    case 2: err = launch_k(qk_norm_rope_any_kernel<2, 4>, grid, threads, 0, stream, true, p); break;
    default: err = launch_k(qk_norm_rope_any_kernel<1, 8>, grid, threads, 0, stream, true, p); break;
  }
  ML_LAUNCH(h, err, "qk_norm_rope launch");
  return MOE_LORA_OK;
}
