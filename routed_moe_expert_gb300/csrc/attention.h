// Shared by the kernels of moe_lora_attention (attention*.cu).
#pragma once

#include "common.cuh"

namespace mlk {

struct AttentionParams {
  const __nv_bfloat16 *q, *k, *v;
  const int32_t *tables, *kv_lens, *offsets;   // offsets null: row b is request b's
  __nv_bfloat16* out;
  float* lse;
  long long q_t, q_h, o_t, o_h, k_p, k_h, k_t, v_p, v_h, v_t, table_stride;
  int T, B, Hq, Hk, G, D;
  int num_pages, page, width;
  int shared_len;
  float scale_log2;                            // scale * log2(e): weights are powers of two
  uint32_t* status;
};

// A request's rows [q0, q0 + n) and its keys, checked: rows within [0, T), at most width * page keys.
struct Request {
  int q0, n, kv;
  bool bad;
};
MLDEV Request request_of(const AttentionParams& p, int b) {
  Request r;
  r.bad = false;
  if (p.offsets == nullptr) {
    r.q0 = b;
    r.n = 1;
  } else {
    const int lo = p.offsets[b], hi = p.offsets[b + 1];
    r.bad = lo < 0 || hi < lo || hi > p.T;
    r.q0 = r.bad ? 0 : lo;
    r.n = r.bad ? 0 : hi - lo;
  }
  const int kv = p.kv_lens[b];
  const long long room = static_cast<long long>(p.width) * p.page;
  r.bad = r.bad || kv < 0 || kv > room;
  r.kv = static_cast<int>(min(static_cast<long long>(max(kv, 0)), room));
  return r;
}

}  // namespace mlk
