// Requests and page pools of the attention calls: argument checks on the host,
// request lookup on the device (not part of the ABI).
#pragma once

#include "internal.h"

namespace moe {

constexpr int kMaxGroup = 64;  // query heads per key head

// Pools and requests as the kernels take them; strides in bytes.
struct KvView {
  uint8_t *k, *v;
  const float *k_scale, *v_scale;
  long long page_stride, head_stride, tok_stride;
  int Hkv, page_shift, npages;
  const int32_t *q_start, *kv_len, *page_table;
  int B, T, table_stride;
};

// MOE_OK and the view when the pools and the requests pass their checks.
inline int kv_view(const moe_kv_pages* p, const moe_kv_batch* b, KvView* out) {
  if (!p || !b || !p->k || !p->v || (p->e4m3 != 0 && p->e4m3 != 1) || p->Hkv < 1 || p->Hkv > 1024 ||
      (p->D != 64 && p->D != 128 && p->D != 256) || p->page < 1 || p->page > 65536 || (p->page & (p->page - 1)) ||
      p->npages < 1 || (p->e4m3 && p->D * p->page < 128))  // the copy engine writes whole 128-byte lines
    return MOE_EINVAL;
  const int size = p->e4m3 ? 1 : 2;
  auto stride_ok = [&](long long s, int n) {
    return n <= 1 || (s >= p->D && s < (1ll << 38) && s * size % 16 == 0);
  };
  if (!stride_ok(p->page_stride, p->npages) || !stride_ok(p->head_stride, p->Hkv) || !stride_ok(p->tok_stride, p->page))
    return MOE_EINVAL;
  if ((reinterpret_cast<uintptr_t>(p->k) & 15) || (reinterpret_cast<uintptr_t>(p->v) & 15)) return MOE_EINVAL;
  if (b->B < 0 || b->T < 0 || b->max_n < 0 || b->table_stride < 0) return MOE_EINVAL;
  if (b->B > 0 && b->T > 0 && (!b->q_start || !b->kv_len || (!b->page_table && b->table_stride > 0))) return MOE_EINVAL;
  out->k = static_cast<uint8_t*>(p->k);
  out->v = static_cast<uint8_t*>(p->v);
  out->k_scale = p->e4m3 ? p->k_scale : nullptr;
  out->v_scale = p->e4m3 ? p->v_scale : nullptr;
  out->page_stride = p->npages > 1 ? p->page_stride * size : 0;
  out->head_stride = p->Hkv > 1 ? p->head_stride * size : 0;
  out->tok_stride = p->page > 1 ? p->tok_stride * size : 0;
  out->Hkv = p->Hkv;
  out->npages = p->npages;
  out->page_shift = 0;
  while ((1 << out->page_shift) < p->page) ++out->page_shift;
  out->q_start = b->q_start;
  out->kv_len = b->kv_len;
  out->page_table = b->page_table;
  out->B = b->B;
  out->T = b->T;
  out->table_stride = b->table_stride;
  return MOE_OK;
}

// Token rows [T][heads][D] of bf16: 16-byte aligned, token stride whole 16-byte pieces.
inline bool rows_ok(const void* p, long long stride, int T, long long width) {
  return p && !(reinterpret_cast<uintptr_t>(p) & 15) && (T <= 1 || (stride >= width && stride % 8 == 0));
}

}  // namespace moe
