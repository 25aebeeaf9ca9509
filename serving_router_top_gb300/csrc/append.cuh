// What the two append kernels share: arguments, their checks, and the stores (not part of the ABI).
#pragma once

#include <float.h>
#include <limits.h>
#include <math.h>

#include "paged.cuh"

struct moe_rope {
  int rot, interleaved;
  uint64_t* turns;  // device [rot/2]
};

namespace moe {
namespace append {

constexpr int kMaxThreads = 256;
constexpr int kMaxPairs = 128;  // rot <= 256

struct Args {
  KvView kv;
  const uint64_t* turns;
  int rot, interleaved;
  const uint16_t *q, *k, *v;
  uint16_t* qo;
  long long qs, qos, ks, vs;
  int Hq;
  int32_t* err;
};

__device__ __forceinline__ void unpack8(uint4 u, float f[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float f[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two values -> two E4M3 bytes (low byte first), to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight columns of one head to where they belong: head < Hq is a query, then keys, then values.
template <bool E4M3>
__device__ __forceinline__ void store8(const Args& a, int t, int head, int col, const float f[8], int D, long long at,
                                       float scale) {
  if (head < a.Hq) {
    *reinterpret_cast<uint4*>(a.qo + (long long)t * a.qos + head * D + col) = pack8(f);
    return;
  }
  if (at < 0) return;
  const bool is_v = head >= a.Hq + a.kv.Hkv;
  const int h = head - a.Hq - (is_v ? a.kv.Hkv : 0);
  uint8_t* dst = (is_v ? a.kv.v : a.kv.k) + at + h * a.kv.head_stride;
  if (!E4M3) {
    *reinterpret_cast<uint4*>(dst + 2 * col) = pack8(f);
  } else {
    // A division for each column, as the code is that of x / scale: times the scale's reciprocal, ties and the
    // smallest scales go elsewhere.  4096 tokens of 32 + 2 x 4 heads of 128 take 17.9 us, with the reciprocal 16.6.
    uint2 u;
    u.x = e4m3x2(f[0] / scale, f[1] / scale) | (e4m3x2(f[2] / scale, f[3] / scale) << 16);
    u.y = e4m3x2(f[4] / scale, f[5] / scale) | (e4m3x2(f[6] / scale, f[7] / scale) << 16);
    *reinterpret_cast<uint2*>(dst + col) = u;
  }
}

// The checks of both calls; `out` is filled and `work` tells whether there is anything to launch.
inline int checked(const moe_kv_pages* kv, const moe_kv_batch* b, const moe_rope* rope, const uint16_t* q, long long q_stride,
            uint16_t* q_out, long long q_out_stride, int Hq, const uint16_t* k, long long k_stride, const uint16_t* v,
            long long v_stride, int32_t* err_dev, Args* out, bool* work) {
  Args& a = *out;
  *work = false;
  const int rc = kv_view(kv, b, &a.kv);
  if (rc) return rc;
  const int T = b->T, D = kv->D;
  if (Hq < 0 || Hq > 1024 * kMaxGroup || (Hq > 0) != (q != nullptr) || (rope && rope->rot > D)) return MOE_EINVAL;
  if (T == 0 || b->B == 0) return MOE_OK;
  if (q && (!rows_ok(q, q_stride, T, (long long)Hq * D) || !rows_ok(q_out, q_out_stride, T, (long long)Hq * D)))
    return MOE_EINVAL;
  if (!rows_ok(k, k_stride, T, (long long)kv->Hkv * D) || !rows_ok(v, v_stride, T, (long long)kv->Hkv * D))
    return MOE_EINVAL;
  a.turns = rope ? rope->turns : nullptr;
  a.rot = rope ? rope->rot : 0;
  a.interleaved = rope ? rope->interleaved : 0;
  a.q = q;
  a.k = k;
  a.v = v;
  a.qo = q_out;
  a.qs = q_stride;
  a.qos = q_out_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.Hq = Hq;
  a.err = err_dev;
  *work = true;
  return MOE_OK;
}

}  // namespace append
}  // namespace moe
