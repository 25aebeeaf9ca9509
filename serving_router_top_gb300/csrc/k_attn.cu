// Attention of the newest tokens of each request over a paged cache.
//
// For a token at position p, query head h and its key head:
//   s_j = scale * q . k_j,  j <= p (and j > p - window);  o = sum exp(s_j) v_j / sum exp(s_j)
// in one pass over the keys with the running maximum and sum of the softmax.
// One CTA per (token, query head): its warps take the keys in turn and their
// parts are joined at the end.
#include "paged.cuh"

struct moe_attn_ws {
  int Hq, Hkv, D;
  int32_t* error;
};

namespace moe {
namespace attn {

constexpr int kWarps = 8;

struct Args {
  KvView kv;
  const uint16_t* q;
  uint16_t* o;
  long long qs, os;
  int Hq, G, window;
  float scale;
  int32_t* err;
};

// Lane's D/32 neighbouring elements of a cache row.
template <bool E4M3, int N>
__device__ __forceinline__ void load_row(const uint8_t* p, int lane, float f[N]) {
  if (E4M3) {
    const uint8_t* e = p + lane * N;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = f16x2_to_f32x2(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(e + i)));
      f[i] = v.x;
      f[i + 1] = v.y;
    }
  } else {
    const uint16_t* e = reinterpret_cast<const uint16_t*>(p) + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = bf16_bits_to_f32(e[i]);
  }
}

template <bool E4M3, int D>
__global__ void __launch_bounds__(32 * kWarps) k_attn(const __grid_constant__ Args a) {
  constexpr int N = D / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int t = blockIdx.x, head = blockIdx.y, h = head / a.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = request_of(a.kv, t);
  if (b < 0) return;
  const long long pos = position_of(a.kv, b, t), cap = (long long)a.kv.table_stride << a.kv.page_shift;
  if (threadIdx.x == 0 && a.kv.kv_len[b] > cap) set_error(a.err, MOE_ERANGE);
  const long long end = pos + 1 < cap ? pos + 1 : cap;
  const long long first = a.window > 0 && pos + 1 > a.window ? pos + 1 - a.window : 0;
  float q[N], o[N];
  const float qk = a.scale * (a.kv.k_scale ? a.kv.k_scale[h] : 1.f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = qk * bf16_bits_to_f32(a.q[(long long)t * a.qs + head * D + lane * N + i]);
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (long long j = first + warp; j < end; j += kWarps) {
    const int id = a.kv.page_table[(long long)b * a.kv.table_stride + (j >> a.kv.page_shift)];
    float k[N], v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) k[i] = v[i] = 0.f;
    if (id >= 0 && id < a.kv.npages) {
      const long long at = id * a.kv.page_stride + h * a.kv.head_stride +
                           (j & ((1 << a.kv.page_shift) - 1)) * a.kv.tok_stride;
      load_row<E4M3, N>(a.kv.k + at, lane, k);
      load_row<E4M3, N>(a.kv.v + at, lane, v);
    } else if (lane == 0) {
      set_error(a.err, MOE_ERANGE);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s);
    const float c = mn == -INFINITY ? 1.f : __expf(m - mn), w = mn == -INFINITY ? 0.f : __expf(s - mn);
    m = mn;
    l = l * c + w;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * c + w * v[i];
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) s_o[warp][lane * N + i] = o[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float mx = -INFINITY, lt = 0.f, ot = 0.f;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w]);
    for (int w = 0; w < kWarps; ++w) {
      const float c = s_m[w] == -INFINITY ? 0.f : __expf(s_m[w] - mx);
      lt += c * s_l[w];
      ot += c * s_o[w][threadIdx.x];
    }
    const float vs = a.kv.v_scale ? a.kv.v_scale[h] : 1.f;
    const float r = end > first ? ot / lt * vs : 0.f;
    a.o[(long long)t * a.os + head * D + threadIdx.x] = __bfloat16_as_ushort(__float2bfloat16_rn(r));
  }
}

template <bool E4M3>
cudaError_t launch(int D, dim3 grid, cudaStream_t s, const Args& a) {
  const dim3 block(32 * kWarps);
  switch (D) {
    case 64: k_attn<E4M3, 64><<<grid, block, 0, s>>>(a); break;
    case 128: k_attn<E4M3, 128><<<grid, block, 0, s>>>(a); break;
    default: k_attn<E4M3, 256><<<grid, block, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace moe

extern "C" int moe_attn_ws_create(moe_attn_ws** out, int Hq, int Hkv, int D) {
  using namespace moe;
  if (!out || Hkv < 1 || Hkv > 1024 || Hq < 1 || Hq % Hkv || Hq / Hkv > kMaxGroup || (D != 64 && D != 128 && D != 256))
    return MOE_EINVAL;
  *out = nullptr;
  moe_attn_ws* w = static_cast<moe_attn_ws*>(calloc(1, sizeof(moe_attn_ws)));
  if (!w) return MOE_ENOMEM;
  w->Hq = Hq;
  w->Hkv = Hkv;
  w->D = D;
  if (cudaMalloc(&w->error, 256) != cudaSuccess) {
    cudaGetLastError();
    free(w);
    return MOE_ENOMEM;
  }
  if (cudaMemset(w->error, 0, 256) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    moe_attn_ws_destroy(w);
    return MOE_ECUDA;
  }
  *out = w;
  return MOE_OK;
}

extern "C" int moe_attn_ws_destroy(moe_attn_ws* w) {
  if (!w) return MOE_OK;
  cudaFree(w->error);
  free(w);
  return MOE_OK;
}

extern "C" int moe_attn_ws_get_view(const moe_attn_ws* w, moe_attn_ws_view* v) {
  if (!w || !v) return MOE_EINVAL;
  v->error = w->error;
  return MOE_OK;
}

extern "C" int moe_attn_sync_status(moe_attn_ws* w, moe_stream_t stream) {
  if (!w) return MOE_EINVAL;
  MOE_CUDA_TRY(cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)));
  int32_t e = 0;
  MOE_CUDA_TRY(cudaMemcpy(&e, w->error, 4, cudaMemcpyDeviceToHost));
  MOE_CUDA_TRY(cudaMemset(w->error, 0, 4));
  return e;
}

extern "C" int moe_paged_attention(const moe_kv_pages* kv, const moe_kv_batch* b, const uint16_t* q, long long q_stride,
                                   int Hq, uint16_t* o, long long o_stride, float scale, int window, moe_attn_ws* ws,
                                   moe_stream_t stream) {
  using namespace moe;
  attn::Args a = {};
  const int rc = kv_view(kv, b, &a.kv);
  if (rc) return rc;
  if (!ws || Hq != ws->Hq || kv->Hkv != ws->Hkv || kv->D != ws->D || window < 0 || !isfinite(scale)) return MOE_EINVAL;
  const int T = b->T;
  if (T == 0 || b->B == 0) return MOE_OK;
  const long long width = (long long)Hq * kv->D;
  if (!rows_ok(q, q_stride, T, width) || !rows_ok(o, o_stride, T, width)) return MOE_EINVAL;
  a.q = q;
  a.o = o;
  a.qs = q_stride;
  a.os = o_stride;
  a.Hq = Hq;
  a.G = Hq / kv->Hkv;
  a.window = window;
  a.scale = scale;
  a.err = ws->error;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(T, Hq);
  if ((kv->e4m3 ? attn::launch<true>(kv->D, grid, s, a) : attn::launch<false>(kv->D, grid, s, a)) != cudaSuccess)
    return MOE_ECUDA;
  return MOE_OK;
}
