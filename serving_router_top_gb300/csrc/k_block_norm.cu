// The norms around a block with its gate and residual add, one pass per token row:
//   z = post ? w_post * y * rsqrt(mean y^2 + eps) : y
//   x' = x + s * g * z,   xn = w_pre * x' * rsqrt(mean x'^2 + eps).
// The row stays in registers between its two sums of squares (both fp32), so x
// and y are read once and x' and xn written once, 12 bytes a column, and memory
// bounds it: 8192 rows of 2048 columns, 201 MB, 32.4 us, 6.2 TB/s (93% of what a
// copy reaches).  One rounding, of xn to bf16.
#include "internal.h"

namespace moe {
namespace bnorm {

constexpr int kMaxH = 16384;

struct Args {
  const float* x;
  float* xo;
  uint16_t* xn;
  const uint16_t *y, *w_post, *gate, *w_pre;
  long long xs, xos, xns, ys, gs;
  int T, H, post, sig;
  float scale, eps;
};

// Over a row's threads: a warp, or the CTA.
template <bool WARP, int N>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (WARP) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float tot = 0.f;
  if (N <= 256) {
#pragma unroll
    for (int w = 0; w < N / 32; ++w) tot += w < int(blockDim.x / 32) ? red[w] : 0.f;
  } else {
#pragma unroll 8
    for (int w = 0; w < int(blockDim.x / 32); ++w) tot += red[w];
  }
  return tot;
}

template <int V>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float f[V]) {
  if (V == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  } else {
    f[0] = bf16_bits_to_f32(*p);
  }
}

// A row has a warp (a CTA's warps take a row each) or a CTA of at most N threads; a thread holds P
// pieces of V columns.  Registers for all of an SM's threads where there is one piece (8192 x 2048 34.1 us
// with 37 registers, 32.4 with 32), and for four CTAs of 512 a column at a time (89, 81).
constexpr int kWarpRows = 4;
template <bool WARP, int N, int P, int V>
__global__ void __launch_bounds__(N, P == 1 ? 2048 / N : V == 1 && N == 512 ? 4 : 1) k_block_norm(const __grid_constant__ Args a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[2][N / 32];
  const int across = WARP ? 32 : blockDim.x;  // threads of a row
  const long long t = WARP ? (long long)blockIdx.x * kWarpRows + threadIdx.y : blockIdx.x;
  if (WARP && t >= a.T) return;
  float x[P][V], z[P][V];
  float ss = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = (threadIdx.x + p * across) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) x[p][i] = z[p][i] = 0.f;
    if (c < a.H) {
      const float* xp = a.x + t * a.xs + c;
      if (V == 8) {
        const float4 u = reinterpret_cast<const float4*>(xp)[0], w = reinterpret_cast<const float4*>(xp)[1];
        x[p][0] = u.x; x[p][1 % V] = u.y; x[p][2 % V] = u.z; x[p][3 % V] = u.w;
        x[p][4 % V] = w.x; x[p][5 % V] = w.y; x[p][6 % V] = w.z; x[p][7 % V] = w.w;
      } else {
        x[p][0] = *xp;
      }
      if (a.y) load_bf16<V>(a.y + t * a.ys + c, z[p]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) ss += z[p][i] * z[p][i];
  }
  if (a.y) {
    float inv = 1.f;
    if (a.post) inv = 1.0f / sqrtf(row_sum<WARP, N>(ss, red[0]) / float(a.H) + a.eps);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (threadIdx.x + p * across) * V;
      if (c < a.H) {
        float w[V], g[V];
        if (a.post && a.w_post) {
          load_bf16<V>(a.w_post + c, w);
#pragma unroll
          for (int i = 0; i < V; ++i) z[p][i] *= w[i];
        }
        if (a.gate) {
          load_bf16<V>(a.gate + t * a.gs + c, g);
#pragma unroll
          for (int i = 0; i < V; ++i) z[p][i] *= a.sig ? sigmoid_f32(g[i]) : g[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) x[p][i] = fmaf(a.scale, z[p][i] * inv, x[p][i]);
      }
    }
  }
  if (a.xo) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (threadIdx.x + p * across) * V;
      if (c < a.H) {
        float* o = a.xo + t * a.xos + c;
        if (V == 8) {
          reinterpret_cast<float4*>(o)[0] = make_float4(x[p][0], x[p][1 % V], x[p][2 % V], x[p][3 % V]);
          reinterpret_cast<float4*>(o)[1] = make_float4(x[p][4 % V], x[p][5 % V], x[p][6 % V], x[p][7 % V]);
        } else {
          *o = x[p][0];
        }
      }
    }
  }
  if (!a.xn) return;
  ss = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < V; ++i) ss += x[p][i] * x[p][i];
  const float inv = 1.0f / sqrtf(row_sum<WARP, N>(ss, red[1]) / float(a.H) + a.eps);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = (threadIdx.x + p * across) * V;
    if (c < a.H) {
      float w[V];
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = 1.f;
      if (a.w_pre) load_bf16<V>(a.w_pre + c, w);
      uint16_t* o = a.xn + t * a.xns + c;
      if (V == 8) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(x[p][(2 * i) % V] * inv * w[(2 * i) % V],
                                                         x[p][(2 * i + 1) % V] * inv * w[(2 * i + 1) % V]);
          u[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(o) = make_uint4(u[0], u[1], u[2], u[3]);
      } else {
        *o = __bfloat16_as_ushort(__float2bfloat16_rn(x[p][0] * inv * w[0]));
      }
    }
  }
}

}  // namespace bnorm
}  // namespace moe

extern "C" int moe_block_norm(const moe_block_norm_desc* d, const float* x, long long x_stride, float* x_out,
                              long long x_out_stride, uint16_t* xn, long long xn_stride, int T, int H,
                              moe_stream_t stream) {
  using namespace moe;
  if (!d || !x || T < 0 || H < 1 || H > bnorm::kMaxH || !(d->eps > 0.f)) return MOE_EINVAL;
  if (!d->y && (d->post_norm || d->gate)) return MOE_EINVAL;
  auto ok = [&](const void* p, long long stride, int size, bool may_be_0) {
    return !p || (!(reinterpret_cast<uintptr_t>(p) % size) && (T <= 1 || stride >= H || (may_be_0 && stride == 0)));
  };
  if (!ok(x, x_stride, 4, false) || !ok(x_out, x_out_stride, 4, false) || !ok(xn, xn_stride, 2, false) ||
      !ok(d->y, d->y_stride, 2, false) || !ok(d->gate, d->gate_stride, 2, true) || !ok(d->w_post, 0, 2, true) ||
      !ok(d->w_pre, 0, 2, true))
    return MOE_EINVAL;
  if (T == 0 || (!x_out && !xn)) return MOE_OK;
  auto wide = [&](const void* p, long long stride) {
    return !p || (!(reinterpret_cast<uintptr_t>(p) & 15) && (T <= 1 || stride % 8 == 0));
  };
  const bool vec = H % 8 == 0 && wide(x, x_stride) && wide(x_out, x_out_stride) && wide(xn, xn_stride) &&
                   wide(d->y, d->y_stride) && wide(d->gate, d->gate_stride) && wide(d->w_post, 0) && wide(d->w_pre, 0);
  bnorm::Args a;
  a.x = x; a.xo = x_out; a.xn = xn;
  a.y = d->y; a.w_post = d->w_post; a.gate = d->gate; a.w_pre = d->w_pre;
  a.xs = x_stride; a.xos = x_out_stride; a.xns = xn_stride; a.ys = d->y_stride; a.gs = d->gate_stride;
  a.T = T; a.H = H; a.post = d->post_norm ? 1 : 0; a.sig = d->gate_sigmoid ? 1 : 0;
  a.scale = d->res_scale; a.eps = d->eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  // One piece a thread as far as a CTA goes, in threads for the row's columns, not a power of two: T rows of
  // H columns with a gate, 8192 x 2048 32.4 us (two pieces 36.5), 4096 x 4096 39.6 (44.4), 2048 x 8192 45.8
  // (49.6), 1024 x 16384 57.5 with two (72.8 with four): 0.93, 0.89, 0.77 and 0.61 of a copy's rate.  A warp a
  // row up to 512 columns: 8192 x 512 12.9 us (CTAs 23.1), 16384 x 256 12.2 (40.4), but 8192 x 1024 28.1 (CTAs
  // 20.2) and 4 x 1024 4.5 (2.3).  Rows that are not aligned go a column at a time: 4096 x 4095 81 us with eight
  // a thread (sixteen 111, four 102), 0.43 of a copy's rate.
  auto threads = [&](int columns) { return dim3((((H - 1) / columns + 1) + 31) / 32 * 32); };
  if (vec) {
    e = H <= 512    ? launch_pdl(bnorm::k_block_norm<true, 32 * bnorm::kWarpRows, 2, 8>, dim3((T - 1) / bnorm::kWarpRows + 1),
                                 dim3(32, bnorm::kWarpRows), 0, s, a)
        : H <= 2048 ? launch_pdl(bnorm::k_block_norm<false, 256, 1, 8>, dim3(T), threads(8), 0, s, a)
        : H <= 4096 ? launch_pdl(bnorm::k_block_norm<false, 512, 1, 8>, dim3(T), threads(8), 0, s, a)
        : H <= 8192 ? launch_pdl(bnorm::k_block_norm<false, 1024, 1, 8>, dim3(T), threads(8), 0, s, a)
                    : launch_pdl(bnorm::k_block_norm<false, 1024, 2, 8>, dim3(T), threads(16), 0, s, a);
  } else {
    e = H <= 4096 ? launch_pdl(bnorm::k_block_norm<false, 512, 8, 1>, dim3(T), threads(8), 0, s, a)
                  : launch_pdl(bnorm::k_block_norm<false, 1024, 16, 1>, dim3(T), threads(16), 0, s, a);
  }
  return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}
