// New keys and values into a paged cache behind norms of each head's queries and keys, at the positions of tree nodes.
//
// Mathematics.  Of a head's D columns x: y = w x / sqrt(mean(x^2) + eps), then the rotation of k_kv_append.cu by the
// node's position base + depth, where its place in the cache is base + index.  All in fp32: the sum of squares, rsqrtf
// (2 units) and the products are far below the one rounding to the stored type that follows.
//
// Layout, as in k_kv_append.cu: a CTA per token, a thread two items of 16 columns of a head, loaded before the chain
// that finds request, page and angles.  The lanes with a head's columns are neighbours (4, 8 or 16), so the sum of
// squares takes two to four exchanges between lanes.  The weights come to shared memory on the side.
#include "append.cuh"

namespace moe {
namespace append {

struct NormArgs {
  Args a;
  const int32_t* depth;  // of the rows in their trees, or null: they follow one another
  int norm;
  const uint16_t *wq, *wk;
  float eps;
};

// 8192 tokens of 32 + 2 x 4 heads of 128 columns, 168 MB: 32.8 us, 5.1 TB/s, with two items a thread and 64 registers (four
// CTAs of 256 threads).  Without the look at sums past fp32 32.3; then with one fp32 at a time 33.3, of which with registers
// for five CTAs 34.3, for six 38.9, without a limit 34.2; with one item a thread 39.6 at its best, three 33.2, four 34.1.  It
// issues on two cycles of three; a third of its instructions find request, page and angles.  4096 into E4M3 21.5 us, of
// which the divisions (append.cuh) are 1.4: the chain and the arithmetic are bf16's, over fewer bytes.
constexpr int kMine = 2, kPerSm = 4;

template <bool E4M3, int D>
__global__ void __launch_bounds__(kMaxThreads, kPerSm) k_kv_append_norm(const __grid_constant__ NormArgs na) {
  const Args& a = na.a;
  constexpr int kItems = D / 16;
  // cos of pairs 8 j + 4 z .. at [0][z][j], sin at [1][z][j]: a lane takes four of each at a time
  __shared__ float4 turn[2][2][kMaxPairs / 8];
  __shared__ uint4 weights[D / 4];         // eight columns each: the queries', then the keys'
  __shared__ int owner, position, begins;
  pdl_trigger();
  pdl_wait();
  const int t = blockIdx.x, step = blockDim.x, pairs = a.rot / 2;
  const int n = (a.Hq + 2 * a.kv.Hkv) * kItems;
  struct Item {
    int head, c0, c1, pair;  // its pairs are 8 pair .. 8 pair + 7; < 0: the columns are not turned
    uint4 v0, v1;            // 8 columns from c0 and from c1 on
    float scale;             // of a key's or value's head, E4M3
  };
  auto fetch = [&](int it, Item& x) {
    x.head = -1;
    if (it >= n) return;
    const int head = it / kItems, j = it - head * kItems;
    const bool turns = head < a.Hq + a.kv.Hkv && 16 * j < a.rot, halves = turns && !a.interleaved;
    x.head = head;
    x.pair = turns ? j : -1;
    x.c0 = halves ? 8 * j : 16 * j;
    x.c1 = halves ? pairs + 8 * j : 16 * j + 8;
    const uint16_t* src = head < a.Hq ? a.q + (long long)t * a.qs + head * D
                          : head < a.Hq + a.kv.Hkv ? a.k + (long long)t * a.ks + (head - a.Hq) * D
                                                   : a.v + (long long)t * a.vs + (head - a.Hq - a.kv.Hkv) * D;
    x.v0 = *reinterpret_cast<const uint4*>(src + x.c0);
    x.v1 = *reinterpret_cast<const uint4*>(src + x.c1);
    if (E4M3) {
      const bool is_v = head >= a.Hq + a.kv.Hkv;
      const float* sc = is_v ? a.kv.v_scale : a.kv.k_scale;
      x.scale = head >= a.Hq && sc ? sc[head - a.Hq - (is_v ? a.kv.Hkv : 0)] : 1.0f;
    }
  };
  Item x[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) fetch(threadIdx.x + i * step, x[i]);
  if (na.norm)
    for (int i = threadIdx.x; i < D / 4; i += step) {  // eight columns a copy
      if (const uint16_t* src = i < D / 8 ? na.wq : na.wk)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(weights + i))),
                     "l"(src + i % (D / 8) * 8)
                     : "memory");
      else
        weights[i] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    }
  const int deep = na.depth ? na.depth[t] : 0;

  // the request whose rows t is one of
  bool found = false;
  for (int b = threadIdx.x; b < a.kv.B; b += step) {
    const int s0 = a.kv.q_start[b], s1 = a.kv.q_start[b + 1], len = a.kv.kv_len[b];
    if (s0 <= t && t < s1) {
      owner = b;
      begins = s0;
      position = int(min(max((long long)len - (s1 - t), (long long)INT_MIN), (long long)INT_MAX));
      found = true;
    }
  }
  found = __syncthreads_or(found);
  if (!found) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  const int b = owner, pos = position;
  long long at = -1;  // byte offset of (page, place) in the pools
  int id = -1;
  if (pos >= 0 && (pos >> a.kv.page_shift) < a.kv.table_stride)
    id = a.kv.page_table[(long long)b * a.kv.table_stride + (pos >> a.kv.page_shift)];
  // a node's place is not its position
  const int turned = na.depth ? int(min(max((long long)pos - (t - begins) + deep, (long long)INT_MIN), (long long)INT_MAX)) : pos;
  for (int i = threadIdx.x; i < pairs; i += step) {
    // a signed fraction of a turn in [-1/2, 1/2); sincospif takes half turns
    const long long frac = (long long)(uint64_t(int64_t(turned)) * a.turns[i]);
    float c, s;
    sincospif(float(frac) * 0x1p-63f, &s, &c);
    reinterpret_cast<float*>(&turn[0][i >> 2 & 1][i >> 3])[i & 3] = c;
    reinterpret_cast<float*>(&turn[1][i >> 2 & 1][i >> 3])[i & 3] = s;
  }
  if (id >= 0 && id < a.kv.npages)
    at = id * a.kv.page_stride + (long long)(pos & ((1 << a.kv.page_shift) - 1)) * a.kv.tok_stride;
  else if (threadIdx.x == 0)
    set_error(a.err, MOE_ERANGE);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  auto put = [&](const Item& x) {
    if (x.head < 0) return;
    float f0[8], f1[8];
    unpack8(x.v0, f0);
    unpack8(x.v1, f1);
    if (na.norm && x.head < a.Hq + a.kv.Hkv) {
      auto squares = [&]() {  // of the head's columns, the same in all its lanes
        float2 both = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 u = make_float2(f0[i], f0[i + 1]), v = make_float2(f1[i], f1[i + 1]);
          both = __ffma2_rn(u, u, __ffma2_rn(v, v, both));
        }
        float sum = both.x + both.y;
        const unsigned mates = ((1u << kItems) - 1) << ((threadIdx.x & 31) / kItems * kItems);
#pragma unroll
        for (int o = 1; o < kItems; o <<= 1) sum += __shfl_xor_sync(mates, sum, o);
        return sum;
      };
      float sum = squares(), eps = na.eps;
      if (sum > FLT_MAX) {  // columns from 2^60 on: 2^-96 of them has the same norm, with eps taken along
#pragma unroll
        for (int i = 0; i < 8; ++i) f0[i] *= 0x1p-96f, f1[i] *= 0x1p-96f;
        sum = squares();
        eps = eps * 0x1p-96f * 0x1p-96f;
      }
      const float inv = rsqrtf(sum * (1.f / D) + eps);
      const int z = x.head >= a.Hq ? D / 8 : 0;
      const float2 inv2 = make_float2(inv, inv);
      float w[8];
      unpack8(weights[z + x.c0 / 8], w);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 r = __fmul2_rn(make_float2(f0[i], f0[i + 1]), __fmul2_rn(make_float2(w[i], w[i + 1]), inv2));
        f0[i] = r.x, f0[i + 1] = r.y;
      }
      unpack8(weights[z + x.c1 / 8], w);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 r = __fmul2_rn(make_float2(f1[i], f1[i + 1]), __fmul2_rn(make_float2(w[i], w[i + 1]), inv2));
        f1[i] = r.x, f1[i + 1] = r.y;
      }
    }
    if (x.pair >= 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 c4 = turn[0][h][x.pair], s4 = turn[1][h][x.pair];
        if (!a.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            float *u = f0 + 4 * h + i, *w = f1 + 4 * h + i;
            const float2 c = i ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y), s = i ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y);
            const float2 uu = make_float2(u[0], u[1]), ww = make_float2(w[0], w[1]), ws = __fmul2_rn(ww, s);
            const float2 r = __ffma2_rn(uu, c, make_float2(-ws.x, -ws.y)), q = __ffma2_rn(uu, s, __fmul2_rn(ww, c));
            u[0] = r.x, u[1] = r.y, w[0] = q.x, w[1] = q.y;
          }
        } else {
          float* f = h ? f1 : f0;
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = f[2 * i], w = f[2 * i + 1];
            f[2 * i] = fmaf(u, c[i], -(w * s[i]));
            f[2 * i + 1] = fmaf(u, s[i], w * c[i]);
          }
        }
      }
    }
    store8<E4M3>(a, t, x.head, x.c0, f0, D, at, x.scale);
    store8<E4M3>(a, t, x.head, x.c1, f1, D, at, x.scale);
  };
#pragma unroll
  for (int i = 0; i < kMine; ++i) put(x[i]);
  for (int it = threadIdx.x + kMine * step; it < n; it += step) {
    fetch(it, x[0]);
    put(x[0]);
  }
}

template <bool E4M3>
cudaError_t launch_norm(int D, int T, cudaStream_t s, const NormArgs& a) {
  const int n = (a.a.Hq + 2 * a.a.kv.Hkv) * (D / 16), each = (n + kMine - 1) / kMine;
  const dim3 block(each >= kMaxThreads ? kMaxThreads : (each + 31) / 32 * 32);
  switch (D) {
    case 64: return launch_pdl(k_kv_append_norm<E4M3, 64>, dim3(T), block, 0, s, a);
    case 128: return launch_pdl(k_kv_append_norm<E4M3, 128>, dim3(T), block, 0, s, a);
    default: return launch_pdl(k_kv_append_norm<E4M3, 256>, dim3(T), block, 0, s, a);
  }
}

}  // namespace append
}  // namespace moe

extern "C" int moe_kv_append_norm(const moe_kv_pages* kv, const moe_kv_batch* b, const moe_tree* tree, const moe_rope* rope,
                                  const moe_head_norm* norm, const uint16_t* q, long long q_stride, uint16_t* q_out,
                                  long long q_out_stride, int Hq, const uint16_t* k, long long k_stride, const uint16_t* v,
                                  long long v_stride, int32_t* err_dev, moe_stream_t stream) {
  using namespace moe;
  append::NormArgs a = {};
  if (norm && (!(norm->eps > 0.f) || !isfinite(norm->eps) || (reinterpret_cast<uintptr_t>(norm->w_q) & 15) ||
               (reinterpret_cast<uintptr_t>(norm->w_k) & 15)))
    return MOE_EINVAL;
  bool work;
  const int rc = append::checked(kv, b, rope, q, q_stride, q_out, q_out_stride, Hq, k, k_stride, v, v_stride, err_dev, &a.a, &work);
  if (rc || !work) return rc;
  if (tree && !tree->depth) return MOE_EINVAL;
  a.depth = tree ? tree->depth : nullptr;
  a.norm = norm != nullptr;
  if (norm) {
    a.wq = norm->w_q;
    a.wk = norm->w_k;
    a.eps = norm->eps;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int T = b->T, D = kv->D;
  const cudaError_t e = kv->e4m3 ? append::launch_norm<true>(D, T, s, a) : append::launch_norm<false>(D, T, s, a);
  return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}
