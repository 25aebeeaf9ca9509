// New keys and values into a paged cache, with the position rotation on the way.
//
// The expert-path pages give no kernel for this step; the mathematics is the
// rotation of column pairs (u, w) by a = p * f_i for a token at position p:
//   u' = u cos a - w sin a,   w' = w cos a + u sin a.
// p * f_i in fp32 is off by p * 2^-24 (0.06 rad at a million tokens), and fp64
// runs at a small fraction of the fp32 rate here.  So f_i is kept as a 64-bit
// fixed-point fraction of a turn: p times it, modulo 2^64, is the angle's
// fraction of a turn with an error of at most p * 2^-65, and only its top bits
// become a float, for sincospif.
#include "append.cuh"

namespace moe {
namespace append {

// One CTA per token; a thread takes kMine items of 16 columns of a head at a time (the two halves'
// vectors of eight pairs, or two neighbours).  The first items' loads are on their way while the
// CTA finds its request, position, page and angles, a chain of dependent loads.  8192 tokens of
// 32 + 2 x 4 heads of 128 columns, 168 MB: 38.9 us with the loads after the chain, 28.1 us now, 6.0 TB/s.
// Four tokens to a CTA, the next one's loads beside the last one's stores, take 101 registers and 47 us;
// one or three items a thread 32.0 and 28.4 us.
constexpr int kMine = 2;

template <bool E4M3, int D>
__global__ void __launch_bounds__(kMaxThreads) k_kv_append(const __grid_constant__ Args a) {
  constexpr int kItems = D / 16;
  // cos, sin of each pair's angle: pair 8 j + i at [i][j], as the lanes of a head read them (64 bytes
  // apart, those met in four banks, and the prompt chunk took 32.2 us)
  __shared__ float2 cs[8][kMaxPairs / 8];
  __shared__ int owner, position;
  pdl_trigger();
  pdl_wait();
  const int t = blockIdx.x, step = blockDim.x, pairs = a.rot / 2;
  const int n = (a.Hq + 2 * a.kv.Hkv) * kItems;
  struct Item {
    int head, c0, c1, pair;  // its pairs are 8 pair .. 8 pair + 7; < 0: the columns stay as they are
    uint4 v0, v1;
    float scale;  // of a key's or value's head, E4M3
  };
  auto fetch = [&](int it, Item& x) {
    x.head = -1;
    if (it >= n) return;
    const int head = it / kItems, j = it - head * kItems;
    const bool turn = head < a.Hq + a.kv.Hkv && 16 * j < a.rot, halves = turn && !a.interleaved;
    x.head = head;
    x.pair = turn ? j : -1;
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

  // the request whose rows t is one of
  bool found = false;
  for (int b = threadIdx.x; b < a.kv.B; b += step) {
    const int s0 = a.kv.q_start[b], s1 = a.kv.q_start[b + 1], len = a.kv.kv_len[b];
    if (s0 <= t && t < s1) {
      owner = b;
      position = int(min(max((long long)len - (s1 - t), (long long)INT_MIN), (long long)INT_MAX));
      found = true;
    }
  }
  if (!__syncthreads_or(found)) return;
  const int b = owner, pos = position;
  long long at = -1;  // byte offset of (page, place) in the pools
  int id = -1;
  if (pos >= 0 && (pos >> a.kv.page_shift) < a.kv.table_stride)
    id = a.kv.page_table[(long long)b * a.kv.table_stride + (pos >> a.kv.page_shift)];
  for (int i = threadIdx.x; i < pairs; i += step) {
    // a signed fraction of a turn in [-1/2, 1/2); sincospif takes half turns
    const long long frac = (long long)(uint64_t(int64_t(pos)) * a.turns[i]);
    float c, s;
    sincospif(float(frac) * 0x1p-63f, &s, &c);
    cs[i & 7][i >> 3] = make_float2(c, s);
  }
  if (id >= 0 && id < a.kv.npages)
    at = id * a.kv.page_stride + (long long)(pos & ((1 << a.kv.page_shift) - 1)) * a.kv.tok_stride;
  else if (threadIdx.x == 0)
    set_error(a.err, MOE_ERANGE);
  __syncthreads();

  auto put = [&](const Item& x) {
    if (x.head < 0) return;
    float f0[8], f1[8];
    unpack8(x.v0, f0);
    unpack8(x.v1, f1);
    if (x.pair >= 0) {
      if (!a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 r = cs[i][x.pair];
          const float u = f0[i], w = f1[i];
          f0[i] = u * r.x - w * r.y;
          f1[i] = w * r.x + u * r.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 r = cs[i][x.pair], r2 = cs[4 + i][x.pair];
          float u = f0[2 * i], w = f0[2 * i + 1];
          f0[2 * i] = u * r.x - w * r.y;
          f0[2 * i + 1] = w * r.x + u * r.y;
          u = f1[2 * i], w = f1[2 * i + 1];
          f1[2 * i] = u * r2.x - w * r2.y;
          f1[2 * i + 1] = w * r2.x + u * r2.y;
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
cudaError_t launch(int D, int T, cudaStream_t s, const Args& a) {
  const int n = (a.Hq + 2 * a.kv.Hkv) * (D / 16), each = (n + kMine - 1) / kMine;
  const dim3 block(each >= kMaxThreads ? kMaxThreads : (each + 31) / 32 * 32);
  switch (D) {
    case 64: return launch_pdl(k_kv_append<E4M3, 64>, dim3(T), block, 0, s, a);
    case 128: return launch_pdl(k_kv_append<E4M3, 128>, dim3(T), block, 0, s, a);
    default: return launch_pdl(k_kv_append<E4M3, 256>, dim3(T), block, 0, s, a);
  }
}

// f / 2 pi, whole turns off, as a 64-bit fraction to nearest.  In integers: divided in a double it is off by 2^-53 of
// itself, 2^-25 of a turn at position 2^31 for f = 1.  192 bits of 1 / 2 pi are enough for any |f| below 2^64.
uint64_t turns_of(double f) {
  constexpr uint64_t kInv[3] = {0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull, 0x28be60db9391054aull};  // 2^192 / (2 pi), low word first
  int ex = 0;
  const uint64_t m = uint64_t(ldexp(frexp(fabs(f), &ex), 53));  // |f| = m 2^(ex - 53)
  uint64_t w[5] = {};  // m 2^192 / (2 pi)
  unsigned __int128 carry = 0;
  for (int i = 0; i < 3; ++i) {
    carry += (unsigned __int128)m * kInv[i];
    w[i] = uint64_t(carry);
    carry >>= 64;
  }
  w[3] = uint64_t(carry);
  const int low = 128 - (ex - 53);  // its bits from `low` on are the fraction
  auto bits = [&](int at) {         // 64 bits from bit `at` on
    const int i = at / 64, s = at % 64;
    return i > 3 ? 0 : s ? w[i] >> s | w[i + 1] << (64 - s) : w[i];
  };
  if (m == 0 || low < 1) return 0;
  const uint64_t frac = bits(low) + (bits(low - 1) & 1);
  return f < 0 ? 0 - frac : frac;
}

}  // namespace append
}  // namespace moe

extern "C" int moe_rope_create(moe_rope** out, int rot, int interleaved, double theta, const double* inv_freq_host) {
  using namespace moe;
  if (!out || rot < 16 || rot > 2 * append::kMaxPairs || rot % 16) return MOE_EINVAL;
  *out = nullptr;
  if (!inv_freq_host && !(theta > 0.0 && isfinite(theta))) return MOE_EINVAL;
  uint64_t turns[append::kMaxPairs];
  for (int i = 0; i < rot / 2; ++i) {
    const double f = inv_freq_host ? inv_freq_host[i] : pow(theta, -2.0 * i / rot);
    if (!isfinite(f)) return MOE_EINVAL;
    turns[i] = append::turns_of(f);
  }
  moe_rope* r = static_cast<moe_rope*>(calloc(1, sizeof(moe_rope)));
  if (!r) return MOE_ENOMEM;
  r->rot = rot;
  r->interleaved = interleaved ? 1 : 0;
  if (cudaMalloc(&r->turns, sizeof(turns)) != cudaSuccess) {
    cudaGetLastError();
    free(r);
    return MOE_ENOMEM;
  }
  if (cudaMemcpy(r->turns, turns, size_t(rot / 2) * 8, cudaMemcpyHostToDevice) != cudaSuccess) {
    cudaGetLastError();
    moe_rope_destroy(r);
    return MOE_ECUDA;
  }
  *out = r;
  return MOE_OK;
}

extern "C" int moe_rope_destroy(moe_rope* r) {
  if (!r) return MOE_OK;
  cudaFree(r->turns);
  free(r);
  return MOE_OK;
}

extern "C" int moe_kv_append(const moe_kv_pages* kv, const moe_kv_batch* b, const moe_rope* rope, const uint16_t* q,
                             long long q_stride, uint16_t* q_out, long long q_out_stride, int Hq, const uint16_t* k,
                             long long k_stride, const uint16_t* v, long long v_stride, int32_t* err_dev,
                             moe_stream_t stream) {
  using namespace moe;
  append::Args a = {};
  bool work;
  const int rc = append::checked(kv, b, rope, q, q_stride, q_out, q_out_stride, Hq, k, k_stride, v, v_stride, err_dev, &a, &work);
  if (rc || !work) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if ((kv->e4m3 ? append::launch<true>(kv->D, b->T, s, a) : append::launch<false>(kv->D, b->T, s, a)) != cudaSuccess)
    return MOE_ECUDA;
  return MOE_OK;
}
