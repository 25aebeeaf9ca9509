// Verification of drafted trees against the target's probabilities (speculative sampling without loss).
//
// Mathematics.  At node v, R = p and s = 1.  A child drawn from q is kept with chance min(1, R(x) / (s q(x))); refused,
// what is left to draw from is max(R / s - q, 0) made a distribution again, kept here as R = max(R - s q, 0) and its
// sum s.  A child that was picked is drawn from a q that is 1 at x: R then only loses R(x), and s as much.  The last
// R is drawn from by its running sum.
//
// Fixed point.  Whether u s q < R, and the first index whose running sum passes u sum R, must not hang on the order
// of a sum: the tokens of two runs, or of a batch and a single request, would part there.  Every value is therefore
// taken as a whole number of 2^-60 (an fp32 above 2^-37 is one exactly), and sums of those are exact in any order.
// fp64 would round them and runs at a sixty-fourth of the rate here.
//
// Movement.  A cluster of CTAs takes a request.  Its first CTA gathers, for every node at once, the two values that
// decide about it, and walks the tree with no further load until a sum over the vocabulary is wanted; then every CTA
// sums its part of the rows, and each writes its sum to all others.  Refused picks need no sum before the last one.
// The draw finds the CTA, the warp and the 128 values that hold the threshold, and reads those alone again.
// Only the first CTA decides what comes next, so no CTA of a cluster waits at another barrier than the rest, whatever
// becomes of the inputs meanwhile.
//
// What bounds it: a chain of trips to memory (requests; parents and tokens; the nodes' values; the rows) and of the
// cluster's barriers, launch beside them.  A chain of 6 drawn nodes over 131072 tokens 8.2 us on sixteen CTAs; 64 picked trees
// of up to 16 nodes over 100001 tokens 16.3 us, 1.6 TB/s of the last nodes' rows, and 64 drawn chains over 131072 29.4 us, 2.3
// TB/s.  Eight CTAs of 256 threads, which read the drawn group again, took 16.8 us for the first and 30.3 for the second.
#include "paged.cuh"

namespace moe {
namespace verify {

using u64 = unsigned long long;

constexpr int kNodes = 256, kThreads = 512, kWarps = kThreads / 32, kMaxCtas = 16, kGroups = 4;
constexpr u64 kOne = 1ull << 60, kMost = 1ull << 62;

struct Args {
  const int32_t* q_start;
  const float *target, *draft;
  long long ts, ds;
  const int32_t *token, *parent;
  const float *u, *u_last;
  int V, T;
  int32_t *path, *count, *next;
  int path_stride;
  int32_t* err;
};

// A probability in units of 2^-60: below 0 and NaN 0, above 1 that.
__device__ __forceinline__ u64 fixed(float x) {
  const uint32_t b = __float_as_uint(fminf(fmaxf(x, 0.f), 1.f)), e = b >> 23;
  return (u64((b & 0x7fffffu) | 0x800000u) << 37) >> min(127u - e, 63u);
}
// A random number in units of 2^-64.
__device__ __forceinline__ u64 chance(float u) {
  const uint32_t b = __float_as_uint(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f)), e = b >> 23;
  return e == 0 ? 0 : (u64((b & 0x7fffffu) | 0x800000u) << 40) >> min(126u - e, 63u);
}
__device__ __forceinline__ u64 times(u64 a, u64 b) {  // of two numbers of 2^-60
  return (__umul64hi(a, b) << 4) | ((a * b) >> 60);
}
__device__ __forceinline__ u64 less(u64 a, u64 b) { return a > b ? a - b : 0; }
__device__ __forceinline__ u64 plus(u64 a, u64 b) { return min(a + b, kMost); }  // of two that are at most kMost

__device__ __forceinline__ uint32_t su32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint32_t my_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t ranks() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {  // the same place in another CTA
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(su32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void put(uint32_t at, u64 x) { asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory"); }
__device__ __forceinline__ void put(uint32_t at, int x) { asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory"); }
__device__ __forceinline__ void meet() {  // all threads of the cluster; what was written before is seen after
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// What the first CTA asks of all: a sum over the row of `node`'s R after `refused` drawn children, or without the
// `gone` picked ones; the last one is drawn from.  node < 0: there is nothing to do.
struct Order {
  int row, refused, gone, last;
};
struct Shared {
  u64 p[kNodes], q[kNodes], u[kNodes];  // of a node: the target's and the draft's value of its token at its parent
  u64 sigma[kNodes + 1];                // s after so many refusals
  u64 part[kMaxCtas], warp[kWarps];     // sums of the cluster's CTAs and of this CTA's warps
  int token[kNodes], gone[kNodes];
  short parent[kNodes];
  Order order;
};

struct Rows {
  const float *p, *q;  // from the 16-byte boundary at or before the target's row; the draft's, if it is read
  int lead, end;       // the row's first and last place, from there
  bool together;       // the draft's row lies the same way
};
// Four places from x on; places outside the row read as zero.
__device__ __forceinline__ void load4(const float* row, const Rows& r, int x, bool whole, float4* out) {
  if (whole && x >= r.lead && x + 4 <= r.end) {
    *out = __ldg(reinterpret_cast<const float4*>(row + x));
    return;
  }
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = x + i >= r.lead && x + i < r.end ? __ldg(row + x + i) : 0.f;
  *out = make_float4(f[0], f[1], f[2], f[3]);
}
// R of a value after `refused` drawn children.
__device__ __forceinline__ u64 rest(float p, float q, int refused, const u64* sigma) {
  u64 r = fixed(p);
  if (refused > 0) {
    const u64 f = fixed(q);
    r = less(r, f);
    for (int k = 1; k < refused; ++k) r = less(r, times(sigma[k], f));
  }
  return r;
}

template <bool DRAWN, int PER_SM>
__global__ void __launch_bounds__(kThreads, PER_SM) k_verify(const __grid_constant__ Args a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = int(my_rank()), C = int(ranks()), b = blockIdx.x / C;
  // no CTA writes to another before all have begun: they meet once the first has its view of the tree
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_trigger();
  pdl_wait();
  const float u_last = a.u_last[b];
  // ------------------------------------------------------------ the first CTA's view of the tree
  int s0 = 0, n = 0;
  if (rank == 0) {
    const RowSpan rows = row_span(a.q_start, b, a.T);
    s0 = rows.s0;
    n = rows.n;
    if (tid == 0 && (n < 0 || n > kNodes)) set_error(a.err, MOE_ERANGE);
    n = min(max(n, 0), kNodes);
    for (int i = tid; i < kNodes; i += kThreads) {
      int up = -1, x = -1;
      u64 p = 0, q = 0, u = 0;
      if (i > 0 && i < n) {
        up = a.parent[s0 + i];
        x = a.token[s0 + i];
        u = chance(a.u[s0 + i]);
        if (up < 0 || up >= i) up = -1;
        if (x < 0 || x >= a.V) x = -1;
        if (up >= 0 && x >= 0) {
          p = fixed(a.target[(s0 + up) * a.ts + x]);
          if (DRAWN) q = fixed(a.draft[(s0 + up) * a.ds + x]);
        }
      }
      sh.parent[i] = short(up);
      sh.token[i] = x;
      sh.p[i] = p;
      sh.q[i] = q;
      sh.u[i] = u;
    }
    for (int d = tid; d < a.path_stride; d += kThreads) a.path[(long long)b * a.path_stride + d] = -1;
    if (tid == 0) a.next[b] = -1;
    __syncthreads();
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // the walk's state, in the first CTA's first warp
  int node = 0, seen = 0, kept = 0, refused = 0, gone = 0;
  u64 sigma = kOne;
  auto arrive_at = [&](int v) {
    node = v;
    seen = v;
    refused = gone = 0;
    sigma = kOne;
    if (lane == 0) a.path[(long long)b * a.path_stride + kept] = v;
    ++kept;
  };
  auto next_child = [&]() {  // of node, after `seen`; -1: none
    if (kept >= a.path_stride) return -1;
    for (int w = (seen + 1) / 32; w < (n + 31) / 32; ++w) {
      const int i = 32 * w + lane;
      const unsigned m = __ballot_sync(0xffffffffu, i > seen && i < n && sh.parent[i] == node);
      if (m) return 32 * w + __ffs(m) - 1;
    }
    return -1;
  };
  if (rank == 0 && warp == 0 && n > 0) arrive_at(0);

  // A warp's lines of 128 places are in four groups, a line of each read at once.  With one line to a group the values
  // stay in registers: further sums over the same row, and the draw, read nothing.
  float4 x[kGroups], y[kGroups];
  int held = -1;         // the row that they are of
  bool held_q = false;   // and of the draft's
  bool own_row = false;  // nothing was left of R: the target's own row is drawn from
  for (;;) {
    if (!own_row) {
      if (rank == 0 && warp == 0) {
        Order o = {-1, 0, 0, 1};
        if (n > 0) {
          if (refused > 0) sigma = sh.sigma[refused];
          for (;;) {
            const int c = next_child();
            if (c < 0) break;
            seen = c;
            u64 r = sh.p[c];
            bool keep;
            if constexpr (DRAWN) {
              const u64 f = sh.q[c];
              if (refused > 0) r = less(r, f);
              for (int k = 1; k < refused; ++k) r = less(r, times(sh.sigma[k], f));
              keep = __umul64hi(sh.u[c], times(sigma, f)) < r;
            } else {
              const int x = sh.token[c];
              bool before = x < 0;
              for (int k = lane; k < gone; k += 32) before |= sh.gone[k] == x;
              if (__any_sync(0xffffffffu, before)) r = 0;
              keep = __umul64hi(sh.u[c], sigma) < r;
              if (!keep && r > 0) {
                sigma = less(sigma, r);
                if (lane == 0) sh.gone[gone] = x;
                __syncwarp();
                ++gone;
              }
            }
            if (keep) {
              arrive_at(c);
            } else if (DRAWN) {
              ++refused;
              break;
            }
          }
          o = {s0 + node, refused, gone, DRAWN ? next_child() < 0 : 1};
          if (lane == 0) a.count[b] = kept;
        } else if (lane == 0) {
          a.count[b] = 0;
        }
        __syncwarp();
        for (int c = lane; c < C; c += 32) {
          const uint32_t to = at_rank(&sh.order, c);
          put(to, o.row);
          put(to + 4, o.refused);
          put(to + 8, o.gone);
          put(to + 12, o.last);
        }
        for (int k = lane; k < o.gone * (C - 1); k += 32) put(at_rank(&sh.gone[k / (C - 1)], 1 + k % (C - 1)), sh.gone[k / (C - 1)]);
      }
      meet();
    }
    Order o = sh.order;
    if (!DRAWN) o.refused = 0;
    else o.gone = 0;
    if (o.row < 0) return;
    if (own_row) o.refused = o.gone = 0;

    // ---------------------------------------------------------- sums
    Rows rows;
    const float* p = a.target + o.row * a.ts;
    rows.lead = int(reinterpret_cast<uintptr_t>(p) >> 2 & 3);
    rows.end = rows.lead + a.V;
    rows.p = p - rows.lead;
    rows.q = nullptr;
    rows.together = true;
    if (o.refused > 0) {
      const float* q = a.draft + o.row * a.ds;
      rows.q = q - rows.lead;
      rows.together = (reinterpret_cast<uintptr_t>(rows.q) & 15) == 0;
    }
    const int lines = (rows.end + 127) / 128, each = (lines + C * kWarps - 1) / (C * kWarps);  // of 128 places; of a warp
    const int line0 = min((rank * kWarps + warp) * each, lines), line1 = min(line0 + each, lines);
    const int deep = (each + kGroups - 1) / kGroups;  // lines of a group
    // Picked tokens that are gone are zeros before anything is added up: taken off a sum that was cut they would leave
    // another one, by what else the sum was of.  A few of a request's warps have any.
    bool lost = false;
    if constexpr (!DRAWN)
      for (int k = 0; k < o.gone; k += 32) {
        const int line = k + lane < o.gone ? (sh.gone[k + lane] + rows.lead) / 128 : -1;
        lost |= __any_sync(0xffffffffu, line >= line0 && line < line1);
      }
    auto drop = [&](int line, float4& v) {
      for (int k = 0; k < o.gone; k += 32) {
        const int t = k + lane < o.gone ? sh.gone[k + lane] + rows.lead : -1;
        for (unsigned here = __ballot_sync(0xffffffffu, t >= 0 && t / 128 == line); here; here &= here - 1) {
          const int at = __shfl_sync(0xffffffffu, t, __ffs(here) - 1) - 128 * line - 4 * lane;
          if (at == 0) v.x = 0.f;
          if (at == 1) v.y = 0.f;
          if (at == 2) v.z = 0.f;
          if (at == 3) v.w = 0.f;
        }
      }
    };
    u64 sum[kGroups] = {};
    for (int l = 0; l < deep; ++l) {
      const bool p_here = deep == 1 && held == o.row, q_here = p_here && held_q;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int line = line0 + g * deep + l;
        if (!p_here) x[g] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!q_here) y[g] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (line < line1) {
          if (!p_here) load4(rows.p, rows, 128 * line + 4 * lane, true, &x[g]);
          if (!q_here && o.refused > 0) load4(rows.q, rows, 128 * line + 4 * lane, rows.together, &y[g]);
        }
      }
      if (!DRAWN && lost)
#pragma unroll
        for (int g = 0; g < kGroups; ++g) drop(line0 + g * deep + l, x[g]);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        // four of at most 2^60 beside at most 2^62: no carry is lost
        sum[g] += rest(x[g].x, y[g].x, o.refused, sh.sigma) + rest(x[g].y, y[g].y, o.refused, sh.sigma) +
                  rest(x[g].z, y[g].z, o.refused, sh.sigma) + rest(x[g].w, y[g].w, o.refused, sh.sigma);
        sum[g] = min(sum[g], kMost);
      }
    }
    held = lost ? -1 : o.row;
    held_q = o.refused > 0;
    auto over_lanes = [](u64 v) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) v = plus(v, __shfl_xor_sync(0xffffffffu, v, d));
      return v;
    };
    const u64 mine = over_lanes(plus(plus(sum[0], sum[1]), plus(sum[2], sum[3])));
    if (lane == 0) sh.warp[warp] = mine;
    __syncthreads();
    if (tid < C) {
      u64 all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) all = plus(all, sh.warp[w]);
      put(at_rank(&sh.part[rank], tid), all);
    }
    meet();
    u64 total = 0, before = 0;
    for (int c = 0; c < C; ++c) {
      if (c == rank) before = total;
      total = plus(total, sh.part[c]);
    }
    if (!o.last) {
      if (tid == 0) sh.sigma[o.refused] = total;
      __syncthreads();
      continue;
    }
    if (total == 0) {
      if (own_row || o.refused + o.gone == 0) return;  // the target's row is empty: no token
      own_row = true;
      meet();  // the sums have been read
      continue;
    }
    // ---------------------------------------------------------- the draw
    u64 t = __umul64hi(chance(u_last), total);
    if (t < before) return;
    t -= before;
    for (int w = 0; w < warp; ++w) {
      if (t < sh.warp[w]) return;
      t -= sh.warp[w];
    }
    if (t >= sh.warp[warp]) return;
    int l0 = line0, end = line1;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const u64 here = over_lanes(sum[g]);
      l0 = line0 + g * deep;
      end = min(l0 + deep, line1);
      if (deep == 1) x[0] = x[g], y[0] = y[g];
      if (t < here) break;
      t -= here;
    }
    for (int l = l0; l < end; ++l) {
      const int at = (l - l0) % kGroups;
      if (deep > 1 && at == 0) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          if (l + g >= end) break;
          load4(rows.p, rows, 128 * (l + g) + 4 * lane, true, &x[g]);
          if (o.refused > 0) load4(rows.q, rows, 128 * (l + g) + 4 * lane, rows.together, &y[g]);
        }
      } else if (at > 0) {  // the next one read
#pragma unroll
        for (int g = 1; g < kGroups; ++g) x[g - 1] = x[g], y[g - 1] = y[g];
      }
      const int x0 = 128 * l + 4 * lane;
      u64 r[4] = {rest(x[0].x, y[0].x, o.refused, sh.sigma), rest(x[0].y, y[0].y, o.refused, sh.sigma),
                  rest(x[0].z, y[0].z, o.refused, sh.sigma), rest(x[0].w, y[0].w, o.refused, sh.sigma)};
      for (int k = 0; k < o.gone; ++k) {
        const int g = sh.gone[k] + rows.lead - x0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (g == i) r[i] = 0;
      }
      const u64 four = min(r[0] + r[1] + r[2] + r[3], kMost);
      u64 upto = four;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 o2 = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto = plus(upto, o2);
      }
      const u64 line = __shfl_sync(0xffffffffu, upto, 31);
      if (t >= line) {
        t -= line;
        continue;
      }
      const unsigned past = __ballot_sync(0xffffffffu, t < upto);
      const u64 earlier = __shfl_up_sync(0xffffffffu, upto, 1);  // at most t where upto is above it, so it was not cut
      if (lane == __ffs(past) - 1) {
        u64 left = lane > 0 ? t - earlier : t;
        int i = 0;
        while (i < 3 && left >= r[i]) left -= r[i++];
        a.next[b] = x0 + i - rows.lead;
      }
      return;
    }
    return;
  }
}

}  // namespace verify
}  // namespace moe

extern "C" int moe_verify_drafts(const moe_kv_batch* b, const moe_verify_desc* d, int32_t* path, int path_stride,
                                 int32_t* count, int32_t* token, int32_t* err_dev, moe_stream_t stream) {
  using namespace moe;
  if (!b || !d || b->B < 0 || b->T < 0 || d->V < 1 || d->V > 1 << 24 || path_stride < 1) return MOE_EINVAL;
  if (b->B == 0) return MOE_OK;
  if (!b->q_start || !path || !count || !token || !d->u_last) return MOE_EINVAL;
  if (b->T > 0 && (!d->target || !d->token || !d->parent || !d->u)) return MOE_EINVAL;
  if (b->T > 1 && (d->target_stride < d->V || (d->draft && d->draft_stride < d->V))) return MOE_EINVAL;
  if ((reinterpret_cast<uintptr_t>(d->target) | reinterpret_cast<uintptr_t>(d->draft)) & 3) return MOE_EINVAL;
  // a request's outputs are written while others still read their tokens and random numbers
  const long long B = b->B, T = b->T;
  const struct {
    const void* p;
    long long n;
  } out[3] = {{path, B * path_stride}, {count, B}, {token, B}},
    in[5] = {{b->q_start, B + 1}, {d->token, T}, {d->parent, T}, {d->u, T}, {d->u_last, B}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& x : in)
      if (!apart(out[i].p, out[i].n, x.p, x.n)) return MOE_EINVAL;
    for (int j = 0; j < i; ++j)
      if (!apart(out[i].p, out[i].n, out[j].p, out[j].n)) return MOE_EINVAL;
  }
  verify::Args a = {b->q_start, d->target, d->draft, b->T > 1 ? d->target_stride : d->V, b->T > 1 ? d->draft_stride : d->V,
                    d->token, d->parent, d->u, d->u_last, d->V, b->T, path, count, token, path_stride, err_dev};
  // CTAs of a request: up to two an SM in all, and no more than have four lines of 128 values a warp to read.  With one, two,
  // four and eight an SM 64 picked trees take 18.4, 16.3, 23.2 and 41.5 us and 64 drawn chains 30.9, 29.5, 35.8 and 55.8, as
  // requests past the second wait for others to end; 32 drawn chains 19.1, 19.3, 32.0 and 32.0.
  const int sms = sm_count();
  if (sms < 1) return MOE_ECUDA;
  const int most = d->V / (128 * verify::kGroups * verify::kWarps) + 1;
  int ctas = verify::kMaxCtas;
  while (ctas > 1 && ((long long)b->B * ctas > 2 * sms || ctas >= 2 * most)) ctas /= 2;
  if ((long long)b->B * ctas > INT32_MAX) return MOE_EINVAL;
  // Registers for one CTA an SM where there are no more, else for two, which spill where drafts are drawn.  With 128 and with
  // 64: one drawn chain 8.2 and 9.2 us, four 9.3 and 12.1, eight drawn trees of 16 29.2 and 32.4, one picked chain 6.6 and
  // 6.7; 64 picked trees 25.0 and 16.3.  Eight drawn chains are the exception, 16.5 and 13.6: at one CTA an SM seven
  // clusters of sixteen find a place.
  const bool alone = (long long)b->B * ctas <= sms;
  auto* kernel = d->draft ? alone ? verify::k_verify<true, 1> : verify::k_verify<true, 2>
                          : alone ? verify::k_verify<false, 1> : verify::k_verify<false, 2>;
  // clusters of sixteen are to be asked for
  if (ctas > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return MOE_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(b->B) * ctas);
  cfg.blockDim = dim3(verify::kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {unsigned(ctas), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? MOE_OK : MOE_ECUDA;
}
