// Attention over a paged cache on the tcgen05 tensor cores (one kernel for new
// tokens, verify windows and prompt chunks) and the join of what it splits.
//
// Mathematics.  For one key head, the query rows of a row tile are R = (token,
// head of the group) pairs, up to NR of them, and the keys come in tiles of 128:
//   S^T = K Q^T            [128 keys x NR]       (M = keys, N = rows)
//   P^T = exp2(c S^T - m)  masked; m per row
//   O^T += V^T P^T         [D x NR]              (M = columns of v, N = rows)
// Keys on the M side keep the tensor core's 128 rows full however few query
// rows there are: a decode step has one to sixteen of them, and the other way
// round all but those rows of the tile would be padding.  It also leaves each
// of the 128 softmax threads one key, so a tile's exponentials are spread over
// all of them.
//
// The running maximum is lazy: m is the exact maximum of a row at the time it
// was last set, and it is set again, with O and the sums rescaled, only when a
// score passes m + 8 (in log2 units), so a weight is at most 2^8 and most
// tiles need one vote instead of a maximum over all threads.  Sums are kept by
// each thread for its keys and added up once, at the end of a piece.
//
// Roundings.  Scores and sums are fp32.  The operands are bf16: q and a bf16
// cache as they are, E4M3 codes exactly, and P rounded once, half a unit of
// 2^-8 relative to each weight however small (f16 would keep three bits more
// of the large weights and lose those 2^-32 below the largest).
//
// Split.  Every (request, key head, row tile) is a unit of tiles; all tiles of
// a call are laid end to end and cut into equal runs, one per SM, whatever the
// lengths.  A run takes its units in pieces; a piece that is not its whole unit
// leaves (m, sum, O) in the scratch, and a second kernel joins the pieces of a
// unit in their order.
#pragma once

#include <limits.h>

#include "paged.cuh"

namespace moe {
namespace attn {

constexpr int kKeys = 128;                    // keys in a tile
constexpr float kUnset = -1e30f;              // m of a row that has seen no key
constexpr float kGrow = 8.0f;                 // m is set again when a score passes it by this (log2)
constexpr unsigned long long kWaitNs = 1000000000ull;
constexpr int kSmem = 232448;
constexpr int kMisc = 6144;                   // barriers, row statistics, schedule

struct Args {
  KvView kv;
  const uint16_t* q;
  uint16_t* o;
  long long qs, os;
  int G, window;
  float scale;
  int32_t* err;
  float* part;  // [2 * CTAs][NR][D] pieces: head piece of CTA c at 2c, tail piece at 2c + 1
  float* ml;    // [2 * CTAs][NR][2] their m and sums
  int4* head;   // [CTAs] head piece: request, key head, row tile; w = 1 when it starts inside its unit
  long long* cut;  // [CTAs][2] that unit's tiles, first and last + 1, in the call's order of tiles
  long long* total;  // [1] tiles of the call
};

template <int D, int NR, bool E4M3>
struct Cfg {
  static constexpr int DS = D < 128 ? D : 128;       // columns in a slot
  static constexpr int H = D / DS;                   // slots of a key or value tile
  static constexpr int SLOT = kKeys * DS * 2;
  static constexpr int QBYTES = NR * D * 2;
  static constexpr int PBYTES = kKeys * NR * 2;
  static constexpr int FREE = kSmem - kMisc - 2 * PBYTES;
  static constexpr int QB = (FREE - 2 * QBYTES) / SLOT >= 5 ? 2 : 1;
  static constexpr int NS = (FREE - QB * QBYTES) / SLOT;
  static constexpr int CW = NR < 32 ? NR : 32;       // rows a softmax warp holds
  static constexpr int SW = 4 * (NR / CW);           // softmax warps
  static constexpr int PW = NR > 64 ? 4 : 8;         // producer warps
  static constexpr int THREADS = 32 * (SW + 1 + PW);
  static constexpr int COLS0 = (2 + H) * NR;
  static constexpr int COLS = COLS0 <= 64 ? 64 : COLS0 <= 128 ? 128 : COLS0 <= 256 ? 256 : 512;
  static_assert(COLS0 <= 512 && NS >= 3 && NS <= 16, "resources of an SM");
};

// ------------------------------------------------------------------ schedule
// One request as the kernels see it; out-of-range entries are cut to what memory holds.
struct Req {
  int s0, n, pos0, kv;
};
__device__ __forceinline__ Req load_req(const KvView& kv, int b) {
  Req r;
  const int s0 = kv.q_start[b], s1 = kv.q_start[b + 1];
  r.kv = max(kv.kv_len[b], 0);
  r.s0 = min(max(s0, 0), kv.T);
  r.n = min(max(s1, r.s0), kv.T) - r.s0;
  r.pos0 = r.kv - r.n;
  return r;
}
struct Span {  // the keys that a row tile's rows see between them: [lo, hi), in nt tiles from tile0
  int i0, i1, lo, hi, tile0, nt;
};
template <int NR>
__device__ __forceinline__ Span span_of(const Req& r, int rt, int G, int window, int cap) {
  Span s;
  s.i0 = rt * NR / G;
  s.i1 = (min((rt + 1) * NR, r.n * G) - 1) / G;
  s.hi = min(max(r.pos0 + s.i1 + 1, 0), cap);
  s.lo = window > 0 ? min(max(r.pos0 + s.i0 - window + 1, 0), s.hi) : 0;
  s.tile0 = s.lo / kKeys;
  s.nt = max(s.hi / kKeys + (s.hi % kKeys != 0) - s.tile0, 1);  // a tile even where nothing is seen: its rows get zeros
  return s;
}
__device__ __forceinline__ int cap_of(const KvView& kv) {
  return int(min((long long)kv.table_stride << kv.page_shift, (long long)INT_MAX - kKeys));
}
template <int NR>
__device__ __forceinline__ long long head_tiles(const Req& r, int G, int window, int cap) {
  long long w = 0;
  for (int rt = 0; rt * NR < r.n * G; ++rt) w += span_of<NR>(r, rt, G, window, cap).nt;
  return w;
}

// A walk over the tiles of a run: the same in every role.
template <int NR>
struct Walk {
  Req r;
  Span s;
  int b, h, rt, j, jbeg, jend;
  long long left;  // tiles after this one
  __device__ __forceinline__ void unit(const Args& a, int cap, int from, long long count) {
    s = span_of<NR>(r, rt, a.G, a.window, cap);
    jbeg = j = from;
    jend = int(min((long long)s.nt, from + count));
    left = count - 1;
  }
  // The run's first tile: tile `off` of request b.
  __device__ __forceinline__ void start(const Args& a, int cap, int b_, long long off, long long count) {
    b = b_;
    r = load_req(a.kv, b);
    const long long per = head_tiles<NR>(r, a.G, a.window, cap);
    h = int(off / per);
    off -= h * per;
    for (rt = 0;; ++rt) {
      const int nt = span_of<NR>(r, rt, a.G, a.window, cap).nt;
      if (off < nt) break;
      off -= nt;
    }
    unit(a, cap, int(off), count);
  }
  __device__ __forceinline__ void next(const Args& a, int cap) {  // left > 0
    if (++j < jend) {
      --left;
      return;
    }
    if ((rt + 1) * NR < r.n * a.G) {
      ++rt;
    } else {
      rt = 0;
      if (++h == a.kv.Hkv) {
        h = 0;
        do {
          r = load_req(a.kv, ++b);
        } while (r.n == 0);
      }
    }
    unit(a, cap, 0, left);
  }
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t su32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// 128-byte swizzle: row r of 128 bytes, 16-byte piece c
__device__ __forceinline__ uint32_t sw128(int r, int c) { return uint32_t(r * 128 + ((c ^ (r & 7)) << 4)); }
__device__ __forceinline__ void bar_init(uint64_t* b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n));
}
__device__ __forceinline__ void arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for the phase with parity `par`; gives up after kWaitNs, and at once when another wait of
// the CTA gave up: every role then runs through its loop without waiting, and the call reports it.
__device__ __forceinline__ void wait(uint64_t* b, uint32_t par, volatile int* fail) {
  unsigned long long t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(su32(b)), "r"(par)
        : "memory");
    if (ok) return;
    if (*fail) return;
    if (i == 0) t0 = now_ns();
    else if ((i & 63) == 0 && now_ns() - t0 > kWaitNs) *fail = 1;
  }
}
__device__ __forceinline__ void commit_to(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(b))
               : "memory");
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc))
      : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void ld16(uint32_t t, float v[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void st16(uint32_t t, const float v[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// True in every softmax thread when it is in any of them.
template <int N>
__device__ __forceinline__ bool vote_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(p)), "n"(N)
      : "memory");
  return r != 0;
}
template <int N>
__device__ __forceinline__ void softmax_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Shared-memory descriptors (start, leading and stride offsets in 16-byte units, version 1).
__device__ __forceinline__ uint64_t desc(uint32_t start, uint32_t lbo, uint32_t sbo, uint64_t swizzle) {
  return uint64_t((start >> 4) & 0x3FFF) | (uint64_t(lbo >> 4) << 16) | (uint64_t(sbo >> 4) << 32) |
         (uint64_t(1) << 46) | (swizzle << 61);
}

struct Misc {
  uint64_t full[16], empty[16], qfull[2], qfree[2], sfull[2], pfull[2], pvdone[2], ofree, drain;
  uint32_t taddr;
  int fail;
  int b;          // the run's first request
  long long off;  // its first tile in it
  long long scan[32];
  float m[128], alpha[128];
  float red[4][128];
  int nbad;
  uint8_t bad[128];  // keys of a tile with values that are not finite
};
static_assert(sizeof(Misc) <= kMisc, "misc");

// ------------------------------------------------------------------ roles

// Byte offset of each of a thread's keys in a pool (-1: nothing there, read as zeros).
template <int RPT>
struct Rows {
  long long off[RPT];
};
template <int RPT, int STEP, int NR>
__device__ __forceinline__ void find_rows(const Args& a, const Walk<NR>& w, int r0, int lane_col, Rows<RPT>& out,
                                          bool report) {
  const KvView& kv = a.kv;
  const int32_t* row = kv.page_table + (long long)w.b * kv.table_stride;
  int id[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int key = (w.s.tile0 + w.j) * kKeys + r0 + i * STEP;
    id[i] = key >= w.s.lo && key < w.s.hi ? row[key >> kv.page_shift] : -2;
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int key = (w.s.tile0 + w.j) * kKeys + r0 + i * STEP;
    if (id[i] >= 0 && id[i] < kv.npages) {
      out.off[i] = id[i] * kv.page_stride + w.h * kv.head_stride +
                   (long long)(key & ((1 << kv.page_shift) - 1)) * kv.tok_stride;
    } else {
      out.off[i] = -1;
      if (report && id[i] != -2) set_error(a.err, MOE_ERANGE);
    }
  }
}

// Two E4M3 codes (low byte first) -> bf16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two) {
  const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2(two));
  return pack2(f.x, f.y);
}

// The query rows of a piece, K-major with the 128-byte swizzle, one 64-column chunk after another.
template <int D, int NR, int THREADS>
__device__ __forceinline__ void load_q(const Args& a, const Walk<NR>& w, uint8_t* dst, int tid) {
  constexpr int CH = D / 8;  // 16-byte pieces of a row
  const int rows = w.r.n * a.G - w.rt * NR;
  for (int p = tid; p < NR * CH; p += THREADS) {
    const int row = p / CH, c = p % CH;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (row < rows) {
      const int rr = w.rt * NR + row, i = rr / a.G, g = rr - i * a.G;
      u = *reinterpret_cast<const uint4*>(a.q + (w.r.s0 + i) * a.qs + (long long)(w.h * a.G + g) * D + c * 8);
    }
    *reinterpret_cast<uint4*>(dst + (c / 8) * (NR * 128) + sw128(row, c % 8)) = u;
  }
}

// Sum of each of W values over the warp's lanes: lane i of every group of W gets value i's.
template <int W>
__device__ __forceinline__ float transpose_sum(float (&v)[W], int lane) {
  if constexpr (W == 1) {
    return v[0];
  } else {
    constexpr int half = W / 2;
    float k[half];
    const bool up = lane & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float mine = up ? v[i + half] : v[i], other = up ? v[i] : v[i + half];
      k[i] = mine + __shfl_xor_sync(0xffffffffu, other, half);
    }
    return transpose_sum<half>(k, lane);
  }
}

template <int D, int NR, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, NR, E4M3>::THREADS, 1) k_attn(const __grid_constant__ Args a) {
  using C = Cfg<D, NR, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  uint8_t* sq = ring + C::NS * C::SLOT;
  uint8_t* sp = sq + C::QB * C::QBYTES;
  Misc& ms = *reinterpret_cast<Misc*>(sp + 2 * C::PBYTES);
  volatile int* fail = &ms.fail;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kMmaWarp = C::SW, kProd0 = 32 * (C::SW + 1), kProd = 32 * C::PW, kSoft = 32 * C::SW;

  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      bar_init(&ms.full[i], C::PW);
      bar_init(&ms.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&ms.qfull[i], C::PW);
      bar_init(&ms.qfree[i], 1);
      bar_init(&ms.sfull[i], 1);
      bar_init(&ms.pfull[i], C::SW);
      bar_init(&ms.pvdone[i], 1);
    }
    bar_init(&ms.ofree, C::SW);
    bar_init(&ms.drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    ms.fail = 0;
    ms.nbad = 0;
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&ms.taddr)),
                 "n"(C::COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();

  // ---- the run: all tiles of the call cut into equal parts
  const int cap = cap_of(a.kv);
  const int B = a.kv.B, per = (B + C::THREADS - 1) / C::THREADS;
  long long mine = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < B) {
      const Req r = load_req(a.kv, b);
      if (blockIdx.x == 0 && r.n > 0 && r.kv > cap) set_error(a.err, MOE_ERANGE);
      mine += a.kv.Hkv * head_tiles<NR>(r, a.G, a.window, cap);
    }
  }
  long long incl = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, x);
    if (lane >= x) incl += y;
  }
  if (lane == 31) ms.scan[warp] = incl;
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t taddr = ms.taddr;
  long long total = 0, before = incl - mine;
  for (int w = 0; w < C::THREADS / 32; ++w) {
    if (w < warp) before += ms.scan[w];
    total += ms.scan[w];
  }
  const int runs = int(min((long long)gridDim.x, total)), run = blockIdx.x;  // no run is empty
  const long long w0 = run < runs ? total * run / runs : 0, w1 = run < runs ? total * (run + 1) / runs : 0;
  const long long count = w1 - w0;
  if (tid == 0) {
    a.head[run].w = 0;
    if (run == 0) *a.total = total;
  }
  if (count > 0 && w0 >= before && w0 < before + mine) {
    long long off = w0 - before;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      const long long n = a.kv.Hkv * head_tiles<NR>(load_req(a.kv, b), a.G, a.window, cap);
      if (off < n) {
        ms.b = b;
        ms.off = off;
        break;
      }
      off -= n;
    }
  }
  __syncthreads();

  if (count > 0) {
    Walk<NR> w;
    w.start(a, cap, ms.b, ms.off, count);
    if (warp == kMmaWarp) {
      // -------------------------------------------------------- tensor cores
      if (lane == 0) {
        // D f32, A and B bf16, N = NR, M = 128; the second product's operands are both MN-major
        constexpr uint32_t kBase = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(NR >> 3) << 17) | (8u << 24);
        constexpr uint32_t kIdescS = kBase, kIdescO = kBase | (1u << 15) | (1u << 16);
        int slot = 0, qn = -1;  // ring position, pieces begun
        uint32_t sph = 0;       // its phase
        auto take = [&]() {
          wait(&ms.full[slot], sph, fail);
          tc_after();
        };
        auto pass = [&]() {
          if (++slot == C::NS) {
            slot = 0;
            sph ^= 1;
          }
        };
        bool first_prev = false;
        int pieces_done = 0;
        for (long long n = 0; n <= count; ++n) {
          bool first = false;
          if (n < count) {
            // S^T(n) = K(n) Q^T
            first = w.j == w.jbeg;
            if (first) {
              ++qn;
              wait(&ms.qfull[qn % C::QB], (qn / C::QB) & 1, fail);
            }
            const uint32_t d = taddr + uint32_t(n & 1) * NR;
            for (int hh = 0; hh < C::H; ++hh) {
              take();
              const uint32_t ka = su32(ring + slot * C::SLOT);
              const uint32_t qa = su32(sq + (qn % C::QB) * C::QBYTES) + hh * (C::DS / 64) * (NR * 128);
              if (!*fail) {
#pragma unroll
                for (int k = 0; k < C::DS / 16; ++k) {
                  const uint32_t ko = (k / 4) * (kKeys * 128) + (k % 4) * 32, qo = (k / 4) * (NR * 128) + (k % 4) * 32;
                  mma(d, desc(ka + ko, 16, 1024, 2), desc(qa + qo, 16, 1024, 2), kIdescS, hh + k > 0);
                }
                commit_to(&ms.empty[slot]);
              }
              pass();
            }
            if (!*fail) {
              commit_to(&ms.sfull[n & 1]);
              if (w.j + 1 == w.jend) commit_to(&ms.qfree[qn % C::QB]);
            }
          }
          if (n > 0) {
            // O^T += V(n-1)^T P(n-1)^T
            const int p = int((n - 1) & 1);
            wait(&ms.pfull[p], ((n - 1) >> 1) & 1, fail);
            if (first_prev && pieces_done > 0) wait(&ms.ofree, (pieces_done - 1) & 1, fail);
            if (first_prev) ++pieces_done;
            const uint32_t pa = su32(sp + p * C::PBYTES);
            for (int hh = 0; hh < C::H; ++hh) {
              take();
              const uint32_t va = su32(ring + slot * C::SLOT);
              if (!*fail) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k) {
                  // D = 64: the upper 64 rows of M read the same columns again and are not used
                  mma(taddr + uint32_t(2 + hh) * NR, desc(va + k * 2048, D < 128 ? 0 : kKeys * 128, 1024, 2),
                      desc(pa + k * 256, 128, 2048, 0), kIdescO, !first_prev || k > 0);
                }
                commit_to(&ms.empty[slot]);
              }
              pass();
            }
            if (!*fail) commit_to(&ms.pvdone[p]);
          }
          first_prev = first;
          if (n + 1 < count) w.next(a, cap);
        }
        commit_to(&ms.drain);
        unsigned long long t0 = now_ns();
        for (uint32_t ok = 0; !ok && now_ns() - t0 < 2 * kWaitNs;)
          asm volatile(
              "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], 0;\n\tselp.u32 %0, 1, 0, p;\n\t}"
              : "=r"(ok)
              : "r"(su32(&ms.drain))
              : "memory");
      }
      __syncwarp();
    } else if (warp > kMmaWarp) {
      // -------------------------------------------------------- producers
      const int pt = tid - kProd0;
      int slot = 0, qn = -1;
      uint32_t sph = 1;  // a fresh slot is empty
      auto pass = [&]() {
        if (++slot == C::NS) {
          slot = 0;
          sph ^= 1;
        }
      };
      auto give = [&](uint64_t* b) {  // this warp's part of a slot is in shared memory
        proxy_fence();
        __syncwarp();
        if (lane == 0) arrive(b);
      };
      auto queries = [&](const Walk<NR>& wk, auto&& before_wait) {
        ++qn;
        if (qn >= C::QB) before_wait();
        if (qn >= C::QB) wait(&ms.qfree[qn % C::QB], (qn / C::QB - 1) & 1, fail);
        load_q<D, NR, kProd>(a, wk, sq + (qn % C::QB) * C::QBYTES, pt);
        give(&ms.qfull[qn % C::QB]);
      };
      if constexpr (!E4M3) {
        // cp.async, 16 bytes a thread; a slot is handed over when kLag newer ones are on their way
        constexpr int CH = C::DS / 8, STEP = kProd / CH, RPT = kKeys / STEP;
        constexpr int kLag = C::NS / 2;
        const int r0 = pt / CH, c = pt % CH;
        Rows<RPT> rk, rv;
        int given = 0, made = 0;  // slots handed over, slots begun
        int gslot = 0;
        auto hand = [&]() {
          proxy_fence();
          __syncwarp();
          if (lane == 0) arrive(&ms.full[gslot]);
          if (++gslot == C::NS) gslot = 0;
          ++given;
        };
        // what has been begun is handed over before a wait that depends on it
        auto flush = [&]() {
          asm volatile("cp.async.wait_all;" ::: "memory");
          while (given < made) hand();
        };
        auto load = [&](const uint8_t* pool, const Rows<RPT>& r) {
          for (int hh = 0; hh < C::H; ++hh) {
            wait(&ms.empty[slot], sph, fail);
            uint8_t* dst = ring + slot * C::SLOT + (c / 8) * (kKeys * 128);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
              const bool ok = r.off[i] >= 0;
              const uint8_t* src = pool + (ok ? r.off[i] + hh * (C::DS * 2) + c * 16 : 0);
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(su32(dst) + sw128(r0 + i * STEP, c % 8)),
                           "l"(src), "r"(ok ? 16 : 0)
                           : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            pass();
            ++made;
            if (made - given > kLag) {
              asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
              hand();
            }
          }
        };
        for (long long n = 0; n <= count; ++n) {
          if (n < count) {
            if (w.j == w.jbeg) queries(w, flush);
            find_rows<RPT, STEP>(a, w, r0, c, rk, c == 0);
            load(a.kv.k, rk);
          }
          if (n > 0) load(a.kv.v, rv);
          rv = rk;
          if (n + 1 < count) w.next(a, cap);
        }
        flush();
      } else {
        // 16 codes a load, turned into bf16 on the way; the loads of kDepth tiles are in flight
        constexpr int CH = C::DS / 16, STEP = kProd / CH, RPT = kKeys / STEP;
        constexpr int kRegs = NR > 16 ? 32 : 64, kTile = C::H * RPT * 8;  // registers for loads, of one tile
        constexpr int kDepth = 4 * kTile <= kRegs ? 4 : 2 * kTile <= kRegs ? 2 : 1;
        const int r0 = pt / CH, c = pt % CH;
        uint4 kb[kDepth][C::H][RPT], vb[kDepth][C::H][RPT];
        Rows<RPT> rk, rv;
        auto load = [&](const uint8_t* pool, const Rows<RPT>& r, uint4 (&buf)[C::H][RPT]) {
#pragma unroll
          for (int hh = 0; hh < C::H; ++hh)
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
              buf[hh][i] = make_uint4(0, 0, 0, 0);
              if (r.off[i] >= 0)
                buf[hh][i] = __ldg(reinterpret_cast<const uint4*>(pool + r.off[i] + hh * C::DS + c * 16));
            }
        };
        auto store = [&](const uint4 (&buf)[C::H][RPT]) {
#pragma unroll
          for (int hh = 0; hh < C::H; ++hh) {
            wait(&ms.empty[slot], sph, fail);
            uint8_t* dst = ring + slot * C::SLOT + (c / 4) * (kKeys * 128);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
              const uint32_t v[4] = {buf[hh][i].x, buf[hh][i].y, buf[hh][i].z, buf[hh][i].w};
              uint32_t f[8];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                f[2 * x] = e4m3x2_to_bf16x2(v[x] & 0xffffu);
                f[2 * x + 1] = e4m3x2_to_bf16x2(v[x] >> 16);
              }
              const int r = r0 + i * STEP;
              *reinterpret_cast<uint4*>(dst + sw128(r, (c % 4) * 2)) = make_uint4(f[0], f[1], f[2], f[3]);
              *reinterpret_cast<uint4*>(dst + sw128(r, (c % 4) * 2 + 1)) = make_uint4(f[4], f[5], f[6], f[7]);
            }
            give(&ms.full[slot]);
            pass();
          }
        };
        Walk<NR> ahead = w;  // kDepth tiles ahead of w
        long long an = 0;    // its tile
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
          if (an < count) {
            find_rows<RPT, STEP>(a, ahead, r0, c, rk, c == 0);
            load(a.kv.k, rk, kb[u]);
            if (u < kDepth - 1) load(a.kv.v, rk, vb[u]);
            rv = rk;
            ++an;
            if (an < count) ahead.next(a, cap);
          }
        }
        for (long long n0 = 0; n0 <= count; n0 += kDepth) {
#pragma unroll
          for (int u = 0; u < kDepth; ++u) {
            const long long n = n0 + u;
            constexpr int kBack = kDepth - 1;
            if (n < count) {
              if (w.j == w.jbeg) queries(w, [] {});
              store(kb[u]);
            }
            // rv: tile n + kDepth - 1, whose values follow; then the keys of tile n + kDepth
            if (n > 0 && n <= count) store(vb[(u + kBack) % kDepth]);
            if (n + kDepth - 1 < count) load(a.kv.v, rv, vb[(u + kBack) % kDepth]);
            if (n + kDepth < count) {
              find_rows<RPT, STEP>(a, ahead, r0, c, rk, c == 0);
              load(a.kv.k, rk, kb[u]);
              rv = rk;
              if (++an < count) ahead.next(a, cap);
            }
            if (n + 1 < count) w.next(a, cap);
          }
        }
      }
    } else {
      // -------------------------------------------------------- softmax
      constexpr int CW = C::CW;
      const int quad = warp & 3, c0 = (warp >> 2) * CW;
      const int krow = quad * 32 + lane;  // this thread's key in a tile, and its column of v
      const uint32_t tl = taddr + (uint32_t(quad * 32) << 16);
      float l[CW];
      float factor = 0.f;  // of the scores, in log2 units
      for (long long n = 0; n < count; ++n) {
        const bool first = w.j == w.jbeg;
        if (first) {
#pragma unroll
          for (int i = 0; i < CW; ++i) l[i] = 0.f;
          factor = a.scale * 1.4426950408889634f * (E4M3 && a.kv.k_scale ? a.kv.k_scale[w.h] : 1.f);
        }
        const int p = int(n & 1);
        const uint32_t ph = (n >> 1) & 1;
        const int key0 = (w.s.tile0 + w.j) * kKeys, key = key0 + krow;
        // every row of the tile sees every key of it
        const bool whole = key0 + kKeys <= min(w.r.pos0 + w.s.i0 + 1, cap) &&
                           (a.window <= 0 || key0 > w.r.pos0 + w.s.i1 - a.window);
        wait(&ms.sfull[p], ph, fail);
        tc_after();
        float s[CW];
#pragma unroll
        for (int i = 0; i < CW; i += 16) ld16(tl + p * NR + c0 + i, s + i);
        ld_wait();
        float over = -INFINITY;
        {
          int i = (w.rt * NR + c0) / a.G, g = (w.rt * NR + c0) - i * a.G;
#pragma unroll
          for (int x = 0; x < CW; ++x) {
            s[x] *= factor;
            if (!whole) {
              const int pos = w.r.pos0 + i;
              if (key > pos || key >= cap || (a.window > 0 && key <= pos - a.window)) s[x] = -INFINITY;
              if (++g == a.G) {
                g = 0;
                ++i;
              }
            }
            if (!first) over = fmaxf(over, s[x] - ms.m[c0 + x]);
          }
        }
        if (vote_any<kSoft>(first || over > kGrow)) {
          // set m: the rows' maxima over the 128 keys
#pragma unroll
          for (int x = 0; x < CW; ++x) {
            const float v = warp_max(s[x]);
            if (lane == (x & 31)) ms.red[quad][c0 + x] = v;
          }
          softmax_sync<kSoft>();
          if (tid < NR) {
            const float old = first ? kUnset : ms.m[tid];
            const float v = fmaxf(fmaxf(fmaxf(ms.red[0][tid], ms.red[1][tid]), fmaxf(ms.red[2][tid], ms.red[3][tid])), old);
            ms.m[tid] = v;
            ms.alpha[tid] = ex2(old - v);
          }
          softmax_sync<kSoft>();
          if (!first) {
#pragma unroll
            for (int x = 0; x < CW; ++x) l[x] *= ms.alpha[c0 + x];
            wait(&ms.pvdone[p ^ 1], ((n - 1) >> 1) & 1, fail);
            tc_after();
            for (int hh = 0; hh < C::H; ++hh)
#pragma unroll
              for (int x = 0; x < CW; x += 16) {
                float o[16];
                ld16(tl + (2 + hh) * NR + c0 + x, o);
                ld_wait();
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] *= ms.alpha[c0 + x + y];
                st16(tl + (2 + hh) * NR + c0 + x, o);
              }
            st_wait();
          }
        }
        if (n >= 2) wait(&ms.pvdone[p], ((n - 2) >> 1) & 1, fail);  // P(n - 2) has been read
        uint8_t* dst = sp + p * C::PBYTES + (krow >> 3) * 128 + (krow & 7) * 16;
#pragma unroll
        for (int x = 0; x < CW; x += 8) {
          uint32_t u[4];
#pragma unroll
          for (int y = 0; y < 8; y += 2) {
            const float e0 = ex2(s[x + y] - ms.m[c0 + x + y]);
            const float e1 = ex2(s[x + y + 1] - ms.m[c0 + x + y + 1]);
            l[x + y] += e0;
            l[x + y + 1] += e1;
            u[y / 2] = pack2(e0, e1);
          }
          *reinterpret_cast<uint4*>(dst + ((c0 + x) >> 3) * 2048) = make_uint4(u[0], u[1], u[2], u[3]);
        }
        // A value that is not finite must not reach a row that does not see its key (0 times it is
        // NaN): where rows differ in what they see, such values are taken out of the tile and added
        // to the rows that do see them.
        bool spoiled = false;
        if (!whole && w.s.i1 > w.s.i0) {
          const long long at = (n + 1 == count ? 2 * count - 1 : 2 * n + 2) * C::H;  // V(n)'s place in the ring's order
          bool bad = false;
          for (int hh = 0; hh < C::H; ++hh) {
            const int slot = int((at + hh) % C::NS);
            wait(&ms.full[slot], uint32_t((at + hh) / C::NS) & 1, fail);
            constexpr uint32_t kExp = 0x7f80u;
#pragma unroll 4
            for (int c = 0; c < C::DS / 8; ++c) {
              uint4* v = reinterpret_cast<uint4*>(ring + slot * C::SLOT + (c / 8) * (kKeys * 128) + sw128(krow, c % 8));
              uint32_t x[4] = {v->x, v->y, v->z, v->w};
              bool here = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((x[i] & kExp) == kExp) x[i] &= 0xffff0000u, here = true;
                if ((x[i] >> 16 & kExp) == kExp) x[i] &= 0xffffu, here = true;
              }
              if (here) *v = make_uint4(x[0], x[1], x[2], x[3]);
              bad |= here;
            }
          }
          if (bad && c0 == 0) ms.bad[atomicAdd(&ms.nbad, 1)] = uint8_t(krow);
          spoiled = vote_any<kSoft>(bad);
        }
        proxy_fence();
        tc_before();
        __syncwarp();
        if (lane == 0) arrive(&ms.pfull[p]);
        if (spoiled) {
          wait(&ms.pvdone[p], ph, fail);
          tc_after();
          const int nbad = *const_cast<volatile int*>(&ms.nbad);
          for (int e = 0; e < nbad; ++e) {
            const int k = key0 + ms.bad[e];
            const int id = a.kv.page_table[(long long)w.b * a.kv.table_stride + (k >> a.kv.page_shift)];
            const uint8_t* v = a.kv.v + id * a.kv.page_stride + w.h * a.kv.head_stride +
                               (long long)(k & ((1 << a.kv.page_shift) - 1)) * a.kv.tok_stride;
            for (int hh = 0; hh < C::H; ++hh) {
              const int col = hh * 128 + krow;
              float add = 0.f;
              if (col < D) {
                if (E4M3) add = f16x2_to_f32x2(e4m3x2_to_f16x2(v[col])).x;
                else add = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(v)[col]);
              }
              if (isfinite(add)) add = 0.f;
              int i = (w.rt * NR + c0) / a.G, g = (w.rt * NR + c0) - i * a.G;
#pragma unroll
              for (int x = 0; x < CW; x += 16) {
                float o[16];
                ld16(tl + (2 + hh) * NR + c0 + x, o);
                ld_wait();
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                  const int pos = w.r.pos0 + i;
                  if (k <= pos && (a.window <= 0 || k > pos - a.window)) o[y] += add;
                  if (++g == a.G) {
                    g = 0;
                    ++i;
                  }
                }
                st16(tl + (2 + hh) * NR + c0 + x, o);
              }
            }
          }
          st_wait();
          tc_before();
          softmax_sync<kSoft>();
          if (tid == 0) ms.nbad = 0;
        }

        if (w.j + 1 == w.jend) {
          // ---- the piece is done: its rows' sums, then O
#pragma unroll
          for (int x = 0; x < CW; x += 16) {
            float v[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) v[y] = l[x + y];
            float t = transpose_sum<16>(v, lane);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            if (lane < 16) ms.red[quad][c0 + x + lane] = t;
          }
          softmax_sync<kSoft>();
          const bool head = w.jbeg > 0, split = head || w.jend < w.s.nt;
          const int rows = min(NR, w.r.n * a.G - w.rt * NR);
          const long long part = 2ll * blockIdx.x + (head ? 0 : 1);
          if (split) {
            if (tid < rows) {
              float2 v = make_float2(ms.m[tid], ms.red[0][tid] + ms.red[1][tid] + ms.red[2][tid] + ms.red[3][tid]);
              reinterpret_cast<float2*>(a.ml)[part * NR + tid] = v;
            }
            if (head && tid == 0) {
              a.head[blockIdx.x] = make_int4(w.b, w.h, w.rt, 1);
              a.cut[2 * blockIdx.x] = w0 - w.jbeg;
              a.cut[2 * blockIdx.x + 1] = w0 - w.jbeg + w.s.nt;
            }
          }
          const float vs = E4M3 && a.kv.v_scale ? a.kv.v_scale[w.h] : 1.f;
          wait(&ms.pvdone[p], ph, fail);
          tc_after();
          for (int hh = 0; hh < C::H; ++hh) {
            const int col = hh * 128 + krow;
            int i = (w.rt * NR + c0) / a.G, g = (w.rt * NR + c0) - i * a.G;
#pragma unroll
            for (int x = 0; x < CW; x += 16) {
              float o[16];
              ld16(tl + (2 + hh) * NR + c0 + x, o);
              ld_wait();
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                const int row = c0 + x + y;
                if (row < rows && col < D) {
                  if (split) {
                    a.part[(part * NR + row) * D + col] = o[y];
                  } else {
                    const float t = ms.red[0][row] + ms.red[1][row] + ms.red[2][row] + ms.red[3][row];
                    const float v = t == 0.f ? 0.f : o[y] / t * vs;
                    a.o[(w.r.s0 + i) * a.os + (long long)(w.h * a.G + g) * D + col] =
                        __bfloat16_as_ushort(__float2bfloat16_rn(v));
                  }
                }
                if (++g == a.G) {
                  g = 0;
                  ++i;
                }
              }
            }
          }
          tc_before();
          softmax_sync<kSoft>();  // m, red and O are free
          if (lane == 0) arrive(&ms.ofree);
        }
        if (n + 1 < count) w.next(a, cap);
      }
    }
  }
  __syncthreads();
  if (tid == 0 && *fail) set_error(a.err, MOE_ETIMEOUT);
  if (warp == kMmaWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(C::COLS));
  }
}

// Joins the pieces of a unit: o = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k, in the order of
// the pieces.  CTA (c, y): the unit that the cut before run c is the first to fall into, rows y, y + 16, ..
constexpr int kJoinThreads = 256;
constexpr int kMaxRuns = 512;
template <int D, int NR>
__global__ void __launch_bounds__(kJoinThreads) k_join(const __grid_constant__ Args a) {
  constexpr int L = D / 4, PG = kJoinThreads / L;  // threads over a row's columns, over its pieces
  __shared__ float f[kMaxRuns + 1], red[kJoinThreads / 32];
  __shared__ float4 acc[kJoinThreads];
  pdl_trigger();
  pdl_wait();
  const long long total = *a.total;
  const int runs = int(min((long long)gridDim.x, total)), c = blockIdx.x, tid = threadIdx.x;
  if (c < 1 || c >= runs) return;
  const int4 hd = a.head[c];
  const long long u0 = a.cut[2 * c], u1 = a.cut[2 * c + 1];
  if (!hd.w || total * (c - 1) / runs > u0) return;
  const Req r = load_req(a.kv, hd.x);
  const int rows = min(NR, r.n * a.G - hd.z * NR);
  int np = 1;  // pieces: the tail of run c - 1, then the heads of the runs that begin before the unit's end
  while (c - 1 + np < runs && total * (c - 1 + np) / runs < u1) ++np;
  auto place = [&](int k) { return 2ll * (c - 1 + k) + (k == 0 ? 1 : 0); };
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    float m = kUnset;
    for (int k = tid; k < np; k += kJoinThreads) m = fmaxf(m, __ldcg(a.ml + (place(k) * NR + row) * 2));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, red[w]);
    float l = 0.f;
    for (int k = tid; k < np; k += kJoinThreads) {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(a.ml) + place(k) * NR + row);
      f[k] = ex2(v.x - m);
      l += f[k] * v.y;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    __syncthreads();  // f is whole, red has been read
    if ((tid & 31) == 0) red[tid >> 5] = l;
    const int col = tid % L, pg = tid / L;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = pg; k < np; k += PG) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part + (place(k) * NR + row) * D) + col);
      const float w = f[k];
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
    acc[tid] = o;
    __syncthreads();
    if (pg == 0) {
      l = 0.f;
      for (int w = 0; w < kJoinThreads / 32; ++w) l += red[w];
      for (int k = 1; k < PG; ++k) {
        const float4 v = acc[k * L + col];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
      }
      const float vs = a.kv.v_scale ? a.kv.v_scale[hd.y] : 1.f;
      const float x = l == 0.f ? 0.f : vs / l;
      const int rr = hd.z * NR + row, i = rr / a.G, g = rr - i * a.G;
      uint2 u;
      u.x = pack2(o.x * x, o.y * x);
      u.y = pack2(o.z * x, o.w * x);
      *reinterpret_cast<uint2*>(a.o + (r.s0 + i) * a.os + (long long)(hd.y * a.G + g) * D + col * 4) = u;
    }
    __syncthreads();
  }
}

// Tile of rows for calls of about `rows` query rows per request and key head.
inline int row_tile(int D, long long rows) { return rows <= 16 ? 16 : rows <= 64 || D == 256 ? 64 : 128; }

template <int D, int NR, bool E4M3>
int launch_one(const Args& a, int ctas, cudaStream_t s) {
  using C = Cfg<D, NR, E4M3>;
  if (launch_pdl(k_attn<D, NR, E4M3>, dim3(ctas), dim3(C::THREADS), kSmem, s, a) != cudaSuccess) return MOE_ECUDA;
  if (launch_pdl(k_join<D, NR>, dim3(ctas, 16), dim3(kJoinThreads), 0, s, a) != cudaSuccess) return MOE_ECUDA;
  return MOE_OK;
}
template <int D, int NR>
int opt_in() {
  return cudaFuncSetAttribute(k_attn<D, NR, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess &&
                 cudaFuncSetAttribute(k_attn<D, NR, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) ==
                     cudaSuccess
             ? MOE_OK
             : MOE_ECUDA;
}

}  // namespace attn
}  // namespace moe
