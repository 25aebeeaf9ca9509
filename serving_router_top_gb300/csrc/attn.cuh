// Attention over a paged cache on the tcgen05 tensor cores (new tokens, verify
// windows, prompt chunks of 256 columns) and the join of what it splits.
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
// weight passes 2^8: most tiles' weights are computed at once, with one vote
// after them instead of a maximum over all threads before them.  Sums are kept
// by each thread for its keys and added up once, at the end of a piece.
//
// Roundings.  Scores and sums are fp32.  A bf16 cache and q are the operands as
// they are; P is rounded once to bf16, half a unit of 2^-8 relative to each
// weight however small (f16 would keep three bits more of the large weights and
// lose those 2^-32 below the largest).
//
// E4M3 caches.  Keys go to the tensor core as they are, against q in two E4M3
// terms: q 2^e = t0 + t1 / 32, with 2^e such that the row's largest is in
// [2^7, 2^8).  A bf16 value has 8 significant bits and a term takes 4, so the two
// are exact for what is within 2^-14 of the row's largest and off by 2^-22 of it
// below.  The terms are 2 NR rows of one product, whose halves the softmax adds.
// Values become bf16, exactly: as many terms of P would lose weights 2^-23 below
// the largest, thousands of which can be half the sum.  With keys converted too,
// the conversions' traffic through shared memory and their turns in the ring took
// longer than the memory: one token of 32 requests of 4096 keys, 128 columns, 63.1
// us with both converted, 51.9 us now; 64 columns 53.6 and 46.5; 16 windows of four
// up to 32768 keys, 256 columns, 50.7 and 48.6.
//
// Movement.  Two warps, one for keys and one for values, ask the copy engine for
// the tiles (a page, or 128 keys of a larger one, by 64 columns a box, swizzled for
// the tensor core); pages that are not there are asked for past the pool's end and
// read as zeros.  E4M3 values land as they are and are turned into bf16 by warps of
// their own, which also write the queries' terms.
//
// What bounds it: memory.  One token over 131071 keys (268 MB) 47.5 us, 5.7 TB/s with
// the join; 32 requests of 4096 keys 84 us, 6.4 TB/s, 95% of what a copy reaches.
// Short units add a softmax's chain at each end, about three tiles' time.
//
// Split.  Every (request, key head, row tile) is a unit: its tiles, and before
// them a cost for its beginning and end (new queries, a maximum from scratch, an
// output) counted in tiles.  All units of a call are laid end to end and cut
// into equal runs, one or two per SM, whatever the lengths.  A run takes its units in
// pieces; a piece that is not its whole unit leaves (m, sum, O) in the scratch,
// and a second kernel joins the pieces of a unit in their order.
#pragma once

#include <cuda.h>
#include <limits.h>

#include "paged.cuh"

namespace moe {
namespace attn {

constexpr int kKeys = 128;                    // keys in a tile
constexpr float kUnset = -3.402823466e38f;    // m of a row that has seen no key: no finite score is below it
constexpr float kMost = 256.0f;               // m is set again when a weight passes this
constexpr float kLost = 0x1p-100f;            // sums from before m grew by this factor are nothing to those after
constexpr unsigned long long kWaitNs = 1000000000ull, kLandNs = 2000000ull;
constexpr int kSmem = 232448;                 // shared memory of one CTA on an SM, and of each of two
constexpr int kSmem2 = 115712;
constexpr int misc_bytes(int nr) { return (2192 + 60 * nr + 127) / 128 * 128; }  // barriers, row statistics, schedule

struct Args {
  CUtensorMap mk, mv, mq;  // pools [page][head][place][column], query rows [token][head][column]
  KvView kv;
  const uint16_t* q;
  uint16_t* o;
  long long qs, os;
  int G, window, tokens;   // query heads a key head; visible keys (0: all); tokens in a row tile
  float scale;
  int phantom;  // a test of the waits: 1 the queries', 2 the weights', 3 the slots' barriers want an arrival that never comes
  int32_t* err;
  float* part;  // [2 * runs][NR][D] pieces: head piece of run c at 2c, tail piece at 2c + 1
  float* ml;    // [2 * runs][NR][2] their m and sums
  int4* join;   // [runs] where run c's first piece is the second of a unit: token, key head, rows, pieces (else 0)
};

template <int D, int NR, bool E4M3>
struct Cfg {
  static constexpr int DS = D < 128 ? D : 128;       // columns in a slot
  static constexpr int H = D / DS;                   // slots of a key or value tile
  static constexpr int SLOT = kKeys * DS * 2;
  static constexpr int RAW = E4M3 ? kKeys * DS : 0;  // a slot's codes
  static constexpr int QBYTES = 2 * NR * D;          // the rows in bf16, or their two E4M3 terms
  static constexpr int PBYTES = kKeys * NR * 2;
  // Two CTAs to an SM where each still has three slots of 128 columns or five of 64: they hide each
  // other's waits (a tile's softmax is a chain of about 1100 clocks whatever its rows, an SM's share of
  // the memory brings 64 columns' 32 KB in 1400) and the ends of units.
  static constexpr int OCC = !E4M3 && (kSmem2 - misc_bytes(NR) - 2 * PBYTES - QBYTES) / SLOT >= (D < 128 ? 5 : 3) && H == 1 ? 2 : 1;
  static constexpr int SMEM = OCC == 2 ? kSmem2 : kSmem;
  static constexpr int FREE = SMEM - misc_bytes(NR) - 2 * PBYTES;
  // E4M3: a ring of bf16 values, the rest for keys and values as they come.  32 requests of 4096 keys, 128
  // columns: two slots of bf16 51.7 us, three 52.7.
  static constexpr int NV = 2;
  static constexpr int codes(int qb) { return E4M3 ? (FREE - qb * QBYTES - NV * SLOT) / (RAW + !E4M3) : 0; }
  static constexpr int QB = OCC == 2 ? 1 : E4M3 ? (codes(2) >= 5 ? 2 : 1) : (FREE - 2 * QBYTES) / SLOT >= 5 ? 2 : 1;
  static constexpr int NS0 = E4M3 ? NV : (FREE - QB * QBYTES) / SLOT, NS = NS0 > 16 ? 16 : NS0;
  static constexpr int NK0 = (codes(QB) + 1) / 2, NK = NK0 > 8 ? 8 : NK0, NR0 = codes(QB) / 2, NRAW = NR0 > 8 ? 8 : NR0;
  static constexpr int SN = E4M3 ? 2 * NR : NR;      // columns of S
  static constexpr int CW = NR < 32 ? NR : 32;                 // rows a softmax warp holds
  static constexpr int SW = 4 * (NR / CW);                      // softmax warps
  // Converting warps: four take 65 us where eight take 53 (128 columns, 16 rows); beside 16 softmax warps
  // eight leave no registers.
  static constexpr int CV = !E4M3 ? 0 : NR > 32 ? 4 : 8;
  static constexpr int THREADS = 32 * (SW + 3 + CV);
  static constexpr int COLS0 = 2 * SN + 2 * H * NR;             // two S, two O
  static constexpr int COLS = COLS0 <= 64 ? 64 : COLS0 <= 128 ? 128 : COLS0 <= 256 ? 256 : 512;
  // What a unit costs beside its tiles, in tiles.  64 requests of 3 to 8192 tokens with 128 columns (64 KB
  // of keys and values a tile): 1, 2, 3 and 4 give 50.1, 44.9, 46.4 and 48.9 us; 48 with 64 columns (32 KB)
  // and a window of 1000: 33.5, 27.8, 25.9 and 26.8 us (at one run an SM).  E4M3, whose ends cost more beside
  // tiles of half the bytes, with 2, 3 and 4: 64 requests of 3 to 8192 tokens, 64 columns (16 KB) 44.2, 40.1
  // and 39.2 us, 128 columns 45.6, 41.4 and 40.8, 256 columns 36.9, 35.3 and 37.6; 16 windows of four over up
  // to 32768 keys 26.5, 24.6 and 24.0, 29.4, 27.0 and 26.2, 42.7, 39.8 and 39.0.  3 is within 3% of the best.
  static constexpr int V = !E4M3 && SLOT * H * 2 >= 65536 ? 2 : 3;
  static_assert(COLS0 <= 512 && (E4M3 ? NK >= 2 && NRAW >= 2 : NS >= 3), "resources of an SM");
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
  r.n = min(s1, kv.T) - r.s0;  // below zero where the starts decrease
  r.pos0 = r.kv - r.n;
  return r;
}
struct Span {  // the keys that a row tile's tokens i0 .. i1 see between them: [lo, hi), in nt tiles from tile0
  int i0, i1, lo, hi, tile0, nt;
};
__device__ __forceinline__ Span span_of(const Req& r, int rt, int tokens, int window, int cap) {
  Span s;
  s.i0 = rt * tokens;
  s.i1 = min(s.i0 + tokens, r.n) - 1;
  s.hi = min(max(r.pos0 + s.i1 + 1, 0), cap);
  s.lo = window > 0 ? min(max(r.pos0 + s.i0 - window + 1, 0), s.hi) : 0;
  s.tile0 = s.lo / kKeys;
  s.nt = max((s.hi + kKeys - 1) / kKeys - s.tile0, 1);  // a tile even where nothing is seen: its rows get zeros
  return s;
}
// Tokens that a request's pages hold, below kMaxTokens: sums of two positions and a window stay in 32 bits.
constexpr int kMaxTokens = 1 << 29;
__host__ __device__ inline int cap_of(const KvView& kv) {
  const long long held = (long long)kv.table_stride << kv.page_shift;
  return held < kMaxTokens ? int(held) : kMaxTokens;
}
// Tiles of a key head of a request, and its units.
struct Load {
  int tiles, units;
};
__device__ __forceinline__ Load head_load(const Req& r, int tokens, int window, int cap) {
  Load w = {0, 0};
  for (; w.units * tokens < r.n; ++w.units) w.tiles += span_of(r, w.units, tokens, window, cap).nt;
  return w;
}
// First place of run c: `total` places in `runs` runs whose lengths differ by one at most.
__device__ __forceinline__ int cut_at(int total, int runs, int c) {
  const int q = total / runs;
  return q * c + min(c, total - q * runs);
}
__device__ __forceinline__ int run_of(int total, int runs, int x) {
  const int q = total / runs, longer = total - q * runs;
  return x < longer * (q + 1) ? x / (q + 1) : longer + (x - longer * (q + 1)) / q;
}

// A walk over the tiles of a run: the same in every role.  A unit takes V places before its tiles.
template <int V>
struct Walk {
  Req r;
  Span s;
  int b, h, rt, j, jbeg, jend;
  int rest;  // places of the run after this unit
  __device__ __forceinline__ void unit(const Args& a, int cap, int off, int places) {
    s = span_of(r, rt, a.tokens, a.window, cap);
    jbeg = j = max(off - V, 0);
    jend = min(max(off + places - V, 0), s.nt);
    rest = off + places - (s.nt + V);
  }
  // The run's first unit, from its place `off` on.
  __device__ __forceinline__ void start(const Args& a, int cap, int4 first, int places) {
    b = first.x;
    h = first.y;
    rt = first.z;
    r = load_req(a.kv, b);
    unit(a, cap, first.w, places);
  }
  __device__ __forceinline__ void next(const Args& a, int cap) {  // a tile follows
    if (++j < jend) return;
    if ((rt + 1) * a.tokens < r.n) {
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
    unit(a, cap, 0, rest);
  }
};
// Place x of a request: its key head, row tile and place in their unit, and the request's tiles before it.
template <int V>
__device__ __forceinline__ int find_place(const Args& a, const Req& r, const Load& per, int cap, int x, int4* unit) {
  const int cost = per.tiles + V * per.units, h = x / cost;
  int t = h * per.tiles, rt = 0;
  x -= h * cost;
  for (;; ++rt) {
    const int nt = span_of(r, rt, a.tokens, a.window, cap).nt;
    if (x < nt + V) break;
    x -= nt + V;
    t += nt;
  }
  unit->y = h;
  unit->z = rt;
  unit->w = x;
  return t + max(x - V, 0);
}

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t su32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// 128-byte swizzle: row r of 128 bytes, 16-byte piece c
__device__ __forceinline__ uint32_t sw64(int r, int c) { return uint32_t(r * 64 + ((c ^ (r >> 1 & 3)) << 4)); }  // rows of 64 bytes
__device__ __forceinline__ uint32_t sw128(int r, int c) { return uint32_t(r * 128 + ((c ^ (r & 7)) << 4)); }
__device__ __forceinline__ void bar_init(uint64_t* b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n));
}
__device__ __forceinline__ void arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
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
#pragma unroll 1
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(su32(b)), "r"(par)
        : "memory");
    if (ok) return;
    if ((i & 15) != 15) continue;
    if (*fail) return;
    if (i == 15) t0 = now_ns();
    else if (now_ns() - t0 > kWaitNs) *fail = 1;
  }
}
// What a CTA does last when a wait gave up.  Tiles that nobody took may be on their way: nothing more is asked for
// once the flag is up, so after this time, a thousand times a copy's, they have landed and the shared memory can go.
__device__ __forceinline__ void give_up(int32_t* err) {
  set_error(err, MOE_ETIMEOUT);
  for (const unsigned long long t0 = now_ns(); now_ns() - t0 < kLandNs;) {
  }
}
// A box of 64 columns (or a slot's codes) of a page from its place `tok` on -> dst, counted on b.
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* tm, int col, int tok, int head, int page,
                                         uint64_t* b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(col), "r"(tok), "r"(head), "r"(page), "r"(su32(b))
      : "memory");
}
__device__ __forceinline__ void load_rows(void* dst, const CUtensorMap* tm, int col, int head, int token, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(col), "r"(head), "r"(token), "r"(su32(b))
      : "memory");
}
// The tensor core's instructions are issued by one lane of a converged warp.
__device__ __forceinline__ void commit_to(uint64_t* b) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(su32(b))
      : "memory");
}
// Four steps of 16 along the contracted dimension; the descriptors advance by A and B (16-byte units).
template <int A, int B>
__device__ __forceinline__ void mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "add.u64 a1, %1, %5;\n\tadd.u64 b1, %2, %6;\n\t"
      "add.u64 a2, %1, %7;\n\tadd.u64 b2, %2, %8;\n\t"
      "add.u64 a3, %1, %9;\n\tadd.u64 b3, %2, %10;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "n"(A), "n"(B), "n"(2 * A), "n"(2 * B), "n"(3 * A), "n"(3 * B)
      : "memory");
}
// Steps of 32 E4M3 codes along the contracted dimension, both operands K-major.
template <int STEPS>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
#pragma unroll
  for (int k = 0; k < STEPS; k += 2)
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 a1, b1;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 b1, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, 1;\n\t}" ::"r"(d),
        "l"(a + 2 * k), "l"(b + 2 * k), "r"(idesc), "r"(k > 0 ? 1u : acc)
        : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void ld16(uint32_t t, float* v) {
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
__device__ __forceinline__ void st16(uint32_t t, const float* v) {
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
// Pairs in one instruction: a = a * f - m, and a += x.
__device__ __forceinline__ void scale_sub2(float& a0, float& a1, float f0, float f1, float m0, float m1) {
  asm("{\n\t.reg .b64 a, f, m;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 f, {%2, %3};\n\tmov.b64 m, {%4, %5};\n\t"
      "fma.rn.f32x2 a, a, f, m;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(f0), "f"(f1), "f"(-m0), "f"(-m1));
}
__device__ __forceinline__ void add2(float& a0, float& a1, float x0, float x1) {
  asm("{\n\t.reg .b64 a, x;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, x;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(x0), "f"(x1));
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
// Two values -> two E4M3 codes (low byte first), to nearest even.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four E4M3 codes (low byte first) -> bf16, exact.
__device__ __forceinline__ void e4m3x4_to_bf16x4(uint32_t four, uint32_t* out) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
  const float2 a = f16x2_to_f32x2(lo), b = f16x2_to_f32x2(hi);
  out[0] = pack2(a.x, a.y);
  out[1] = pack2(b.x, b.y);
}

// Shared-memory descriptors (start, leading and stride offsets in 16-byte units, version 1).
__device__ __forceinline__ uint64_t desc(uint32_t start, uint32_t lbo, uint32_t sbo, uint64_t swizzle) {
  return uint64_t((start >> 4) & 0x3FFF) | (uint64_t(lbo >> 4) << 16) | (uint64_t(sbo >> 4) << 32) |
         (uint64_t(1) << 46) | (swizzle << 61);
}

struct PlanShared {
  int4 first;    // the run's first request, key head and row tile, and its first place in their unit
  int tiles[2];  // the call's tiles before the run and before the next one
  int2 scan[32];
};
struct Plan {
  int total, runs, x0, x1, count;  // places and runs of the call; the run's places and tiles
};
// The run: all units of the call, end to end, cut into equal parts.  Called by every thread of the CTA;
// its two barriers also end the CTA's set-up.
template <int V, int THREADS>
__device__ __forceinline__ Plan plan_run(const Args& a, int cap, PlanShared& sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = a.kv.B, per = (B + THREADS - 1) / THREADS;
  int2 mine = make_int2(0, 0);  // places and tiles of this thread's requests
  bool falls = false;           // q_start decreases: the requests could then have more rows than the count has room for
  Req r = {};
  Load ld = {};  // the last of them
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < B) {
      r = load_req(a.kv, b);
      falls |= r.n < 0;
      if (blockIdx.x == 0 && r.n > 0 && r.kv > cap) set_error(a.err, MOE_ERANGE);
      ld = head_load(r, a.tokens, a.window, cap);
      mine.x += a.kv.Hkv * (ld.tiles + V * ld.units);
      mine.y += a.kv.Hkv * ld.tiles;
    }
  }
  int2 before = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const int y0 = __shfl_up_sync(0xffffffffu, before.x, x), y1 = __shfl_up_sync(0xffffffffu, before.y, x);
    if (lane >= x) {
      before.x += y0;
      before.y += y1;
    }
  }
  falls = __any_sync(0xffffffffu, falls);
  if (lane == 31) sh.scan[warp] = falls ? make_int2(INT_MIN, 0) : before;
  before.x -= mine.x;
  before.y -= mine.y;
  tc_before();
  __syncthreads();
  tc_after();
  const int2 sum = lane < THREADS / 32 ? sh.scan[lane] : make_int2(0, 0);
  falls = __any_sync(0xffffffffu, sum.x == INT_MIN);
  if (falls && blockIdx.x == 0 && tid == 0) set_error(a.err, MOE_ERANGE);
  before.x += __reduce_add_sync(0xffffffffu, lane < warp ? sum.x : 0);
  before.y += __reduce_add_sync(0xffffffffu, lane < warp ? sum.y : 0);
  Plan p;
  const int run = blockIdx.x;
  p.total = falls ? 0 : __reduce_add_sync(0xffffffffu, sum.x);
  p.runs = min(int(gridDim.x), p.total);
  p.x0 = run < p.runs ? cut_at(p.total, p.runs, run) : p.total;
  p.x1 = run < p.runs ? cut_at(p.total, p.runs, run + 1) : p.total;
  if (mine.x > 0 && !falls) {  // a cut falls into the requests of one thread
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      int x = (e ? p.x1 : p.x0) - before.x, t = before.y, b = tid * per;
      if (x < 0 || x >= mine.x) continue;
      for (; per > 1; ++b) {
        r = load_req(a.kv, b);
        ld = head_load(r, a.tokens, a.window, cap);
        const int c = a.kv.Hkv * (ld.tiles + V * ld.units);
        if (x < c) break;
        x -= c;
        t += a.kv.Hkv * ld.tiles;
      }
      int4 unit = make_int4(b, 0, 0, 0);
      sh.tiles[e] = t + find_place<V>(a, r, ld, cap, x, &unit);
      if (e == 0) sh.first = unit;
    }
  }
  if (tid == THREADS - 1 && p.x1 == p.total) sh.tiles[1] = before.y + mine.y;
  __syncthreads();
  p.count = run < p.runs ? sh.tiles[1] - sh.tiles[0] : 0;
  return p;
}
// What the join needs of the unit that a run's first piece, begun at tile jbeg, is the second piece of.
template <int V>
__device__ __forceinline__ int4 join_record(const Args& a, const Plan& p, const Walk<V>& w) {
  // the unit's tiles take the places from `at` on; its first piece is the run's that has place `at`
  const int run = blockIdx.x, at = p.x0 - w.jbeg;
  if (w.jbeg == 0 || cut_at(p.total, p.runs, run - 1) > at) return make_int4(0, 0, 0, 0);
  return make_int4(w.r.s0 + w.s.i0, w.h, (w.s.i1 - w.s.i0 + 1) * a.G, run_of(p.total, p.runs, at + w.s.nt - 1) - run + 2);
}

template <int NR>
struct Misc {
  uint64_t full[16], empty[16], kfull[8], kempty[8], rfull[8], rempty[8], factors[2], qfull[2], qfree[2], sfull[2], pfull[2], pvdone[2], ofree[2], drain;
  uint32_t taddr;
  int fail;
  PlanShared plan;
  alignas(16) float m[NR];   // of the rows, log2 units
  alignas(16) float alpha[NR];
  alignas(16) float qf[4][NR];  // E4M3: factors of four pieces' rows (queries run three pieces ahead at most)
  float inv[NR];             // 1 / sum of a finished piece's rows
  float red[4][NR], sum[4][NR];
  int page[2][kKeys];        // pages of a tile's boxes, for keys and for values
  int nbad;
  uint8_t bad[kKeys];  // keys of a tile with values that are not finite
};

// Whether a key's row of N columns in a slot has a value that is not finite: 0 times it is NaN.
template <int N>
__device__ __forceinline__ bool not_finite(const uint8_t* slot, int key) {
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  __nv_bfloat162 t = zero;
#pragma unroll 4
  for (int c = 0; c < N / 8; ++c) {
    const uint4 x = *reinterpret_cast<const uint4*>(slot + (c / 8) * (kKeys * 128) + sw128(key, c % 8));
    t = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), zero, t);
    t = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), zero, t);
    t = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), zero, t);
    t = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), zero, t);
  }
  return __hisnan(t.x) || __hisnan(t.y);
}
// Those values become zeros.
template <int N>
__device__ __forceinline__ void drop_not_finite(uint8_t* slot, int key) {
#pragma unroll 1
  for (int c = 0; c < N; ++c) {
    uint16_t* v = reinterpret_cast<uint16_t*>(slot + (c / 64) * (kKeys * 128) + sw128(key, c % 64 / 8)) + c % 8;
    if ((*v & 0x7f80u) == 0x7f80u) *v = 0;
  }
}

// A place in a ring of N slots.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase;
  __device__ __forceinline__ explicit Ring(uint32_t ph) : phase(ph) {}
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};

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
__global__ void __launch_bounds__(Cfg<D, NR, E4M3>::THREADS, Cfg<D, NR, E4M3>::OCC) k_attn(const __grid_constant__ Args a) {
  using C = Cfg<D, NR, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;                         // keys and values, or values alone
  uint8_t* kring = ring + C::NS * C::SLOT;      // E4M3: keys
  uint8_t* raw = kring + C::NK * C::RAW;        // E4M3: values as they come
  uint8_t* sq = raw + C::NRAW * C::RAW;
  uint8_t* sp = sq + C::QB * C::QBYTES;
  using Ms = Misc<NR>;
  static_assert(sizeof(Ms) <= misc_bytes(NR), "misc");
  Ms& ms = *reinterpret_cast<Ms*>(sp + 2 * C::PBYTES);
  volatile int* fail = &ms.fail;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  constexpr int kMmaWarp = C::SW, kLoadWarp = C::SW + 1, kSoft = 32 * C::SW;  // loads: keys, then values

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&ms.taddr)),
                 "n"(C::COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    // not before: a kernel further on that takes tensor memory too could hold what this one waits for
    pdl_trigger();
  } else if (tid == 32 * kLoadWarp) {
    for (int i = 0; i < C::NS; ++i) {
      bar_init(&ms.full[i], E4M3 ? C::CV : 1);
      bar_init(&ms.empty[i], 1 + (a.phantom == 3));
    }
    for (int i = 0; i < C::NK; ++i) {
      bar_init(&ms.kfull[i], 1);
      bar_init(&ms.kempty[i], 1 + (a.phantom == 3));
    }
    for (int i = 0; i < C::NRAW; ++i) {
      bar_init(&ms.rfull[i], 1);
      bar_init(&ms.rempty[i], C::CV);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&ms.qfull[i], (E4M3 ? C::CV : 1) + (a.phantom == 1));
      bar_init(&ms.qfree[i], 1);
      bar_init(&ms.factors[i], 1);
      bar_init(&ms.sfull[i], 1);
      bar_init(&ms.pfull[i], C::SW + (a.phantom == 2));
      bar_init(&ms.pvdone[i], 1);
      bar_init(&ms.ofree[i], C::SW);
    }
    bar_init(&ms.drain, 1);
    for (const CUtensorMap* m : {&a.mk, &a.mv, &a.mq})
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    ms.fail = 0;
    ms.nbad = 0;
  }
  pdl_wait();

  constexpr int V = C::V;
  const int cap = cap_of(a.kv);
  const Plan plan = plan_run<V, C::THREADS>(a, cap, ms.plan);
  const uint32_t taddr = ms.taddr;
  const int run = blockIdx.x, count = plan.count;
  if (count == 0 && tid == 0) a.join[run] = make_int4(0, 0, 0, 0);

  if (count > 0) {
    Walk<V> w;
    w.start(a, cap, ms.plan.first, plan.x1 - plan.x0);
    if (warp == kMmaWarp) {
      // -------------------------------------------------------- tensor cores
      // D f32, A and B bf16, N = NR, M = 128; the second product's operands are both MN-major
      constexpr uint32_t kBase = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(NR >> 3) << 17) | (8u << 24);
      constexpr uint32_t kIdescS = kBase, kIdescO = kBase | (1u << 15) | (1u << 16);
      constexpr uint32_t kIdescQ = (1u << 4) | (uint32_t(C::SN >> 3) << 17) | (8u << 24);  // E4M3 both, N = 2 NR
      Ring<E4M3 ? C::NK : 1> kr(0);
      Ring<C::NS> rg(0);
      int qn = -1;             // pieces begun, less one
      int pieces = -1;         // pieces whose O has been begun, less one
      bool first_prev = false;
      for (int n = 0; n <= count; ++n) {
        bool first = false;
        if (n < count) {
          // S^T(n) = K(n) Q^T
          first = w.j == w.jbeg;
          if (first) {
            ++qn;
            wait(&ms.qfull[qn % C::QB], (qn / C::QB) & 1, fail);
            if (E4M3 && lane == 0) arrive(&ms.factors[qn & 1]);
            __syncwarp();
          }
          const uint32_t d = taddr + uint32_t(n & 1) * C::SN;
          // rows of 128 bytes, swizzled so; 64 codes make 64
          constexpr bool k64 = E4M3 && C::DS == 64;
          const uint64_t qd = desc(su32(sq + (qn % C::QB) * C::QBYTES), 16, k64 ? 512 : 1024, k64 ? 4 : 2);
#pragma unroll
          for (int hh = 0; hh < C::H; ++hh) {
            if constexpr (E4M3) {
              wait(&ms.kfull[kr.slot], kr.phase, fail);
              tc_after();
              mma_e4m3<C::DS / 32>(d, desc(su32(kring + kr.slot * C::RAW), 16, k64 ? 512 : 1024, k64 ? 4 : 2),
                                   qd + hh * (C::SN * C::DS >> 4), kIdescQ, hh > 0);
              commit_to(&ms.kempty[kr.slot]);
              kr.next();
              continue;
            }
            wait(&ms.full[rg.slot], rg.phase, fail);
            tc_after();
            const uint64_t kd = desc(su32(ring + rg.slot * C::SLOT), 16, 1024, 2);
#pragma unroll
            for (int k = 0; k < C::DS / 64; ++k)
              mma4<2, 2>(d, kd + k * (kKeys * 128 >> 4), qd + (hh * (C::DS / 64) + k) * (NR * 128 >> 4), kIdescS,
                         hh + k > 0);
            commit_to(&ms.empty[rg.slot]);
            rg.next();
          }
          commit_to(&ms.sfull[n & 1]);
          if (w.j + 1 == w.jend) commit_to(&ms.qfree[qn % C::QB]);
        }
        if (n > 0) {
          // O^T += V(n-1)^T P(n-1)^T
          const int p = (n - 1) & 1;
          wait(&ms.pfull[p], ((n - 1) >> 1) & 1, fail);
          if (first_prev) {
            ++pieces;
            if (pieces >= 2) wait(&ms.ofree[pieces & 1], ((pieces >> 1) - 1) & 1, fail);
          }
          const uint32_t od = taddr + uint32_t(2 * C::SN + (pieces & 1) * C::H * NR);
          const uint64_t pd = desc(su32(sp + p * C::PBYTES), 128, 2048, 0);
#pragma unroll
          for (int hh = 0; hh < C::H; ++hh) {
            wait(&ms.full[rg.slot], rg.phase, fail);
            tc_after();
            // D = 64: the upper 64 rows of M read the same columns again and are not used
            const uint64_t vd = desc(su32(ring + rg.slot * C::SLOT), D < 128 ? 0 : kKeys * 128, 1024, 2);
#pragma unroll
            for (int k = 0; k < kKeys / 64; ++k)
              mma4<128, 16>(od + uint32_t(hh) * NR, vd + k * 512, pd + k * 64, kIdescO, !first_prev || k > 0);
            commit_to(&ms.empty[rg.slot]);
            rg.next();
          }
          commit_to(&ms.pvdone[p]);
        }
        first_prev = first;
        if (n + 1 < count) w.next(a, cap);
      }
      commit_to(&ms.drain);
      const unsigned long long t0 = now_ns();
      for (uint32_t ok = 0; !ok && now_ns() - t0 < 2 * kWaitNs;)
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], 0;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(su32(&ms.drain))
            : "memory");
    } else if (warp == kLoadWarp || warp == kLoadWarp + 1) {
      // -------------------------------------------------------- loads
      // In the ring, as the products take them: K(0) K(1) V(0) K(2) V(1) .. K(last) V(last - 1) V(last).
      const bool keys = warp == kLoadWarp;
      const KvView& kv = a.kv;
      const int box_shift = min(kv.page_shift, 7), boxes = kKeys >> box_shift;  // keys in a box, boxes in a tile
      const CUtensorMap* tm = keys ? &a.mk : &a.mv;
      int* page = ms.page[keys ? 0 : 1];
      // pages of a tile's boxes: up to four a lane
      int id[4];
      auto find = [&]() {
        const int32_t* row = kv.page_table + (long long)w.b * kv.table_stride;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = lane + 32 * i, key = (w.s.tile0 + w.j) * kKeys + (x << box_shift);
          id[i] = -2;
          if (x < boxes && key < w.s.hi && key + (1 << box_shift) > w.s.lo) id[i] = row[key >> kv.page_shift];
        }
      };
      Ring<C::NS> rg(1);  // a fresh slot is empty
      Ring<E4M3 ? C::NK : 1> kr(1);
      Ring<E4M3 ? C::NRAW : 1> rr(1);
      auto skip = [&]() {
#pragma unroll
        for (int hh = 0; hh < C::H; ++hh) rg.next();
      };
      int qn = -1;
      find();
      if (!keys) {
        skip();
        if (count > 1) skip();
      }
#pragma unroll 1
      for (int n = 0; n < count; ++n) {
        if (!E4M3 && keys && w.j == w.jbeg) {
          ++qn;
          if (qn >= C::QB) wait(&ms.qfree[qn % C::QB], (qn / C::QB - 1) & 1, fail);
          if (lane == 0 && !*fail) {
            uint64_t* b = &ms.qfull[qn % C::QB];
            expect(b, uint32_t(a.tokens * a.G * D * 2));
            for (int c = 0; c < D / 64; ++c)
              load_rows(sq + (qn % C::QB) * C::QBYTES + c * (NR * 128), &a.mq, c * 64, w.h * a.G, w.r.s0 + w.s.i0, b);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = lane + 32 * i;
          if (x < boxes) {
            const bool ok = id[i] >= 0 && id[i] < kv.npages;
            if (!ok && id[i] != -2) set_error(a.err, MOE_ERANGE);
            page[x] = ok ? id[i] : kv.npages;  // past the end: zeros
          }
        }
        __syncwarp();
        const int h = w.h, tok = ((w.s.tile0 + w.j) * kKeys) & ((1 << kv.page_shift) - 1);  // of a page larger than a tile
        if (n + 1 < count) {
          w.next(a, cap);
          find();  // on their way while this tile is asked for
        }
#pragma unroll 1
        for (int hh = 0; hh < C::H; ++hh) {
          // E4M3: keys and values have rings of their own
          const int slot = !E4M3 ? rg.slot : keys ? kr.slot : rr.slot;
          uint64_t* full = (!E4M3 ? ms.full : keys ? ms.kfull : ms.rfull) + slot;
          wait((!E4M3 ? ms.empty : keys ? ms.kempty : ms.rempty) + slot, !E4M3 ? rg.phase : keys ? kr.phase : rr.phase, fail);
          if (__any_sync(0xffffffffu, *fail)) break;  // for the warp: its lanes meet below
          if (lane == 0) expect(full, E4M3 ? C::RAW : C::SLOT);
          __syncwarp();
          constexpr int CHUNKS = E4M3 ? 1 : C::DS / 64;
#pragma unroll 1
          for (int x = lane; x < boxes * CHUNKS; x += 32) {
            const int p = x & (boxes - 1), c = x >> (7 - box_shift);
            uint8_t* dst = E4M3 ? (keys ? kring : raw) + slot * C::RAW + (p << box_shift) * C::DS
                                : ring + slot * C::SLOT + c * (kKeys * 128) + (p << box_shift) * 128;
            load_box(dst, tm, hh * C::DS + c * 64, tok, h, page[p], full);
          }
          __syncwarp();
          if (!E4M3) rg.next();
          else if (keys) kr.next();
          else rr.next();
        }
        if (!E4M3 && (keys ? n > 0 : n + 2 != count)) skip();
      }
    } else if (warp > kLoadWarp + 1) {
      // -------------------------------------------------------- E4M3 codes -> bf16
      if constexpr (E4M3) {
        const int vw = warp - kLoadWarp - 2, vt = vw * 32 + lane;
        constexpr int CH = C::DS / 8, STEP = 32 * C::CV / CH;  // 8 codes a thread make one 16-byte piece
        const int r0 = vt / CH, c = vt % CH;
        Ring<C::NRAW> in(0);
        Ring<C::NS> out(1);
        int qn = -1;
        // The rows of a piece as two terms, a warp a row, and the factors of their scores.
        auto queries = [&](const Walk<V>& k) {
          ++qn;
          if (qn >= C::QB) wait(&ms.qfree[qn % C::QB], (qn / C::QB - 1) & 1, fail);
          // eight columns a thread: L threads a row, `AT` rows at a time
          constexpr int L = D / 8, AT = 32 * C::CV / L, STEPS = (NR + AT - 1) / AT, AHEAD = STEPS < 4 ? STEPS : 4;
          const int rows = (k.s.i1 - k.s.i0 + 1) * a.G, at = vt % L * 8;
          const float base = a.scale * 1.4426950408889634f * (a.kv.k_scale ? a.kv.k_scale[k.h] : 1.f);
          const uint16_t* src = a.q + (long long)(k.r.s0 + k.s.i0) * a.qs + (long long)k.h * a.G * D + at;
          uint8_t* dst = sq + (qn % C::QB) * C::QBYTES + at / C::DS * (C::SN * C::DS) + at % 16;
          auto load = [&](int r) {
            const int i = r / a.G;
            return r < rows ? *reinterpret_cast<const uint4*>(src + i * a.qs + (r - i * a.G) * D) : make_uint4(0, 0, 0, 0);
          };
          int r = vt / L;
          uint4 u[AHEAD];
#pragma unroll
          for (int y = 0; y < AHEAD; ++y) u[y] = load(r + y * AT);
#pragma unroll 1
          for (; r < NR; r += AT) {
            const uint32_t w4[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int y = 0; y + 1 < AHEAD; ++y) u[y] = u[y + 1];
            if constexpr (STEPS > AHEAD) u[AHEAD - 1] = load(r + AHEAD * AT);
            float f[8], most = 0.f;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              f[x] = __uint_as_float(x & 1 ? w4[x / 2] & 0xffff0000u : w4[x / 2] << 16);
              most = fmaxf(most, fabsf(f[x]));
            }
#pragma unroll
            for (int x = 1; x < L; x <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
            const uint32_t e = __float_as_uint(most) >> 23;
            const float up = __uint_as_float(min(261u - e, 237u) << 23);  // the largest in [2^7, 2^8)
            if (at == 0) ms.qf[qn & 3][r] = base / up;
            uint32_t t[2][4];
#pragma unroll
            for (int x = 0; x < 8; x += 2) {
              // an infinity becomes NaN, as its scores' softmax would be
              const float v0 = fabsf(f[x]) < INFINITY ? f[x] * up : NAN, v1 = fabsf(f[x + 1]) < INFINITY ? f[x + 1] * up : NAN;
              t[0][x / 2] = e4m3x2(v0, v1);
              const float2 b = f16x2_to_f32x2(e4m3x2_to_f16x2(uint16_t(t[0][x / 2])));
              t[1][x / 2] = e4m3x2((v0 - b.x) * 32.f, (v1 - b.y) * 32.f);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int row = z * NR + r;
              *reinterpret_cast<uint2*>(dst + (C::DS == 64 ? sw64(row, at % C::DS / 16) : sw128(row, at % C::DS / 16))) =
                  make_uint2(t[z][0] | t[z][1] << 16, t[z][2] | t[z][3] << 16);
            }
          }
          proxy_fence();
          __syncwarp();
          if (lane == 0) arrive(&ms.qfull[qn % C::QB]);
        };
        queries(w);
#pragma unroll 1
        for (int n = 0; n < count; ++n) {
          if (n + 1 < count) {
            w.next(a, cap);
            if (w.j == w.jbeg) queries(w);  // before this tile's values: S of the next tile comes first
          }
#pragma unroll 1
          for (int hh = 0; hh < C::H; ++hh) {
            wait(&ms.rfull[in.slot], in.phase, fail);
            wait(&ms.empty[out.slot], out.phase, fail);
            const uint8_t* src = raw + in.slot * C::RAW + c * 8;
            uint8_t* dst = ring + out.slot * C::SLOT + (c / 8) * (kKeys * 128);
#pragma unroll 4
            for (int i = 0; i < kKeys / STEP; ++i) {
              const uint2 v = *reinterpret_cast<const uint2*>(src + (r0 + i * STEP) * C::DS);
              uint32_t o[4];
              e4m3x4_to_bf16x4(v.x, o);
              e4m3x4_to_bf16x4(v.y, o + 2);
              *reinterpret_cast<uint4*>(dst + sw128(r0 + i * STEP, c % 8)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            proxy_fence();
            __syncwarp();
            if (lane == 0) {
              arrive(&ms.full[out.slot]);
              arrive(&ms.rempty[in.slot]);
            }
            in.next();
            out.next();
          }
        }
      }
    } else {
      // -------------------------------------------------------- softmax
      constexpr int CW = C::CW, CK = CW == 16 || E4M3 ? 16 : 32;  // rows of a warp, and at a time
      const int quad = warp & 3, c0 = (warp >> 2) * CW;
      const int krow = quad * 32 + lane;  // this thread's key in a tile, and its column of v
      const uint32_t tl = taddr + (uint32_t(quad * 32) << 16);
      float l[CW];
      float factor = 0.f, v_factor = 1.f;  // of the scores, in log2 units, and of the values
      // a finished piece whose O is still to be written
      int piece = -1, d_token = 0, d_head = 0, d_rows = 0, d_part = -1;
      bool pending = false;
      int newest = 0, oldest = 0, whole0 = 0, whole1 = 0;
      if (tid == 0) a.join[run] = join_record<V>(a, plan, w);
      // Rows x0 .. x0 + CK - 1 of tile n (p = n & 1): scores in log2 units, less m where asked.
      auto scores = [&](int p, int x0, float* s, bool less_m) {
#pragma unroll
        for (int i = 0; i < CK; i += 16) ld16(tl + p * C::SN + c0 + x0 + i, s + i);
        float second[E4M3 ? CK : 1];
        if constexpr (E4M3) {
#pragma unroll
          for (int i = 0; i < CK; i += 16) ld16(tl + p * C::SN + NR + c0 + x0 + i, second + i);
        }
        ld_wait();
#pragma unroll
        for (int x = 0; x < CK; x += 4) {
          float4 m = make_float4(0.f, 0.f, 0.f, 0.f), f = make_float4(factor, factor, factor, factor);
          if (less_m) m = *reinterpret_cast<const float4*>(&ms.m[c0 + x0 + x]);
          if constexpr (E4M3) {
            f = *reinterpret_cast<const float4*>(&ms.qf[piece & 3][c0 + x0 + x]);
#pragma unroll
            for (int y = 0; y < 4; ++y) s[x + y] = fmaf(second[x + y], 0x1p-5f, s[x + y]);
          }
          scale_sub2(s[x], s[x + 1], f.x, f.y, m.x, m.y);
          scale_sub2(s[x + 2], s[x + 3], f.z, f.w, m.z, m.w);
        }
      };
      // Weights of the tile, in bf16 for the product and into the sums; true when a score passes m by
      // kGrow.  hide: sets hidden scores to -inf.  sums: 0 where m was given up as too small, 1 everywhere.
      auto weights = [&](int p, auto hide, bool sums) {
        uint8_t* dst = sp + p * C::PBYTES + (krow >> 3) * 128 + (krow & 7) * 16;
        __nv_bfloat162 most = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
        for (int x0 = 0; x0 < CW; x0 += CK) {
          float s[CK];
          scores(p, x0, s, true);
          hide(x0, s);
#pragma unroll
          for (int x = 0; x < CK; x += 8) {
            uint32_t u[4];
#pragma unroll
            for (int y = 0; y < 8; y += 2) {
              const float e0 = ex2(s[x + y]), e1 = ex2(s[x + y + 1]);
              if (sums) {
                add2(l[x0 + x + y], l[x0 + x + y + 1], e0, e1);
              } else {
                if (ms.alpha[c0 + x0 + x + y] <= kLost) l[x0 + x + y] += e0;
                if (ms.alpha[c0 + x0 + x + y + 1] <= kLost) l[x0 + x + y + 1] += e1;
              }
              u[y / 2] = pack2(e0, e1);
              most = __hmax2(most, *reinterpret_cast<const __nv_bfloat162*>(&u[y / 2]));
            }
            *reinterpret_cast<uint4*>(dst + ((c0 + x0 + x) >> 3) * 2048) = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
        return fmaxf(__low2float(most), __high2float(most)) > kMost;
      };
      // S of tile n is there and P(n - 2) has been read.
      auto ready = [&](int n) {
        wait(&ms.sfull[n & 1], (n >> 1) & 1, fail);
        tc_after();
        if (n >= 2) wait(&ms.pvdone[n & 1], ((n - 2) >> 1) & 1, fail);
      };
#pragma unroll 1
      for (int n = 0; n <= count; ++n) {
        bool over = false;
        if (n < count && !pending && w.j > w.jbeg) {
          // Tiles inside a piece of which every row sees every key, with the m there is; it holds for all
          // but a few.  A loop of its own: the code of all that a tile may need beside this is far apart,
          // and fetching past it cost 600 clocks a tile (E4M3, 64 columns: 60.1 us, 46.9 so).
          const int to = min(w.jend - 1, whole1);
          if (w.j >= whole0) {
#pragma unroll 1
            for (; w.j < to; ++w.j, ++n) {
              ready(n);
              const bool high = weights(n & 1, [](int, float*) {}, true);
              proxy_fence();
              over = vote_any<kSoft>(high);
              if (over) break;
              tc_before();
              __syncwarp();
              if (lane == 0) arrive(&ms.pfull[n & 1]);
            }
          }
        }
        const int p = n & 1;
        const uint32_t ph = (n >> 1) & 1;
        if (n < count) {
          const bool first = w.j == w.jbeg;
          if (first) {
            ++piece;
#pragma unroll
            for (int i = 0; i < CW; ++i) l[i] = 0.f;
            factor = a.scale * 1.4426950408889634f;
            if (E4M3 && a.kv.v_scale) v_factor = a.kv.v_scale[w.h];
            if (E4M3) wait(&ms.factors[piece & 1], (piece >> 1) & 1, fail);
            // the row tile's tokens; the tiles of which every row sees every key
            newest = w.r.pos0 + w.s.i1, oldest = w.r.pos0 + w.s.i0;
            whole1 = max(min(oldest + 1, cap), 0) / kKeys - w.s.tile0;
            whole0 = a.window > 0 ? max(newest - a.window + kKeys, 0) / kKeys - w.s.tile0 : 0;
          }
          const uint32_t to = tl + uint32_t(2 * C::SN + (piece & 1) * C::H * NR);  // O of this piece
          const int key0 = (w.s.tile0 + w.j) * kKeys, key = key0 + krow;
          const bool whole = w.j >= whole0 && w.j < whole1;
          auto hide = [&](int x0, float* s) {
            if (whole) return;
            // rows are in the order of their tokens: rows from .. to - 1 see this key
            const int i_from = max(key - oldest, 0), i_to = a.window > 0 ? key - oldest + a.window : a.tokens;
            const int from = key >= cap || i_from > a.tokens ? INT_MAX : i_from * a.G;
            const int to_row = i_to >= a.tokens ? INT_MAX : i_to * a.G;
#pragma unroll
            for (int x = 0; x < CK; ++x)
              if (c0 + x0 + x < from || c0 + x0 + x >= to_row) s[x] = -INFINITY;
          };
          ready(n);
          bool set = first || over;
#pragma unroll 1
          for (bool again = set;; again = true) {
            if (again) {
              // set m: the rows' maxima over the 128 keys
#pragma unroll
              for (int x0 = 0; x0 < CW; x0 += CK) {
                float s[CK];
                scores(p, x0, s, false);
                hide(x0, s);
#pragma unroll
                for (int x = 0; x < CK; ++x) {
                  const float v = warp_max(s[x]);
                  if (lane == x) ms.red[quad][c0 + x0 + x] = v;
                }
              }
              softmax_sync<kSoft>();
              if (tid < NR) {
                const float old = first ? kUnset : ms.m[tid];
                const float v = fmaxf(fmaxf(fmaxf(ms.red[0][tid], ms.red[1][tid]), fmaxf(ms.red[2][tid], ms.red[3][tid])), old);
                // Rows past the unit's own are another request's, or what shared memory held: their weights are
                // nothing, whatever they score, so they never ask for a new m of the rows beside them.
                const bool own = tid < (w.s.i1 - w.s.i0 + 1) * a.G;
                ms.m[tid] = own ? v : INFINITY;
                ms.alpha[tid] = own ? ex2(old - v) : 1.f;
              }
              softmax_sync<kSoft>();
              if (!first) {
                // The sums hold this tile's weights against the old m already.  Where m grew by so much
                // that those may have overflowed, what was there before them is nothing against them.
#pragma unroll
                for (int x = 0; x < CW; ++x) l[x] = ms.alpha[c0 + x] > kLost ? l[x] * ms.alpha[c0 + x] : 0.f;
                wait(&ms.pvdone[p ^ 1], ((n - 1) >> 1) & 1, fail);
                tc_after();
#pragma unroll 1
                for (int x = 0; x < C::H * CW; x += 16) {
                  const int hh = x / CW, y0 = x % CW;
                  float o[16];
                  ld16(to + hh * NR + c0 + y0, o);
                  ld_wait();
#pragma unroll
                  for (int y = 0; y < 16; ++y) o[y] *= ms.alpha[c0 + y0 + y];
                  st16(to + hh * NR + c0 + y0, o);
                }
                st_wait();
              }
            }
            const bool high = weights(p, hide, first || !again);
            if (again) break;
            if (whole) proxy_fence();
            set = vote_any<kSoft>(high);
            if (!set) break;
          }
          // Values at hidden keys may hold anything, and 0 times what is not finite is NaN.  Those that
          // no row sees become zeros; where some rows see a key and some do not, values that are not
          // finite are taken out of the tile and added to the rows that do see them.
          bool spoiled = false;
          if (!whole) {
            const bool gone = key < w.s.lo || key >= w.s.hi, mixed = w.s.i1 > w.s.i0;
            const bool some = !gone && mixed && (key > oldest || (a.window > 0 && key <= newest - a.window));
            const int at = (E4M3 ? n : n + 1 == count ? 2 * count - 1 : 2 * n + 2) * C::H;  // V(n)'s place in the ring's order
            bool bad = false;
            // V(n)'s slots may still be held by V(n - 1), or in a ring for both by K(n + 1): see those filled
            // first, so that the slots' phases tell V(n)'s.  With more slots it was an older tile.
            if (C::NS < (E4M3 ? 2 : 3) * C::H && n >= 1) wait(&ms.pvdone[p ^ 1], ((n - 1) >> 1) & 1, fail);
            if (!E4M3 && C::NS < 3 * C::H && n + 1 < count) wait(&ms.sfull[p ^ 1], ((n + 1) >> 1) & 1, fail);
#pragma unroll 1
            for (int hh = 0; hh < C::H; ++hh) {
              const int slot = (at + hh) % C::NS;
              wait(&ms.full[slot], uint32_t((at + hh) / C::NS) & 1, fail);
              if (c0 > 0 || !(gone || some)) continue;
              uint8_t* row = ring + slot * C::SLOT;
              if (gone) {
#pragma unroll 4
                for (int c = 0; c < C::DS / 8; ++c)
                  *reinterpret_cast<uint4*>(row + (c / 8) * (kKeys * 128) + sw128(krow, c % 8)) = make_uint4(0, 0, 0, 0);
              } else if (not_finite<C::DS>(row, krow)) {
                bad = true;
                drop_not_finite<C::DS>(row, krow);
              }
            }
            if (mixed) {
              if (bad) ms.bad[atomicAdd(&ms.nbad, 1)] = uint8_t(krow);
              spoiled = vote_any<kSoft>(bad);
            }
          }
          if (!whole || set) proxy_fence();
          tc_before();
          __syncwarp();
          if (lane == 0) arrive(&ms.pfull[p]);
          if (spoiled) {
            wait(&ms.pvdone[p], ph, fail);
            tc_after();
            const int nbad = *const_cast<volatile int*>(&ms.nbad);
#pragma unroll 1
            for (int e = 0; e < nbad * C::H; ++e) {
              const int k = key0 + ms.bad[e / C::H], hh = e % C::H, col = hh * 128 + krow;
              const int id = a.kv.page_table[(long long)w.b * a.kv.table_stride + (k >> a.kv.page_shift)];
              const uint8_t* v = a.kv.v + id * a.kv.page_stride + w.h * a.kv.head_stride +
                                 (long long)(k & ((1 << a.kv.page_shift) - 1)) * a.kv.tok_stride;
              float add = 0.f;
              // pages that are not there read as zeros, also where a wait gave up and the slot holds something else
              if (col < D && id >= 0 && id < a.kv.npages) {
                if (E4M3) add = f16x2_to_f32x2(e4m3x2_to_f16x2(v[col])).x;
                else add = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(v)[col]);
              }
              if (isfinite(add)) add = 0.f;
#pragma unroll 1
              for (int x = 0; x < CW; x += 16) {
                float o[16];
                ld16(to + hh * NR + c0 + x, o);
                ld_wait();
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                  const int pos = oldest + (c0 + x + y) / a.G;
                  if (k <= pos && (a.window <= 0 || k > pos - a.window)) o[y] += add;
                }
                st16(to + hh * NR + c0 + x, o);
              }
            }
            st_wait();
            tc_before();
            softmax_sync<kSoft>();
            if (tid == 0) ms.nbad = 0;
          }
        }
        if (pending) {
          // ---- O of the piece that ended with tile n - 1: its last product ran beside this tile's softmax
          wait(&ms.pvdone[p ^ 1], ((n - 1) >> 1) & 1, fail);
          tc_after();
          const int d_piece = n < count ? piece - 1 : piece;
          const uint32_t from = tl + uint32_t(2 * C::SN + (d_piece & 1) * C::H * NR);
#pragma unroll 1
          for (int x = 0; x < C::H * CW; x += 16) {
            const int hh = x / CW, row0 = c0 + x % CW, col = hh * 128 + krow;
            if (row0 >= d_rows) continue;
            float o[16];
            ld16(from + hh * NR + row0, o);
            ld_wait();
            if (d_part >= 0) {
              float* out = a.part + ((long long)d_part * NR + row0) * D + col;
#pragma unroll
              for (int y = 0; y < 16; ++y)
                if (row0 + y < d_rows && col < D) out[y * D] = o[y];
            } else {
              const int i = row0 / a.G;
              int g = row0 - i * a.G;
              uint16_t* out = a.o + (long long)(d_token + i) * a.os + (long long)(d_head * a.G + g) * D + col;
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                // a sum of zero is a row that sees no key; its O is zeros
                if (row0 + y < d_rows && col < D) *out = __bfloat16_as_ushort(__float2bfloat16_rn(o[y] * ms.inv[row0 + y]));
                out += D;
                if (++g == a.G) {
                  g = 0;
                  out += a.os - (long long)a.G * D;
                }
              }
            }
          }
          tc_before();
          __syncwarp();
          if (lane == 0) arrive(&ms.ofree[d_piece & 1]);
          pending = false;
        }
        if (n < count) {
          if (w.j + 1 == w.jend) {
            // ---- the piece is done: its rows' sums
#pragma unroll
            for (int x = 0; x < CW; x += 16) {
              float v[16];
#pragma unroll
              for (int y = 0; y < 16; ++y) v[y] = l[x + y];
              float t = transpose_sum<16>(v, lane);
              t += __shfl_xor_sync(0xffffffffu, t, 16);
              if (lane < 16) ms.sum[quad][c0 + x + lane] = t;
            }
            softmax_sync<kSoft>();
            const bool head = w.jbeg > 0, split = head || w.jend < w.s.nt;
            d_token = w.r.s0 + w.s.i0;
            d_head = w.h;
            d_rows = (w.s.i1 - w.s.i0 + 1) * a.G;
            d_part = split ? 2 * run + (head ? 0 : 1) : -1;
            pending = true;
            if (tid < NR) {
              const float t = ms.sum[0][tid] + ms.sum[1][tid] + ms.sum[2][tid] + ms.sum[3][tid];
              if (split && tid < d_rows)
                reinterpret_cast<float2*>(a.ml)[(long long)d_part * NR + tid] = make_float2(ms.m[tid], t);
              ms.inv[tid] = t == 0.f ? 0.f : v_factor / t;
            }
            // read after the two waits of the next piece's first tile
            if (n + 1 == count) softmax_sync<kSoft>();
          }
          if (n + 1 < count) w.next(a, cap);
        }
      }
    }
  }
  __syncthreads();
  if (tid == 0 && *fail) give_up(a.err);
  if (warp == kMmaWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(C::COLS));
  }
}

// Joins the pieces of a unit: o = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k, in the order of
// the pieces.  CTA (c, y): the unit whose second piece is run c's first.  A warp takes R rows and P
// pieces of each at a time (R P = 8 loads of 16 bytes in flight a lane), so no warp waits for another:
// a CTA a row took 33 us for prompt chunks' 128 rows of 152 units, a row a warp 9.
constexpr int kJoinThreads = 128;
constexpr int join_y(int nr) { return nr > 64 ? 16 : nr > 32 ? 8 : nr / 4; }

template <int D, int NR, int R>
__device__ __forceinline__ void join_rows(const Args& a, const int4& unit, int row0) {
  constexpr int L = D / 4, P = 8 / R, C = (L + 31) / 32;  // four columns a lane
  const int c = blockIdx.x, lane = threadIdx.x & 31, rows = unit.z, np = unit.w;
  // pieces: the tail of run c - 1, then the heads of np - 1 runs
  auto place = [&](int k) { return (2ll * (c - 1 + k) + (k == 0 ? 1 : 0)) * NR; };
  const float2* ml = reinterpret_cast<const float2*>(a.ml);
  float m[R], l[R];
  float4 o[R][C];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = kUnset;
    l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) o[r][i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row0 + r < rows)
      for (int k = lane; k < np; k += 32) m[r] = fmaxf(m[r], __ldcg(&ml[place(k) + row0 + r]).x);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) m[r] = warp_max(m[r]);
  for (int k0 = 0; k0 < np; k0 += P) {
    float2 mine[R];  // of piece k0 + lane
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mine[r] = make_float2(kUnset, 0.f);
      if (lane < P && k0 + lane < np && row0 + r < rows) mine[r] = __ldcg(&ml[place(k0 + lane) + row0 + r]);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = i * 32 + lane;
      float4 v[R][P];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < P; ++k)
          if (k0 + k < np && col < L && row0 + r < rows)
            v[r][k] = __ldcg(reinterpret_cast<const float4*>(a.part + (place(k0 + k) + row0 + r) * D) + col);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float w = ex2(mine[r].x - m[r]);
#pragma unroll
        for (int k = 0; k < P; ++k)
          if (k0 + k < np && row0 + r < rows) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            if (i == 0) l[r] = fmaf(wk, __shfl_sync(0xffffffffu, mine[r].y, k), l[r]);
            if (col < L) {
              o[r][i].x = fmaf(wk, v[r][k].x, o[r][i].x);
              o[r][i].y = fmaf(wk, v[r][k].y, o[r][i].y);
              o[r][i].z = fmaf(wk, v[r][k].z, o[r][i].z);
              o[r][i].w = fmaf(wk, v[r][k].w, o[r][i].w);
            }
          }
      }
    }
  }
  const float vs = a.kv.v_scale ? a.kv.v_scale[unit.y] : 1.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (row0 + r >= rows) break;
    const float x = l[r] == 0.f ? 0.f : vs / l[r];
    const int i = (row0 + r) / a.G, g = row0 + r - i * a.G;
    uint16_t* out = a.o + (long long)(unit.x + i) * a.os + (long long)(unit.y * a.G + g) * D;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int col = j * 32 + lane;
      if (col < L)
        reinterpret_cast<uint2*>(out)[col] =
            make_uint2(pack2(o[r][j].x * x, o[r][j].y * x), pack2(o[r][j].z * x, o[r][j].w * x));
    }
  }
}

template <int D, int NR>
__global__ void __launch_bounds__(kJoinThreads) k_join(const __grid_constant__ Args a) {
  constexpr int W = join_y(NR) * kJoinThreads / 32;  // warps of a unit
  pdl_trigger();
  pdl_wait();
  const int4 unit = __ldcg(a.join + blockIdx.x);
  const int first = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5);
  if (NR > W && unit.w <= 2) {  // more rows than warps, and few pieces
    constexpr int R = NR / W > 4 ? 4 : NR / W;
    for (int row = R * first; row < unit.z; row += R * W) join_rows<D, NR, R>(a, unit, row);
  } else {
    for (int row = first; row < unit.z; row += W) join_rows<D, NR, 1>(a, unit, row);
  }
}

// The same for 16-row tiles and units of many pieces: a CTA takes a row, its warps take eight pieces in
// turn and the first adds up what they found.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) k_join_many(const __grid_constant__ Args a) {
  constexpr int L = D / 4, W = kJoinThreads / 32, P = 8, C = (L + 31) / 32, NR = 16;
  __shared__ float4 acc[W][L];
  __shared__ float2 stat[W];
  pdl_trigger();
  pdl_wait();
  const int4 unit = __ldcg(a.join + blockIdx.x);
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, np = unit.w;
  for (int row = blockIdx.y; row < unit.z; row += gridDim.y) {
    auto place = [&](int k) { return (2ll * (c - 1 + k) + (k == 0 ? 1 : 0)) * NR + row; };
    const float2* ml = reinterpret_cast<const float2*>(a.ml);
    float m = kUnset, l = 0.f;  // of this warp's pieces
    float4 o[C];
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = P * warp; k0 < np; k0 += P * W) {
      float2 mine = make_float2(kUnset, 0.f);
      if (lane < P && k0 + lane < np) mine = __ldcg(&ml[place(k0 + lane)]);
      float4 v[C][P];
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int k = 0; k < P; ++k)
          if (k0 + k < np && i * 32 + lane < L)
            v[i][k] = __ldcg(reinterpret_cast<const float4*>(a.part + place(k0 + k) * D) + i * 32 + lane);
      const float top = fmaxf(m, warp_max(mine.x)), keep = ex2(m - top), w = ex2(mine.x - top);
      m = top;
      l *= keep;
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] = make_float4(o[i].x * keep, o[i].y * keep, o[i].z * keep, o[i].w * keep);
#pragma unroll
      for (int k = 0; k < P; ++k)
        if (k0 + k < np) {
          const float wk = __shfl_sync(0xffffffffu, w, k);
          l = fmaf(wk, __shfl_sync(0xffffffffu, mine.y, k), l);
#pragma unroll
          for (int i = 0; i < C; ++i)
            if (i * 32 + lane < L) {
              o[i].x = fmaf(wk, v[i][k].x, o[i].x);
              o[i].y = fmaf(wk, v[i][k].y, o[i].y);
              o[i].z = fmaf(wk, v[i][k].z, o[i].z);
              o[i].w = fmaf(wk, v[i][k].w, o[i].w);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i * 32 + lane < L) acc[warp][i * 32 + lane] = o[i];
    if (lane == 0) stat[warp] = make_float2(m, l);
    __syncthreads();
    if (threadIdx.x < L) {
      float top = kUnset;
      for (int w = 0; w < W; ++w) top = fmaxf(top, stat[w].x);
      l = 0.f;
      float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < W; ++w) {
        const float f = ex2(stat[w].x - top);
        const float4 v = acc[w][threadIdx.x];
        l = fmaf(f, stat[w].y, l);
        r.x = fmaf(f, v.x, r.x);
        r.y = fmaf(f, v.y, r.y);
        r.z = fmaf(f, v.z, r.z);
        r.w = fmaf(f, v.w, r.w);
      }
      const float vs = a.kv.v_scale ? a.kv.v_scale[unit.y] : 1.f, x = l == 0.f ? 0.f : vs / l;
      const int i = row / a.G, g = row - i * a.G;
      uint16_t* out = a.o + (long long)(unit.x + i) * a.os + (long long)(unit.y * a.G + g) * D;
      reinterpret_cast<uint2*>(out)[threadIdx.x] = make_uint2(pack2(r.x * x, r.y * x), pack2(r.z * x, r.w * x));
    }
    __syncthreads();
  }
}

// Rows of a unit for calls of about n new tokens a request and G query heads a key head: the smallest
// tile that holds a request's rows, and above 64 rows the two 128-row tiles of attn_chunk.cuh where it
// applies, from the first size on: 8 requests of 9 tokens of 8 heads (72 rows) over 4000 E4M3 keys, 128
// columns 28.6 us (33.8 in 64-row tiles), 64 columns 21.3 (25.8).  A tile holds the heads of whole tokens.
constexpr int kChunkRows = 256;
inline int row_tile(int D, int G, int n) {
  return 16 / G >= n ? 16 : 32 / G >= n ? 32 : 64 / G >= n || D > 128 ? 64 : kChunkRows;
}

template <int D, int NR, bool E4M3>
int launch_one(const Args& a, int sms, cudaStream_t s) {
  using C = Cfg<D, NR, E4M3>;
  // So few units that each is cut into more than sixteen pieces even at one run an SM: one run then, as
  // every further piece is another to join, and the join for many.  One token over 131071 keys: 52.4 us
  // at two runs an SM, 49.6 at one, 46.9 with this join.
  const bool many = NR == 16 && (long long)a.kv.B * a.kv.Hkv * 16 < sms && cap_of(a.kv) > 16 * kKeys;
  const int ctas = many ? sms : sms * C::OCC;
  if (launch_pdl(k_attn<D, NR, E4M3>, dim3(ctas), dim3(C::THREADS), C::SMEM, s, a) != cudaSuccess) return MOE_ECUDA;
  const cudaError_t e = NR == 16 && many ? launch_pdl(k_join_many<D>, dim3(ctas, a.G < 16 ? a.G : 16), dim3(kJoinThreads), 0, s, a)
                                         : launch_pdl(k_join<D, NR>, dim3(ctas, join_y(NR)), dim3(kJoinThreads), 0, s, a);
  if (e != cudaSuccess) return MOE_ECUDA;
  return MOE_OK;
}
template <int D, int NR, bool E4M3>
int opt_in() {
  // the join keeps the split of L1 and shared memory that the kernel before it had
  return cudaFuncSetAttribute(k_join<D, NR>, cudaFuncAttributePreferredSharedMemoryCarveout, 100) == cudaSuccess &&
                 cudaFuncSetAttribute(k_join_many<D>, cudaFuncAttributePreferredSharedMemoryCarveout, 100) == cudaSuccess &&
                 cudaFuncSetAttribute(k_attn<D, NR, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, NR, E4M3>::SMEM) ==
                     cudaSuccess
             ? MOE_OK
             : MOE_ECUDA;
}

}  // namespace attn
}  // namespace moe
