// Attention of prompt chunks: the same split, pages and join as attn.cuh, with the rows on the lanes.
//
// With 128 rows and more there is nothing to pad, and the other way round then costs less:
//   S = Q K^T      [128 rows x 128 keys]   (M = rows)
//   O += P V       [128 rows x D]          P from tensor memory
// A thread has one row, so its maximum and sum need no other thread; P never passes through shared
// memory; and a tile of keys and values is read from shared memory once as an N-side operand for
// each 128 rows.  attn.cuh's form at 128 rows moves 224 KB of shared memory a tile (K and V in and out,
// Q, P in and out), 1800 clocks of 128 bytes, beside 1250 clocks of products, and takes 2450; this form
// moves 128 KB.
//
// A CTA holds two row tiles of whole tokens, each with its own softmax warps: while one's weights are
// computed, the tensor core works for the other.  m is lazy as in attn.cuh, but a row's own: it is set
// again when a score passes it by 8 (log2).  P overwrites its S in tensor memory (64 of the 128
// columns), so the next S of a row tile waits for the product that reads it.
//
// What bounds it: that chain, S, weights, O, of two row tiles in turn, 3000 clocks for 256 rows by 128
// keys of 128 columns, with the tensor pipe busy 47% of the time.  Two chunks of up to 512 tokens of 32
// heads over up to 6000 keys: 73.1 us with the join, 959 TFLOP/s; with 64 columns 63 us.
//
// E4M3: four warps turn the tiles into bf16, exactly, in the ring's order.  A tile serves 256 rows here, so
// that is hidden but for 0.3 of a tile's time: the same chunks 83.7 us, 67.0 with 64 columns (attn.cuh's form at
// 64 rows 166.7 and 129.3).
#pragma once

#include "attn.cuh"

namespace moe {
namespace attn {
namespace chunk {

constexpr float kGrow = 8.0f;  // log2

struct Misc {
  uint64_t full[8], empty[8], rfull[8], rempty[8], qfull, qfree, sfull[2], pfull[2], pvdone[2], ofree[2], drain;
  uint32_t taddr;
  int fail;
  PlanShared plan;
  int page[2][kKeys];
  int nbad[4];  // keys of a tile with values that are not finite, of four tiles in turn
  uint8_t bad[4][kKeys];
};
constexpr int kMisc = (sizeof(Misc) + 127) / 128 * 128;

template <int D, bool E4M3>
struct Cfg {
  static constexpr int SLOT = kKeys * D * 2, QTILE = 128 * D * 2, RAW = E4M3 ? kKeys * D : 0;
  // even: keys and values in turn.  E4M3: a ring of bf16 and one of the codes as they come.
  static constexpr int FREE = kSmem - kMisc - 2 * QTILE, NS0 = E4M3 ? 4 : FREE / SLOT, NS = NS0 > 8 ? 8 : NS0 / 2 * 2;
  static constexpr int NR0 = E4M3 ? (FREE - NS * SLOT) / (RAW + !E4M3) : 0, NRAW = NR0 > 8 ? 8 : NR0 / 2 * 2;
  static constexpr int MMA = 8, LOAD = 9, CONVERT = 12;  // warps 0-3 and 4-7: softmax of a row tile each
  static constexpr int THREADS = 32 * (E4M3 ? 16 : 11);
  static constexpr int V = SLOT >= 32768 ? 2 : 3;  // as in attn.cuh, by the bytes of a tile
  static_assert(NS >= 4 && (!E4M3 || NRAW >= 2), "shared memory of an SM");
};

// Four steps of 16 keys: A (P) from tensor memory, eight columns a step, B (V) 2048 bytes on.
__device__ __forceinline__ void mma4_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a2, a3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u64 b1, %2, 128;\n\t"
      "add.u32 a2, %1, 16;\n\tadd.u64 b2, %2, 256;\n\t"
      "add.u32 a3, %1, 24;\n\tadd.u64 b3, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void st16u(uint32_t t, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Of four lanes with four groups of four values each: lane i gets the lanes' groups i, in their order.
__device__ __forceinline__ void turn4(float (&v)[16], int lane) {
#pragma unroll
  for (int d = 1; d < 4; d <<= 1)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (!(g & d)) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // this lane's group that belongs to the other one, against the other's
          const float give = up ? v[4 * g + i] : v[4 * (g | d) + i];
          const float got = __shfl_xor_sync(0xffffffffu, give, d);
          if (up) v[4 * g + i] = got;
          else v[4 * (g | d) + i] = got;
        }
      }
}

// Bit j of seen: node i sees key key0 + j, of 32 WORDS keys.
template <int WORDS>
__device__ __forceinline__ void tree_keys(const Args& a, const Req& r, int i, int key0, int cap, uint32_t* seen) {
  const int deep = a.window > 0 ? a.depth[r.s0 + i] : 0;
  seen_keys<WORDS>(a.above + (long long)(r.s0 + i) * a.words, a.words, a.depth + r.s0, deep, a.window, key0 - r.pos0,
                   min(cap, r.kv) - key0, seen);
}

// Registers a thread from here on, of a warpgroup.
template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void leave_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D, bool E4M3, bool TREE>
__global__ void __launch_bounds__(Cfg<D, E4M3>::THREADS, 1) k_chunk(const __grid_constant__ Args a) {
  using C = Cfg<D, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  uint8_t* sq = ring + C::NS * C::SLOT;
  uint8_t* raw = sq + 2 * C::QTILE;  // E4M3: tiles as they come
  Misc& ms = *reinterpret_cast<Misc*>(raw + C::NRAW * C::RAW);
  volatile int* fail = &ms.fail;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (warp == C::MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&ms.taddr)), "n"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    // not before: a kernel further on that takes tensor memory too could hold what this one waits for
    pdl_trigger();
  } else if (tid == 32 * C::LOAD) {
    for (int i = 0; i < C::NS; ++i) {
      bar_init(&ms.full[i], E4M3 ? 4 : 1);
      bar_init(&ms.empty[i], 1 + (a.phantom == 3));
    }
    for (int i = 0; i < C::NRAW; ++i) {
      bar_init(&ms.rfull[i], 1);
      bar_init(&ms.rempty[i], 4);
    }
    bar_init(&ms.qfull, 1 + (a.phantom == 1));
    bar_init(&ms.qfree, 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(&ms.sfull[i], 1);
      bar_init(&ms.pfull[i], 4 + (a.phantom == 2));
      bar_init(&ms.pvdone[i], 1);
      bar_init(&ms.ofree[i], 4);
    }
    bar_init(&ms.drain, 1);
    for (const CUtensorMap* m : {&a.mk, &a.mv, &a.mq})
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    ms.fail = 0;
    for (int i = 0; i < 4; ++i) ms.nbad[i] = 0;
  }
  pdl_wait();
  // trees' units end in tiles of masks: four trees of 256 nodes 155.1, 153.7, 153.0 and 153.9 us with 2, 3, 4 and 6, 32 of
  // 17 nodes 109.2, 108.1, 109.5 and 111.5
  constexpr int V = TREE ? 3 : C::V;
  const int cap = cap_of(a.kv);
  const Plan plan = plan_run<V, C::THREADS, TREE>(a, cap, ms.plan);
  const uint32_t taddr = ms.taddr;
  const int run = blockIdx.x, count = plan.count;
  if (count == 0 && tid == 0) a.join[run] = make_int4(0, 0, 0, 0);

  if (count > 0) {
    Walk<V, TREE> w;
    w.start(a, cap, ms.plan.first, plan.x1 - plan.x0);
    const int half = a.tokens / 2;  // tokens of a row tile
    auto both = [&]() { return w.s.i1 - w.s.i0 + 1 > half; };  // the unit has rows for the second row tile
    if (warp >= C::MMA) {
      if (E4M3) leave_registers<72>();
      if (warp == C::MMA) {
      // -------------------------------------------------------- tensor cores
      // D f32, A and B bf16, M = 128; S: N = 128 keys, both K-major; O: N = D, B (V) MN-major
      constexpr uint32_t kBase = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);
      constexpr uint32_t kIdescS = kBase | (uint32_t(kKeys >> 3) << 17), kIdescO = kBase | (uint32_t(D >> 3) << 17) | (1u << 16);
      Ring<C::NS> kr(0), vr(0);
      vr.next();
      int scores[2] = {0, 0}, pieces[2] = {0, 0}, qn = 0;  // S products and pieces of each row tile, pieces of the run
      auto put_s = [&](int x) {  // S = Q K(n)^T; its columns hold the last P until that product is done
        if (scores[x] > 0) wait(&ms.pvdone[x], (scores[x] - 1) & 1, fail);
        ++scores[x];
        tc_after();
        const uint64_t qd = desc(su32(sq + x * C::QTILE), 16, 1024, 2), kd = desc(su32(ring + kr.slot * C::SLOT), 16, 1024, 2);
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
          mma4<2, 2>(taddr + x * 128, qd + k * (128 * 128 >> 4), kd + k * (kKeys * 128 >> 4), kIdescS, k > 0);
        commit_to(&ms.sfull[x]);
      };
      auto begin = [&]() {  // the tile's keys are there, and the queries of its piece
        if (w.j == w.jbeg) wait(&ms.qfull, qn++ & 1, fail);
        wait(&ms.full[kr.slot], kr.phase, fail);
      };
      auto end = [&]() {
        commit_to(&ms.empty[kr.slot]);
        if (w.j + 1 == w.jend) commit_to(&ms.qfree);
        kr.next();
        kr.next();
      };
      begin();
      put_s(0);
      if (both()) put_s(1);
      end();
#pragma unroll 1
      for (int n = 0; n < count; ++n) {
        const bool first = w.j == w.jbeg, two = both(), more = n + 1 < count;
        auto put_o = [&](int x) {  // O += P V(n)
          wait(&ms.pfull[x], (scores[x] - 1) & 1, fail);
          if (first && pieces[x]++ > 0) wait(&ms.ofree[x], (pieces[x] - 2) & 1, fail);
          tc_after();
          const uint64_t vd = desc(su32(ring + vr.slot * C::SLOT), kKeys * 128, 1024, 2);
#pragma unroll
          for (int k = 0; k < kKeys / 64; ++k)
            mma4_ta(taddr + 256 + x * D, taddr + x * 128 + k * 32, vd + k * 512, kIdescO, !first || k > 0);
          commit_to(&ms.pvdone[x]);
        };
        wait(&ms.full[vr.slot], vr.phase, fail);
        put_o(0);
        if (more) {
          w.next(a, cap);
          begin();
          put_s(0);
        }
        if (two) put_o(1);
        commit_to(&ms.empty[vr.slot]);
        vr.next();
        vr.next();
        if (more) {
          if (both()) put_s(1);
          end();
        }
      }
      commit_to(&ms.drain);
      const unsigned long long t0 = now_ns();
      for (uint32_t ok = 0; !ok && now_ns() - t0 < 2 * kWaitNs;)
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], 0;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(su32(&ms.drain))
            : "memory");
    } else if (warp == C::LOAD || warp == C::LOAD + 1) {
      // -------------------------------------------------------- loads: keys and queries, values
      const bool keys = warp == C::LOAD;
      const KvView& kv = a.kv;
      const int box_shift = min(kv.page_shift, 7), boxes = kKeys >> box_shift;  // keys in a box, boxes in a tile
      const CUtensorMap* tm = keys ? &a.mk : &a.mv;
      int* page = ms.page[keys ? 0 : 1];
      Ring<E4M3 ? C::NRAW : C::NS> rg(1);
      if (!keys) rg.next();
      int qn = 0;
#pragma unroll 1
      for (int n = 0; n < count; ++n) {
        if (keys && w.j == w.jbeg) {
          if (qn > 0) wait(&ms.qfree, (qn - 1) & 1, fail);
          ++qn;
          if (lane == 0 && !*fail) {
            const int tiles = both() ? 2 : 1;
            expect(&ms.qfull, uint32_t(tiles * half * a.G * D * 2));
            for (int x = 0; x < tiles; ++x)
              for (int c = 0; c < D / 64; ++c)
                load_rows(sq + x * C::QTILE + c * (128 * 128), &a.mq, c * 64, w.h * a.G, w.r.s0 + w.s.i0 + x * half,
                          &ms.qfull);
          }
        }
        const int key0 = (w.s.tile0 + w.j) * kKeys;
        const int32_t* row = kv.page_table + (long long)w.b * kv.table_stride;
        for (int x = lane; x < boxes; x += 32) {
          const int key = key0 + (x << box_shift);
          int id = -2;
          if (key < w.s.hi && key + (1 << box_shift) > w.s.lo) id = row[key >> kv.page_shift];
          const bool ok = id >= 0 && id < kv.npages;
          if (!ok && id != -2) set_error(a.err, MOE_ERANGE);
          page[x] = ok ? id : kv.npages;  // past the end: zeros
        }
        __syncwarp();
        const int tok = key0 & ((1 << kv.page_shift) - 1);  // of a page larger than a tile
        uint64_t* full = (E4M3 ? ms.rfull : ms.full) + rg.slot;
        wait((E4M3 ? ms.rempty : ms.empty) + rg.slot, rg.phase, fail);
        if (!__any_sync(0xffffffffu, *fail)) {  // for the warp: its lanes meet inside
          if (lane == 0) expect(full, E4M3 ? C::RAW : C::SLOT);
          __syncwarp();
          constexpr int CHUNKS = E4M3 ? 1 : D / 64;
#pragma unroll 1
          for (int x = lane; x < boxes * CHUNKS; x += 32) {
            const int p = x & (boxes - 1), c = x >> (7 - box_shift);
            uint8_t* dst = E4M3 ? raw + rg.slot * C::RAW + (p << box_shift) * D
                                : ring + rg.slot * C::SLOT + c * (kKeys * 128) + (p << box_shift) * 128;
            load_box(dst, tm, c * 64, tok, w.h, page[p], full);
          }
        }
        __syncwarp();
        rg.next();
        rg.next();
        if (n + 1 < count) w.next(a, cap);
      }
    } else if (warp >= C::CONVERT) {
      // -------------------------------------------------------- E4M3 codes -> bf16, in the ring's order
      if constexpr (E4M3) {
        const int vt = tid - 32 * C::CONVERT;
        constexpr int CH = D / 8, STEP = 128 / CH;  // 8 codes a thread make one 16-byte piece
        const int r0 = vt / CH, c = vt % CH;
        Ring<C::NRAW> in(0);
        Ring<C::NS> out(1);
#pragma unroll 1
        for (int n = 0; n < 2 * count; ++n) {
          wait(&ms.rfull[in.slot], in.phase, fail);
          wait(&ms.empty[out.slot], out.phase, fail);
          const uint8_t* src = raw + in.slot * C::RAW + c * 8;
          uint8_t* dst = ring + out.slot * C::SLOT + (c / 8) * (kKeys * 128);
#pragma unroll 4
          for (int i = 0; i < kKeys / STEP; ++i) {
            const uint2 v = *reinterpret_cast<const uint2*>(src + (r0 + i * STEP) * D);
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
      // A row a thread takes more than the 128 registers that 512 threads start with; the others need few.
      static_assert(!E4M3 || 256 * (176 + 72) <= C::THREADS * 128, "registers of the launch");
      if (E4M3) take_registers<176>();
      // -------------------------------------------------------- softmax, a row a thread
      const int x = warp >> 2, quad = warp & 3, krow = quad * 32 + lane;  // row tile; row in it, and key in a tile
      const uint32_t ts = taddr + (uint32_t(quad * 32) << 16) + x * 128, to = taddr + (uint32_t(quad * 32) << 16) + 256 + x * D;
      float factor = a.scale * 1.4426950408889634f;
      const int mine = x * half + krow / a.G;  // the row's token in its unit
      float m = kUnset, l = 0.f;
      int spoiled_key0 = 0;
      int k = 0;         // tiles of this row tile
      int spoiled = -1;  // a tile that may have lost values that are not finite, once its product is done
      // Adds them to this row where it sees their keys.
      auto restore = [&]() {
        const int nbad = *const_cast<volatile int*>(&ms.nbad[spoiled & 3]);
        const int pos = min(w.r.pos0 + w.s.i0 + mine, w.r.pos0 + w.s.i1);
#pragma unroll 1
        for (int e = 0; e < nbad; ++e) {
          const int key = spoiled_key0 + ms.bad[spoiled & 3][e];
          if (key >= w.s.hi) continue;  // only where a wait gave up: a place of the list not written yet
          const int id = a.kv.page_table[(long long)w.b * a.kv.table_stride + (key >> a.kv.page_shift)];
          if (id < 0 || id >= a.kv.npages) continue;  // the same: the slot of a page that reads as zeros
          const uint8_t* v = a.kv.v + id * a.kv.page_stride + w.h * a.kv.head_stride +
                             (long long)(key & ((1 << a.kv.page_shift) - 1)) * a.kv.tok_stride;
          const bool sees = TREE ? tree_sees(a, w.r, pos - w.r.pos0, key) : key <= pos && (a.window <= 0 || key > pos - a.window);
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            ld16(to + c, o);
            ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float add = E4M3 ? f16x2_to_f32x2(e4m3x2_to_f16x2(v[c + i])).x
                                     : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(v)[c + i]);
              if (sees && !isfinite(add)) o[i] += add;
            }
            st16(to + c, o);
          }
        }
        if (nbad) st_wait();
        spoiled = -1;
      };
      if (tid == 0) a.join[run] = join_record(a, plan, w);
#pragma unroll 1
      for (int n = 0; n < count; ++n) {
        const bool active = x == 0 || both();
        if (active) {
          const bool first = w.j == w.jbeg;
          if (first) m = kUnset, l = 0.f;
          if (E4M3 && first) factor = a.scale * 1.4426950408889634f * (a.kv.k_scale ? a.kv.k_scale[w.h] : 1.f);
          const int newest = w.r.pos0 + w.s.i1, oldest = w.r.pos0 + w.s.i0;
          const int pos = min(w.r.pos0 + w.s.i0 + mine, newest);
          const int key0 = (w.s.tile0 + w.j) * kKeys;
          const bool whole = key0 + kKeys <= min(TREE ? w.r.pos0 : oldest + 1, cap) && (a.window <= 0 || key0 > newest - a.window);
          wait(&ms.sfull[x], k & 1, fail);
          tc_after();
          if (spoiled >= 0) restore();  // S follows the product of the tile before it
          float s[kKeys];
#pragma unroll
          for (int i = 0; i < kKeys; i += 16) ld16(ts + i, s + i);
          ld_wait();
          float f = factor;
          if (!whole || factor <= 0.f) {
            // Hidden scores stay -infinity where the factor is positive.  It is multiplied in with m, in one
            // multiply-add as in whole tiles: the product's part below m's last bit, which that keeps, is then the
            // same in all of a row's weights.  With factors that are not, every tile takes the product first.
            const float once = factor > 0.f ? 1.f : factor;
            f = factor > 0.f ? factor : 1.f;
            if constexpr (TREE) {
              uint32_t seen[kKeys / 32];  // of the tile's keys, by this row
              tree_keys<kKeys / 32>(a, w.r, pos - w.r.pos0, key0, cap, seen);
#pragma unroll
              for (int i = 0; i < kKeys; ++i) s[i] = seen[i / 32] >> (i % 32) & 1 ? s[i] * once : -INFINITY;
            } else {
              const int from = a.window > 0 ? pos - a.window + 1 - key0 : INT_MIN, to_key = min(pos + 1, cap) - key0;
#pragma unroll
              for (int i = 0; i < kKeys; ++i) s[i] = i < from || i >= to_key ? -INFINITY : s[i] * once;
            }
          }
          float top = -INFINITY, top1 = -INFINITY;  // the row's largest score
#pragma unroll
          for (int i = 0; i < kKeys; i += 2) top = fmaxf(top, s[i]), top1 = fmaxf(top1, s[i + 1]);
          top = fmaxf(top, top1) * f;
          const bool grow = top > m + kGrow;  // true for the first that a row sees: m is unset
          if (__any_sync(0xffffffffu, grow)) {
            const float old = m;
            if (grow) m = top;
            const float alpha = grow ? ex2(old - m) : 1.f;
            l *= alpha;
            if (!first) {
              wait(&ms.pvdone[x], (k - 1) & 1, fail);
              tc_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                float o[16];
                ld16(to + c, o);
                ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= alpha;
                st16(to + c, o);
              }
              st_wait();
            }
          }
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t u[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              scale_sub2(s[c + i], s[c + i + 1], f, f, m, m);
              const float e0 = ex2(s[c + i]), e1 = ex2(s[c + i + 1]);
              add2(sum0, sum1, e0, e1);
              u[i / 2] = pack2(e0, e1);
            }
            st16u(ts + c / 2, u);
          }
          l += sum0 + sum1;
          // Values at hidden keys, as in attn.cuh: zeros where no row sees the key; where some do, what is
          // not finite leaves the tile and goes to their rows below.  The first row tile's threads, one a
          // key, do it for both: its product comes first.
          const bool mixed = !whole && (TREE || w.s.i1 > w.s.i0);
          if (!whole && x == 0) {
            if (mixed && krow == 0) ms.nbad[n & 3] = 0;
            if (mixed) asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
            const int key = key0 + krow, slot = (2 * n + 1) % C::NS;
            const bool gone = key < w.s.lo || key >= w.s.hi;
            const bool some = !gone && mixed && ((TREE ? key >= w.r.pos0 : key > oldest) || (a.window > 0 && key <= newest - a.window));
            wait(&ms.full[slot], uint32_t((2 * n + 1) / C::NS) & 1, fail);  // V(n - NS / 2) has been used
            uint8_t* row = ring + slot * C::SLOT;
            if (gone) {
#pragma unroll 4
              for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4*>(row + (c / 8) * (kKeys * 128) + sw128(krow, c % 8)) = make_uint4(0, 0, 0, 0);
            } else if (some && not_finite<D>(row, krow)) {
              drop_not_finite<D>(row, krow);
              ms.bad[n & 3][atomicAdd(&ms.nbad[n & 3], 1)] = uint8_t(krow);
            }
            proxy_fence();
            if (mixed) asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
          }
          st_wait();
          tc_before();
          __syncwarp();
          if (lane == 0) arrive(&ms.pfull[x]);
          if (mixed) spoiled = n, spoiled_key0 = key0;
          if (w.j + 1 == w.jend) {
            wait(&ms.pvdone[x], k & 1, fail);
            tc_after();
            if (mixed) restore();
            // ---- the piece is done
            const bool head = w.jbeg > 0, split = head || w.jend < w.s.nt;
            const int unit_row = x * half * a.G + krow, rows = min(half, w.s.i1 - w.s.i0 + 1 - x * half) * a.G;
            const long long part = (2ll * run + (head ? 0 : 1)) * kChunkRows + unit_row;
            if (split && krow < rows) reinterpret_cast<float2*>(a.ml)[part] = make_float2(m, l);
            const float vs = E4M3 && a.kv.v_scale ? a.kv.v_scale[w.h] : 1.f;
            const float inv = split ? 1.f : l == 0.f ? 0.f : vs / l;  // a sum of zero is a row that sees no key; its O is zeros
            unsigned long long row = reinterpret_cast<unsigned long long>(a.part + part * D);
            if (!split)
              row = reinterpret_cast<unsigned long long>(a.o + (long long)(w.r.s0 + w.s.i0 + mine) * a.os +
                                                         (long long)(w.h * a.G + krow % a.G) * D);
            if (krow >= rows) row = 0;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              ld16(to + c, o);
              ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= inv;
              // Four lanes turn their four rows' pieces round and write each row's together: a row a
              // thread, 16 bytes at a time, took 10000 clocks.
              turn4(o, lane);
#pragma unroll
              for (int r = 0; r < 4; ++r) {  // row r of the four, columns c + 4 (lane % 4) ..
                const unsigned long long at = __shfl_sync(0xffffffffu, row, lane / 4 * 4 + r);
                if (!at) continue;
                if (split)
                  *reinterpret_cast<float4*>(at + (c + lane % 4 * 4) * 4) = make_float4(o[4 * r], o[4 * r + 1], o[4 * r + 2], o[4 * r + 3]);
                else
                  *reinterpret_cast<uint2*>(at + (c + lane % 4 * 4) * 2) = make_uint2(pack2(o[4 * r], o[4 * r + 1]), pack2(o[4 * r + 2], o[4 * r + 3]));
              }
            }
            tc_before();
            __syncwarp();
            if (lane == 0) arrive(&ms.ofree[x]);
          }
          ++k;
        }
        if (n + 1 < count) w.next(a, cap);
      }
    }
  }
  __syncthreads();
  if (tid == 0 && *fail) give_up(a.err);
  if (warp == C::MMA) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(512));
  }
}

template <int D, bool E4M3, bool TREE>
int launch(const Args& a, int ctas, cudaStream_t s) {
  if (launch_pdl(k_chunk<D, E4M3, TREE>, dim3(ctas), dim3(Cfg<D, E4M3>::THREADS), kSmem, s, a) != cudaSuccess) return MOE_ECUDA;
  return launch_join<D>(a, kChunkRows, false, ctas, s);
}
template <int D, bool E4M3, bool TREE>
int opt_in() {
  return cudaFuncSetAttribute(k_chunk<D, E4M3, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess ? MOE_OK
                                                                                                                   : MOE_ECUDA;
}

}  // namespace chunk
}  // namespace attn
}  // namespace moe
