// Attention of drafted trees of more than 32 rows a key head with 256 columns: rows on the lanes, as in attn_chunk.cuh.
//
//   S = Q K^T      [128 rows x 128 keys]   (M = rows)
//   O += P V       [128 rows x 256]        P from tensor memory
// O takes half of tensor memory, so there is one row tile, whose scores have the other half twice: while the weights of
// one tile of keys are computed, the tensor core multiplies the last one's with the values and makes the next one's
// scores.  Two threads share a row, 64 keys each: a vote of all 256 of them a tile tells whether a maximum has to be set
// again (m is a row's own, and lazy), and lets P take the place of scores that both have read.
//
// Shared memory holds the queries (64 KB) and a ring of half tiles, 128 keys by 128 columns, that is filled and used in
// the order K(0) K(1) V(0) K(2) V(1) ..: five slots, so that half a tile and more is on its way while one is used.
// E4M3 tiles come as they are into a ring of their own, and eight warps turn them into bf16, exactly.
//
// attn.cuh's form takes these rows 64 at a time, reads keys and values as often, and has no slot to spare beside a key
// and a value tile.  16 trees of up to 32 nodes of 8 heads over 512 to 32768 tokens (22 rows' worth of nodes on average):
// bf16 64.1 us, E4M3 69.7 with the join; in 64-row tiles 96 and 111.
//
// What bounds it: memory's way.  Without the conversions E4M3 takes 61 us, without exponentials or maxima, or with half the
// products, what it takes with them; bf16 over pages that the L2 holds 50.4.  The join is 8 to 12 us of either: each of 152
// runs leaves one or two pieces of 128 x 256 sums.  In E4M3, with 96 registers a thread at launch, 228 bytes a thread of the
// softmax are spilled.
#pragma once

#include "attn_chunk.cuh"

namespace moe {
namespace attn {
namespace wide {

using chunk::kGrow;
using chunk::leave_registers;
using chunk::mma4_ta;
using chunk::st16u;
using chunk::take_registers;
using chunk::tree_keys;
using chunk::turn4;

constexpr int kRows = kWideRows, D = 256, HALF = 128;  // columns in a slot

struct Misc {
  uint64_t full[5], empty[5], rfull[4], rempty[4], qfull, qfree, sfull[2], pfull[2], pvdone[2], ofree, drain;
  uint32_t taddr;
  int fail;
  PlanShared plan;
  int page[2][kKeys];
  float red[2][kRows];  // the rows' maxima of a tile, or their sums, by half of the keys
  int nbad;
  uint8_t bad[kKeys];   // keys of a tile with values that are not finite
};
constexpr int kMisc = (sizeof(Misc) + 127) / 128 * 128;

template <bool E4M3>
struct Cfg {
  static constexpr int SLOT = kKeys * HALF * 2, QBYTES = kRows * D * 2, RAW = kKeys * HALF;
  static constexpr int NS = E4M3 ? 3 : 5, NRAW = E4M3 ? 4 : 0;  // slots of bf16; of codes
  static constexpr int SOFT = 8, MMA = 8, LOAD = 9, CONVERT = 12, CV = 8;  // warps
  static constexpr int THREADS = 32 * (E4M3 ? 20 : 11);
  static_assert(NS * SLOT + NRAW * RAW + QBYTES + kMisc <= kSmem, "shared memory of an SM");
};
constexpr int kSoftThreads = 256;
// What a unit costs beside its tiles, in tiles: 2, 3, 5 and 8 give 71.4, 69.3, 70.5 and 72.9 us (E4M3), 68.9, 63.8, 69.1 and
// 65.7 (bf16).  Four converting warps 88.8 us, eight 69.3.
constexpr int V = 3;

template <bool E4M3>
__global__ void __launch_bounds__(Cfg<E4M3>::THREADS, 1) k_wide(const __grid_constant__ Args a) {
  using C = Cfg<E4M3>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  uint8_t* sq = ring + C::NS * C::SLOT;
  uint8_t* raw = sq + C::QBYTES;  // E4M3: half tiles as they come
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
      bar_init(&ms.full[i], E4M3 ? C::CV : 1);
      bar_init(&ms.empty[i], 1 + (a.phantom == 3));
    }
    for (int i = 0; i < C::NRAW; ++i) {
      bar_init(&ms.rfull[i], 1);
      bar_init(&ms.rempty[i], C::CV);
    }
    bar_init(&ms.qfull, 1 + (a.phantom == 1));
    bar_init(&ms.qfree, 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(&ms.sfull[i], 1);
      bar_init(&ms.pfull[i], C::SOFT + (a.phantom == 2));
      bar_init(&ms.pvdone[i], 1);
    }
    bar_init(&ms.ofree, C::SOFT);
    bar_init(&ms.drain, 1);
    for (const CUtensorMap* m : {&a.mk, &a.mv, &a.mq})
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    ms.fail = 0;
    ms.nbad = 0;
  }
  pdl_wait();
  const int cap = cap_of(a.kv);
  const Plan plan = plan_run<V, C::THREADS, true>(a, cap, ms.plan);
  const uint32_t taddr = ms.taddr;
  const int run = blockIdx.x, count = plan.count;
  if (count == 0 && tid == 0) a.join[run] = make_int4(0, 0, 0, 0);

  if (count > 0) {
    Walk<V, true> w;
    w.start(a, cap, ms.plan.first, plan.x1 - plan.x0);
    if (warp >= C::MMA) {
      if (E4M3) leave_registers<80>();
      if (warp == C::MMA) {
        // -------------------------------------------------------- tensor cores
        // D f32, A and B bf16, M = N = 128; S: both K-major; O: B (V) MN-major
        constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24) | (uint32_t(kKeys >> 3) << 17);
        constexpr uint32_t kIdescO = kIdescS | (1u << 16);
        Ring<C::NS> rg(0);
        int qn = 0, pieces = 0;  // pieces whose scores, and whose O, have been begun
        auto put_s = [&](int n) {  // S(n) = Q K(n)^T, where P(n - 2) has been read
          if (w.j == w.jbeg) wait(&ms.qfull, qn++ & 1, fail);
          if (n >= 2) wait(&ms.pvdone[n & 1], ((n - 2) >> 1) & 1, fail);
          const uint64_t qd = desc(su32(sq), 16, 1024, 2);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            wait(&ms.full[rg.slot], rg.phase, fail);
            tc_after();
            const uint64_t kd = desc(su32(ring + rg.slot * C::SLOT), 16, 1024, 2);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              mma4<2, 2>(taddr + (n & 1) * 128, qd + (2 * hh + k) * (kRows * 128 >> 4), kd + k * (kKeys * 128 >> 4), kIdescS,
                         hh + k > 0);
            commit_to(&ms.empty[rg.slot]);
            rg.next();
          }
          commit_to(&ms.sfull[n & 1]);
          if (w.j + 1 == w.jend) commit_to(&ms.qfree);
        };
        bool first = true;  // of tile n
        put_s(0);
#pragma unroll 1
        for (int n = 0; n < count; ++n) {
          bool next_first = false;
          if (n + 1 < count) {
            w.next(a, cap);
            next_first = w.j == w.jbeg;
            put_s(n + 1);
          }
          // O += P(n) V(n)
          wait(&ms.pfull[n & 1], (n >> 1) & 1, fail);
          if (first && pieces++ > 0) wait(&ms.ofree, (pieces - 2) & 1, fail);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            wait(&ms.full[rg.slot], rg.phase, fail);
            tc_after();
            const uint64_t vd = desc(su32(ring + rg.slot * C::SLOT), kKeys * 128, 1024, 2);
#pragma unroll
            for (int k = 0; k < kKeys / 64; ++k)
              mma4_ta(taddr + 256 + hh * HALF, taddr + (n & 1) * 128 + k * 32, vd + k * 512, kIdescO, !first || k > 0);
            commit_to(&ms.empty[rg.slot]);
            rg.next();
          }
          commit_to(&ms.pvdone[n & 1]);
          first = next_first;
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
        auto skip = [&]() {
          rg.next();
          rg.next();
        };
        if (!keys) {
          skip();
          if (count > 1) skip();
        }
        int qn = 0;
#pragma unroll 1
        for (int n = 0; n < count; ++n) {
          if (keys && w.j == w.jbeg) {
            if (qn > 0) wait(&ms.qfree, (qn - 1) & 1, fail);
            ++qn;
            if (lane == 0 && !*fail) {
              expect(&ms.qfull, uint32_t(a.tokens * a.G * D * 2));
              for (int c = 0; c < D / 64; ++c)
                load_rows(sq + c * (kRows * 128), &a.mq, c * 64, w.h * a.G, w.r.s0 + w.s.i0, &ms.qfull);
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
#pragma unroll 1
          for (int hh = 0; hh < 2; ++hh) {
            uint64_t* full = (E4M3 ? ms.rfull : ms.full) + rg.slot;
            wait((E4M3 ? ms.rempty : ms.empty) + rg.slot, rg.phase, fail);
            if (__any_sync(0xffffffffu, *fail)) break;  // for the warp: its lanes meet below
            if (lane == 0) expect(full, E4M3 ? C::RAW : C::SLOT);
            __syncwarp();
            constexpr int CHUNKS = E4M3 ? 1 : HALF / 64;
#pragma unroll 1
            for (int x = lane; x < boxes * CHUNKS; x += 32) {
              const int p = x & (boxes - 1), c = x >> (7 - box_shift);
              uint8_t* dst = E4M3 ? raw + rg.slot * C::RAW + (p << box_shift) * HALF
                                  : ring + rg.slot * C::SLOT + c * (kKeys * 128) + (p << box_shift) * 128;
              load_box(dst, tm, hh * HALF + c * 64, tok, w.h, page[p], full);
            }
            __syncwarp();
            rg.next();
          }
          if (keys ? n > 0 : n + 2 != count) skip();
          if (n + 1 < count) w.next(a, cap);
        }
      } else if (warp >= C::CONVERT) {
        // -------------------------------------------------------- E4M3 codes -> bf16, in the ring's order
        if constexpr (E4M3) {
          const int vt = tid - 32 * C::CONVERT;
          constexpr int CH = HALF / 8, STEP = 32 * C::CV / CH;  // 8 codes a thread make one 16-byte piece
          const int r0 = vt / CH, c = vt % CH;
          Ring<C::NRAW> in(0);
          Ring<C::NS> out(1);
#pragma unroll 1
          for (int n = 0; n < 4 * count; ++n) {
            wait(&ms.rfull[in.slot], in.phase, fail);
            wait(&ms.empty[out.slot], out.phase, fail);
            const uint8_t* src = raw + in.slot * C::RAW + c * 8;
            uint8_t* dst = ring + out.slot * C::SLOT + (c / 8) * (kKeys * 128);
#pragma unroll 4
            for (int i = 0; i < kKeys / STEP; ++i) {
              const uint2 v = *reinterpret_cast<const uint2*>(src + (r0 + i * STEP) * HALF);
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
      static_assert(!E4M3 || kSoftThreads * 120 + (C::THREADS - kSoftThreads) * 80 <= C::THREADS * 96, "registers of the launch");
      if (E4M3) take_registers<120>();
      // -------------------------------------------------------- softmax, two threads a row
      constexpr int HK = kKeys / 2;
      const int half = warp >> 2, quad = warp & 3, krow = quad * 32 + lane;  // half of the keys, and of O's columns; row
      const uint32_t tl = taddr + (uint32_t(quad * 32) << 16), to = tl + 256 + half * HALF;
      float factor = a.scale * 1.4426950408889634f;
      const int mine = krow / a.G;  // the row's token in its unit
      float m = kUnset, l = 0.f;
      if (tid == 0) a.join[run] = join_record(a, plan, w);
#pragma unroll 1
      for (int n = 0; n < count; ++n) {
        const int p = n & 1;
        const bool first = w.j == w.jbeg;
        if (first) {
          m = kUnset, l = 0.f;
          if (E4M3) factor = a.scale * 1.4426950408889634f * (a.kv.k_scale ? a.kv.k_scale[w.h] : 1.f);
        }
        const int node = min(w.s.i0 + mine, w.s.i1), newest = w.r.pos0 + w.s.i1;
        const int key0 = (w.s.tile0 + w.j) * kKeys;
        const bool whole = key0 + kKeys <= min(w.r.pos0, cap) && (a.window <= 0 || key0 > newest - a.window);
        uint32_t seen[HK / 32];  // of this thread's keys, by its row
        if (!whole) tree_keys<HK / 32>(a, w.r, node, key0 + half * HK, cap, seen);
        wait(&ms.sfull[p], (n >> 1) & 1, fail);
        tc_after();
        float s[HK];
#pragma unroll
        for (int i = 0; i < HK; i += 16) ld16(tl + p * 128 + half * HK + i, s + i);
        ld_wait();
        float f = factor;
        if (!whole || factor <= 0.f) {
          // as in attn_chunk.cuh: hidden scores stay -infinity where the factor is positive
          const float once = factor > 0.f ? 1.f : factor;
          f = factor > 0.f ? factor : 1.f;
#pragma unroll
          for (int i = 0; i < HK; ++i) s[i] = whole || (seen[i / 32] >> (i % 32) & 1) ? s[i] * once : -INFINITY;
        }
        float top = -INFINITY, top1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < HK; i += 2) top = fmaxf(top, s[i]), top1 = fmaxf(top1, s[i + 1]);
        top = fmaxf(top, top1) * f;
        tc_before();
        const bool any = vote_any<kSoftThreads>(top > m + kGrow);  // true for the first tile that a row sees: m is unset
        tc_after();
        if (any) {
          ms.red[half][krow] = top;
          softmax_sync<kSoftThreads>();
          top = fmaxf(ms.red[0][krow], ms.red[1][krow]);
          const bool grow = top > m + kGrow;
          const float alpha = grow ? ex2(m - top) : 1.f;
          if (grow) m = top;
          l *= alpha;
          if (!first) {
            wait(&ms.pvdone[p ^ 1], ((n - 1) >> 1) & 1, fail);
            tc_after();
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll 1
              for (int c = 0; c < HALF; c += 16) {
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
        }
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int c = 0; c < HK; c += 32) {
          uint32_t u[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            scale_sub2(s[c + i], s[c + i + 1], f, f, m, m);
            const float e0 = ex2(s[c + i]), e1 = ex2(s[c + i + 1]);
            add2(sum0, sum1, e0, e1);
            u[i / 2] = pack2(e0, e1);
          }
          st16u(tl + p * 128 + half * (HK / 2) + c / 2, u);
        }
        l += sum0 + sum1;
        // Values at hidden keys, as in attn.cuh: zeros where no row sees the key; what is not finite elsewhere leaves the
        // tile and goes to the rows that see it.  The first half's threads, one a key, look at both slots.
        bool spoiled = false;
        if (!whole) {
          const int key = key0 + krow;
          const bool gone = key < w.s.lo || key >= w.s.hi;
          const bool some = !gone && (key >= w.r.pos0 || (a.window > 0 && key <= newest - a.window));
          const int at = (n + 1 == count ? 2 * count - 1 : 2 * n + 2) * 2;  // V(n)'s place in the ring's order
          // V(n)'s slots may still be held by V(n - 1), or by K(n + 1) in a ring of three: see those filled first, so that the
          // slots' phases tell V(n)'s
          if (n >= 1) wait(&ms.pvdone[p ^ 1], ((n - 1) >> 1) & 1, fail);
          if (E4M3 && n + 1 < count) wait(&ms.sfull[p ^ 1], ((n + 1) >> 1) & 1, fail);
          bool bad = false;
#pragma unroll 1
          for (int hh = 0; hh < 2; ++hh) {
            const int slot = (at + hh) % C::NS;
            wait(&ms.full[slot], uint32_t((at + hh) / C::NS) & 1, fail);
            if (half > 0 || !(gone || some)) continue;
            uint8_t* row = ring + slot * C::SLOT;
            if (gone) {
#pragma unroll 4
              for (int c = 0; c < HALF / 8; ++c)
                *reinterpret_cast<uint4*>(row + (c / 8) * (kKeys * 128) + sw128(krow, c % 8)) = make_uint4(0, 0, 0, 0);
            } else if (not_finite<HALF>(row, krow)) {
              bad = true;
              drop_not_finite<HALF>(row, krow);
            }
          }
          if (bad) ms.bad[atomicAdd(&ms.nbad, 1)] = uint8_t(krow);
          spoiled = vote_any<kSoftThreads>(bad);
          proxy_fence();
        }
        st_wait();
        tc_before();
        __syncwarp();
        if (lane == 0) arrive(&ms.pfull[p]);
        const bool last = w.j + 1 == w.jend;
        if (spoiled || last) {
          wait(&ms.pvdone[p], (n >> 1) & 1, fail);
          tc_after();
        }
        if (spoiled) {
          const int nbad = *const_cast<volatile int*>(&ms.nbad);
#pragma unroll 1
          for (int e = 0; e < nbad; ++e) {
            const int key = key0 + ms.bad[e];
            if (key >= w.s.hi) continue;  // only where a wait gave up
            const int id = a.kv.page_table[(long long)w.b * a.kv.table_stride + (key >> a.kv.page_shift)];
            if (id < 0 || id >= a.kv.npages) continue;  // the same: the slot of a page that reads as zeros
            const uint8_t* v = a.kv.v + id * a.kv.page_stride + w.h * a.kv.head_stride +
                               (long long)(key & ((1 << a.kv.page_shift) - 1)) * a.kv.tok_stride;
            const bool sees = tree_sees(a, w.r, node, key);
#pragma unroll 1
            for (int c = 0; c < HALF; c += 16) {
              float o[16];
              ld16(to + c, o);
              ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int col = half * HALF + c + i;
                const float add = E4M3 ? f16x2_to_f32x2(e4m3x2_to_f16x2(v[col])).x
                                       : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(v)[col]);
                if (sees && !isfinite(add)) o[i] += add;
              }
              st16(to + c, o);
            }
          }
          st_wait();
          tc_before();
          softmax_sync<kSoftThreads>();
          if (tid == 0) ms.nbad = 0;
        }
        if (last) {
          // ---- the piece is done
          const bool head = w.jbeg > 0, split = head || w.jend < w.s.nt;
          const int rows = (w.s.i1 - w.s.i0 + 1) * a.G;
          ms.red[half][krow] = l;
          softmax_sync<kSoftThreads>();
          const float total = ms.red[0][krow] + ms.red[1][krow];
          const long long part = (2ll * run + (head ? 0 : 1)) * kRows + krow;
          if (split && half == 0 && krow < rows) reinterpret_cast<float2*>(a.ml)[part] = make_float2(m, total);
          const float vs = E4M3 && a.kv.v_scale ? a.kv.v_scale[w.h] : 1.f;
          const float inv = split ? 1.f : total == 0.f ? 0.f : vs / total;  // a sum of zero is a row that sees no key
          unsigned long long row = reinterpret_cast<unsigned long long>(a.part + part * D + half * HALF);
          if (!split)
            row = reinterpret_cast<unsigned long long>(a.o + (long long)(w.r.s0 + w.s.i0 + mine) * a.os +
                                                       (long long)(w.h * a.G + krow % a.G) * D + half * HALF);
          if (krow >= rows) row = 0;
#pragma unroll 1
          for (int c = 0; c < HALF; c += 16) {
            float o[16];
            ld16(to + c, o);
            ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= inv;
            turn4(o, lane);  // four lanes write each of their rows together
#pragma unroll
            for (int r = 0; r < 4; ++r) {
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
          if (lane == 0) arrive(&ms.ofree);
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

template <bool E4M3>
int launch(const Args& a, int ctas, cudaStream_t s) {
  if (launch_pdl(k_wide<E4M3>, dim3(ctas), dim3(Cfg<E4M3>::THREADS), kSmem, s, a) != cudaSuccess) return MOE_ECUDA;
  return launch_join<D>(a, kRows, false, ctas, s);
}
template <bool E4M3>
int opt_in() {
  return cudaFuncSetAttribute(k_wide<E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess ? MOE_OK : MOE_ECUDA;
}

}  // namespace wide
}  // namespace attn
}  // namespace moe
