// Keys and values that move inside a cache, in every layer's pools at once: the kept nodes of drafted trees to
// the front of their tree, and copies of pages.
//
// What bounds them: memory for copies, and for kept nodes, whose few rows are a megabyte a layer at most, the
// chain count, path, table, row, store.  One launch holds the pools of 128 layers, so a step pays for that chain once.
#include <stdlib.h>

#include "paged.cuh"

namespace moe {
namespace move {

constexpr int kPools = 256;    // of a launch: keys and values of 128 layers
constexpr int kMaxLayers = 4096;

struct Args {
  KvView kv;  // geometry and requests; its k and v are not used
  int vecs;   // 16-byte pieces of a head's row
  const int32_t *path, *count;
  int path_stride;
  int32_t *len, *err;
  const int32_t *src, *dst, *tokens;
  int blocks;  // of a page
  int pools, first;  // of the launch; the call's first launch
  uint8_t* pool[kPools];
};

// ------------------------------------------------------------------ kept nodes
// A CTA takes a request in several pools.  A thread moves 16-byte columns of a head through all kept nodes in their order,
// kAhead loads before their stores: as kept indices rise, path[d] >= d, and no place is written before the thread has read
// it.  Nodes that are kept in their places are the path's first.
//
// 64 trees' up to six nodes in 24 layers, 28 MB in rows of 256 bytes: 8.8 us; up to twelve, 66 MB, 15.9 us, 4.2 TB/s: rows
// that lie far apart.  With two, three and four columns a thread at a time 9.0 to 10.4 us, and a CTA for each pool 14.0.
constexpr int kThreads = 256, kSteps = 256, kAhead = 8, kCompactPerSm = 4;

__global__ void __launch_bounds__(kThreads, kCompactPerSm) k_compact(const __grid_constant__ Args a) {
  __shared__ long long from[kSteps], to[kSteps];
  __shared__ int bad, moved;  // the first index that does not rise; the first that moves
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x;
  const KvView& kv = a.kv;
  const int rows = row_span(kv.q_start, b, kv.T).n, n = max(rows, 0);
  const long long base = (long long)kv.kv_len[b] - n;
  int want = a.count[b];
  want = min(max(want, 0), min(n, a.path_stride));
  const int32_t* path = a.path + (long long)b * a.path_stride;
  const bool speaks = a.first && blockIdx.y == 0 && tid == 0;
  // this CTA's pools, and their columns of all heads
  const int each = (a.pools + gridDim.y - 1) / gridDim.y, pool0 = blockIdx.y * each, pools = min(each, a.pools - pool0);
  const int cols = kv.Hkv * a.vecs;
  auto place = [&](long long p) -> long long {  // byte offset of a position in the pool, < 0: there is none
    if (p < 0 || (p >> kv.page_shift) >= kv.table_stride) return -1;
    const int id = kv.page_table[(long long)b * kv.table_stride + (p >> kv.page_shift)];
    return id >= 0 && id < kv.npages ? id * kv.page_stride + (p & ((1 << kv.page_shift) - 1)) * kv.tok_stride : -1;
  };
  int kept = want;
  for (int d0 = 0; d0 < kept; d0 += kSteps) {
    if (tid == 0) bad = moved = want;
    __syncthreads();
    const int d = d0 + tid;
    int node = 0;
    if (d < kept) {
      node = path[d];
      if (node < 0 || node >= n || (d > 0 && node <= path[d - 1])) atomicMin(&bad, d);
    }
    __syncthreads();
    kept = min(kept, bad);
    if (d < kept && node != d) {
      atomicMin(&moved, d);
      const long long at = place(base + node), into = place(base + d);
      if (at < 0 || into < 0) set_error(a.err, MOE_ERANGE);
      from[tid] = at < 0 || into < 0 ? -1 : at;
      to[tid] = into;
    }
    __syncthreads();
    const int step0 = max(moved - d0, 0), steps = min(kept - d0, kSteps);
    for (int c = tid; c < pools * cols; c += kThreads) {
      const int pool = c / cols, head = (c - pool * cols) / a.vecs;
      uint8_t* col = a.pool[pool0 + pool] + head * kv.head_stride + (c - pool * cols - head * a.vecs) * 16;
      for (int e0 = step0; e0 < steps; e0 += kAhead) {
        uint4 x[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          if (e0 + e < steps && from[e0 + e] >= 0) x[e] = *reinterpret_cast<const uint4*>(col + from[e0 + e]);
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          if (e0 + e < steps && from[e0 + e] >= 0) *reinterpret_cast<uint4*>(col + to[e0 + e]) = x[e];
      }
    }
    __syncthreads();
  }
  if (speaks) {
    if (kept < want || rows < 0) set_error(a.err, MOE_ERANGE);
    if (a.len) a.len[b] = int(min(max(base + kept, (long long)INT32_MIN), (long long)INT32_MAX));
  }
}

// ------------------------------------------------------------------ pages
// A CTA takes kPiece 16-byte pieces of a page in one pool, all of a thread's loads before its stores.  96 pages of 64 KB in 32
// layers, 805 MB read and written: 117 us, 6.9 TB/s, what a plain copy reaches; one page of 128 KB in 32 layers 5.4 us.
constexpr int kCopyThreads = 256, kEach = 8, kPiece = kCopyThreads * kEach;

__global__ void __launch_bounds__(kCopyThreads) k_copy(const __grid_constant__ Args a) {
  pdl_trigger();
  pdl_wait();
  const KvView& kv = a.kv;
  const int i = blockIdx.x / a.blocks, part = blockIdx.x - i * a.blocks;
  const int src = a.src[i], dst = a.dst[i];
  int most = 1 << kv.page_shift;
  if (a.tokens) most = min(a.tokens[i], most);
  if (src < 0 || src >= kv.npages || dst < 0 || dst >= kv.npages) {
    if (part == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_error(a.err, MOE_ERANGE);
    return;
  }
  const int total = (kv.Hkv << kv.page_shift) * a.vecs;
  const uint8_t* in = a.pool[blockIdx.y] + src * kv.page_stride;
  uint8_t* out = a.pool[blockIdx.y] + dst * kv.page_stride;
  uint4 x[kEach];
  long long at[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int v = part * kPiece + e * kCopyThreads + threadIdx.x, row = v / a.vecs, tok = row & ((1 << kv.page_shift) - 1);
    at[e] = -1;
    if (v >= total || tok >= most) continue;
    at[e] = (row >> kv.page_shift) * kv.head_stride + tok * kv.tok_stride + (v - row * a.vecs) * 16;
    x[e] = *reinterpret_cast<const uint4*>(in + at[e]);
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    if (at[e] >= 0) *reinterpret_cast<uint4*>(out + at[e]) = x[e];
}

// Whether the layers' pools are of one geometry.
bool alike(const moe_kv_pages* kv, int L) {
  for (int l = 1; l < L; ++l) {
    const moe_kv_pages &p = kv[0], &x = kv[l];
    if (x.e4m3 != p.e4m3 || x.Hkv != p.Hkv || x.D != p.D || x.page != p.page || x.npages != p.npages ||
        x.page_stride != p.page_stride || x.head_stride != p.head_stride || x.tok_stride != p.tok_stride || !x.k || !x.v ||
        (reinterpret_cast<uintptr_t>(x.k) & 15) || (reinterpret_cast<uintptr_t>(x.v) & 15))
      return false;
  }
  return true;
}

// Addresses that have been met, in an open table of at least twice as many places.
struct Met {
  uint8_t** at;
  int bits = 2;
  explicit Met(int n) {
    while (1 << bits < 2 * n) ++bits;
    at = static_cast<uint8_t**>(calloc(size_t(1) << bits, sizeof(uint8_t*)));
  }
  ~Met() { free(at); }
  bool first(uint8_t* p) {
    uint64_t h = (reinterpret_cast<uintptr_t>(p) >> 4) * 0x9e3779b97f4a7c15ull >> (64 - bits);
    for (; at[h]; h = (h + 1) & ((1ull << bits) - 1))
      if (at[h] == p) return false;
    at[h] = p;
    return true;
  }
};

// Every pool once, also where layers, or a layer's keys and values, share it: a second move would find places that the
// first has written.  y: CTAs over the pools of a launch, 0: one each.
template <typename Kernel>
int over_layers(Kernel kernel, Args& a, const moe_kv_pages* kv, int L, unsigned x, int y, int threads, cudaStream_t s) {
  Met met(2 * L);
  if (!met.at) return MOE_ENOMEM;
  a.first = 1;
  a.pools = 0;
  for (int i = 0; i < 2 * L; ++i) {
    uint8_t* p = static_cast<uint8_t*>(i & 1 ? kv[i / 2].v : kv[i / 2].k);
    if (met.first(p)) a.pool[a.pools++] = p;
    if (a.pools < kPools && (i + 1 < 2 * L || a.pools == 0)) continue;
    if (launch_pdl(kernel, dim3(x, y > 0 && y < a.pools ? y : a.pools), dim3(threads), 0, s, a) != cudaSuccess) return MOE_ECUDA;
    a.first = a.pools = 0;
  }
  return MOE_OK;
}

}  // namespace move
}  // namespace moe

extern "C" int moe_kv_compact(const moe_kv_pages* kv, int L, const moe_kv_batch* b, const int32_t* path, int path_stride,
                              const int32_t* count, int32_t* kv_len_out, int32_t* err_dev, moe_stream_t stream) {
  using namespace moe;
  move::Args a = {};
  if (!kv || L < 1 || L > move::kMaxLayers) return MOE_EINVAL;
  const int rc = kv_view(kv, b, &a.kv);
  if (rc) return rc;
  if (!move::alike(kv, L) || path_stride < 1 || (kv_len_out && kv_len_out == b->kv_len)) return MOE_EINVAL;
  if (b->B == 0) return MOE_OK;
  if (!path || !count || !b->q_start || !b->kv_len || (!b->page_table && b->table_stride > 0)) return MOE_EINVAL;
  // the lengths are written while other CTAs, and the launches of later layers, still read what they go by
  const long long B = b->B;
  if (kv_len_out && !(apart(kv_len_out, B, b->kv_len, B) && apart(kv_len_out, B, count, B) &&
                      apart(kv_len_out, B, path, B * path_stride) && apart(kv_len_out, B, b->q_start, B + 1) &&
                      apart(kv_len_out, B, b->page_table, B * b->table_stride)))
    return MOE_EINVAL;
  a.vecs = kv->D * (kv->e4m3 ? 1 : 2) / 16;
  a.path = path;
  a.count = count;
  a.path_stride = path_stride;
  a.len = kv_len_out;
  a.err = err_dev;
  const int places = sm_count() * move::kCompactPerSm;
  if (places < 1) return MOE_ECUDA;
  // CTAs for one turn of the GPU, each over several pools: the chain before the first row is paid once
  const int y = places > b->B ? places / b->B : 1;
  return move::over_layers(move::k_compact, a, kv, L, unsigned(b->B), y, move::kThreads, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_kv_copy_pages(const moe_kv_pages* kv, int L, const int32_t* src, const int32_t* dst,
                                 const int32_t* tokens, int n, int32_t* err_dev, moe_stream_t stream) {
  using namespace moe;
  move::Args a = {};
  if (!kv || L < 1 || L > move::kMaxLayers || n < 0 || n > 1 << 20) return MOE_EINVAL;
  const moe_kv_batch none = {};
  const int rc = kv_view(kv, &none, &a.kv);
  if (rc) return rc;
  if (!move::alike(kv, L)) return MOE_EINVAL;
  if (n == 0) return MOE_OK;
  if (!src || !dst) return MOE_EINVAL;
  a.vecs = kv->D * (kv->e4m3 ? 1 : 2) / 16;
  const long long pieces = (long long)kv->Hkv * kv->page * a.vecs;
  if (pieces > INT32_MAX - move::kPiece) return MOE_EINVAL;
  a.blocks = int((pieces + move::kPiece - 1) / move::kPiece);
  if ((long long)n * a.blocks > INT32_MAX) return MOE_EINVAL;
  a.src = src;
  a.dst = dst;
  a.tokens = tokens;
  a.err = err_dev;
  return move::over_layers(move::k_copy, a, kv, L, unsigned(n * a.blocks), 0, move::kCopyThreads,
                           reinterpret_cast<cudaStream_t>(stream));
}
