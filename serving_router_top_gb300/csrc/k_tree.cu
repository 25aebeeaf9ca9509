// Depths and masks of drafted token trees, for all layers of a step.
//
// A node's row of `above` holds the nodes on its way to the root, itself among them.  Ways double: after
// step r a node knows the 2^r nodes next above it and the node after those, so eight steps reach the root
// of any tree of 256 nodes.  `below` is the transpose, 32 x 32 bits a vote.  A CTA a request.
//
// What bounds it: launch and the chain q_start, parent, steps: 2.3 us for one tree of 16 nodes, 2.4 for 64 trees.  In
// attention each row or key would walk up a chain of loads in every layer; a mask is one load.
#include "paged.cuh"

namespace moe {
namespace tree {

constexpr int kWords = 8, kNodes = 32 * kWords;

struct Args {
  const int32_t *q_start, *parent;
  int32_t* depth;
  uint32_t *above, *below;
  int T, words;
  int32_t* err;
};

__global__ void __launch_bounds__(kNodes) k_tree(const __grid_constant__ Args a) {
  __shared__ uint32_t mask[kNodes][kWords + 1];
  __shared__ short next[kNodes], far[kNodes];  // the node after those known, and the steps to it (or to the root)
  pdl_trigger();
  pdl_wait();
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5, W = a.words;
  const RowSpan rows = row_span(a.q_start, blockIdx.x, a.T);
  const int s0 = rows.s0, n = rows.n;
  if (n < 0 && i == 0) set_error(a.err, MOE_ERANGE);
  if (n <= 0) return;
  const int m = min(n, 32 * W);
  int up = -1;
  if (i < m) {
    up = a.parent[s0 + i];
    if (up < -1 || up >= i) {
      set_error(a.err, MOE_ERANGE);
      up = -1;
    }
  }
#pragma unroll
  for (int w = 0; w < kWords; ++w) mask[i][w] = w == warp ? 1u << lane : 0u;
  next[i] = short(up);
  far[i] = up >= 0;
  while (__syncthreads_or(up >= 0)) {
    uint32_t more[kWords];
    int steps = 0, to = -1;
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) more[w] = mask[up][w];
      steps = far[up];
      to = next[up];
    }
    __syncthreads();
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) mask[i][w] |= more[w];
      far[i] += short(steps);
      next[i] = short(to);
      up = to;
    }
  }
  if (i < m) a.depth[s0 + i] = far[i];
  for (int x = i; x < m * W; x += kNodes) a.above[(long long)s0 * W + x] = mask[x / W][x % W];
  // blocks of 32 nodes: below[j] bit k = above[k] bit j
  for (int x = warp; x < W * W; x += kWords) {
    const int jw = x / W, kw = x % W, j = 32 * jw + lane;
    if (32 * jw >= m) break;
    const uint32_t mine = kw >= jw && 32 * kw + lane < m ? mask[32 * kw + lane][jw] : 0u;
    uint32_t row = 0;
#pragma unroll
    for (int b = 0; b < 32; ++b) {
      const uint32_t v = __ballot_sync(0xffffffffu, mine >> b & 1);
      if (lane == b) row = v;
    }
    if (j < m) a.below[(long long)(s0 + j) * W + kw] = row;
  }
  if (n > m) {
    if (i == 0) set_error(a.err, MOE_ERANGE);
    for (int x = m + i; x < n; x += kNodes) {
      a.depth[s0 + x] = 0;
      for (int w = 0; w < W; ++w) a.above[(long long)(s0 + x) * W + w] = a.below[(long long)(s0 + x) * W + w] = 0;
    }
  }
}

}  // namespace tree
}  // namespace moe

extern "C" int moe_tree_prepare(const moe_kv_batch* b, const moe_tree* t, int32_t* err_dev, moe_stream_t stream) {
  using namespace moe;
  if (!b || !t || b->B < 0 || b->T < 0 || t->words < 1 || t->words > tree::kWords) return MOE_EINVAL;
  if (b->T == 0 || b->B == 0) return MOE_OK;
  if (!b->q_start || !t->parent || !t->depth || !t->above || !t->below) return MOE_EINVAL;
  const tree::Args a = {b->q_start, t->parent, t->depth, t->above, t->below, b->T, t->words, err_dev};
  return launch_pdl(tree::k_tree, dim3(b->B), dim3(tree::kNodes), 0, reinterpret_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? MOE_OK
             : MOE_ECUDA;
}
