// Keys that a drafted tree's node sees, as bits (not part of the ABI).  Plain C++: the host runs it too.
#pragma once

#include <limits.h>
#include <stdint.h>

#ifdef __CUDACC__
#define MOE_BOTH __host__ __device__ __forceinline__
#else
#define MOE_BOTH inline
#endif

namespace moe {
namespace attn {

// Of the 32 nodes from 32 w on: bits of a node's row of a mask.  Before the first are keys that every node sees.
MOE_BOTH uint32_t mask_word(const uint32_t* row, int words, int w) {
  return w < 0 ? 0xffffffffu : w < words ? row[w] : 0u;
}
// 32 bits of two words, from bit `by` < 32 of the low one on.
MOE_BOTH uint32_t shift_pair(uint32_t low, uint32_t high, int by) {
#ifdef __CUDA_ARCH__
  return __funnelshift_r(low, high, by);
#else
  return uint32_t((uint64_t(high) << 32 | low) >> by);
#endif
}
MOE_BOTH int lowest_bit(uint32_t x) {
#ifdef __CUDA_ARCH__
  return __ffs(x) - 1;
#else
  return __builtin_ctz(x);
#endif
}
MOE_BOTH int lesser(int a, int b) { return a < b ? a : b; }

// Bit j of seen: a node sees key j of 32 WORDS keys, of which the first is node node0's (before the tree: below 0) and
// those from `end` on are not there.  row, words, deep: the node's mask of itself and those above it, and its depth;
// depth: of its request's nodes.
template <int WORDS>
MOE_BOTH void seen_keys(const uint32_t* row, int words, const int32_t* depth, int deep, int window, int node0, int end,
                        uint32_t* seen) {
  // the first key that it may see: before the tree as far as the window goes, without one any (32 k below that is a number too)
  const int begin = window > 0 ? lesser(deep - window + 1, 0) - node0 : INT_MIN / 2;
  uint32_t low = mask_word(row, words, node0 >> 5);
#ifdef __CUDA_ARCH__
#pragma unroll
#endif
  for (int k = 0; k < WORDS; ++k) {
    const uint32_t high = mask_word(row, words, (node0 >> 5) + k + 1);
    uint32_t m = shift_pair(low, high, node0 & 31);
    low = high;
    const int last = end - 32 * k, first = begin - 32 * k;
    m = last >= 32 ? m : last <= 0 ? 0u : m & ((1u << last) - 1);
    m = first <= 0 ? m : first >= 32 ? 0u : m & (0xffffffffu << first);
    if (window > 0 && deep >= window) {  // a window smaller than the tree is deep: nodes, one by one
      for (uint32_t rest = m; rest; rest &= rest - 1) {
        const int node = node0 + 32 * k + lowest_bit(rest);
        if (node >= 0 && depth[node] <= deep - window) m &= ~(rest & (0u - rest));
      }
    }
    seen[k] = m;
  }
}

}  // namespace attn
}  // namespace moe
