// moe_paged_attention for heads of 64 columns: the kernels of attn.cuh at their tiles of rows, and of attn_chunk.cuh.
#include "attn.cuh"
#include "attn_chunk.cuh"

namespace moe {
namespace attn {

int launch_d64(const Args& a, int e4m3, int nr, int sms, cudaStream_t s) {
  if (e4m3) {
    switch (nr) {
      case 16: return launch_one<64, 16, true, false>(a, sms, s);
      case 32: return launch_one<64, 32, true, false>(a, sms, s);
      case 64: return launch_one<64, 64, true, false>(a, sms, s);
      default: return chunk::launch<64, true, false>(a, sms, s);
    }
  } else {
    switch (nr) {
      case 16: return launch_one<64, 16, false, false>(a, sms, s);
      case 32: return launch_one<64, 32, false, false>(a, sms, s);
      case 64: return launch_one<64, 64, false, false>(a, sms, s);
      default: return chunk::launch<64, false, false>(a, sms, s);
    }
  }
}

int opt_in_d64() {
  // the join keeps the split of L1 and shared memory that the kernel before it had
  auto as_before = [](auto* join) {
    return cudaFuncSetAttribute(join, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess;
  };
  return opt_in<64, 16, false, false>() ||
                 opt_in<64, 32, false, false>() ||
                 opt_in<64, 64, false, false>() ||
                 opt_in<64, 16, true, false>() ||
                 opt_in<64, 32, true, false>() ||
                 opt_in<64, 64, true, false>() ||
                 chunk::opt_in<64, false, false>() ||
                 chunk::opt_in<64, true, false>() ||
                 as_before(k_join<64, 16>) ||
                 as_before(k_join<64, 32>) ||
                 as_before(k_join<64, 48>) ||
                 as_before(k_join<64, 64>) ||
                 as_before(k_join<64, 256>) ||
                 as_before(k_join_many<64>)
             ? MOE_ECUDA
             : MOE_OK;
}

template <>
int launch_join<64>(const Args& a, int nr, bool many, int ctas, cudaStream_t s) {
  const dim3 threads(kJoinThreads);
  cudaError_t e;
  if (many) e = launch_pdl(k_join_many<64>, dim3(ctas, a.G < 16 ? a.G : 16), threads, 0, s, a);
  else if (nr == 16) e = launch_pdl(k_join<64, 16>, dim3(ctas, join_y(16)), threads, 0, s, a);
  else if (nr == 32) e = launch_pdl(k_join<64, 32>, dim3(ctas, join_y(32)), threads, 0, s, a);
  else if (nr == 48) e = launch_pdl(k_join<64, 48>, dim3(ctas, join_y(48)), threads, 0, s, a);
  else if (nr == 64) e = launch_pdl(k_join<64, 64>, dim3(ctas, join_y(64)), threads, 0, s, a);
  else e = launch_pdl(k_join<64, kChunkRows>, dim3(ctas, join_y(kChunkRows)), threads, 0, s, a);
  return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}

}  // namespace attn
}  // namespace moe
