// moe_paged_attention for heads of 256 columns: the kernels of attn.cuh at their tiles of rows.
#include "attn.cuh"

namespace moe {
namespace attn {

int launch_d256(const Args& a, int e4m3, int nr, int sms, cudaStream_t s) {
  if (e4m3) {
    switch (nr) {
      case 16: return launch_one<256, 16, true, false>(a, sms, s);
      case 32: return launch_one<256, 32, true, false>(a, sms, s);
      default: return launch_one<256, 64, true, false>(a, sms, s);
    }
  } else {
    switch (nr) {
      case 16: return launch_one<256, 16, false, false>(a, sms, s);
      case 32: return launch_one<256, 32, false, false>(a, sms, s);
      default: return launch_one<256, 64, false, false>(a, sms, s);
    }
  }
}

int opt_in_d256() {
  // the join keeps the split of L1 and shared memory that the kernel before it had
  auto as_before = [](auto* join) {
    return cudaFuncSetAttribute(join, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess;
  };
  return opt_in<256, 16, false, false>() ||
                 opt_in<256, 32, false, false>() ||
                 opt_in<256, 64, false, false>() ||
                 opt_in<256, 16, true, false>() ||
                 opt_in<256, 32, true, false>() ||
                 opt_in<256, 64, true, false>() ||
                 as_before(k_join<256, 16>) ||
                 as_before(k_join<256, 32>) ||
                 as_before(k_join<256, 64>) ||
                 as_before(k_join<256, 128>) ||
                 as_before(k_join_many<256>)
             ? MOE_ECUDA
             : MOE_OK;
}

template <>
int launch_join<256>(const Args& a, int nr, bool many, int ctas, cudaStream_t s) {
  const dim3 threads(kJoinThreads);
  cudaError_t e;
  if (many) e = launch_pdl(k_join_many<256>, dim3(ctas, a.G < 16 ? a.G : 16), threads, 0, s, a);
  else if (nr == 16) e = launch_pdl(k_join<256, 16>, dim3(ctas, join_y(16)), threads, 0, s, a);
  else if (nr == 32) e = launch_pdl(k_join<256, 32>, dim3(ctas, join_y(32)), threads, 0, s, a);
  else if (nr == 64) e = launch_pdl(k_join<256, 64>, dim3(ctas, join_y(64)), threads, 0, s, a);
  else e = launch_pdl(k_join<256, 128>, dim3(ctas, join_y(128)), threads, 0, s, a);
  return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}

}  // namespace attn
}  // namespace moe
