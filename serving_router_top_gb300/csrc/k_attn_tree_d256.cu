// moe_tree_attention for heads of 256 columns: the kernels of attn.cuh at their tiles of rows, and of attn_wide.cuh.
#include "attn_wide.cuh"

namespace moe {
namespace attn {

int launch_tree_d256(const Args& a, int e4m3, int nr, int sms, cudaStream_t s) {
  if (e4m3) {
    switch (nr) {
      case 16: return launch_one<256, 16, true, true>(a, sms, s);
      case 32: return launch_one<256, 32, true, true>(a, sms, s);
      default: return wide::launch<true>(a, sms, s);
    }
  } else {
    switch (nr) {
      case 16: return launch_one<256, 16, false, true>(a, sms, s);
      case 32: return launch_one<256, 32, false, true>(a, sms, s);
      default: return wide::launch<false>(a, sms, s);
    }
  }
}

int opt_in_tree_d256() {
  return opt_in<256, 16, false, true>() ||
                 opt_in<256, 32, false, true>() ||
                 opt_in<256, 16, true, true>() ||
                 opt_in<256, 32, true, true>() ||
                 wide::opt_in<false>() ||
                 wide::opt_in<true>()
             ? MOE_ECUDA
             : MOE_OK;
}

}  // namespace attn
}  // namespace moe
