// moe_paged_attention for heads of 256 columns: the kernels of attn.cuh at their tiles of rows.
#include "attn.cuh"

namespace moe {
namespace attn {

int launch_d256(const Args& a, int e4m3, int nr, int sms, cudaStream_t s) {
  if (e4m3) {
    switch (nr) {
      case 16: return launch_one<256, 16, true>(a, sms, s);
      case 32: return launch_one<256, 32, true>(a, sms, s);
      default: return launch_one<256, 64, true>(a, sms, s);
    }
  } else {
    switch (nr) {
      case 16: return launch_one<256, 16, false>(a, sms, s);
      case 32: return launch_one<256, 32, false>(a, sms, s);
      default: return launch_one<256, 64, false>(a, sms, s);
    }
  }
}

int opt_in_d256() {
  return opt_in<256, 16, false>() ||
                 opt_in<256, 32, false>() ||
                 opt_in<256, 64, false>() ||
                 opt_in<256, 16, true>() ||
                 opt_in<256, 32, true>() ||
                 opt_in<256, 64, true>()
             ? MOE_ECUDA
             : MOE_OK;
}

}  // namespace attn
}  // namespace moe
