// moe_paged_attention for heads of 256 columns: the kernels of attn.cuh at their tiles of rows.
#include "attn.cuh"

namespace moe {
namespace attn {

int launch_d256(const Args& a, int e4m3, int nr, int ctas, cudaStream_t s) {
  switch (nr) {
    case 16: return e4m3 ? launch_one<256, 16, true>(a, ctas, s) : launch_one<256, 16, false>(a, ctas, s);
    default: return e4m3 ? launch_one<256, 64, true>(a, ctas, s) : launch_one<256, 64, false>(a, ctas, s);
  }
}

int opt_in_d256() {
  return opt_in<256, 16>() || opt_in<256, 64>() ? MOE_ECUDA : MOE_OK;
}

}  // namespace attn
}  // namespace moe
