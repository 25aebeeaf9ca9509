// moe_tree_attention for heads of 64 columns: the kernels of attn.cuh at their tiles of rows, and of attn_chunk.cuh.
#include "attn.cuh"
#include "attn_chunk.cuh"

namespace moe {
namespace attn {

int launch_tree_d64(const Args& a, int e4m3, int nr, int sms, cudaStream_t s) {
  if (e4m3) {
    switch (nr) {
      case 16: return launch_one<64, 16, true, true>(a, sms, s);
      case 32: return launch_one<64, 32, true, true>(a, sms, s);
      case 64: return launch_one<64, 64, true, true>(a, sms, s);
      default: return chunk::launch<64, true, true>(a, sms, s);
    }
  } else {
    switch (nr) {
      case 16: return launch_one<64, 16, false, true>(a, sms, s);
      case 32: return launch_one<64, 32, false, true>(a, sms, s);
      case 48: return launch_one<64, 48, false, true>(a, sms, s);
      case 64: return launch_one<64, 64, false, true>(a, sms, s);
      default: return chunk::launch<64, false, true>(a, sms, s);
    }
  }
}

int opt_in_tree_d64() {
  return opt_in<64, 16, false, true>() ||
                 opt_in<64, 32, false, true>() ||
                 opt_in<64, 64, false, true>() ||
                 opt_in<64, 48, false, true>() ||
                 opt_in<64, 16, true, true>() ||
                 opt_in<64, 32, true, true>() ||
                 opt_in<64, 64, true, true>() ||
                 chunk::opt_in<64, false, true>() ||
                 chunk::opt_in<64, true, true>()
             ? MOE_ECUDA
             : MOE_OK;
}

}  // namespace attn
}  // namespace moe
