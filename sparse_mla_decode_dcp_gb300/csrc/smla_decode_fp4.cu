// Sparse decode over the 416-byte fp4 cache: the launchers of the kernel in
// smla_decode_kernel.cuh for that row format.
#define SMLA_WAITS_OUT_OF_LINE  // see wait_phase
#include "smla_decode_kernel.cuh"

namespace smla {

size_t fp4_decode_workspace_bytes(int32_t T, int32_t H, int32_t K) {
  return ws_layout(T, H, plan_splits(T, K, kMaxList).splits).total;
}

cudaError_t launch_decode_fp4(const DecodeArgs& a, cudaStream_t s) {
  return launch_impl<kModeSlots, Fp4Rows>(a, s);
}

cudaError_t launch_decode_fused_fp4(const DecodeArgs& args, cudaStream_t s) {
  DecodeArgs a = args;
  set_divisors(a);
  return launch_impl<kModeTopk, Fp4Rows>(a, s);
}

cudaError_t decode_fp4_error_word(uint32_t* flags, bool clear) {
  return read_error_word(flags, clear);
}

}  // namespace smla
