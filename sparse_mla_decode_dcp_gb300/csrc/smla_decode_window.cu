// Windowed decode with sinks over either cache: the launcher of the kernel in
// smla_decode_kernel.cuh for generated rows with a gap.
#define SMLA_WAITS_OUT_OF_LINE  // see wait_phase
#include "smla_decode_kernel.cuh"

namespace smla {

size_t window_decode_workspace_bytes(int32_t T, int32_t H, int32_t K) {
  return ws_layout(T, H, plan_splits(T, K, kWindowList).splits).total;
}

cudaError_t launch_decode_window(const DecodeArgs& args, bool fp4, cudaStream_t s) {
  DecodeArgs a = args;
  set_divisors(a);
  return fp4 ? launch_impl<kModeWindow, Fp4Rows>(a, s) : launch_impl<kModeWindow, Fp8Rows>(a, s);
}

cudaError_t decode_window_error_word(uint32_t* flags, bool clear) {
  return read_error_word(flags, clear);
}

}  // namespace smla
