// Sparse and dense decode over the 656-byte fp8_ds_mla cache: the launchers of
// the kernel in smla_decode_kernel.cuh for that row format, and the decode
// with library-owned scratch.
#include "smla_decode_kernel.cuh"

namespace smla {

size_t decode_workspace_bytes(int32_t T, int32_t H, int32_t K) {
  return ws_layout(T, H, decode_splits(T, K)).total;
}

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s) {
  return launch_impl<kModeSlots>(a, s);
}

cudaError_t launch_decode_fused(const DecodeArgs& args, cudaStream_t s) {
  DecodeArgs a = args;
  set_divisors(a);
  return launch_impl<kModeTopk>(a, s);
}

cudaError_t launch_decode_dense(const DecodeArgs& args, cudaStream_t s) {
  DecodeArgs a = args;
  set_divisors(a);
  return launch_impl<kModeDense>(a, s);
}

// ---------------------------------------------------------------------------
// Decode with library-owned scratch, for callers that cannot allocate device
// memory themselves.  The split-K scratch lives in this file-scope array; every
// GPU that loads the library holds it until the process exits.  Host code
// must not pass the array's name to a kernel (on the host it names a stand-in,
// not device memory): its device address is looked up once per device with
// cudaGetSymbolAddress, with that device current, on the first call there.
static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];

namespace {

std::mutex g_noalloc_mutex;
void* g_noalloc_ptr[kMaxDevices] = {};

cudaError_t noalloc_scratch_ptr(void** ptr) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_noalloc_mutex);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess) return e;
    g_noalloc_ptr[dev] = p;
  }
  *ptr = g_noalloc_ptr[dev];
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_decode_noalloc(const DecodeArgs& args, cudaStream_t s) {
  const WsLayout w = ws_layout(args.T, args.H, decode_splits(args.T, args.K));
  if (w.total > kNoAllocScratchBytes) return cudaErrorInvalidValue;  // caller checks first
  DecodeArgs a = args;
  a.workspace = nullptr;
  a.workspace_bytes = 0;
  if (w.total > 0) {
    void* scratch = nullptr;
    cudaError_t e = noalloc_scratch_ptr(&scratch);
    if (e != cudaSuccess) return e;
    // the arrival counters must start at zero; a call that gave up part-way
    // could have left them otherwise
    const size_t rows = size_t(args.T < kTickRows ? args.T : kTickRows);
    e = cudaMemsetAsync(scratch, 0, rows * 2 * sizeof(int32_t), s);
    if (e != cudaSuccess) return e;
    a.workspace = scratch;
    a.workspace_bytes = w.total;
  }
  return launch_impl<kModeSlots>(a, s);
}

cudaError_t decode_error_word(uint32_t* flags, bool clear) {
  return read_error_word(flags, clear);
}

}  // namespace smla
