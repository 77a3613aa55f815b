// Activations to 8 bits: rows of bf16 in groups of 128 columns, each group as
// e4m3 codes and an fp32 scale, in the rounding of the 8-bit cache's rows:
//   scale = fp32(max |x| / 448),   code = e4m3(x / scale), each rounded once.
//
// Three bytes move for an element, so memory bounds it; sixteen lanes take a
// group, eight values each.  The quotient is rounded to e4m3 from fp32: with
// y = 1 / scale, q = x y corrected by its residual is within an ulp of x /
// scale and equal to it where that is an fp32 number.  Rounding q would go
// wrong only where q is halfway between two codes and the quotient is not;
// there the sign of the residual x - q scale tells its side, and q moves one
// ulp to it.
#include <cuda_fp8.h>

#include "../../include/smla.h"
#include "smla_verify.h"

namespace smla {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16;   // of a group
constexpr int kPer = 8;      // values of a lane

__device__ __forceinline__ float quotient(float x, float scale, float inv) {
  float q = x * inv;
  q = fmaf(fmaf(-q, scale, x), inv, q);
  // halves between codes have at most five significant bits
  if ((__float_as_uint(q) & 0x3ffffu) == 0) {
    const float r = fmaf(-q, scale, x);
    if (r != 0.f && q != 0.f)
      q = __uint_as_float(__float_as_uint(q) + ((r < 0.f) == (q < 0.f) ? 1u : ~0u));
  }
  return q;
}

__global__ void __launch_bounds__(kThreads) fp8_quantise_kernel(const QuantiseArgs a, int64_t groups,
                                                                int32_t row_groups, bool vec) {
  const int sub = threadIdx.x & (kLanes - 1);
  griddep_launch_dependents();
  griddep_wait();
  const int64_t step = int64_t(gridDim.x) * (kThreads / kLanes);
  for (int64_t i0 = int64_t(blockIdx.x) * (kThreads / kLanes); i0 < groups; i0 += step) {
    const int64_t i = i0 + threadIdx.x / kLanes;
    const bool live = i < groups;
    const int64_t row = live ? i / row_groups : 0;
    const int32_t kb = int32_t(live ? i - row * row_groups : 0);
    const int64_t g = row / a.M;
    const int64_t m = row - g * a.M;
    const int32_t col = kb * 128 + sub * kPer;
    const int32_t n = live ? min(max(a.K - col, 0), kPer) : 0;
    const uint16_t* x = a.x + g * a.xs.batch + m * a.xs.rows + col;
    float v[kPer];
    if (vec && n == kPer) {
      const uint4 w = *reinterpret_cast<const uint4*>(x);
      const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(p[j] << 16);
        v[2 * j + 1] = __uint_as_float(p[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = j < n ? __uint_as_float(uint32_t(x[j]) << 16) : 0.f;
    }
    // magnitudes order as their bits do, infinities and NaNs above the rest
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool finite = top < 0x7f800000u;
    const float scale = finite ? __fdiv_rn(__uint_as_float(top), 448.f) : __uint_as_float(0x7fc00000u);
    const bool coded = finite && scale >= 0x1p-126f;
    uint32_t code[kPer / 4] = {};
    if (coded) {
      // small groups are taken 2^64 larger, where residuals are exact too
      const float up = scale < 0x1p-60f ? 0x1p64f : 1.f;
      const float unit = scale * up;
      const float inv = __frcp_rn(unit);
#pragma unroll
      for (int j = 0; j < kPer; j += 2) {
        const float2 q = make_float2(quotient(v[j] * up, unit, inv), quotient(v[j + 1] * up, unit, inv));
        code[j / 4] |= uint32_t(__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3)) << (8 * (j & 2));
      }
    }
    if (n > 0) {
      uint8_t* c = a.codes + g * a.cs.batch + m * a.cs.rows + col;
      if (n == kPer && (reinterpret_cast<uintptr_t>(c) & 7) == 0) {
        *reinterpret_cast<uint2*>(c) = make_uint2(code[0], code[1]);
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (j < n) c[j] = uint8_t(code[j / 4] >> (8 * (j & 3)));
      }
    }
    if (live && sub == 0) a.scales[g * a.ss.batch + m * a.ss.rows + kb * a.ss.cols] = scale;
  }
}

}  // namespace

cudaError_t launch_fp8_quantise(const QuantiseArgs& a, cudaStream_t s) {
  const int32_t row_groups = int32_t((int64_t(a.K) + 127) / 128);
  const int64_t groups = int64_t(a.G) * a.M * row_groups;
  const int64_t per = kThreads / kLanes;
  const int64_t need = (groups + per - 1) / per;
  const unsigned grid = unsigned(need < 152 * 64 ? need : 152 * 64);
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && a.xs.batch % 8 == 0 && a.xs.rows % 8 == 0;
  return launch_overlapped(fp8_quantise_kernel, grid, kThreads, 0, s, a, groups, row_groups, vec);
}

}  // namespace smla
