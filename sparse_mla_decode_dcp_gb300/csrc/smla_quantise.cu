// Activations to 8 bits: rows of bf16 in groups of 128 columns, each group as
// e4m3 codes and an fp32 scale, in the rounding of the 8-bit cache's rows:
//   scale = fp32(max |x| / 448),   code = e4m3(x / scale), each rounded once.
//
// Three bytes move for an element, so memory should bound it, and a value may
// cost few instructions: a product and half a conversion.  That is enough
// because x and the largest value, top, have 8 significant bits: let the
// quotient of x and top / 448 be compared with a number halfway between two
// codes, whose significand M has at most 5 bits.  With the significands X and T
// that is 7 X 2^k against M T: if they differ, the quotient is at least 2^-13 of
// itself away from the halfway number, far more than any rounding here.  If they
// are equal, x / scale is as far from it as the rounded scale is from top / 448:
//   * the scale is below: the quotient is above, by less than 2^-23 (and below
//     it the other way): the reciprocal is taken 2^-20 larger (smaller),
//     which decides these and no others;
//   * the scale is exact (7 divides T): the quotient is the halfway number
//     itself and goes to the even code: the product is rounded to 14 bits first.
#include <cuda_fp8.h>

#include "../../include/smla.h"
#include "smla_verify.h"

namespace smla {
namespace {

constexpr int kThreads = 256;
// Lanes of a group, values of a lane.  What a lane does once for its group (its
// place, the maximum, scale and reciprocal) costs as much as several values.
constexpr int kLanes = 8;
constexpr int kPer = 16;

// top / 448, rounded once: a product by the rounded reciprocal, corrected by its
// residual, is that for every bf16 top (all 256 significands were tried)
// whose quotient is normal.
__device__ __forceinline__ float over_448(float top) {
  if (top < 0x1p-116f) return __fdiv_rn(top, 448.f);
  constexpr float kInv = 1.f / 448.f;
  const float s = top * kInv;
  return fmaf(fmaf(-s, 448.f, top), kInv, s);
}

// A thread block's groups lie `step` apart in the list of all of them; the
// place of the next (column block, row, batch) follows by carries.
struct Walk {
  int64_t groups, step;
  int32_t row_groups, d_kb, d_m, d_g;  // step as column blocks, rows, batches
};

__global__ void __launch_bounds__(kThreads) fp8_quantise_kernel(const QuantiseArgs a, const Walk walk, bool vec) {
  const int sub = threadIdx.x & (kLanes - 1);
  griddep_launch_dependents();
  griddep_wait();
  int64_t i = int64_t(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  int32_t kb, m, g;
  if (walk.groups <= INT32_MAX) {
    const uint32_t row = uint32_t(i) / uint32_t(walk.row_groups);
    kb = int32_t(uint32_t(i) - row * uint32_t(walk.row_groups));
    g = int32_t(row / uint32_t(a.M));
    m = int32_t(row - uint32_t(g) * uint32_t(a.M));
  } else {
    const int64_t row = i / walk.row_groups;
    kb = int32_t(i - row * walk.row_groups);
    g = int32_t(row / a.M);
    m = int32_t(row - int64_t(g) * a.M);
  }
  // both halves of a warp stay while either has a group
  for (; __any_sync(0xffffffffu, i < walk.groups); i += walk.step) {
    const bool live = i < walk.groups;
    const int32_t col = kb * 128 + sub * kPer;
    const int32_t n = live ? min(max(a.K - col, 0), kPer) : 0;
    const uint16_t* x = a.x + g * a.xs.batch + m * a.xs.rows + col;
    float v[kPer];
    if (vec && n == kPer) {
      const uint4 w0 = reinterpret_cast<const uint4*>(x)[0], w1 = reinterpret_cast<const uint4*>(x)[1];
      const uint32_t p[kPer / 2] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int j = 0; j < kPer / 2; ++j) {
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
    const float scale = finite ? over_448(__uint_as_float(top)) : __uint_as_float(0x7fc00000u);
    uint32_t code[kPer / 4] = {};
    if (finite && scale >= 0x1p-126f) {
      const float off = fmaf(-scale, 448.f, __uint_as_float(top));  // exact
      float inv = __fdividef(1.f, scale);
      if (off == 0.f) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const float q = __fmul_rn(v[j], inv), c = __fmul_rn(q, 1025.f);
          v[j] = __fsub_rn(c, __fsub_rn(c, q));
        }
        inv = 1.f;
      } else {
        inv = fmaf(inv, copysignf(0x1p-20f, off), inv);
      }
#pragma unroll
      for (int j = 0; j < kPer; j += 2)
        code[j / 4] |= uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(v[j] * inv, v[j + 1] * inv), __NV_SATFINITE,
                                                         __NV_E4M3))
                       << (8 * (j & 2));
    }
    if (n > 0) {
      uint8_t* c = a.codes + g * a.cs.batch + m * a.cs.rows + col;
      if (n == kPer && (reinterpret_cast<uintptr_t>(c) & 15) == 0) {
        *reinterpret_cast<uint4*>(c) = make_uint4(code[0], code[1], code[2], code[3]);
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (j < n) c[j] = uint8_t(code[j / 4] >> (8 * (j & 3)));
      }
    }
    if (live && sub == 0) a.scales[g * a.ss.batch + m * a.ss.rows + kb * a.ss.cols] = scale;
    kb += walk.d_kb;
    int32_t carry = kb >= walk.row_groups;
    kb -= carry ? walk.row_groups : 0;
    m += walk.d_m + carry;
    carry = m >= a.M;
    m -= carry ? a.M : 0;
    g += walk.d_g + carry;
  }
}

}  // namespace

cudaError_t launch_fp8_quantise(const QuantiseArgs& a, cudaStream_t s) {
  Walk w;
  w.row_groups = int32_t((int64_t(a.K) + 127) / 128);
  w.groups = int64_t(a.G) * a.M * w.row_groups;
  const int64_t per = kThreads / kLanes;
  const int64_t need = (w.groups + per - 1) / per;
  const unsigned grid = unsigned(need < 152 * 6 ? need : 152 * 6);
  w.step = int64_t(grid) * per;
  const int64_t rows = w.step / w.row_groups;
  w.d_kb = int32_t(w.step - rows * w.row_groups);
  w.d_g = int32_t(rows / a.M);
  w.d_m = int32_t(rows - int64_t(w.d_g) * a.M);
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && a.xs.batch % 8 == 0 && a.xs.rows % 8 == 0;
  return launch_overlapped(fp8_quantise_kernel, grid, kThreads, 0, s, a, w, vec);
}

}  // namespace smla
