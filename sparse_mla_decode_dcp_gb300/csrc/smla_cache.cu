// The packed cache's other side: writing a step's latent rows into it (norm,
// rotary positions, quantisation and scatter in one pass) and gathering rows
// back to bf16 or fp32.
//
// Write.  For token t with latent x (512) and rope part z (64):
//   y = x g / sqrt(mean(x^2) + eps)          (g = gamma; y = x without one)
//   rope pair (a, b) at angle (c, s) -> (a c - b s, a s + b c)
//   fp8 row: per 128 dims scale = fp32(max|y| / 448), code = e4m3(y / scale)
//   fp4 row: per 16 dims scale = e4m3(max|y| / 6), code = e2m1(y / scale)
// Every rounding to a code or a stored scale is of the exact quotient: the
// products x g of two bf16 are exact in fp32, and everything else runs in
// pairs of fp32 (value and remainder), about 45 bits, rounded to odd before
// the conversion, so that a quotient next to a rounding border lands on the
// side 64-bit arithmetic puts it.  An fp32 quotient would put about one code
// in 10^6 on the other side, a whole step of e2m1 (up to a third of the
// value).  fp64 would do too but runs at about 1/60 of the fp32 rate here.
//
// One warp per row: a lane owns 16 consecutive latent dims (one fp4 group, an
// eighth of an fp8 group) and one rope pair.  Measured with norm and rotation,
// rows to random slots: 64 rows 2.0 us (fp4) and 2.6 (fp8), about a launch;
// 16,384 rows 9.4 and 11.1; 65,536 rows 33.1 and 39.2, 3.6 and 3.5 TB/s, where
// the issue slots are 73-75% busy with the exact sums and quotients, not HBM.
// Rows without a slot leave their warps' places empty: 16,384 of which one in
// four is written 4.9 and 5.5, 4,096 that all are 4.3 and 5.1.
//
// Gather.  One warp per row, 8 dims per lane and step, so that every store is
// 16 consecutive bytes a lane; kRows rows at once keep their loads in flight
// together.  Bound by HBM: row + 4 bytes in, 1152 (bf16) or 2304 (fp32) out.
// Measured on random rows: 4,001 to bf16 2.6 us (fp8 and fp4), 131,072 38.3
// and 33.4 us, 262,144 73.8 and 64.5 (6.4 TB/s, 96% of a plain copy's rate); to
// fp32 138 and 131 (5.5 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "../../include/smla.h"
#include "smla_internal.h"

namespace smla {
namespace {

__device__ unsigned int g_cache_error;

constexpr int kWarps = 8;

// Two fp32 side by side, in the packed instructions that issue once for both:
// a write is bound by its instructions (fp4: 424 a row instead of 505, 16,384
// rows 9.4 -> 8.5 us).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void f2_split(F2 a, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 f2_sub(F2 a, F2 b) { return f2_fma(b, f2(-1.f, -1.f), a); }

// A value as the unevaluated sum of two fp32.
struct Pair {
  float hi, lo;
};

// Exact sum of two fp32 (Knuth's two-sum).
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}

// a + b, hi not rounded again: lo stays the sum of the parts cut off so far.
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return {s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo))};
}

// hi + lo with hi the nearest fp32 (|lo| well below |hi|).
__device__ __forceinline__ Pair pair_norm(Pair a) {
  const float hi = __fadd_rn(a.hi, a.lo);
  return {hi, __fsub_rn(a.lo, __fsub_rn(hi, a.hi))};
}

// a / d for an fp32 divisor; hi is the nearest fp32.
__device__ __forceinline__ Pair pair_div(Pair a, float d) {
  const float q = __fdiv_rn(a.hi, d);
  const float rem = __fadd_rn(__fmaf_rn(-q, d, a.hi), a.lo);  // zero when q is exact
  const float c = __fdividef(rem, d);
  const float hi = __fadd_rn(q, c);
  return {hi, __fsub_rn(c, __fsub_rn(hi, q))};
}

// x * p for an fp32 factor.
__device__ __forceinline__ Pair pair_mul(float x, Pair p) {
  const float v = __fmul_rn(x, p.hi);
  return {v, __fadd_rn(__fmaf_rn(x, p.hi, -v), __fmul_rn(x, p.lo))};
}

// hi + lo rounded to odd in fp32: truncated toward zero, last bit set when
// anything was cut off.  Rounding that once more to a format of at most 22
// bits equals rounding hi + lo itself.
__device__ __forceinline__ float round_odd(Pair p) {
  if (p.lo == 0.f) return p.hi;
  uint32_t b = __float_as_uint(p.hi);
  if ((p.lo < 0.f) != (p.hi < 0.f)) --b;  // |hi + lo| < |hi|
  return __uint_as_float(b | 1u);
}

// a / d rounded to odd, inv = 1 / d in fp32: the quotient is corrected once,
// to the nearest fp32, and what is left of a then has the sign of the part
// that was cut off (zero, exactly, when nothing was).
__device__ __forceinline__ float quotient_odd(Pair a, float d, float inv) {
  const float v = __fmul_rn(a.hi, inv);
  const float q = __fmaf_rn(__fadd_rn(__fmaf_rn(-v, d, a.hi), a.lo), inv, v);
  if (q == 0.f) return a.hi;  // zero, or too small for fp32: its sign is what counts
  return round_odd({q, __fadd_rn(__fmaf_rn(-q, d, a.hi), a.lo)});
}

// 1 / sqrt(m): one Newton step from the fp32 reciprocal square root, its
// residual 1 - m r^2 formed exactly enough with fused multiply-adds.
__device__ __forceinline__ Pair pair_rsqrt(Pair m) {
  const float r = rsqrtf(m.hi);
  const float t = __fmul_rn(r, r);
  const float te = __fmaf_rn(r, r, -t);
  float u = __fmaf_rn(-m.hi, t, 1.f);
  u = __fsub_rn(u, __fmaf_rn(m.hi, te, __fmul_rn(m.lo, t)));
  return {r, 0.5f * r * u};
}

// The codes of a lane's 16 values y r / d, packed into kWords words by
// pack(v0, v1, pair index).  In fp32 alone a quotient is within 2^-21 of its
// exact value, so where the codes of v (1 - 2^-20) and v (1 + 2^-20) agree they
// are the exact quotient's; a warp with a value that close to a border (about
// one fp8 row in 100, one fp4 row in 500) takes the exact quotients.  Called by
// whole warps.
template <int kWords, class Pack>
__device__ __forceinline__ void quantise(const F2* y, Pair r, float d, float inv, uint32_t* w,
                                         Pack pack) {
  constexpr int kPairs = 8 / kWords;  // pairs of values a word
  const float t = __fmul_rn(r.hi, inv);
  const float tb = __fmul_rn(t, 1.f - 0x1p-20f), ta = __fmul_rn(t, 1.f + 0x1p-20f);
  const F2 below = f2(tb, tb), above = f2(ta, ta);
  uint32_t near = 0;
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float a, b;
      f2_split(f2_mul(y[kPairs * k + i], below), a, b);
      lo |= pack(a, b, i);
      f2_split(f2_mul(y[kPairs * k + i], above), a, b);
      hi |= pack(a, b, i);
    }
    w[k] = lo;
    near |= lo ^ hi;
  }
  if (!__any_sync(0xffffffffu, near != 0)) return;
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    w[k] = 0;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float a, b;
      f2_split(y[kPairs * k + i], a, b);
      w[k] |= pack(quotient_odd(pair_mul(a, r), d, inv), quotient_odd(pair_mul(b, r), d, inv), i);
    }
  }
}

// A plain load, not through the read-only path (see launch_overlapped).
template <class T>
__device__ __forceinline__ T load(const T* p) {
  return *p;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A lane's 16 fp8 codes of the values y r / d.
__device__ __forceinline__ uint4 fp8_codes(const F2* y, Pair r, float d) {
  uint32_t w[4];
  quantise<4>(
      y, r, d, __frcp_rn(d), w,
      [](float a, float b, int i) {
        return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3))
               << (16 * (i & 1));
      });
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The row's 16 codes of each lane, and a group's scale from its first lane.
__device__ __forceinline__ void store_fp8(uint8_t* dst, int lane, uint4 codes, float scale) {
  *reinterpret_cast<uint4*>(dst + 16 * lane) = codes;
  if ((lane & 7) == 0) *reinterpret_cast<float*>(dst + 512 + 4 * (lane >> 3)) = scale;
}

// The latent part of an fp8 row with a group that is zero, not finite or near
// the low end of fp32, apart from the path of the others; it reads its inputs
// again.  Near the low end products and remainders would lose bits,
// and r / scale overflow: such a group (its scale below 2^-59 or so) is
// quantised 2^64 times as large, its values formed so that they are exact at
// that size.  Called by whole warps.
__noinline__ __device__ void write_fp8_special(const uint16_t* src, const uint16_t* gamma, uint8_t* dst,
                                               Pair r, int lane) {
  uint32_t x[8], g[8];
  float amax = 0.f, zero = 0.f;  // zero stays so unless a value is not finite
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[k] = reinterpret_cast<const volatile uint32_t*>(src)[8 * lane + k];
    g[k] = gamma ? reinterpret_cast<const volatile uint32_t*>(gamma)[8 * lane + k] : 0x3f803f80u;  // ones
    const float u = __fmul_rn(bf16_lo(x[k]), bf16_lo(g[k])), v = __fmul_rn(bf16_hi(x[k]), bf16_hi(g[k]));
    amax = fmaxf(amax, fmaxf(fabsf(u), fabsf(v)));
    zero = __fmaf_rn(u, 0.f, __fmaf_rn(v, 0.f, zero));
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    zero += __shfl_xor_sync(0xffffffffu, zero, o);
  }
  const bool tiny = !(__fmul_rn(amax, r.hi) >= 0x1p-51f && amax >= 0x1p-100f);
  const float up = tiny ? 0x1p64f : 1.f;
  auto product = [&](float v, float gv) {  // the smaller factor takes the 2^64
    return fabsf(v) < 1.f ? __fmul_rn(__fmul_rn(v, up), gv) : __fmul_rn(v, __fmul_rn(gv, up));
  };
  F2 y[8];
  amax = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float u = product(bf16_lo(x[k]), bf16_lo(g[k])), v = product(bf16_hi(x[k]), bf16_hi(g[k]));
    amax = fmaxf(amax, fmaxf(fabsf(u), fabsf(v)));
    y[k] = f2(u, v);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float scale = __fmul_rn(pair_div(pair_mul(amax, r), 448.f).hi, tiny ? 0x1p-64f : 1.f);
  // below the normal fp32 range: the group is stored as zeros
  if (scale < 0x1p-126f) scale = 0.f;
  const bool finite = isfinite(r.hi) && isfinite(r.lo) && zero == 0.f && isfinite(scale);
  const bool keep = finite && scale > 0.f;
  const uint4 codes = fp8_codes(y, r, keep ? __fmul_rn(scale, up) : 1.f);
  store_fp8(dst, lane, keep ? codes : make_uint4(0u, 0u, 0u, 0u),
            finite ? scale : __int_as_float(0x7fc00000));
}

// Five CTAs an SM (48 registers): with the call of write_fp8_special the
// compiler would take 52, and 65,536 fp8 rows 10% longer.
template <bool kFp4>
__global__ void __launch_bounds__(kWarps * 32, 5) cache_write_kernel(const CacheWriteArgs a) {
  constexpr int kRowBytes = kFp4 ? SMLA_FP4_ROW_BYTES : SMLA_ROW_BYTES;
  constexpr int kRope = kRowBytes - 128;
  const int lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  griddep_launch_dependents();
  if (t >= a.T) return;
  griddep_wait();
  const int32_t slot = load(a.slots + t);
  const int32_t pos = a.cos_sin ? load(a.positions + t) : 0;
  if (slot < 0) return;
  const bool bad_slot = slot >= a.num_slots;
  const bool bad_pos = a.cos_sin && (pos < 0 || pos >= a.num_positions);
  if (bad_slot || bad_pos) {
    if (lane == 0)
      atomicOr(&g_cache_error, (bad_slot ? SMLA_DEVERR_SLOT_RANGE : 0u) |
                                   (bad_pos ? SMLA_DEVERR_POSITION : 0u));
    return;
  }
  const uint16_t* src = a.kv + t * a.kv_row_stride;
  uint8_t* dst = a.kv_cache + int64_t(slot) * kRowBytes;

  // every load of the row first
  uint32_t x[8], g[8];
  {
    const uint4 v0 = load(reinterpret_cast<const uint4*>(src) + 2 * lane);
    const uint4 v1 = load(reinterpret_cast<const uint4*>(src) + 2 * lane + 1);
    x[0] = v0.x, x[1] = v0.y, x[2] = v0.z, x[3] = v0.w;
    x[4] = v1.x, x[5] = v1.y, x[6] = v1.z, x[7] = v1.w;
  }
  // the lane's rope pair: values 2 lane, 2 lane + 1, or lane, lane + 32
  const uint16_t* zs = src + SMLA_V_DIM;
  uint32_t z;
  if (a.rope_pairs)
    z = load(reinterpret_cast<const uint32_t*>(zs) + lane);
  else
    z = uint32_t(load(zs + lane)) | uint32_t(load(zs + 32 + lane)) << 16;
  float co = 1.f, si = 0.f;
  if (a.cos_sin) {
    co = load(a.cos_sin + int64_t(pos) * 64 + lane);
    si = load(a.cos_sin + int64_t(pos) * 64 + 32 + lane);
  }
  if (a.gamma) {
    const uint4 v0 = load(reinterpret_cast<const uint4*>(a.gamma) + 2 * lane);
    const uint4 v1 = load(reinterpret_cast<const uint4*>(a.gamma) + 2 * lane + 1);
    g[0] = v0.x, g[1] = v0.y, g[2] = v0.z, g[3] = v0.w;
    g[4] = v1.x, g[5] = v1.y, g[6] = v1.z, g[7] = v1.w;
  }

  F2 y[8];  // x g, exact
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = f2(bf16_lo(x[k]), bf16_hi(x[k]));
  Pair r = {1.f, 0.f};
  if (a.gamma) {
    // the even and the odd values' sums of squares, each with what its
    // additions cut off
    F2 sum = f2_mul(y[0], y[0]), cut = f2(0.f, 0.f);
#pragma unroll
    for (int k = 1; k < 8; ++k) {
      const F2 q = f2_mul(y[k], y[k]);
      const F2 s = f2_add(sum, q);
      const F2 qq = f2_sub(s, sum);
      cut = f2_add(cut, f2_add(f2_sub(sum, f2_sub(s, qq)), f2_sub(q, qq)));
      sum = s;
    }
    Pair even, odd;
    f2_split(sum, even.hi, odd.hi);
    f2_split(cut, even.lo, odd.lo);
    Pair ss = pair_add(even, odd);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      ss = pair_add(ss, {__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)});
    ss = pair_norm(ss);
    const Pair m = two_sum(__fmul_rn(ss.hi, 1.f / 512.f), a.eps);
    r = pair_rsqrt({m.hi, __fadd_rn(m.lo, __fmul_rn(ss.lo, 1.f / 512.f))});
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = f2_mul(y[k], f2(bf16_lo(g[k]), bf16_hi(g[k])));
  }
  // the group's largest magnitude; a value that is not finite (an infinite
  // or NaN input, or a sum of squares past fp32) makes the group's scale NaN
  float amax = 0.f;
  F2 zero = f2(0.f, 0.f);  // stays zero unless a value is not finite
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float u, v;
    f2_split(y[k], u, v);
    amax = fmaxf(amax, fmaxf(fabsf(u), fabsf(v)));
    zero = f2_fma(y[k], f2(0.f, 0.f), zero);
  }
  float z0, z1;
  f2_split(zero, z0, z1);
  if (!kFp4) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const Pair largest = pair_mul(amax, r);
    // 2^-51 or more and finite, by its bits
    const bool plain = uint32_t(__float_as_int(largest.hi) - 0x26000000) < 0x7f800000u - 0x26000000u &&
                       amax >= 0x1p-100f && z0 == 0.f && z1 == 0.f;
    const bool all_plain = __all_sync(0xffffffffu, plain);
    const float scale = pair_div(largest, 448.f).hi;
    const uint4 codes = fp8_codes(y, r, scale);
    if (all_plain)
      store_fp8(dst, lane, codes, scale);
    else
      write_fp8_special(src, a.gamma, dst, r, lane);
  } else {
    const bool finite = isfinite(r.hi) && isfinite(r.lo) && z0 == 0.f && z1 == 0.f;
    const Pair s = pair_div(pair_mul(amax, r), 6.f);
    const uint32_t sc = __nv_cvt_float_to_fp8(round_odd(s), __NV_SATFINITE, __NV_E4M3);
    const float scale = __half2float(__half(__nv_cvt_fp8_to_halfraw(sc, __NV_E4M3)));
    const float d = scale > 0.f ? scale : 1.f;
    const float inv = __frcp_rn(d);
    uint32_t w[2];
    quantise<2>(
        y, r, d, inv, w,
        [](float a, float b, int i) {
          return uint32_t(__nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest))
                 << (8 * (i & 3));
        });
    const bool keep = scale > 0.f && finite;
    *reinterpret_cast<uint2*>(dst + 8 * lane) = keep ? make_uint2(w[0], w[1]) : make_uint2(0u, 0u);
    dst[256 + lane] = finite ? uint8_t(sc) : uint8_t(0x7f);
  }

  // rope
  const float za = bf16_lo(z), zb = bf16_hi(z);
  const uint32_t o = a.cos_sin ? bf16x2_bits(__fmaf_rn(za, co, -__fmul_rn(zb, si)),
                                             __fmaf_rn(za, si, __fmul_rn(zb, co)))
                               : z;
  if (a.rope_pairs) {
    *reinterpret_cast<uint32_t*>(dst + kRope + 4 * lane) = o;
  } else {
    *reinterpret_cast<uint16_t*>(dst + kRope + 2 * lane) = uint16_t(o);
    *reinterpret_cast<uint16_t*>(dst + kRope + 64 + 2 * lane) = uint16_t(o >> 16);
  }
}

// 8 consecutive values of a row to its output (bf16 or fp32).
template <bool kFp32>
__device__ __forceinline__ void store8(void* out, int64_t at, const float* v) {
  if (kFp32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    __stcs(o, make_float4(v[0], v[1], v[2], v[3]));
    __stcs(o + 1, make_float4(v[4], v[5], v[6], v[7]));
  } else {
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at),
           make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]),
                      bf16x2_bits(v[6], v[7])));
  }
}

__device__ __forceinline__ void e4m3x2(uint32_t c, float& a, float& b) {
  const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(c & 0xffffu), __NV_E4M3));
  a = __low2float(h);
  b = __high2float(h);
}

// c s, rounded to fp32, or (kOdd, where bf16 follows) rounded to odd, so that
// the rounding to bf16 is of the product itself: the product is exact, or lies
// between two neighbouring fp32 of which one has an odd last bit.
template <bool kOdd>
__device__ __forceinline__ float times(float c, float s) {
  if (!kOdd) return __fmul_rn(c, s);
  const float lo = __fmul_rd(c, s), hi = __fmul_ru(c, s);
  return (__float_as_uint(lo) & 1u) ? lo : hi;
}

constexpr int kRows = 4;

template <bool kFp4, bool kFp32>
__global__ void __launch_bounds__(kWarps * 32) cache_gather_kernel(const CacheGatherArgs a) {
  constexpr int kRowBytes = kFp4 ? SMLA_FP4_ROW_BYTES : SMLA_ROW_BYTES;
  constexpr int kRope = kRowBytes - 128;
  constexpr int kCodeBytes = kFp4 ? 4 : 8;  // 8 dims
  const int lane = threadIdx.x & 31;
  const int64_t n0 = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kRows;
  griddep_launch_dependents();
  if (n0 >= a.N) return;
  griddep_wait();
  int32_t slot[kRows];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    slot[i] = n0 + i < a.N ? load(a.slots + n0 + i) : -1;
    if (slot[i] >= a.num_slots) {
      bad = true;
      slot[i] = -1;
    }
  }
  uint2 code[kRows][2];
  float scale[kRows][2];
  uint32_t rope[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    code[i][0] = code[i][1] = make_uint2(0, 0);
    scale[i][0] = scale[i][1] = 0.f;
    rope[i] = 0;
    if (slot[i] >= 0) {
      const uint8_t* src = a.kv_cache + int64_t(slot[i]) * kRowBytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* p = src + kCodeBytes * (32 * h + lane);
        if (kFp4) {
          code[i][h].x = load(reinterpret_cast<const uint32_t*>(p));
          scale[i][h] = __half2float(
              __half(__nv_cvt_fp8_to_halfraw(load(src + 256 + 16 * h + (lane >> 1)), __NV_E4M3)));
        } else {
          code[i][h] = load(reinterpret_cast<const uint2*>(p));
          scale[i][h] = load(reinterpret_cast<const float*>(src + 512) + 2 * h + (lane >> 4));
        }
      }
      rope[i] = load(reinterpret_cast<const uint32_t*>(src + kRope) + lane);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (n0 + i >= a.N) break;
    const int64_t row = (n0 + i) * a.out_row_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
      if (kFp4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2 c = __half2(__nv_cvt_fp4x2_to_halfraw2(
              __nv_fp4x2_storage_t((code[i][h].x >> (8 * k)) & 0xffu), __NV_E2M1));
          v[2 * k] = __low2float(c) * scale[i][h];
          v[2 * k + 1] = __high2float(c) * scale[i][h];
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t w = k < 2 ? code[i][h].x : code[i][h].y;
          e4m3x2(w >> (16 * (k & 1)), v[2 * k], v[2 * k + 1]);
          v[2 * k] = times<!kFp32>(v[2 * k], scale[i][h]);
          v[2 * k + 1] = times<!kFp32>(v[2 * k + 1], scale[i][h]);
        }
      }
      store8<kFp32>(a.out, row + 256 * h + 8 * lane, v);
    }
    if (kFp32)
      __stcs(reinterpret_cast<float2*>(static_cast<float*>(a.out) + row + 512) + lane,
             make_float2(bf16_lo(rope[i]), bf16_hi(rope[i])));
    else
      __stcs(reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row + 512) + lane, rope[i]);
  }
  if (bad && lane == 0) atomicOr(&g_cache_error, SMLA_DEVERR_SLOT_RANGE);
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs& a, bool fp4, cudaStream_t s) {
  const unsigned grid = unsigned((int64_t(a.T) + kWarps - 1) / kWarps);
  return launch_overlapped(fp4 ? cache_write_kernel<true> : cache_write_kernel<false>, grid, kWarps * 32,
                           0, s, a);
}

cudaError_t launch_cache_gather(const CacheGatherArgs& a, bool fp4, bool fp32, cudaStream_t s) {
  const unsigned grid = unsigned((int64_t(a.N) + kWarps * kRows - 1) / (kWarps * kRows));
  const auto kernel = fp4 ? (fp32 ? cache_gather_kernel<true, true> : cache_gather_kernel<true, false>)
                          : (fp32 ? cache_gather_kernel<false, true> : cache_gather_kernel<false, false>);
  return launch_overlapped(kernel, grid, kWarps * 32, 0, s, a);
}

cudaError_t cache_error_word(uint32_t* flags, bool clear) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_cache_error, sizeof(v));
  if (e != cudaSuccess) return e;
  *flags |= v;
  if (clear) {
    v = 0;
    e = cudaMemcpyToSymbol(g_cache_error, &v, sizeof(v));
  }
  return e;
}

}  // namespace smla
