// 8-bit integer quantisation of rows, shared by the quantiser and the few-token kernels.
//
// Row x of n elements: D = max(max_i |x_i|, 127 * 2^-126), scale = D / 127 (one fp32 division) and
// q_i = the whole number nearest to the real quotient 127 x_i / D, ties to even, so |q_i| <= 127. The
// floor on D keeps the scale a normal number (an all-zero row gets 2^-126 and zeros). A row that
// holds a NaN or an infinity gets scale NaN and q = 0: whatever is computed from it is NaN.
//
// The quotient is rounded exactly, without a division per element: bf16 rows do hold ties (half of
// the row's largest value is 63.5), and a product with the rounded reciprocal of D would take them
// either way. q0 = rint(fl(127 x) fl(1/D)) is the nearest whole number or, within about 2^-16 of
// a tie, a neighbour; the sign of 2|127 x - q0 D| - D, computed exactly near a tie (fma), tells which.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr float kQ8Floor = 127.0f * 0x1p-126f;

// magnitude bits of v, which order as the magnitudes do, NaN above infinity
__device__ __forceinline__ unsigned mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct Q8Row {
  float c127, D, rD, scale;   // 127 c, D c, 1 / (D c), D / 127; c = 2^-10 for rows near the type's top
  bool bad;
  Q8Row() = default;
  __device__ __forceinline__ explicit Q8Row(unsigned amax_bits) {
    bad = amax_bits >= 0x7f800000u;
    const float d = bad ? 1.0f : fmaxf(__uint_as_float(amax_bits), kQ8Floor);
    const float c = d >= 0x1p100f ? 0x1p-10f : 1.0f;   // 127 x stays finite; a power of two is exact
    c127 = 127.0f * c;
    D = d * c;
    rD = 1.0f / D;
    scale = bad ? __uint_as_float(0x7fc00000u) : d / 127.0f;
  }
};

// q of N elements (a multiple of 4) as N packed bytes. F32: x may be any fp32 value (127 x is then
// rounded, and its rounding error enters the sign test); otherwise x holds bf16 values (127 x exact).
template <bool F32, int N>
__device__ __forceinline__ void q8_pack(const float (&x)[N], const Q8Row& r, unsigned (&out)[N / 4]) {
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: the sum's low mantissa bits are the integer
  unsigned m[N];
  bool fix = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float th = x[i] * r.c127;
    const float s = __builtin_fmaf(th, r.rD, kMagic);
    m[i] = __float_as_uint(s);
    const float q = s - kMagic;
    const float d = __builtin_fmaf(-q, r.D, th);
    float e = __builtin_fmaf(2.0f, fabsf(d), -r.D);
    if constexpr (F32) e = __builtin_fmaf(2.0f, copysignf(1.0f, d) * __builtin_fmaf(x[i], r.c127, -th), e);
    fix |= e >= 0.0f;
  }
  if (fix) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float th = x[i] * r.c127;
      const float q = __uint_as_float(m[i]) - kMagic;
      const float d = __builtin_fmaf(-q, r.D, th);
      float e = __builtin_fmaf(2.0f, fabsf(d), -r.D);
      if constexpr (F32) e = __builtin_fmaf(2.0f, copysignf(1.0f, d) * __builtin_fmaf(x[i], r.c127, -th), e);
      if (e > 0.0f || (e == 0.0f && (m[i] & 1u))) m[i] += d >= 0.0f ? 1u : ~0u;
    }
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const unsigned lo = __builtin_amdgcn_perm(m[4 * i + 1], m[4 * i], 0x0c0c0400u);
    const unsigned hi = __builtin_amdgcn_perm(m[4 * i + 3], m[4 * i + 2], 0x04000c0cu);
    out[i] = r.bad ? 0u : (lo | hi);
  }
}

// w silu(a) b of the 8-bit layer, for few tokens and many alike, so that a token's h has the same bits in either
// (with two accuracies, bytes of h near a tie differed). silu(a) = a / (1 + e^-a) with e^-a = 2^t e^c: t = -a log2 e as
// rounded (by up to 2^-18 at the ends, which alone would cost e^-a 30 units in the last place), c = -a - t ln 2 what
// the rounding left out, e^c = 1 + c. The hardware's power of two and reciprocal are good to one unit, the whole to
// 1.5 to 3. Below a = -88, where the power would leave fp32, 0. The gate/up product of 131072 pairs of 768 values takes
// 454 us with the plain power and reciprocal, 492 so, and 522 with expf and a division.
__device__ __forceinline__ float weighted_swiglu8(float w, float a, float b) {
  constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147182f, kLn2Low = -1.90465430e-9f;
  const float z = __builtin_amdgcn_fmed3f(-a, -104.0f, 88.0f);
  const float t = z * kLog2e;
  const float c = __builtin_fmaf(-t, kLn2Low, __builtin_fmaf(-t, kLn2, z));
  const float p = __builtin_amdgcn_exp2f(t);
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(p, c, p));
  return w * (a * (a < -88.0f ? 0.0f : s) * b);
}

}  // namespace moe
