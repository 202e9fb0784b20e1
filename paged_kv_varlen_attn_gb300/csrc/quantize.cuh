// Quantization of K/V values into e4m3 and 4-bit pools, shared by the cache writers.
#pragma once

#include "device_common.cuh"

namespace pa {

// x / s correctly rounded to float32 wherever the quotient decides an e4m3
// code, from y = RN(1/s): q0 = RN(x y), the remainder r = x - q0 s (exact,
// one FMA) and q = RN(q0 + r y). By Markstein's theorem (y within half an
// ulp of 1/s and q0 within one ulp of x/s make RN(q0 + r y) the correctly
// rounded quotient, as long as r neither underflows nor the quotient
// overflows), q is RN(x/s). Zero, |q0| >= 512, infinite and NaN products
// take q0 (a zero product keeps its sign, which q0 + r y would lose for
// -0; where r = 0 otherwise, q0 + r y is q0 anyway; every quotient of at
// least 464 saturates to the same code). With 2^-32 <= |s| <= 2^32 the
// reciprocal is normal and every quotient of at least 2^-11 (below that the
// code is a signed zero either way) has a normal, hence exact, remainder;
// other scales take the IEEE division. The product and the two FMAs run on
// two values at a time (f32x2): three instructions per pair of values
// besides the selects, instead of two divisions.
struct ScaleDiv {
  float s, ns, y;   // the scale, its negation and RN(1 / s)
  bool fast;        // |s| in [2^-32, 2^32]
};

__device__ __forceinline__ ScaleDiv scale_div(float s) {
  const float as = fabsf(s);
  return {s, -s, __frcp_rn(s), as >= 0x1p-32f && as <= 0x1p32f};
}

__device__ __forceinline__ float pick_quotient(float q0, float q) {
  return (q0 != 0.f && fabsf(q0) < 512.f) ? q : q0;
}

// The e4m3 bytes of 8 floats divided by the scale.
__device__ __forceinline__ uint2 quantize8(float (&v)[8], const ScaleDiv& d) {
  if (d.fast) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      float q0a, q0b, ra, rb, qa, qb;
      ffma2(q0a, q0b, v[k], v[k + 1], d.y, d.y, -0.f, -0.f);     // RN(x y)
      ffma2(ra, rb, q0a, q0b, d.ns, d.ns, v[k], v[k + 1]);       // x - q0 s
      ffma2(qa, qb, ra, rb, d.y, d.y, q0a, q0b);                 // q0 + r y
      v[k] = pick_quotient(q0a, qa);
      v[k + 1] = pick_quotient(q0b, qb);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __fdiv_rn(v[k], d.s);
  }
  const uint32_t w0 = f32x2_to_e4m3x2(v[0], v[1]) | (f32x2_to_e4m3x2(v[2], v[3]) << 16);
  const uint32_t w1 = f32x2_to_e4m3x2(v[4], v[5]) | (f32x2_to_e4m3x2(v[6], v[7]) << 16);
  return make_uint2(w0, w1);
}

// The same of 8 bf16 or f16 values of a 16-byte vector.
template <bool F16>
__device__ __forceinline__ uint2 quantize8(uint4 x, const ScaleDiv& d) {
  const uint32_t h[4] = {x.x, x.y, x.z, x.w};
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = Elem<F16>::unpack(h[k]);
    v[2 * k] = a.x;
    v[2 * k + 1] = a.y;
  }
  return quantize8(v, d);
}

// The 4-bit codes of a head's row, 8 consecutive elements per lane, LPH lanes
// per row (see pa.h for the format and its roundings): a word of this lane's 8
// codes, and in *params the row's f16 scale (low half) and minimum. The
// quotient is a product with the float32 reciprocal of the rounded scale, and
// adding 1.5 * 2^23 rounds it to the nearest integer, ties to even, into the low
// bits of the sum; eight multiply-adds (modulo 2^32) place those, and what the
// exponents add up to is a constant. A NaN anywhere in the row makes scale and
// minimum NaN, hence the row's values.
template <int LPH>
__device__ __forceinline__ uint32_t quantize8_int4(const float (&x)[8], int lane,
                                                   uint32_t* params) {
  constexpr float kTop = 32752.f;   // (2 * kTop) / 15 and kTop are f16 numbers' size
  float f[8], lo = INFINITY, hi = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    nan |= isnan(x[k]);
    f[k] = fminf(fmaxf(x[k], -kTop), kTop);
    lo = fminf(lo, f[k]);
    hi = fmaxf(hi, f[k]);
  }
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const uint32_t row = ((LPH == 32 ? 0u : 1u << LPH) - 1u) << (lane / LPH * LPH);
  nan = (__ballot_sync(0xffffffffu, nan) & row) != 0;
  const __half s = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 1.f / 15.f));
  const __half m = __float2half_rn(lo);
  *params = nan ? 0x7fff7fffu
                : static_cast<uint32_t>(__half_as_ushort(s)) |
                      static_cast<uint32_t>(__half_as_ushort(m)) << 16;
  const float sf = __half2float(s), mf = __half2float(m);
  const float inv = sf > 0.f && !nan ? __frcp_rn(sf) : 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float q = fminf(fmaxf(__fmul_rn(__fsub_rn(f[k], mf), inv), 0.f), 15.f);
    w += __float_as_uint(__fadd_rn(q, 12582912.f)) << (4 * (k >> 1) + 16 * (k & 1));
  }
  // Eight times the bits of 1.5 * 2^23, each at its shift.
  constexpr uint32_t kBase = 0x4B400000u * 0x11111111u;
  return w - kBase;
}

}  // namespace pa
