// Quantization of K/V values into e4m3 pools, shared by the cache writers.
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

}  // namespace pa
