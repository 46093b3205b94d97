// What the two products of e4m3.cuh do with finished sums: four neighbouring columns of
// a row at a time.
#pragma once

#include "e4m3.cuh"

namespace tb {

// SiLU(gate)·up.  The quotient is __fdividef (2 ulp; 0 for gates below -87, where SiLU
// is under 1e-35): the division of the language takes a slow path for a numerator of 0
// or below 2^-126, which rows of zeros meet everywhere (333 rows of 2048 outputs from
// 768: 28.8 -> 9.5 us, with the issuing warp's change).
__device__ __forceinline__ float gated(float g, float u) { return __fdividef(g, 1.0f + expf(-g)) * u; }

// The same where the result is rounded to 16 bits or fewer and there are many: 2^x and 1/x as
// the hardware has them.  The exponent's rounding shifts e^-g by up to |g|·2^-23, which SiLU
// feels by at most 0.28·|g|·2^-23 (and relative to its size by |g|·2^-23, for gates far below
// zero), and the two functions add 2^-21 of its size.  Below -87 1/x is 0, as above.
__device__ __forceinline__ float gated_short(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * r * u;
}

__device__ __forceinline__ void put4(void* y, int y_dtype, size_t at, float4 v) {
  if (y_dtype == TB_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(y) + at) = v;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<bf16*>(y) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}
// The fours at at(0), ..., at(B - 1).  (All are requested before the first is converted: with
// the type told apart for each, 512 x 4096 x 14336 took 52.0 us, 37.7 so.)
template <int B, typename At> __device__ __forceinline__ void get4(float4 (&v)[B], const void* y, int y_dtype, At at) {
  if (y_dtype == TB_F32) {
#pragma unroll
    for (int b = 0; b < B; ++b) v[b] = *reinterpret_cast<const float4*>(static_cast<const float*>(y) + at(b));
    return;
  }
  uint2 w[B];
#pragma unroll
  for (int b = 0; b < B; ++b) w[b] = *reinterpret_cast<const uint2*>(static_cast<const bf16*>(y) + at(b));
#pragma unroll
  for (int b = 0; b < B; ++b)
    v[b] = make_float4(__uint_as_float(w[b].x << 16), __uint_as_float(w[b].x & 0xffff0000u), __uint_as_float(w[b].y << 16),
                       __uint_as_float(w[b].y & 0xffff0000u));
}

// Up to four exponent bytes of consecutive K blocks as one word, the first in the low
// byte; `n` of them exist.  Missing ones read as 2^0.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* p, int n) {
  if (n >= 4 && ((uintptr_t)p & 3u) == 0) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t w = 0x7f7f7f7fu;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) w = (w & ~(0xffu << (8 * i))) | (uint32_t)p[i] << (8 * i);
  return w;
}

}  // namespace tb
