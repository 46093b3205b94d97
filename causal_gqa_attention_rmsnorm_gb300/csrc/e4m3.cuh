// Rows and weights of 8-bit floating-point codes (e4m3) with power-of-two scales:
// what the kernels of the 8-bit projections share, and their launchers.
//
// A block is 128 columns of one row, or 128 x 128 of a weight matrix.  Its scale is
// 2^e, held as the byte e + 127, with e the smallest integer in [kScaleMin, kScaleMax]
// for which the block's largest finite magnitude is at most 448·2^e; a value x is held
// as the code of x / 2^e, which is exact before the rounding to the code's 4 bits.
#pragma once

#include "common.cuh"

namespace tb {

constexpr int kBlk = 128;          // columns (and rows of weights) per scale

// The upper end leaves no finite fp32 value to saturate; the lower end keeps 2^-e and
// the scales' product with any code far from fp32's subnormals.
constexpr int kScaleMin = -100, kScaleMax = 120;

// Smallest e in range with top <= 448·2^e (448 = 1.75·2^8); top finite and not negative.
__device__ __forceinline__ int block_exponent(float top) {
  const int b = __float_as_int(top);
  const int e = (b >> 23) - 127 - 8 + ((b & 0x7fffff) > 0x600000 ? 1 : 0);
  return min(max(e, kScaleMin), kScaleMax);
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Four values, already divided by their scale, to codes.  NaN stays NaN.
__device__ __forceinline__ uint32_t codes_of4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// |x| for a block's largest magnitude: infinities and NaN do not count.
__device__ __forceinline__ float finite_mag(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}
// x / 2^e before its rounding to a code; an infinity becomes NaN (the conversion
// would saturate it).
__device__ __forceinline__ float to_code(float x, float inv) { return fabsf(x) < INFINITY ? x * inv : NAN; }

// Rows of codes [rows, cols] with scales [rows, ceil(cols / 128)], or weights
// [rows, cols] with scales [ceil(rows / 128), ceil(cols / 128)].
struct Coded {
  const uint8_t* codes;
  const uint8_t* scale;
};

// e4m3_rows.cu
struct RowsArgs {
  const void* x;         // [M, d]
  const void* r;         // [M, d], or null
  void* h;               // [M, d] x + r, where r is given
  const void* g;         // [d]
  float eps;
  int M, d;
  uint8_t* codes;        // [M, d]
  uint8_t* scale;        // [M, ceil(d / 128)]
};
constexpr int kNormMax = 32768;    // widest row whose mean square one CTA forms in registers
cudaError_t launch_norm_e4m3(const RowsArgs& a, int x_dtype, int r_dtype, cudaStream_t s);
cudaError_t launch_quant_e4m3(const RowsArgs& a, int x_dtype, cudaStream_t s);
// w [K, N] ([in, out]) -> codes [N, K], scales [ceil(N / 128), ceil(K / 128)]
cudaError_t launch_pack_e4m3(const void* w, int dtype, int K, int N, uint8_t* codes, uint8_t* scale, cudaStream_t s);

// The products.  x: rows [M, K]; w (and w3): weights [N, K]; y [M, N].
struct GemmArgs {
  Coded x, w, w3;        // w3: the gated product's second matrix
  int M, N, K;
  const void* res;       // [M, N] of y's type, added to the product, or null
  void* y;               // [M, N] fp32 or bf16 (y_dtype), or codes with y_scale
  uint8_t* y_scale;
  int y_dtype;
};
// e4m3_gemm_few.cu: any sizes; tiles of 16, 32, 64 or (not gated) 128 rows; the rule
int e4m3_few_tile(int M, int N, int K, int mats, bool light, int sms);
cudaError_t launch_gemm_e4m3_few(const GemmArgs& a, int tile, cudaStream_t s);
cudaError_t launch_gated_e4m3_few(const GemmArgs& a, int tile, cudaStream_t s);
// e4m3_gemm_many.cu: CTA pairs, any sizes
cudaError_t launch_gemm_e4m3_many(const GemmArgs& a, bool one, cudaStream_t s);
cudaError_t launch_gated_e4m3_many(const GemmArgs& a, bool one, cudaStream_t s);

}  // namespace tb
