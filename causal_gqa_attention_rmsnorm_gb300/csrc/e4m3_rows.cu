// Rows to e4m3 codes with one power-of-two scale per 128 columns: RMSNorm (with the
// residual's addition on the way) or the rows as they are; and weights to codes with
// one scale per 128 x 128.
//
//   h = x + r,  y = h / sqrt(mean h² + eps) * g,  codes of y per block of 128
//
// One pass over memory: a row lies in the registers of 32 to 1024 threads, eight
// neighbouring columns to a thread, so that 16 lanes of a warp hold the 128 columns of
// a block and its largest magnitude takes four shuffles.  The sum, the mean square and
// the quotients are fp32; y is never rounded to anything but its code.
//
// Bound by memory: 32768 x 4096 of bf16 with a residual of bf16 133 us, 7.1 TB/s of what it
// has to move, as fast as memory is copied; 8192 x 11008 of fp32 alone 64 us (7.0); 3777 x
// 768 of fp32 7.4 us (4.3: a short launch, most of it start and end); one row 2.1 us.
#include <algorithm>

#include "e4m3.cuh"
#include "gemm_tc.cuh"
#include "sm100_ptx.cuh"

namespace tb {
namespace {

// Eight neighbouring values as they lie in memory, and as fp32.  (Plain loads: the
// kernel before may still be writing other memory while this grid is resident, so
// nothing is read as constant.)
template <typename T> struct Eight {
  static constexpr int N = Vec16<T>::N;
  Vec16<T> u[8 / N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) u[i].raw = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) u[i].raw = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float get(int i) const { return u[i / N].get(i % N); }
};
template <> struct Eight<void> {};
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) {
  uint4 w;
  uint32_t* u = &w.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = w;
}

// The codes of a thread's eight values v·s·g of a block that 16 lanes hold (g: or all
// ones); the first of the 16 also stores the scale.  t = v·g comes first, so that the
// row's s and the block's 2^-e are one factor: s·2^-e is exact, and the largest |t|·s is
// the largest |t·s| (rounding keeps the order).  A block whose largest |t|·s is no finite
// number (an infinity in it, v·g beyond fp32 where v·s·g is not, a row without a finite
// s) is done again in the other order and with infinities told from values; a NaN is
// passed over by the maximum and kept by the conversion.
template <typename T, bool NORM>
__device__ __forceinline__ void put_block(const float (&v)[8], float s, const Eight<T>& g, bool in, uint8_t* codes,
                                          uint8_t* scale) {
  float t[8], top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = NORM ? v[i] * g.get(i) : v[i];
#pragma unroll
  for (int i = 0; i < 8; i += 2) top = ptx::fmax3(top, fabsf(t[i]), fabsf(t[i + 1]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float f = s;
  if (__any_sync(0xffffffffu, !(top * s < INFINITY))) {
    top = 0.f;
    f = 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (NORM) t[i] = v[i] * s * g.get(i);
      top = fmaxf(top, finite_mag(t[i]));
      if (fabsf(t[i]) == INFINITY) t[i] = NAN;
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (!in) return;
  const int e = block_exponent(top * f);
  f *= pow2i(-e);
  *reinterpret_cast<uint2*>(codes) = make_uint2(codes_of4(t[0] * f, t[1] * f, t[2] * f, t[3] * f),
                                                codes_of4(t[4] * f, t[5] * f, t[6] * f, t[7] * f));
  if ((threadIdx.x & 15) == 0) *scale = (uint8_t)(e + 127);
}

// RT: the type of r (void: none).  A row takes `tpr` threads (a multiple of 32), NV
// eights each, a CTA blockDim.x / tpr rows; with NORM that is one, or a row per warp.
// Without NORM, blockIdx.y counts pieces of tpr·NV·8 columns.
template <typename T, typename RT, int NV> constexpr bool kLean = sizeof(T) == 2 && NV == 4 && std::is_same<RT, void>::value;
// (64 registers without r keep four CTAs of 256 on an SM: 16384 x 4096 of bf16 54 -> 45
// us.  Elsewhere no number of CTAs is asked for, which is not the same as one: 16384 x
// 4096 of fp32 with r 123 and 147 us.)
template <typename T, typename RT, bool NORM, int NV>
__global__ void __launch_bounds__(NV == 1 ? 1024 : kLean<T, RT, NV> ? 256 : 512, kLean<T, RT, NV> ? 4 : 0) k_rows_e4m3(RowsArgs a, int tpr) {
  constexpr bool RES = !std::is_same<RT, void>::value;
  __shared__ float part[32];
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int col0 = (NORM ? 0 : (int)blockIdx.y * tpr * NV * 8) + (int)(threadIdx.x % tpr) * 8;
  const size_t row = (size_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr, base = row * a.d;
  pdl_wait();
  if (row >= a.M) return;              // (whole warps; with a barrier ahead, whole CTAs)
  Eight<T> x[NV];
  Eight<RT> r[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = col0 + i * tpr * 8;
    x[i].zero();                       // (columns past the row read as zeros throughout)
    if constexpr (RES) r[i].zero();
    if (c < a.d) {
      x[i].load(static_cast<const T*>(a.x) + base + c);
      if constexpr (RES) r[i].load(static_cast<const RT*>(a.r) + base + c);
    }
  }
  float v[NV][8], q = 0.f, s = 1.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = x[i].get(j);
      if constexpr (RES) v[i][j] += r[i].get(j);
      q = fmaf(v[i][j], v[i][j], q);
    }
  Eight<T> g[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = col0 + i * tpr * 8;
    g[i].zero();
    if (NORM && c < a.d) g[i].load(static_cast<const T*>(a.g) + c);
  }
  if constexpr (NORM) {
    q = warp_sum(q);
    if (tpr > 32) {
      // the sums of the row's warps, added by each warp in the same order
      if (lane == 0) part[threadIdx.x >> 5] = q;
      __syncthreads();
      q = warp_sum(lane < tpr / 32 ? part[lane] : 0.f);
    }
    s = 1.0f / sqrtf(q / (float)a.d + a.eps);
  }
  const int blocks = (a.d + kBlk - 1) / kBlk;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = col0 + i * tpr * 8;
    put_block<T, NORM>(v[i], s, g[i], c < a.d, a.codes + base + c, a.scale + row * blocks + c / kBlk);
  }
  // (last: 32768 x 4096 of bf16 132 us, 141 with h stored before the sum)
  if constexpr (RES) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col0 + i * tpr * 8;
      if (c < a.d) store8(static_cast<T*>(a.h) + base + c, v[i]);
    }
  }
}

// Codes [N, K] of w [K, N]: a CTA takes a block of 128 x 128, keeps it in shared memory
// as fp32 (rows of w, one word of padding, so that both ways of reading it are free of
// conflicts) and writes it transposed.  Done once per weight set.
template <typename T> __global__ void __launch_bounds__(256) k_pack_e4m3(const T* w, int K, int N, uint8_t* codes, uint8_t* scale) {
  extern __shared__ float tile[];      // [128][129]
  __shared__ float tops[8];
  const int k0 = blockIdx.x * kBlk;
  for (int n0 = blockIdx.y * kBlk; n0 < N; n0 += gridDim.y * kBlk) {
    float top = 0.f;
    for (int i = threadIdx.x; i < kBlk * kBlk; i += 256) {
      const int k = i / kBlk, n = i % kBlk;
      const float v = k0 + k < K && n0 + n < N ? to_f(w[(size_t)(k0 + k) * N + n0 + n]) : 0.f;
      tile[k * 129 + n] = v;
      top = fmaxf(top, finite_mag(v));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
    top = 0.f;
    for (int i = 0; i < 8; ++i) top = fmaxf(top, tops[i]);
    const int e = block_exponent(top);
    const float inv = pow2i(-e);
    if (threadIdx.x == 0) scale[(size_t)(n0 / kBlk) * gridDim.x + blockIdx.x] = (uint8_t)(e + 127);
    for (int i = threadIdx.x; i < kBlk * (kBlk / 4); i += 256) {
      const int n = i / (kBlk / 4), k = i % (kBlk / 4) * 4;
      if (n0 + n < N && k0 + k < K)    // (K is a multiple of 16)
        *reinterpret_cast<uint32_t*>(codes + (size_t)(n0 + n) * K + k0 + k) =
            codes_of4(to_code(tile[k * 129 + n], inv), to_code(tile[(k + 1) * 129 + n], inv),
                      to_code(tile[(k + 2) * 129 + n], inv), to_code(tile[(k + 3) * 129 + n], inv));
    }
    __syncthreads();
  }
}

// Eights per thread.  Few rows: one, for the shortest chain.  Narrow rows: as many as let
// a warp hold the row.  Else what measured best (h stored before the sum): bf16 with a
// residual of bf16, 32768 x 4096, 1, 2, 3, 4 and 8 of them 223, 148, 152, 141 and 146 us; fp32 with fp32, 16384 x
// 4096, 145, 123, 132, 139 and 177 us; 8192 x 14336 of bf16, 4 and 8 172 and 147 us.
// (Rows in turn through a CTA, the next one requested ahead, and rows copied to shared
// memory in a ring, came to 151 and 160 us for the first.)
template <typename T, bool NORM> int eights_per_thread(int M, int eights) {
  if (M <= 2 * sm_count() && eights <= 1024) return 1;
  if (eights <= 128 && (sizeof(T) == 2 || !NORM)) return (eights + 31) / 32;
  if (sizeof(T) == 4) return eights <= 128 ? 1 : !NORM || eights <= 1024 ? 2 : eights <= 2048 ? 4 : 8;
  return !NORM || eights <= 1024 ? 4 : 8;
}

template <typename T, typename RT, bool NORM> cudaError_t rows(const RowsArgs& a, cudaStream_t s) {
  if (a.M <= 0) return cudaSuccess;
  const int eights = a.d / 8, nv = eights_per_thread<T, NORM>(a.M, eights);
  const int tpr = std::min(((eights + nv - 1) / nv + 31) / 32 * 32, NORM ? 1024 : 256);
  const int per_cta = NORM ? (tpr > 32 ? 1 : 8) : 256 / tpr;
  const dim3 grid((unsigned)(((long long)a.M + per_cta - 1) / per_cta),
                  NORM ? 1 : (unsigned)((eights + tpr * nv - 1) / (tpr * nv)));
  const dim3 block(tpr * per_cta);
  switch (nv) {
    case 1: return launch_pdl(k_rows_e4m3<T, RT, NORM, 1>, grid, block, 0, s, a, tpr);
    case 2: return launch_pdl(k_rows_e4m3<T, RT, NORM, 2>, grid, block, 0, s, a, tpr);
    case 3: return launch_pdl(k_rows_e4m3<T, RT, NORM, 3>, grid, block, 0, s, a, tpr);
    case 4: return launch_pdl(k_rows_e4m3<T, RT, NORM, 4>, grid, block, 0, s, a, tpr);
    default: return launch_pdl(k_rows_e4m3<T, RT, NORM, 8>, grid, block, 0, s, a, tpr);
  }
}

}  // namespace

cudaError_t launch_norm_e4m3(const RowsArgs& a, int x_dtype, int r_dtype, cudaStream_t s) {
  if (x_dtype == TB_F32) {
    if (!a.r) return rows<float, void, true>(a, s);
    return r_dtype == TB_F32 ? rows<float, float, true>(a, s) : rows<float, bf16, true>(a, s);
  }
  if (!a.r) return rows<bf16, void, true>(a, s);
  return r_dtype == TB_F32 ? rows<bf16, float, true>(a, s) : rows<bf16, bf16, true>(a, s);
}

cudaError_t launch_quant_e4m3(const RowsArgs& a, int x_dtype, cudaStream_t s) {
  return x_dtype == TB_F32 ? rows<float, void, false>(a, s) : rows<bf16, void, false>(a, s);
}

cudaError_t launch_pack_e4m3(const void* w, int dtype, int K, int N, uint8_t* codes, uint8_t* scale, cudaStream_t s) {
  const dim3 grid((K + kBlk - 1) / kBlk, std::min((N + kBlk - 1) / kBlk, 65535));
  constexpr size_t smem = kBlk * 129 * sizeof(float);
  auto go = [&](auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    const cudaError_t e = cudaFuncSetAttribute(k_pack_e4m3<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    k_pack_e4m3<T><<<grid, 256, smem, s>>>(static_cast<const T*>(w), K, N, codes, scale);
    return cudaGetLastError();
  };
  return dtype == TB_F32 ? go((float*)nullptr) : go((bf16*)nullptr);
}

}  // namespace tb
