// Rows to e4m3 codes with one power-of-two scale per 128 columns: RMSNorm (with the
// residual's addition on the way) or the rows as they are; and weights to codes with
// one scale per 128 x 128.
//
//   h = x + r,  y = h / sqrt(mean h² + eps) * g,  codes of y per block of 128
//
// One pass over memory: a row lies in the registers of 32 to 512 threads, eight
// neighbouring columns to a thread, so that 16 lanes of a warp hold the 128 columns of
// a block and its largest magnitude takes four shuffles.  The sum, the mean square and
// the quotients are fp32; y is never rounded to anything but its code.
#include <algorithm>

#include "e4m3.cuh"

namespace tb {
namespace {

// Eight neighbouring values as fp32.  (Plain loads: the kernel before may still be
// writing other memory while this grid is resident, so nothing is read as constant.)
template <typename T> __device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  constexpr int N = Vec16<T>::N;
#pragma unroll
  for (int u = 0; u < 8 / N; ++u) {
    Vec16<T> t;
    t.raw = reinterpret_cast<const uint4*>(p)[u];
#pragma unroll
    for (int i = 0; i < N; ++i) v[u * N + i] = t.get(i);
  }
}
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

// The codes of a thread's eight values of a block that 16 lanes hold; lane 0 of the 16
// also stores the scale.
__device__ __forceinline__ void put_block(const float (&v)[8], bool in, uint8_t* codes, uint8_t* scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_mag(v[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (!in) return;
  const int e = block_exponent(top);
  const float inv = pow2i(-e);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = to_code(v[i], inv);
  *reinterpret_cast<uint2*>(codes) = make_uint2(codes_of4(q[0], q[1], q[2], q[3]), codes_of4(q[4], q[5], q[6], q[7]));
  if ((threadIdx.x & 15) == 0) *scale = (uint8_t)(e + 127);
}

// RT: the type of r (void: none).  A row takes `tpr` threads (a multiple of 32), NV
// eights each; a CTA takes blockDim.x / tpr rows.  Without NORM, blockIdx.y counts
// pieces of tpr·NV·8 columns of a row.
template <typename T, typename RT, bool NORM, int NV>
__global__ void __launch_bounds__(512) k_rows_e4m3(RowsArgs a, int tpr) {
  constexpr bool RES = !std::is_same<RT, void>::value;
  __shared__ float part[16];
  pdl_trigger();
  const int t = threadIdx.x % tpr;
  const long long row = (long long)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < a.M;
  const long long base = row * a.d;
  const int col0 = NORM ? 0 : (int)blockIdx.y * tpr * NV * 8;
  pdl_wait();
  float v[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = col0 + (i * tpr + t) * 8;
    if (live && c < a.d) {
      load8(static_cast<const T*>(a.x) + base + c, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
  if constexpr (RES) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * 8;
      if (live && c < a.d) {
        float r[8];
        load8(static_cast<const RT*>(a.r) + base + c, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += r[j];
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * 8;
      if (live && c < a.d) store8(static_cast<T*>(a.h) + base + c, v[i]);
    }
  }
  float s = 1.f;
  if constexpr (NORM) {
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) q = fmaf(v[i][j], v[i][j], q);
    q = warp_sum(q);
    if (tpr > 32) {
      // the partial sums of a row's warps, in order
      const int w0 = threadIdx.x / tpr * (tpr / 32);
      if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = q;
      __syncthreads();
      q = 0.f;
      for (int w = 0; w < tpr / 32; ++w) q += part[w0 + w];
    }
    s = 1.0f / sqrtf(q / (float)a.d + a.eps);
  }
  if (!live) return;                   // (whole warps: a warp holds one row)
  const int blocks = (a.d + kBlk - 1) / kBlk;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = col0 + (i * tpr + t) * 8;
    const bool in = live && c < a.d;
    if constexpr (NORM) {
      if (in) {
        float g[8];
        load8(static_cast<const T*>(a.g) + c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= s * g[j];
      }
    }
    put_block(v[i], in, a.codes + base + c, a.scale + row * blocks + c / kBlk);
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

int sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

template <typename T, typename RT, bool NORM> cudaError_t rows(const RowsArgs& a, cudaStream_t s) {
  if (a.M <= 0) return cudaSuccess;
  const int eights = a.d / 8;
  const int nv = a.M <= 2 * sms() && eights <= 512 ? 1 : eights > 2048 ? 8 : 4;
  const int want = ((eights + nv - 1) / nv + 31) / 32 * 32;
  const int tpr = std::min(want, NORM ? 512 : 256);
  const int per_cta = std::max(1, 256 / tpr);
  const dim3 grid((unsigned)((a.M + per_cta - 1) / per_cta), NORM ? 1 : (unsigned)((eights + tpr * nv - 1) / (tpr * nv)));
  const dim3 block(tpr * per_cta);
  switch (nv) {
    case 1: return launch_pdl(k_rows_e4m3<T, RT, NORM, 1>, grid, block, 0, s, a, tpr);
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
