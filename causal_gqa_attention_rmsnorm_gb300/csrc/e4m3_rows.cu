// Rows to e4m3 codes with one power-of-two scale per 128 columns: RMSNorm (with the
// residual's addition on the way) or the rows as they are; and weights to codes with
// one scale per 128 x 128.
//
//   h = x + r,  y = h / sqrt(mean h² + eps) * g,  codes of y per block of 128
//
// One pass over memory: a row lies in the registers of 32 to 1024 threads, in eights of
// neighbouring columns, so that 16, 8 or 4 lanes of a warp hold the 128 columns of a block
// and its largest magnitude takes four, three or two shuffles.  The sum, the mean square
// and the quotients are fp32; y is never rounded to anything but its code.
//
// Bound by memory: 32768 x 4096 of bf16 with a residual of bf16 133 us, 7.1 TB/s of what it
// has to move, as fast as memory is copied; 16384 x 4096 of bf16 alone 35 us (5.8: fewer
// bytes to cover a row's chain); the codes alone of 8192 x 11008 of fp32 64 us (7.0); 3777 x
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

// The codes of a thread's P eights y = v·s·g of a block that 16/P neighbouring lanes hold
// (columns c + 128/P·p on, those below d); the first of the lanes also stores the scale.
// v·g comes first, so that the row's s and the block's 2^-e are one factor: s·2^-e is exact
// (for s below 2^28, as e is -100 or more), and the largest |v·g|·s is the largest |v·g·s|
// (rounding keeps the order).  False if the largest |v·g|·s is no finite number, or if s is
// 2^28 or more, where s·2^-e may be infinite (zeros would become NaN) and v·g below fp32's
// normal numbers where v·s·g is not: put_wild then writes the block again.  A NaN is passed
// over by the maximum and kept by the conversion.
template <typename T, bool NORM, int P>
__device__ __forceinline__ bool put_block(const float (&v)[P][8], float s, const Eight<T> (&g)[P], int c, int d, uint8_t* codes,
                                          uint8_t* scale) {
  float t[P][8], top = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[p][i] = NORM ? v[p][i] * g[p].get(i) : v[p][i];
#pragma unroll
    for (int i = 0; i < 8; i += 2) top = ptx::fmax3(top, fabsf(t[p][i]), fabsf(t[p][i + 1]));
  }
#pragma unroll
  for (int o = 8 / P; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  top *= s;
  const int e = block_exponent(top);
  const float f = s * pow2i(-e);
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (c + p * (kBlk / P) < d)
      *reinterpret_cast<uint2*>(codes + c + p * (kBlk / P)) =
          make_uint2(codes_of4(t[p][0] * f, t[p][1] * f, t[p][2] * f, t[p][3] * f),
                     codes_of4(t[p][4] * f, t[p][5] * f, t[p][6] * f, t[p][7] * f));
  if (threadIdx.x % (16 / P) == 0 && c < d) scale[c / kBlk] = (uint8_t)(e + 127);
  return top < INFINITY && s < 0x1p28f;
}

// The same of a block with an infinity in it, with v·g beyond fp32 where v·s·g is not, or of
// a row whose s is 2^28 or more (its mean square + eps below 2^-56: rows of 3.7e-9, or zeros,
// with an eps of next to nothing) or no finite number: in the order v·s·g, infinities told from values one by one, and
// from memory once more, so that put_block need not keep its values.  By whole warps (the
// shuffles); `mine`: whether this thread's block is one.
template <typename T, typename RT, bool NORM, int P>
__device__ __noinline__ void put_wild(const T* x, const RT* r, const T* g, float s, int c, int d, uint8_t* codes, uint8_t* scale,
                                      bool mine) {
  auto y = [&](int at) {
    float v = to_f(x[at]);
    if constexpr (!std::is_same<RT, void>::value) v += to_f(r[at]);
    return NORM ? v * s * to_f(g[at]) : v;
  };
  float top = 0.f;
#pragma unroll 1
  for (int i = 0; i < 8 * P; ++i) {
    const int at = c + i / 8 * (kBlk / P) + i % 8;
    if (mine && at < d) top = fmaxf(top, finite_mag(y(at)));
  }
#pragma unroll
  for (int o = 8 / P; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (!mine) return;
  const int e = block_exponent(top);
  const float f = pow2i(-e);
#pragma unroll 1
  for (int i = 0; i < 2 * P; ++i) {
    const int at = c + i / 2 * (kBlk / P) + i % 2 * 4;
    if (at < d)
      *reinterpret_cast<uint32_t*>(codes + at) = codes_of4(to_code(y(at), f), to_code(y(at + 1), f), to_code(y(at + 2), f), to_code(y(at + 3), f));
  }
  if (threadIdx.x % (16 / P) == 0 && c < d) scale[c / kBlk] = (uint8_t)(e + 127);
}

// RT: the type of r (void: none).  A row takes `tpr` threads (a multiple of 32), NV
// eights each, a CTA blockDim.x / tpr rows; with NORM that is one, or a row per warp.
// Without NORM, blockIdx.y counts pieces of tpr·NV·8 columns.
template <typename RT> constexpr bool kRes = !std::is_same<RT, void>::value;
// A thread's eights of one block.  More of them share the block's maximum, exponent and
// shuffles (16384 x 4096 of bf16 37.1 us with P 2, 34.9 with 4), while few rows want the
// shorter chain, and r leaves no registers for 4 (8192 x 11008 of bf16 111 us, 106 with 2).
template <typename RT, int NV> constexpr int kP = NV % 2 ? 1 : NV == 4 && !kRes<RT> ? 4 : 2;
// bf16 without r stays as it was read until it is divided (half the registers), and CTAs of
// 48 to 64 registers a thread lie on an SM: 8192 x 11008 91 -> 48 us.
template <typename T, typename RT, int NV> constexpr bool kLean = sizeof(T) == 2 && NV % 2 == 0 && !kRes<RT>;
template <typename T, typename RT, int NV> constexpr int kThreads = NV == 1 ? 1024 : sizeof(T) == 2 && (NV == 4 || (NV == 2 && !kRes<RT>)) ? 256 : 512;
// (32768 x 4096 of bf16 with r 134.1 us where no number of CTAs is asked for, 132.7 with 3,
// 137.6 with 4)
template <typename T, typename RT, int NV>
constexpr int kCtas = kLean<T, RT, NV> ? (NV == 2 ? 6 : NV == 4 ? 5 : 2) : sizeof(T) == 2 && NV == 4 ? 3 : 0;
// g is read when it is needed where its registers would keep CTAs away: 16384 x 4096 of fp32
// 59.5 -> 53.9 us, 8192 x 11008 with r of bf16 205 -> 151; early elsewhere, where it shortens
// a row's chain (16384 x 4096 of fp32 with r of fp32 132 -> 124.5, bf16 with r 137 -> 134).
template <typename T, typename RT, int NV>
constexpr bool kLate = NV % 2 == 0 && (!kRes<RT> || NV == 8 || (sizeof(T) == 4 && NV == 4));
template <typename T, typename RT, bool NORM, int NV>
__global__ void __launch_bounds__(kThreads<T, RT, NV>, kCtas<T, RT, NV>) k_rows_e4m3(RowsArgs a, int tpr) {
  constexpr bool RES = kRes<RT>;
  constexpr bool LEAN = kLean<T, RT, NV>, LATE = NORM && kLate<T, RT, NV>;
  constexpr int P = kP<RT, NV>, G = 16 / P, NB = NV / P;
  __shared__ float part[32];
  pdl_trigger();
  const int lane = threadIdx.x & 31, t = threadIdx.x % tpr;
  const int col0 = (NORM ? 0 : (int)blockIdx.y * tpr * NV * 8) + t / G * kBlk + t % G * 8;
  auto col = [&](int i) { return col0 + i / P * (tpr / G * kBlk) + i % P * (8 * G); };
  const size_t row = (size_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr, base = row * a.d;
  pdl_wait();
  if (row >= a.M) return;              // (whole warps; with a barrier ahead, whole CTAs)
  Eight<T> x[NV];
  Eight<RT> r[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x[i].zero();                       // (columns past the row read as zeros throughout)
    if constexpr (RES) r[i].zero();
    if (col(i) < a.d) {
      x[i].load(static_cast<const T*>(a.x) + base + col(i));
      if constexpr (RES) r[i].load(static_cast<const RT*>(a.r) + base + col(i));
    }
  }
  float v[NB][P][8], q = 0.f, s = 1.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i / P][i % P][j] = x[i].get(j);
      if constexpr (RES) v[i / P][i % P][j] += r[i].get(j);
      if (NORM) q = fmaf(v[i / P][i % P][j], v[i / P][i % P][j], q);
    }
  Eight<T> g[NB][P];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    g[i / P][i % P].zero();
    if (NORM && !LATE && col(i) < a.d) g[i / P][i % P].load(static_cast<const T*>(a.g) + col(i));
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
  uint32_t wild = 0;
  const RT* res = nullptr;
  if constexpr (RES) res = static_cast<const RT*>(a.r) + base;
  if constexpr (LEAN) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      asm volatile("" : "+r"(x[i].u[0].raw.x), "+r"(x[i].u[0].raw.y), "+r"(x[i].u[0].raw.z), "+r"(x[i].u[0].raw.w));
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if constexpr (LATE || LEAN) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (NORM && LATE && col(b * P + p) < a.d) g[b][p].load(static_cast<const T*>(a.g) + col(b * P + p));
        if constexpr (LEAN)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[b][p][j] = x[b * P + p].get(j);
      }
    }
    if (!put_block<T, NORM, P>(v[b], s, g[b], col(b * P), a.d, a.codes + base, a.scale + row * blocks)) wild |= 1u << b;
  }
  if (__any_sync(0xffffffffu, wild != 0)) {
#pragma unroll 1
    for (int b = 0; b < NB; ++b)
      put_wild<T, RT, NORM, P>(static_cast<const T*>(a.x) + base, res, static_cast<const T*>(a.g), s, col(b * P), a.d, a.codes + base,
                               a.scale + row * blocks, wild >> b & 1);
  }
  // (last: 32768 x 4096 of bf16 132 us, 141 with h stored before the sum)
  if constexpr (RES) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (col(i) < a.d) store8(static_cast<T*>(a.h) + base + col(i), v[i / P][i % P]);
  }
}

// Codes [N, K] of w [K, N]: a CTA takes a block of 128 x 128, keeps it in shared memory
// as fp32 (rows of w, one word of padding, so that both ways of reading it are free of
// conflicts) and writes it transposed.  Done once per weight set.
template <typename T> __global__ void __launch_bounds__(256) k_pack_e4m3(const T* w, int K, int N, uint8_t* codes, uint8_t* scale) {
  extern __shared__ float tile[];      // [128][129]
  __shared__ float tops[8];
  const int k0 = blockIdx.x * kBlk;
  // (blocks are counted, not columns of w: these and the grid's step go beyond 31 bits together)
  const int blocks = (N + kBlk - 1) / kBlk;
  for (int nb = blockIdx.y; nb < blocks; nb += gridDim.y) {
    const int n0 = nb * kBlk;
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
    if (threadIdx.x == 0) scale[(size_t)nb * gridDim.x + blockIdx.x] = (uint8_t)(e + 127);
    for (int i = threadIdx.x; i < kBlk * (kBlk / 4); i += 256) {
      const int n = i / (kBlk / 4), k = i % (kBlk / 4) * 4;
      if (n0 + n < N && k0 + k < K)    // (K is a multiple of 16)
        *reinterpret_cast<uint32_t*>(codes + (size_t)(n0 + n) * K + k0 + k) =
            codes_of4(to_code(tile[k * 129 + n], inv), to_code(tile[(k + 1) * 129 + n], inv),
                      to_code(tile[(k + 2) * 129 + n], inv), to_code(tile[(k + 3) * 129 + n], inv));
    }
    __syncthreads();
  }
  // A product may request these before this grid's end has been waited for (common.cuh): what
  // lets it in is that the CTAs are through, so they are once their codes can be seen.
  asm volatile("fence.acq_rel.gpu;\n\tfence.proxy.async.global;" ::: "memory");
}

// Eights per thread.  Few rows: one, for the shortest chain.  Narrow rows: as many as let
// a warp hold the row.  Else what measured best, us, by eights per thread:
//                                       1     2     4     8
//   norm, bf16:        1 x 4096, r bf16 2.3  2.3   2.4   3.5     608 x 4096:   6.4   5.1   5.4   6.5
//     304 x 8192, r bf16  7.2   -    5.7   6.6
//     4096 x 2048       -    -    8.2   7.5                      2048 x 2048:   -     -    4.7   5.1
//     16384 x 4096     64.3 44.1 34.9  34.2                      4096 x 4096:   -     -   11.6  12.9
//     16384 x 6144      -    -   54.4  49.3                      8192 x 8192:   -     -   37.2  34.5
//     32768 x 4096, r bf16       241   144   133   134           8192 x 8192:   -     -   68.6  70.0
//   norm, fp32:        16384 x 4096  78.6 53.6  51.2  55.0       8192 x 14336:  -     -   103   105
//     r bf16, 8192 x 8192              -   124   108   117       8192 x 14336:  -     -   236   207
//     r fp32, 16384 x 4096           161   124   127   129       8192 x 8192:   -   144   154   132
//   quantisation:      8192 x 11008 fp32 69.9 64.6 64.2          16384 x 4096 bf16: 41.1 29.9 29.8
// (Rows in turn through a CTA, the next one requested ahead, and rows copied to shared
// memory in a ring, came to 151 and 160 us for 32768 x 4096 with r.)
template <typename T, typename RT, bool NORM> int eights_per_thread(int M, int eights) {
  constexpr bool RES = kRes<RT>;
  const int narrow = (eights + 31) / 32;
  if (M <= 2 * sm_count() && eights <= (NORM && sizeof(T) == 2 ? 512 : 1024)) return 1;
  if (!NORM) return narrow <= 2 ? narrow : sizeof(T) == 4 ? 2 : 4;
  if (sizeof(T) == 2) {
    if (narrow <= 4) return narrow;
    if (RES) return eights <= 1024 ? 4 : 8;
    return narrow <= 8 ? (M > 2048 ? 8 : 4) : eights <= 640 ? 4 : 8;
  }
  if (narrow <= 4) return !RES && M > 2048 ? narrow : 1;
  if (!RES) return eights <= 1536 ? 4 : 8;
  return eights <= 512 ? 2 : std::is_same<RT, bf16>::value && eights <= 1536 ? 4 : 8;
}

template <typename T, typename RT, bool NORM> cudaError_t rows(const RowsArgs& a, cudaStream_t s) {
  if (a.M <= 0) return cudaSuccess;
  const int eights = a.d / 8, nv = eights_per_thread<T, RT, NORM>(a.M, eights);
  const int tpr = std::min(((eights + nv - 1) / nv + 31) / 32 * 32, NORM ? 1024 : 256);
  const int per_cta = NORM ? (tpr > 32 ? 1 : 8) : 256 / tpr;
  const dim3 grid((unsigned)(((long long)a.M + per_cta - 1) / per_cta),
                  NORM ? 1 : (unsigned)((eights + tpr * nv - 1) / (tpr * nv)));
  const dim3 block(tpr * per_cta);
  if (nv == 1) return launch_pdl(k_rows_e4m3<T, RT, NORM, 1>, grid, block, 0, s, a, tpr);
  if (nv == 2) return launch_pdl(k_rows_e4m3<T, RT, NORM, 2>, grid, block, 0, s, a, tpr);
  if constexpr (NORM && (sizeof(T) == 2 || !kRes<RT>))
    if (nv == 3) return launch_pdl(k_rows_e4m3<T, RT, NORM, 3>, grid, block, 0, s, a, tpr);
  if constexpr (NORM)
    if (nv == 8) return launch_pdl(k_rows_e4m3<T, RT, NORM, 8>, grid, block, 0, s, a, tpr);
  if constexpr ((NORM && sizeof(T) == 2) || !std::is_same<RT, float>::value)
    if constexpr (NORM || sizeof(T) == 2) return launch_pdl(k_rows_e4m3<T, RT, NORM, 4>, grid, block, 0, s, a, tpr);
  return cudaErrorInvalidValue;
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
