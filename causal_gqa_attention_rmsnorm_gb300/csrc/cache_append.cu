// Appending rows to a KV cache with the position rotation applied on the way.
//
// Row i of sequence b sits at position p = start[b] + i; each adjacent pair
// (x0, x1) of its q and k becomes (x0·c - x1·s, x0·s + x1·c) with (c, s) from
// row p of a table formed in fp64.  Every product and sum rounds to fp32 on its
// own (no contraction), so that the stored bits do not depend on how a compiler
// fuses them; the result is rounded once to the stored type.
#include <algorithm>

#include "cache.cuh"

namespace tb {
namespace {

constexpr int kVec = 8;                 // elements per thread and step: four pairs

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    Vec16<T> v;
    v.raw = *reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v.get(i);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint4 w;
    uint32_t* u = &w.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    *reinterpret_cast<uint4*>(p) = w;
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  }
}
// Four pairs turned by cs[0..3] (two float4: cos, sin, cos, sin).
__device__ __forceinline__ void rotate8(float (&x)[8], const float4 (&cs)[2]) {
  const float* t = &cs[0].x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c = t[2 * i], s = t[2 * i + 1], a = x[2 * i], b = x[2 * i + 1];
    x[2 * i] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    x[2 * i + 1] = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
  }
}
__device__ __forceinline__ void load_cs(const AppendArgs& a, int pos, int e, float4 (&cs)[2]) {
  const float4* p = reinterpret_cast<const float4*>(a.rope + (size_t)pos * (a.c.dh >> 1) + (e >> 1));
  cs[0] = __ldg(p);
  cs[1] = __ldg(p + 1);
}

// Position of sequence b's first new row and how many rows it gets; nn = -1
// where they do not fit.
struct Place {
  int t0, nn;
};
__device__ __forceinline__ Place place_of(const AppendArgs& a, int b) {
  Place p;
  p.t0 = a.start ? a.start[b] : a.c.lens[b];
  p.nn = a.n_new ? min(max(a.n_new[b], 0), a.n) : a.n;
  if (p.t0 < 0 || p.t0 > a.c.T - p.nn) p.nn = -1;
  return p;
}
// The new length, by one thread per sequence.  With start == nullptr the
// lengths are the positions the other CTAs read, so a later launch does it.
__device__ __forceinline__ void set_len(const AppendArgs& a, int b) {
  const Place p = place_of(a, b);
  if (p.nn < 0)
    atomicOr(a.c.err, TB_DEVERR_CACHE_FULL);
  else
    a.c.lens[b] = p.t0 + p.nn;
}
__global__ void k_append_lens(AppendArgs a) {
  pdl_wait();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < a.c.B) set_len(a, b);
}

// q, k and v rows of 16- and 32-bit types.  A thread holds one eight-element
// piece of a token's head and that piece's four (cos, sin) pairs, and walks the
// heads of the token: H of q (if any), then Hkv of k and of v.
template <typename T>
__global__ void __launch_bounds__(256) k_append_rope(AppendArgs a, int with_kv) {
  pdl_trigger();
  pdl_wait();
  const int pieces = a.c.dh / kVec;
  const int per = blockDim.x / pieces;                  // heads in step
  const int e = (threadIdx.x % pieces) * kVec, h0 = threadIdx.x / pieces;
  const int b = blockIdx.y, i = blockIdx.x;
  if (a.start && i == 0 && threadIdx.x == 0) set_len(a, b);
  const Place p = place_of(a, b);
  if (i >= p.nn || h0 >= per) return;
  const int pos = p.t0 + i, Hkv = a.c.Hkv, H = a.q ? a.H : 0, dh = a.c.dh;
  float4 cs[2];
  load_cs(a, pos, e, cs);
  const int total = H + (with_kv ? 2 * Hkv : 0);
  for (int h = h0; h < total; h += per) {
    float x[8];
    if (h < H) {
      load8((const T*)a.q + b * a.q_seq + i * a.q_tok + (size_t)h * dh + e, x);
      rotate8(x, cs);
      store8((T*)a.q_out + (((size_t)b * a.n + i) * H + h) * dh + e, x);
      continue;
    }
    const bool is_k = h < H + Hkv;
    const int hk = h - H - (is_k ? 0 : Hkv);
    load8(is_k ? (const T*)a.k + b * a.k_seq + i * a.k_tok + (size_t)hk * dh + e
               : (const T*)a.v + b * a.v_seq + i * a.v_tok + (size_t)hk * dh + e,
          x);
    if (is_k) rotate8(x, cs);
    const long long row = cache_row(a.c, b, hk, pos);
    if (row >= 0) store8((T*)(is_k ? a.c.k : a.c.v) + row * dh + e, x);
  }
}

// ---- e4m3 blocks -----------------------------------------------------------

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// Smallest e in [kE4Min, kE4Max] with top <= 448·2^e (448 = 1.75·2^8).
__device__ __forceinline__ int block_exp(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kE4Min), kE4Max);
}
// An infinity is stored as NaN: the code has none.
__device__ __forceinline__ float no_inf(float x) { return fabsf(x) <= 3.402823466e38f ? x : NAN; }

// One CTA per (block of the cache, KV head, sequence and K or V): the largest
// magnitude of the block's new rows, the scale, then the codes; the rows are
// read twice, the second time from L1/L2.
__global__ void __launch_bounds__(256) k_append_e4m3(AppendArgs a) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.z >> 1, is_v = blockIdx.z & 1, h = blockIdx.y;
  const Place p = place_of(a, b);
  if (p.nn <= 0) return;
  const int bs = a.c.ps, dh = a.c.dh;
  const int blk = p.t0 / bs + blockIdx.x;
  const int t_lo = max(p.t0, blk * bs), t_hi = min(p.t0 + p.nn, (blk + 1) * bs);
  if (t_lo >= t_hi) return;
  long long sc;
  const long long row0 = cache_row(a.c, b, h, blk * bs, &sc);
  if (row0 < 0) return;
  const bf16* src = is_v ? (const bf16*)a.v + b * a.v_seq + (size_t)h * dh : (const bf16*)a.k + b * a.k_seq + (size_t)h * dh;
  const long long tok = is_v ? a.v_tok : a.k_tok;
  uint8_t* dst = (uint8_t*)(is_v ? a.c.v : a.c.k) + row0 * dh;
  float* scale = (is_v ? a.c.vs : a.c.ks) + sc;
  const int pieces = dh / kVec, n_pieces = (t_hi - t_lo) * pieces;
  auto fetch = [&](int i, float (&x)[8]) {
    const int t = t_lo + i / pieces, e = (i % pieces) * kVec;
    load8(src + (long long)(t - p.t0) * tok + e, x);
    if (!is_v) {
      float4 cs[2];
      load_cs(a, t, e, cs);
      rotate8(x, cs);
    }
  };
  float top = 0.f;
  for (int i = threadIdx.x; i < n_pieces; i += blockDim.x) {
    float x[8];
    fetch(i, x);
#pragma unroll
    for (int u = 0; u < 8; ++u) top = fmaxf(top, fabsf(no_inf(x[u])));     // fmaxf drops NaN
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  __shared__ float red[8];
  __shared__ float was_s;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
  if (threadIdx.x == 0) was_s = *scale;
  __syncthreads();
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) top = fmaxf(top, red[i]);
  const bool partial = t_lo > blk * bs;                  // the block holds older rows of the sequence
  const float need = pow2(block_exp(top));
  const float s = partial ? fmaxf(was_s, need) : need;
  const float inv = 1.0f / s;                            // exact: s is a power of two
  if (threadIdx.x == 0) *scale = s;
  if (partial && s > was_s) {
    const float ratio = was_s / s;                       // a power of two, below 1
    for (int i = threadIdx.x; i < (t_lo - blk * bs) * pieces; i += blockDim.x) {
      uint2* at = reinterpret_cast<uint2*>(dst + (size_t)i * kVec);
      uint2 c = *at;
      uint16_t* w = reinterpret_cast<uint16_t*>(&c);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 f = from_e4m3x2(w[u]);
        w[u] = (uint16_t)e4m3x2(f.x * ratio, f.y * ratio);
      }
      *at = c;
    }
  }
  for (int i = threadIdx.x; i < n_pieces; i += blockDim.x) {
    float x[8];
    fetch(i, x);
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = no_inf(x[u]) * inv;
    uint2 w;
    w.x = e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16;
    w.y = e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16;
    const int t = t_lo + i / pieces, e = (i % pieces) * kVec;
    *reinterpret_cast<uint2*>(dst + (size_t)(t - blk * bs) * dh + e) = w;
  }
}

}  // namespace

cudaError_t launch_append_rope(const AppendArgs& a, cudaStream_t s) {
  const bool e4 = a.c.dtype == TB_E4M3;
  cudaError_t e = cudaSuccess;
  const dim3 grid((unsigned)a.n, (unsigned)a.c.B);
  if (a.c.dtype == TB_F32)
    e = launch_pdl(k_append_rope<float>, grid, dim3(256), 0, s, a, 1);
  else
    e = launch_pdl(k_append_rope<bf16>, grid, dim3(256), 0, s, a, e4 ? 0 : 1);
  if (e == cudaSuccess && e4) {
    const int nb = (a.n + a.c.ps - 2) / a.c.ps + 1;        // blocks that n rows can reach from any start
    const int rows = std::min(a.n, a.c.ps);
    const int threads = std::min(256, (rows * (a.c.dh / kVec) + 31) / 32 * 32);
    e = launch_pdl(k_append_e4m3, dim3((unsigned)nb, a.c.Hkv, 2 * a.c.B), dim3(threads), 0, s, a);
  }
  if (e == cudaSuccess && !a.start)
    e = launch_pdl(k_append_lens, dim3((a.c.B + 127) / 128), dim3(128), 0, s, a);
  return e;
}

}  // namespace tb
