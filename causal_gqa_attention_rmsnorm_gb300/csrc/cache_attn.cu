// Attention of the last tokens of each sequence over its cache, with a sliding
// window and sinks, over fp32, bf16 and e4m3 rows, contiguous or paged.
//
//   o = Σ_j p_j v_j / Σ_j p_j,  p_j = exp(scale·q·k_j - m),  j over the keys the
//   query at position p sees: j <= p and (W = 0 or j > p - W or j < S).
//
// k_attn_row: one warp per query row, 32 keys per step.
#include <math.h>

#include "cache.cuh"

namespace tb {
namespace {

// Row `row` of the cache, element e, as fp32 (without its block's scale).
__device__ __forceinline__ float cache_elem(const CacheView& c, const void* base, long long row, int e) {
  if (c.dtype == TB_F32) return __ldg((const float*)base + row * c.dh + e);
  if (c.dtype == TB_BF16) return to_f(((const bf16*)base)[row * c.dh + e]);
  const uint8_t code = __ldg((const uint8_t*)base + row * c.dh + e);
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

// One query row by one warp, exactly as the formula reads: masked keys are not
// touched at all.  q points to dh elements of type TQ; every lane returns with
// out[u] = o[lane + 32u] (u < dh / 32, at least one).
template <typename TQ>
__device__ void attend_row(const AttnArgs& a, int b, int hkv, int pos, const TQ* q, float (&out)[4]) {
  const int lane = threadIdx.x & 31, dh = a.c.dh;
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  const int lo = win_lo(pos, a.window);
  const int sinks = min(a.sinks, lo);
  const int nkeys = pos < 0 ? 0 : sinks + pos + 1 - lo;
  for (int j0 = 0; j0 < nkeys; j0 += 32) {
    const int jj = j0 + lane;
    const bool in = jj < nkeys;
    const int j = in ? (jj < sinks ? jj : jj - sinks + lo) : 0;
    long long sc = 0;
    const long long row = in ? cache_row(a.c, b, hkv, j, &sc) : -1;
    float s = 0.f;
    if (row >= 0) {
      for (int e = 0; e < dh; ++e) s = fmaf(to_f(q[e]), cache_elem(a.c, a.c.k, row, e), s);
      if (a.c.dtype == TB_E4M3) s *= a.c.ks[sc];
    }
    s = in ? s * a.scale_log2 : -INFINITY;
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - base);
    const float p = in ? exp2f(s - base) : 0.f;
    m = mn;
    l = l * f + warp_sum(p);
#pragma unroll
    for (int u = 0; u < 4; ++u) acc[u] *= f;
    const float vs = row >= 0 && a.c.dtype == TB_E4M3 ? a.c.vs[sc] : 1.f;
    const int steps = min(32, nkeys - j0);
    for (int k = 0; k < steps; ++k) {
      const float pk = __shfl_sync(0xffffffffu, p, k) * __shfl_sync(0xffffffffu, vs, k);
      const long long rk = __shfl_sync(0xffffffffu, row, k);
      if (rk < 0) continue;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = lane + 32 * u;
        if (e < dh) acc[u] = fmaf(pk, cache_elem(a.c, a.c.v, rk, e), acc[u]);
      }
    }
  }
  const bool none = l == 0.f;             // no visible key
#pragma unroll
  for (int u = 0; u < 4; ++u) out[u] = none ? 0.f : acc[u] / l;
}

template <typename TQ>
__global__ void __launch_bounds__(256) k_attn_row(AttnArgs a) {
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * 8 + warp;
  if (r >= (long long)a.c.B * a.n * a.H) return;
  const int h = (int)(r % a.H), i = (int)(r / a.H % a.n), b = (int)(r / a.H / a.n);
  const SeqRange sr = seq_range(a, b);
  if (i >= sr.nn) return;
  float out[4];
  attend_row<TQ>(a, b, h / (a.H / a.c.Hkv), sr.first + i, (const TQ*)a.q + (size_t)r * a.c.dh, out);
  __syncwarp();                          // o may be q
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (lane + 32 * u < a.c.dh) ((TQ*)a.o)[(size_t)r * a.c.dh + lane + 32 * u] = from_f<TQ>(out[u]);
}

}  // namespace

size_t cache_attn_workspace(const AttnArgs& a) {
  (void)a;
  return 0;
}

cudaError_t launch_cache_attn(const AttnArgs& a, void* ws, cudaStream_t s) {
  (void)ws;
  const long long rows = (long long)a.c.B * a.n * a.H;
  const unsigned grid = (unsigned)((rows + 7) / 8);
  if (a.c.dtype == TB_F32) return launch_pdl(k_attn_row<float>, dim3(grid), dim3(256), 0, s, a);
  return launch_pdl(k_attn_row<bf16>, dim3(grid), dim3(256), 0, s, a);
}

}  // namespace tb
