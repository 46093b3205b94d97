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

namespace {
// fp32 queries: one warp per row; else by the rows that share a KV head.
bool few(const AttnArgs& a) { return a.n * (a.H / a.c.Hkv) <= kFewRows; }
}  // namespace

size_t cache_attn_workspace(const AttnArgs& a) {
  if (a.c.dtype == TB_F32) return 0;
  return few(a) ? cache_attn_few_workspace(a) : cache_attn_many_workspace(a);
}

cudaError_t launch_cache_attn(const AttnArgs& a, void* ws, cudaStream_t s) {
  if (a.c.dtype == TB_F32) {
    const long long rows = (long long)a.c.B * a.n * a.H;
    return launch_pdl(k_attn_row<float>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, a);
  }
  return few(a) ? launch_cache_attn_few(a, ws, s) : launch_cache_attn_many(a, ws, s);
}

}  // namespace tb
