// Attention of the last tokens of each sequence over its cache, with a sliding
// window and sinks, over fp32, bf16 and e4m3 rows, contiguous or paged.
//
//   o = Σ_j p_j v_j / Σ_j p_j,  p_j = exp(scale·q·k_j - m),  j over the keys the
//   query at position p sees: j <= p and (W = 0 or j > p - W or j < S).
//
// This file: which kernel takes a call, and the fp32 path.
//
// fp32 (k_attn_f32): a CTA takes eight of the n·G rows (tokens x query heads) that
// share a KV head, and a range of their visible keys; each of its warps walks 32
// keys at a time.  Scores: a lane holds one key and reads its K row in 16-byte
// pieces, the rows' queries come from shared memory as broadcasts.  Values: a lane
// holds dims lane, lane + 32, ..., the 32 weights come by shuffle, and a weight of
// a hidden key is never multiplied (a NaN there stays where it is).  The warps'
// (max, sum, weighted sum of v) are joined in shared memory, the key ranges' by
// k_f32_merge, both in order.  No tensor-core type holds fp32, so a key costs its
// 4·dh operations per row on the FMA pipes.
//
// Measured (GPU time): 3 tokens of 2 sequences, window 500, 8 and 2 heads of 64: 10.4
// us; one token of 8001 keys, 32 and 8 heads of 128: 41 us (its bytes take 10), of 32
// sequences of up to 8k 499 us (169); 512 tokens at the end of 4096 2.58 ms, 12.5
// TFLOP/s.  Neither bytes nor FMA bound it yet: one CTA of 142 registers a thread per
// SM waits for its own loads (a lane reads its key's row in 16-byte pieces) and, at
// the end, for its slowest warp (one token of 32 sequences, window 500: issue slots 26 %
// and DRAM 18 % busy), and one token of four query heads fills four of the eight rows.
#include <math.h>

#include <algorithm>

#include "cache.cuh"
#include "gemm_tc.cuh"

namespace tb {
namespace {

constexpr int kRows = 8;              // rows per CTA
constexpr int kFWarps = 8;
constexpr int kKeys = 32;             // keys per warp and step

struct F32Args {
  AttnArgs a;
  int n_tiles;            // row tiles of a (sequence, KV head)
  int n_range;            // key ranges
  float* part;            // [B][Hkv][n_tiles][n_range][kRows][dh + 2]: O, max, sum (n_range > 1)
};

// The visible 32-key runs of the rows of tile rt of sequence b.
__device__ __forceinline__ KeyRuns tile_runs(const F32Args& f, const SeqRange& sr, int rt) {
  const int i0 = rt * kRows >> f.a.g_sh, i1 = min((rt * kRows + kRows - 1) >> f.a.g_sh, sr.nn - 1);
  if (i0 >= sr.nn) return KeyRuns{0, 0, 0};
  return key_runs(sr.first + i1 + 1, sr.first + i0, f.a.window, f.a.sinks, kKeys);
}

// *p, or 0: a predicated load spelled out up to 64 dims (one token of 32 sequences of
// up to 8k rows, 8 and 2 heads of 64: 90 us, from the plain expression 108), left to
// the compiler at 128 (32 and 8 heads: 503 us, spelled out 512).
template <int DH>
__device__ __forceinline__ float load_if(bool in, const float* p) {
  if constexpr (DH == 128) return in ? *p : 0.f;
  float v = 0.f;
  asm("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p ld.global.f32 %0, [%1];\n\t}" : "+f"(v) : "l"(p), "r"((int)in));
  return v;
}

template <int DH>
__global__ void __launch_bounds__(kFWarps * 32) k_attn_f32(const F32Args f) {
  pdl_trigger();
  pdl_wait();
  constexpr int D = (DH + 31) / 32;   // dims per lane
  const AttnArgs& a = f.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = blockIdx.x % f.n_range, rt = blockIdx.x / f.n_range, h = blockIdx.y, b = blockIdx.z;
  const int G = 1 << a.g_sh;
  const SeqRange sr = seq_range(a, b);
  const int rows = min(kRows, sr.nn * G - rt * kRows);      // of real tokens
  if (rows <= 0) return;
  const KeyRuns kr = tile_runs(f, sr, rt);
  const int g0 = (int)((long long)kr.count * rg / f.n_range), g1 = (int)((long long)kr.count * (rg + 1) / f.n_range);

  __shared__ __align__(16) float q_s[kRows][DH];
  __shared__ float m_s[kFWarps][kRows], l_s[kFWarps][kRows];
  __shared__ float acc_s[kFWarps][kRows][DH];
  auto row_at = [&](int r) {          // where row r's q and o lie
    const int t = rt * kRows + r;
    return (((size_t)b * a.n + (t >> a.g_sh)) * a.H + h * G + (t & (G - 1))) * DH;
  };
  for (int i = threadIdx.x; i < kRows * DH; i += kFWarps * 32)
    q_s[i / DH][i % DH] = i / DH < rows ? ((const float*)a.q)[row_at(i / DH) + i % DH] * a.scale_log2 : 0.f;
  __syncthreads();
  int pos[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) pos[r] = r < rows ? sr.first + ((rt * kRows + r) >> a.g_sh) : -1;

  float m[kRows], l[kRows], acc[kRows][D];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int u = 0; u < D; ++u) acc[r][u] = 0.f;
  }
  for (int g = g0 + warp; g < g1; g += kFWarps) {
    const int key = run_index(kr, g) * kKeys + lane;
    bool any = false;
    uint32_t vis[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const bool see = key <= pos[r] && (key >= win_lo(pos[r], a.window) || key < a.sinks);
      any |= see;
      vis[r] = __ballot_sync(0xffffffffu, see);
    }
    const long long row = any ? cache_row(a.c, b, h, key) : -1;
    float s[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) s[r] = 0.f;
    if (row >= 0) {
      const float4* kp = reinterpret_cast<const float4*>((const float*)a.c.k + row * DH);
#pragma unroll 8
      for (int e = 0; e < DH / 4; ++e) {
        const float4 kv = kp[e];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float4 qv = *reinterpret_cast<const float4*>(&q_s[r][4 * e]);
          s[r] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[r]))));
        }
      }
    }
    float p[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float z = (vis[r] >> lane) & 1u ? s[r] : -INFINITY;
      float mx = z;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn;
      const float fac = exp2f(m[r] - base);
      p[r] = exp2f(z - base);
      l[r] = fmaf(l[r], fac, p[r]);   // per lane; summed at the end
#pragma unroll
      for (int u = 0; u < D; ++u) acc[r][u] *= fac;
      m[r] = mn;
    }
    // eight keys' values on their way at a time
#pragma unroll 1
    for (int k0 = 0; k0 < kKeys; k0 += 8) {
      float v[8][D];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const long long vr = __shfl_sync(0xffffffffu, row, k0 + k);
#pragma unroll
        for (int u = 0; u < D; ++u)        // (-1: seen by no row, or a page outside the pool)
          v[k][u] = load_if<DH>(vr >= 0 && (DH >= 32 || lane < DH), (const float*)a.c.v + vr * DH + lane + 32 * u);
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float pk = __shfl_sync(0xffffffffu, p[r], k0 + k);
          if ((vis[r] >> (k0 + k)) & 1u) {
#pragma unroll
            for (int u = 0; u < D; ++u) acc[r][u] = fmaf(pk, v[k][u], acc[r][u]);
          }
        }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float ls = warp_sum(l[r]);
    if (lane == 0) {
      m_s[warp][r] = m[r];
      l_s[warp][r] = ls;
    }
#pragma unroll
    for (int u = 0; u < D; ++u)
      if (DH >= 32 || lane < DH) acc_s[warp][r][lane + 32 * u] = acc[r][u];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * DH; i += kFWarps * 32) {
    const int r = i / DH, e = i % DH;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFWarps; ++w) M = fmaxf(M, m_s[w][r]);
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f, A = 0.f;
#pragma unroll
    for (int w = 0; w < kFWarps; ++w) {
      const float wgt = exp2f(m_s[w][r] - base);
      L = fmaf(l_s[w][r], wgt, L);
      A = fmaf(acc_s[w][r][e], wgt, A);
    }
    if (f.n_range == 1) {
      // zeros for a negative position, which sees no key; where keys are seen and all
      // scores are -inf the sum is 0 too, and 0 / 0 the answer
      ((float*)a.o)[row_at(r) + e] = sr.first + ((rt * kRows + r) >> a.g_sh) < 0 ? 0.f : A / L;
    } else {
      float* p = f.part + ((((((size_t)b * a.c.Hkv + h) * f.n_tiles + rt) * f.n_range + rg) * kRows) + r) * (DH + 2);
      p[e] = A;
      if (e == 0) {
        p[DH] = M;
        p[DH + 1] = L;
      }
    }
  }
}

// Joins the key ranges of a row, one warp per row.
template <int DH>
__global__ void __launch_bounds__(256) k_f32_merge(const F32Args f) {
  pdl_trigger();
  pdl_wait();
  constexpr int D = (DH + 31) / 32;
  const AttnArgs& a = f.a;
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;         // kRows warps
  const int rt = blockIdx.x, h = blockIdx.y, b = blockIdx.z, G = 1 << a.g_sh;
  const SeqRange sr = seq_range(a, b);
  const int t = rt * kRows + r;
  if (t >= sr.nn * G) return;
  const float* p0 = f.part + (((((size_t)b * a.c.Hkv + h) * f.n_tiles + rt) * f.n_range) * kRows + r) * (DH + 2);
  const size_t step = (size_t)kRows * (DH + 2);
  constexpr int U = 8;                  // ranges in flight, under a running maximum
  float M = -INFINITY, L = 0.f, acc[D];
#pragma unroll
  for (int u = 0; u < D; ++u) acc[u] = 0.f;
  for (int i = 0; i < f.n_range; i += U) {
    float m[U], l[U], v[U][D];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const float* p = p0 + (i + j) * step;
      const bool in = i + j < f.n_range;
      m[j] = in ? p[DH] : -INFINITY;
      l[j] = in ? p[DH + 1] : 0.f;
#pragma unroll
      for (int u = 0; u < D; ++u) v[j][u] = in && (DH >= 32 || lane < DH) ? p[lane + 32 * u] : 0.f;
    }
    float mx = M;
#pragma unroll
    for (int j = 0; j < U; ++j) mx = fmaxf(mx, m[j]);
    const float base = mx == -INFINITY ? 0.f : mx, fac = exp2f(M - base);
    L *= fac;
#pragma unroll
    for (int u = 0; u < D; ++u) acc[u] *= fac;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const float wgt = exp2f(m[j] - base);
      L = fmaf(l[j], wgt, L);
#pragma unroll
      for (int u = 0; u < D; ++u) acc[u] = fmaf(v[j][u], wgt, acc[u]);
    }
    M = mx;
  }
  float* out = (float*)a.o + (((size_t)b * a.n + (t >> a.g_sh)) * a.H + h * G + (t & (G - 1))) * DH;
#pragma unroll
  for (int u = 0; u < D; ++u)
    if (DH >= 32 || lane < DH) out[lane + 32 * u] = sr.first + (t >> a.g_sh) < 0 ? 0.f : acc[u] / L;
}

// Row tiles, and key ranges: so many that the CTAs fill the GPU twice, with a
// step of all eight warps (256 keys) in each at least.
F32Args f32_plan(const AttnArgs& a, void* ws) {
  F32Args f;
  f.a = a;
  f.part = (float*)ws;
  const int G = a.H / a.c.Hkv;
  f.n_tiles = (a.n * G + kRows - 1) / kRows;
  const long long base = (long long)f.n_tiles * a.c.Hkv * a.c.B;
  long long keys = a.c.T;                                    // a tile's keys at most
  if (a.window > 0) keys = std::min<long long>(keys, (long long)a.window + a.sinks + kRows + 2 * kKeys);
  const long long most = (keys + kFWarps * kKeys - 1) / (kFWarps * kKeys);
  f.n_range = (int)std::max<long long>(1, std::min<long long>(most, (2LL * sm_count() + base - 1) / std::max<long long>(base, 1)));
  return f;
}

template <int DH>
cudaError_t run_f32(const AttnArgs& a, void* ws, cudaStream_t s) {
  const F32Args f = f32_plan(a, ws);
  cudaError_t e = launch_pdl(k_attn_f32<DH>, dim3((unsigned)(f.n_tiles * f.n_range), a.c.Hkv, a.c.B),
                             dim3(kFWarps * 32), 0, s, f);
  if (e == cudaSuccess && f.n_range > 1)
    e = launch_pdl(k_f32_merge<DH>, dim3((unsigned)f.n_tiles, a.c.Hkv, a.c.B), dim3(kRows * 32), 0, s, f);
  return e;
}

// Few rows per KV head stream the cache through warp-level MMAs, more take the
// tensor-core kernel, whose work does not grow with the rows up to 128.  bf16,
// 20 and 32 rows against that kernel: 53 and 56 against 60 us (4 sequences of 16k,
// 8 KV heads of 128), 63 and 66 against 76 (one of 64k), 89 and 92 against 94 (32 of
// 4k); e4m3: 50 and 53 against 64, 57 and 59 against 81, 81 and 84 against 110.
bool few(const AttnArgs& a) { return a.n * (a.H / a.c.Hkv) <= kFewRows; }

}  // namespace

bool cache_attn_fits(const AttnArgs& a) { return a.c.dtype == TB_F32 || !few(a) || cache_attn_few_fits(a); }

size_t cache_attn_workspace(const AttnArgs& a) {
  if (a.c.dtype != TB_F32) return few(a) ? cache_attn_few_workspace(a) : cache_attn_many_workspace(a);
  if (a.c.B == 0 || a.n == 0) return 0;
  const F32Args f = f32_plan(a, nullptr);
  return f.n_range == 1 ? 0
                        : (size_t)a.c.B * a.c.Hkv * f.n_tiles * f.n_range * kRows * (a.c.dh + 2) * sizeof(float);
}

// The most that any call of up to a.n tokens needs.  Streaming calls need less
// where their rows are dealt differently, fp32 ones where there are tiles enough
// to leave the keys whole; the tensor-core kernel's need grows with n.
size_t cache_attn_workspace_upto(const AttnArgs& a) {
  size_t most = cache_attn_workspace(a);
  const int G = a.H / a.c.Hkv;
  AttnArgs b = a;
  const int step = a.c.dtype == TB_F32 ? kRows / std::min(G, kRows) : 1;
  const int rows = a.c.dtype == TB_F32 ? 2 * sm_count() * kRows : kFewRows;
  for (b.n = step; b.n < a.n && b.n * G <= rows; b.n += step) most = std::max(most, cache_attn_workspace(b));
  return most;
}

cudaError_t launch_cache_attn(const AttnArgs& a, void* ws, cudaStream_t s) {
  if (a.c.dtype != TB_F32) return few(a) ? launch_cache_attn_few(a, ws, s) : launch_cache_attn_many(a, ws, s);
  switch (a.c.dh) {
    case 16: return run_f32<16>(a, ws, s);
    case 32: return run_f32<32>(a, ws, s);
    case 64: return run_f32<64>(a, ws, s);
    case 128: return run_f32<128>(a, ws, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tb
