// Internal interface of the cache operators: appending rows with the rotation
// applied, and attention of several tokens over a cache.
#pragma once

#include "common.cuh"

namespace tb {

// Everything that lies in global memory is read with plain loads: these grids are
// resident before the kernel in front of them ends (pdl_trigger), which may still be
// writing lengths, rows, scales or the rotation table, and a non-coherent load
// (ld.global.nc) wants memory that nobody writes while its grid lives.

// A cache as the kernels see it.  Row t of (sequence b, KV head h):
//   contiguous (bt == nullptr): row (b·Hkv + h)·T + t
//   paged: row (page·Hkv + h)·ps + t % ps, page = bt[b·per + t / ps]
// The e4m3 scale of the row: index (b·Hkv + h)·per + t / ps, or page·Hkv + h.
struct CacheView {
  void* k = nullptr;
  void* v = nullptr;
  float* ks = nullptr;
  float* vs = nullptr;
  const int32_t* bt = nullptr;
  int32_t* lens = nullptr;
  int B = 0, Hkv = 0, T = 0, dh = 0;
  int ps = 1;              // rows per page, or per scale block of a contiguous e4m3 cache
  int ps_sh = -1;          // log2 of it where it is a power of two
  int per = 0;             // pages (or blocks) per sequence
  int num_pages = 0;
  int dtype = TB_BF16;
  int* err = nullptr;
};

// x / n where sh is log2 n or -1: the look-ups below stand in chains of latencies.
__device__ __forceinline__ int div_sh(int x, int n, int sh) { return sh >= 0 ? x >> sh : x / n; }
inline int shift_of(int n) { return n > 0 && (n & (n - 1)) == 0 ? __builtin_ctz((unsigned)n) : -1; }
// Page (or scale block) of a sequence that token t lies in, and its row there.
__device__ __forceinline__ int block_of(const CacheView& c, int t) { return div_sh(t, c.ps, c.ps_sh); }
__device__ __forceinline__ int in_block(const CacheView& c, int t) { return t - block_of(c, t) * c.ps; }

// Page of token t of sequence b; -1 (flagged) for an id outside the pool.
__device__ __forceinline__ int cache_page(const CacheView& c, int b, int t) {
  const int page = c.bt[(size_t)b * c.per + block_of(c, t)];
  if (page >= 0 && page < c.num_pages) return page;
  atomicOr(c.err, TB_DEVERR_BAD_PAGE);
  return -1;
}

// Row index (in rows of dh) of token t and, with `sc`, the index of its scale;
// -1 for a bad page.
__device__ __forceinline__ long long cache_row(const CacheView& c, int b, int h, int t, long long* sc = nullptr) {
  if (!c.bt) {
    const long long plane = (long long)b * c.Hkv + h;
    if (sc) *sc = plane * c.per + block_of(c, t);
    return plane * c.T + t;
  }
  const int page = cache_page(c, b, t);
  if (page < 0) return -1;
  const long long plane = (long long)page * c.Hkv + h;
  if (sc) *sc = plane;
  return plane * c.ps + in_block(c, t);
}

// e4m3 block scales are 2^e with e in [kE4Min, kE4Max]: the block's largest
// finite magnitude is at most 448·2^e.  The lower end keeps full precision for
// blocks down to ~1e-9, and the two ends lie less than 2^96 apart, so that the
// ratio of any two scales stays far inside fp32 in the attention's exponents.
constexpr int kE4Min = -24, kE4Max = 60;

// Four e4m3 codes as fp16, exactly, two pairs.  (Moving the bits with logic
// operations instead, seven for four codes, ran slower: 156 against 126 us for
// 32 sequences of a 16k cache.)
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Two values to e4m3 codes (low byte: lo), saturating, NaN staying NaN; and back.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  float2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}
// 2^-e with x·2^-e in [0.5, 1) for a normal x > 0, held to normal powers of two; 1 otherwise.
__device__ __forceinline__ float pow2_frame(float x) {
  if (!(x > 0.f)) return 1.f;
  const int e = max(-126, min(126, (int)((__float_as_uint(x) >> 23) & 0xffu) - 126));
  return __uint_as_float((uint32_t)(127 - e) << 23);
}
// bf16 queries as two e4m3 terms, q = q1 + q2, under a power of two that brings a
// row's largest element into [128, 256): q1 takes the leading four bits of an
// element, the rest is at most half a step of q1 and has four bits itself, so the
// split is exact for elements down to 2^-2 and off by 2^-10 at most below (2^-17
// of the row's largest).  Both terms multiply the K codes as they lie in the
// cache.  The power of two: NaN for a row with an infinity, which must not
// saturate.
__device__ __forceinline__ float split_frame(float amax) {
  return amax <= 3.402823466e38f ? pow2_frame(fmaxf(amax, 0x1p-118f)) * 256.f : NAN;
}
// Four bf16 elements (two words), times fr: codes of both terms.
__device__ __forceinline__ void split4(uint32_t a, uint32_t b, float fr, uint32_t& t1, uint32_t& t2) {
  const float v[4] = {__uint_as_float(a << 16) * fr, __uint_as_float(a & 0xffff0000u) * fr, __uint_as_float(b << 16) * fr,
                      __uint_as_float(b & 0xffff0000u) * fr};
  const uint32_t c0 = e4m3x2(v[0], v[1]), c1 = e4m3x2(v[2], v[3]);
  const float2 f0 = from_e4m3x2(c0), f1 = from_e4m3x2(c1);
  t1 = c0 | c1 << 16;
  t2 = e4m3x2(v[0] - f0.x, v[1] - f0.y) | e4m3x2(v[2] - f1.x, v[3] - f1.y) << 16;
}

// Shared memory by 32-bit address: a pointer that went through an integer would
// be taken for a generic one.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
// log2 of a block scale, and its inverse.
__device__ __forceinline__ float scale_exp(float s) { return (float)((int)(__float_as_uint(s) >> 23) - 127); }
__device__ __forceinline__ float scale_inv(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

struct AttnArgs {
  CacheView c;
  const void* q = nullptr;         // [B, n, H, dh]
  void* o = nullptr;
  const int32_t* n_new = nullptr;
  int n = 0, H = 0;
  int g_sh = 0;                    // log2 of G = H/Hkv
  int window = 0, sinks = 0;
  float scale_log2 = 0.f;          // score scale · log2 e
};

// The queries of sequence b: `nn` of them, the first at position `first`
// (negative positions see nothing), over `len` rows.
struct SeqRange {
  int len, nn, first;
};
__device__ __forceinline__ SeqRange seq_range(const AttnArgs& a, int b) {
  SeqRange r;
  r.len = a.c.lens[b];
  if (r.len > a.c.T) {
    atomicOr(a.c.err, TB_DEVERR_CACHE_FULL);
    r.len = a.c.T;
  }
  if (r.len < 0) r.len = 0;
  r.nn = a.n_new ? min(max(a.n_new[b], 0), a.n) : a.n;
  r.first = r.len - r.nn;
  return r;
}
// A query at position p sees keys [win_lo, p] and, below win_lo, the sinks.
__device__ __forceinline__ int win_lo(int p, int window) { return window > 0 && p >= window ? p - window + 1 : 0; }

// The runs of `unit` keys (aligned) that hold every key some query of a
// sequence sees: the first `ns`, then from `wl` on; `count` in all, none beyond
// the sequence.  Run g of the list starts at key run_key(r, g).
struct KeyRuns {
  int ns, wl, count;
};
__device__ __forceinline__ KeyRuns key_runs(int len, int first, int window, int sinks, int unit) {
  KeyRuns r{0, 0, 0};
  if (len <= 0) return r;
  r.wl = win_lo(first, window) / unit;
  r.ns = min((min(sinks, len) + unit - 1) / unit, r.wl);
  r.count = r.ns + (len - 1) / unit - r.wl + 1;
  return r;
}
__device__ __forceinline__ int run_index(const KeyRuns& r, int g) { return g < r.ns ? g : g - r.ns + r.wl; }

// cache_append.cu
struct AppendArgs {
  CacheView c;
  const void *q, *k, *v;
  void* q_out;
  long long q_tok, q_seq, k_tok, k_seq, v_tok, v_seq;
  int H, n;
  int pieces, piece_sh, hkv_sh;    // eight-element pieces of a row, log2 of them or -1, of Hkv or -1
  const int32_t *start, *n_new;    // start == nullptr: lens
  const float2* rope;
};
cudaError_t launch_append_rope(const AppendArgs& a, cudaStream_t s);

// cache_attn_few.cu: up to kFewRows query rows (tokens x heads) per KV head,
// 16-bit queries over bf16 or e4m3 rows of dh 64 or 128.
constexpr int kFewRows = 32;
// Whether the stages of one sequence can be numbered (at most 2^30).
bool cache_attn_few_fits(const AttnArgs& a);
size_t cache_attn_few_workspace(const AttnArgs& a);
cudaError_t launch_cache_attn_few(const AttnArgs& a, void* ws, cudaStream_t s);
// cache_attn_many.cu: any number of rows, same types and widths.
size_t cache_attn_many_workspace(const AttnArgs& a);
cudaError_t launch_cache_attn_many(const AttnArgs& a, void* ws, cudaStream_t s);

// One bf16 query row by one warp, as the formula reads: keys it does not see are
// not touched at all.  For rows whose fast result is not finite (a weight of 0
// times an infinity or NaN in a row that the query does not see, or a value that
// really is not finite).  q points to DH elements; every lane returns with
// out[u] = o[lane·DH/32 + u].
__device__ __forceinline__ void eight_of(const CacheView& c, const void* base, long long row, int e, float (&x)[8]) {
  if (c.dtype == TB_BF16) {
    Vec16<bf16> v;
    v.raw = *reinterpret_cast<const uint4*>((const bf16*)base + row * c.dh + e);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v.get(i);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>((const uint8_t*)base + row * c.dh + e);
    uint32_t h[4];
    codes4(w.x, h[0], h[1]);
    codes4(w.y, h[2], h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
          : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
          : "r"(h[i]));
  }
}
template <int DH>
__device__ __noinline__ void attend_row(const AttnArgs& a, int b, int hkv, int pos, const bf16* q, float (&out)[DH / 32]) {
  constexpr int D = DH / 32;              // output dims per lane: part of one eight
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f, acc[D];
#pragma unroll
  for (int u = 0; u < D; ++u) acc[u] = 0.f;
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
      for (int e = 0; e < DH; e += 8) {
        Vec16<bf16> qv;
        qv.raw = *reinterpret_cast<const uint4*>(q + e);
        float k[8];
        eight_of(a.c, a.c.k, row, e, k);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(qv.get(i), k[i], s);
      }
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
    for (int u = 0; u < D; ++u) acc[u] *= f;
    const float pv = p * (row >= 0 && a.c.dtype == TB_E4M3 ? a.c.vs[sc] : 1.f);
    const int steps = min(32, nkeys - j0);
    for (int k = 0; k < steps; ++k) {
      const float pk = __shfl_sync(0xffffffffu, pv, k);
      const long long rk = __shfl_sync(0xffffffffu, row, k);
      if (rk < 0) continue;
      float v[8];
      eight_of(a.c, a.c.v, rk, lane * D & ~7, v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((i & ~(D - 1)) == (lane * D & 7)) acc[i & (D - 1)] = fmaf(pk, v[i], acc[i & (D - 1)]);
    }
  }
#pragma unroll
  for (int u = 0; u < D; ++u) out[u] = nkeys == 0 ? 0.f : acc[u] / l;     // (0 / 0 where all scores are -inf)
}

// cache_attn.cu
bool cache_attn_fits(const AttnArgs& a);
size_t cache_attn_workspace(const AttnArgs& a);
size_t cache_attn_workspace_upto(const AttnArgs& a);
cudaError_t launch_cache_attn(const AttnArgs& a, void* ws, cudaStream_t s);

}  // namespace tb
