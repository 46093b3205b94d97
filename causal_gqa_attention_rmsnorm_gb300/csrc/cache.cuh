// Internal interface of the cache operators: appending rows with the rotation
// applied, and attention of several tokens over a cache.
#pragma once

#include "common.cuh"

namespace tb {

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
  int per = 0;             // pages (or blocks) per sequence
  int num_pages = 0;
  int dtype = TB_BF16;
  int* err = nullptr;
};

// Page of token t of sequence b; -1 (flagged) for an id outside the pool.
__device__ __forceinline__ int cache_page(const CacheView& c, int b, int t) {
  const int page = c.bt[(size_t)b * c.per + t / c.ps];
  if (page >= 0 && page < c.num_pages) return page;
  atomicOr(c.err, TB_DEVERR_BAD_PAGE);
  return -1;
}

// Row index (in rows of dh) of token t and, with `sc`, the index of its scale;
// -1 for a bad page.
__device__ __forceinline__ long long cache_row(const CacheView& c, int b, int h, int t, long long* sc = nullptr) {
  if (!c.bt) {
    const long long plane = (long long)b * c.Hkv + h;
    if (sc) *sc = plane * c.per + t / c.ps;
    return plane * c.T + t;
  }
  const int page = cache_page(c, b, t);
  if (page < 0) return -1;
  const long long plane = (long long)page * c.Hkv + h;
  if (sc) *sc = plane;
  return plane * c.ps + t % c.ps;
}

// e4m3 block scales are 2^e with e in [kE4Min, kE4Max]: the block's largest
// finite magnitude is at most 448·2^e.  The lower end keeps full precision for
// blocks down to ~1e-9, and the two ends lie less than 2^96 apart, so that the
// ratio of any two scales stays far inside fp32 in the attention's exponents.
constexpr int kE4Min = -24, kE4Max = 60;

struct AttnArgs {
  CacheView c;
  const void* q = nullptr;         // [B, n, H, dh]
  void* o = nullptr;
  const int32_t* n_new = nullptr;
  int n = 0, H = 0;
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
// Keys a query at position p sees: [0, sink_end) and [win_lo, p], disjoint.
__device__ __forceinline__ int win_lo(int p, int window) { return window > 0 && p >= window ? p - window + 1 : 0; }

// cache_append.cu
struct AppendArgs {
  CacheView c;
  const void *q, *k, *v;
  void* q_out;
  long long q_tok, q_seq, k_tok, k_seq, v_tok, v_seq;
  int H, n;
  const int32_t *start, *n_new;    // start == nullptr: lens
  const float2* rope;
};
cudaError_t launch_append_rope(const AppendArgs& a, cudaStream_t s);

// cache_attn.cu
size_t cache_attn_workspace(const AttnArgs& a);
cudaError_t launch_cache_attn(const AttnArgs& a, void* ws, cudaStream_t s);

}  // namespace tb
