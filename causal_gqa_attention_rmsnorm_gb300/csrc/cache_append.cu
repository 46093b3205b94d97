// Appending rows to a KV cache with the position rotation applied on the way.
//
// Row i of sequence b sits at position p = start[b] + i; each adjacent pair
// (x0, x1) of its q and k becomes (x0·c - x1·s, x0·s + x1·c) with (c, s) from
// row p of a table formed in fp64.  Every product and sum rounds to fp32 on its
// own (no contraction), so that the stored bits do not depend on how a compiler
// fuses them; the result is rounded once to the stored type.
//
// The bytes bound it: every row is read and written once, the table's rows are
// reused by all heads of a token.  Measured: 4 x 4096 bf16 rows of 32 + 2·8 heads
// of 128 into 64-row pages, 60 us, 0.82 of the copy bandwidth; 3 x 1371 rows of
// 12 + 2·12 heads of 64 into e4m3 blocks of 64, 9.3 us (0.43: a CTA reads its block,
// reduces and writes, and nothing overlaps one block's reduction with the next one's
// reads), 4 x 4096 rows of 32 + 2·8 heads of 128 into e4m3 pages of 64 78 us (0.58);
// fp32, 4 x 2048 rows, 63 us (0.77); one token 2.0 us, fp32 2.4, a launch.
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
  cs[0] = p[0];
  cs[1] = p[1];
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

// Eight elements as they lie in memory.
template <typename T> struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = sizeof(T) == 4 ? __uint_as_float((&v[0].x)[i])
                            : __uint_as_float(i & 1 ? (&v[0].x)[i >> 1] & 0xffff0000u : (&v[0].x)[i >> 1] << 16);
  }
};

// The rows of one token, by a group of threads (`me` of `group`): q, and for
// 16- and 32-bit caches (with_kv) k and v.  A thread holds one eight-element piece
// of a head and that piece's four (cos, sin) pairs and walks the heads of the
// token, H of q (if any), then Hkv of k and of v, three of them on their way at a
// time: the angles and the page are looked up once per thread, not once per head,
// and the first rows are asked for before the position is known.
constexpr int kAhead = 3;
// Threads of a group: a power of two that holds a head, and the token's `total`
// heads kAhead to a thread where 256 threads can.
int group_of(int dh, int total) {
  const int pieces = dh / kVec;
  int g = 32;
  while (g < 256 && (g < pieces || g * kAhead < total * pieces)) g *= 2;
  return g;
}
template <typename T>
__device__ __forceinline__ void rotate_token(const AppendArgs& a, int b, int i, int me, int group, bool with_kv) {
  const int per = div_sh(group, a.pieces, a.piece_sh);  // heads in step
  const int h0 = div_sh(me, a.pieces, a.piece_sh), e = (me - h0 * a.pieces) * kVec;
  if (h0 >= per) return;
  const int Hkv = a.c.Hkv, H = a.q ? a.H : 0, dh = a.c.dh;
  const T* src_q = (const T*)a.q + b * a.q_seq + i * a.q_tok + e;
  const T* src_k = (const T*)a.k + b * a.k_seq + i * a.k_tok + e;
  const T* src_v = (const T*)a.v + b * a.v_seq + i * a.v_tok + e;
  const int total = H + (with_kv ? 2 * Hkv : 0);
  Raw8<T> raw[kAhead];
  auto load = [&](int hb) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = hb + u * per;
      if (h < total)
        raw[u].load(h < H ? src_q + (size_t)h * dh
                          : h < H + Hkv ? src_k + (size_t)(h - H) * dh : src_v + (size_t)(h - H - Hkv) * dh);
    }
  };
  load(h0);             // on their way while the position, the page and the angles arrive
  const Place p = place_of(a, b);
  if (i >= p.nn) return;
  const int pos = p.t0 + i;
  float4 cs[2];
  load_cs(a, pos, e, cs);
  // (plane of KV head 0, row in it): the same page for all heads
  long long plane0 = (long long)b * Hkv;
  int in_plane = pos, plane_rows = a.c.T;
  if (with_kv && a.c.bt) {
    const int page = cache_page(a.c, b, pos);
    plane0 = page < 0 ? -1 : (long long)page * Hkv;
    in_plane = in_block(a.c, pos);
    plane_rows = a.c.ps;
  }
  T* dst_q = (T*)a.q_out + ((size_t)b * a.n + i) * H * dh + e;
  for (int hb = h0; hb < total; hb += kAhead * per) {
    if (hb != h0) load(hb);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = hb + u * per;
      if (h >= total) break;
      if (h < H + Hkv) {                                // (v is stored as it came)
        float x[8];
        raw[u].get(x);
        rotate8(x, cs);
        if (h < H) {
          store8(dst_q + (size_t)h * dh, x);
          continue;
        }
        if (plane0 >= 0) store8((T*)a.c.k + ((plane0 + h - H) * plane_rows + in_plane) * dh + e, x);
      } else if (plane0 >= 0) {
        raw[u].store((T*)a.c.v + ((plane0 + h - H - Hkv) * plane_rows + in_plane) * dh + e);
      }
    }
  }
}

// Five CTAs per SM: 59.9 us for the 4 x 4096 rows, against 61.5 with six and 75.9
// with seven (fewer registers than the rows on their way need).
template <typename T>
__global__ void __launch_bounds__(256, 5) k_append_rope(AppendArgs a, int group) {
  pdl_trigger();
  pdl_wait();
  const int sh = 31 - __clz(group), i = blockIdx.x * (blockDim.x >> sh) + (threadIdx.x >> sh), me = threadIdx.x & (group - 1);
  if (i >= a.n) return;
  if (a.start && i == 0 && me == 0) set_len(a, blockIdx.y);
  rotate_token<T>(a, blockIdx.y, i, me, group, true);
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

// The blocks first, then q: of a sequence's CTAs the first n_blocks take one block
// of the cache, one KV head and K or V each, the others q's tokens.
// For a block: the largest magnitude of its new rows, the scale, then the codes.
// With NP > 0 a thread holds its NP eight-element pieces, rotated, from the one
// pass to the other (32 bits each); with NP = 0 (blocks of more rows) the rows are
// read twice, the second time from L1/L2.
template <int NP>
__global__ void __launch_bounds__(256) k_append_e4m3(AppendArgs a, int n_blocks, int group) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y, c = blockIdx.x;
  if (c >= n_blocks) {
    const int sh = 31 - __clz(group), i = (c - n_blocks) * (blockDim.x >> sh) + (threadIdx.x >> sh);
    if (i < a.n) rotate_token<bf16>(a, b, i, threadIdx.x & (group - 1), group, false);
    return;
  }
  const int half = div_sh(c, a.c.Hkv, a.hkv_sh), h = c - half * a.c.Hkv, is_v = half & 1, bi = half >> 1;
  if (a.start && h == 0 && is_v == 0 && bi == 0 && threadIdx.x == 0) set_len(a, b);
  const Place p = place_of(a, b);
  if (p.nn <= 0) return;
  const int bs = a.c.ps, dh = a.c.dh;
  const int blk = block_of(a.c, p.t0) + bi;
  const int t_lo = max(p.t0, blk * bs), t_hi = min(p.t0 + p.nn, (blk + 1) * bs);
  if (t_lo >= t_hi) return;
  // (the page's look-up, and with it the scale's, is on its way with the rows)
  long long sc = 0;
  const long long row0 = cache_row(a.c, b, h, blk * bs, &sc);
  const bf16* src = is_v ? (const bf16*)a.v + b * a.v_seq + (size_t)h * dh : (const bf16*)a.k + b * a.k_seq + (size_t)h * dh;
  const long long tok = is_v ? a.v_tok : a.k_tok;
  const int n_pieces = (t_hi - t_lo) * a.pieces;
  auto fetch = [&](int i, float (&x)[8]) {
    const int r = div_sh(i, a.pieces, a.piece_sh), t = t_lo + r, e = (i - r * a.pieces) * kVec;
    load8(src + (long long)(t - p.t0) * tok + e, x);
    if (!is_v) {
      float4 cs[2];
      load_cs(a, t, e, cs);
      rotate8(x, cs);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = no_inf(x[u]);
  };
  float held[NP > 0 ? NP : 1][8];
  float top = 0.f;
  auto take = [&](const float (&x)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) top = fmaxf(top, fabsf(x[u]));     // fmaxf drops NaN
  };
  if constexpr (NP > 0) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      if (i < n_pieces) {
        fetch(i, held[j]);
        take(held[j]);
      }
    }
  } else {
    for (int i = threadIdx.x; i < n_pieces; i += blockDim.x) {
      fetch(i, held[0]);
      take(held[0]);
    }
  }
  if (row0 < 0) return;                                  // a page outside the pool
  uint8_t* dst = (uint8_t*)(is_v ? a.c.v : a.c.k) + row0 * dh;
  float* scale = (is_v ? a.c.vs : a.c.ks) + sc;
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
    for (int i = threadIdx.x; i < (t_lo - blk * bs) * a.pieces; i += blockDim.x) {
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
  auto put = [&](int i, const float (&x)[8]) {
    uint2 w;
    w.x = e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16;
    w.y = e4m3x2(x[4] * inv, x[5] * inv) | e4m3x2(x[6] * inv, x[7] * inv) << 16;
    const int r = div_sh(i, a.pieces, a.piece_sh), t = t_lo + r, e = (i - r * a.pieces) * kVec;
    *reinterpret_cast<uint2*>(dst + (size_t)(t - blk * bs) * dh + e) = w;
  };
  if constexpr (NP > 0) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      if (i < n_pieces) put(i, held[j]);
    }
  } else {
    for (int i = threadIdx.x; i < n_pieces; i += blockDim.x) {
      fetch(i, held[0]);
      put(i, held[0]);
    }
  }
}

}  // namespace

cudaError_t launch_append_rope(const AppendArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.c.dtype != TB_E4M3) {
    const int group = group_of(a.c.dh, (a.q ? a.H : 0) + 2 * a.c.Hkv);
    int threads = group;
    while (threads < 256 && threads / group < a.n) threads *= 2;
    const dim3 grid((unsigned)((a.n + threads / group - 1) / (threads / group)), (unsigned)a.c.B);
    e = a.c.dtype == TB_F32 ? launch_pdl(k_append_rope<float>, grid, dim3(threads), 0, s, a, group)
                            : launch_pdl(k_append_rope<bf16>, grid, dim3(threads), 0, s, a, group);
  } else {
    const int nb = (int)(((long long)a.n + a.c.ps - 2) / a.c.ps) + 1;        // blocks that n rows can reach from any start
    const int pieces = std::min(a.n, a.c.ps) * (a.c.dh / kVec);      // of a block, at most
    // (a step of few rows per block has many small CTAs: q takes no more than half
    // of the usual threads there)
    int group = group_of(a.c.dh, a.q ? a.H : 0);
    if (pieces <= 128) group = std::min(group, 128);
    // a power of two, so that whole groups of q's tokens fill a CTA
    int threads = 32;
    while (threads < 256 && (threads < pieces || (a.q && threads < group))) threads *= 2;
    const long long blocks = 2LL * a.c.Hkv * nb;
    const long long tokens = a.q ? (a.n + threads / group - 1) / (threads / group) : 0;
    if (blocks + tokens > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)(blocks + tokens), (unsigned)a.c.B);
    const int first = (int)blocks;
    const int np = (pieces + threads - 1) / threads;
    if (np <= 1)
      e = launch_pdl(k_append_e4m3<1>, grid, dim3(threads), 0, s, a, first, group);
    else if (np <= 2)
      e = launch_pdl(k_append_e4m3<2>, grid, dim3(threads), 0, s, a, first, group);
    else if (np <= 4)
      e = launch_pdl(k_append_e4m3<4>, grid, dim3(threads), 0, s, a, first, group);
    else if (np <= 8)
      e = launch_pdl(k_append_e4m3<8>, grid, dim3(threads), 0, s, a, first, group);
    else
      e = launch_pdl(k_append_e4m3<0>, grid, dim3(threads), 0, s, a, first, group);
  }
  if (e == cudaSuccess && !a.start)
    e = launch_pdl(k_append_lens, dim3((a.c.B + 127) / 128), dim3(128), 0, s, a);
  return e;
}

}  // namespace tb
