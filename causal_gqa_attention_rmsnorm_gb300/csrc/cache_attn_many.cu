// Attention of many query rows over a bf16 or e4m3 cache on the 5th-generation
// tensor cores: chunks of a prompt, and drafts of more rows than the streaming
// kernel takes.
//
//   The n·G rows (tokens x query heads of a KV head, G = H/Hkv, token-major) of
//   a (sequence, KV head) are packed into tiles of 128, so that every K/V tile
//   staged in shared memory serves all heads of the group; a CTA works on two
//   row tiles ("slots") over the same key tiles:
//     S_g = Q_g·Kᵀ into tensor memory (M = 128, N = 128 keys), softmax in fp32
//     by one thread per row, P back over S in 16 bits, O_g += P_g·V.
//   Roles: warps 0..7 softmax (four per slot), warp 8 copies and hands the pieces
//   of work to the others, warp 9 issues the MMAs, warp 10 (over e4m3 and 11) sees
//   to V tiles that cannot be used as they land.  Where there is but one row tile,
//   both slots work on it, each on every second key tile, and slot 0 joins the two.
//   The MMA order per key tile is P·V of slot 0, S of slot 0 for the next tile, the
//   same of slot 1, so that the tensor pipe works on one slot during the other's
//   softmax.
//
//   Key tiles are 128 aligned keys: those with sinks, then those of the union of
//   the two slots' windows, up to the last query; a slot sits out tiles that
//   none of its rows sees.  Only tiles at a border are masked by element.  Rows
//   of V that no query of the item sees are zeroed in shared memory (0·NaN is
//   NaN inside an MMA), and pages that hold only such rows are not read.
//
//   Balance: an item (a pair of row tiles) costs its key tiles plus one; all
//   items form one line that is cut into equal parts, one per CTA, whatever the
//   lengths.  An item that a cut leaves whole is written out directly; pieces of
//   a cut one leave (max, sum, O) in the workspace and k_many_merge joins them in
//   order.  The line's prefix sums come from k_many_plan.
//
//   e4m3: S is an 8-bit MMA on the K codes as they lie in the cache, the queries
//   split into two e4m3 terms (split4), at twice the 16-bit rate.  P has no such
//   split that pays, so V becomes fp16 (exactly): TMA brings 32-key chunks of codes
//   through a ring and conversion warps write them into the swizzled V tile.  K scales multiply the scores per 16
//   keys; V scales 2^e enter the exponent, p' = 2^(z + e - m'), so that
//   O = Σ p'·code and l = Σ p'·2^-e (see the streaming kernel).
//
// Over bf16 the weights enter P·V rounded to bf16, their sum is taken before: one
// MMA has one type for both operands, and v's range does not fit fp16.  (A chunk of
// 2 x 8192 tokens: error against 64 bits 0.0020 of the output, 0.0016 of it the
// output's own rounding.)
//
// What bounds it: per key tile and slot the chain S ready -> row maximum ->
// exponentials -> P ready, half of which hides behind the other slot's MMAs; and
// the instruction cache, which all roles share: waits that give up live out of
// line, masks are applied by a rolled pass over S in tensor memory before the
// unrolled softmax, which then has one form (conversion waits inline: 545 against
// 472 us; a copy of the softmax for border tiles: 852 against 734; MMAs issued by a
// whole warp instead of one lane: 836 against 734).
// Measured, 32 + 8 heads of 128: 2 x 8192 bf16 tokens, window 4096, 128 sinks, pages
// of 64: 728 us, 1156 TFLOP/s, 0.61 of the 8192-cubed bf16 matrix product; 2048
// tokens at the end of 16000: bf16 389 us, 1292 TFLOP/s, e4m3 432 us, 1163.
//
// Rows whose result is not finite are computed once more by k_many_merge, key by
// key, so that what a masked row holds never matters.
#include <math.h>

#include <algorithm>

#include "cache.cuh"
#include "gemm_tc.cuh"
#include "sm100_ptx.cuh"

namespace tb {
namespace {

using namespace ptx;

constexpr int kBM = 128, kBN = 128;
constexpr float kRescale = 8.f;
constexpr int kChunk = 32;                     // keys per chunk of V codes
constexpr int kRaw = 8;                        // chunks in the ring: two V tiles
constexpr int kScTiles = 8;                    // tiles whose block scales are kept
constexpr int kConv = 2;                       // conversion warps
constexpr float kParts = 1.3f;                 // see parts_of
template <bool E4> constexpr int kVWarps = E4 ? kConv : 1;

template <int DH, bool E4> struct ManyCfg {
  static constexpr int NB = DH / 64;                       // 64-column blocks of a 16-bit row
  static constexpr uint32_t Q_BYTES = kBM * DH * 2;        // a slot's queries, 16-bit
  static constexpr uint32_t QT_BYTES = kBM * DH;           // E4: one term of them
  static constexpr uint32_t K_BYTES = kBN * DH * (E4 ? 1 : 2);
  static constexpr uint32_t V_BYTES = kBN * DH * 2;
  static constexpr uint32_t RAW = kChunk * DH;             // bytes of a chunk of codes
  // E4: the terms of rows of 128 dims replace the row in place (each of its two
  // 128-byte halves); those of 64 dims have tiles of their own
  static constexpr uint32_t OFF_QT = E4 && DH == 64 ? 2 * Q_BYTES : 0;
  static constexpr uint32_t OFF_K = OFF_QT + 2 * Q_BYTES;
  static constexpr uint32_t OFF_V = OFF_K + 2 * K_BYTES;
  static constexpr uint32_t OFF_RAW = OFF_V + 2 * V_BYTES;
  static constexpr uint32_t OFF_SC = OFF_RAW + (E4 ? kRaw * RAW : 0);      // [kScTiles][8 runs]{K scale, log2 of V's}
  static constexpr uint32_t OFF_BAR = OFF_SC + (E4 ? kScTiles * 64 : 0);
  static constexpr uint32_t OFF_DESC = OFF_BAR + 512;
  static constexpr uint32_t OFF_JOIN = OFF_DESC + 1024;    // [128] {max, sum} of slot 1, then slot 0's query factors
  static constexpr size_t SMEM = OFF_JOIN + 1536 + 1024;
  static constexpr uint32_t TMEM_O = 2 * kBN;
  static constexpr int THREADS = E4 ? 384 : 352;
};

struct MergeRec {
  int b, h, p, valid;
  long long start;         // its place on the line
};

struct ManyArgs {
  AttnArgs a;
  int pairs;               // row-tile pairs of a sequence of n tokens
  int tpt;                 // tokens per row tile: 128 / G
  int n_cta;
  int box;                 // keys per box of a 16-bit tile, or of K codes
  int vbox;                // keys per box of V codes
  bool negate;             // the score scale is negative: the scores are negated, its magnitude applied
  long long* pre;          // [B·pairs + 1] line position of (sequence, pair) within its KV head
  MergeRec* rec;    // [n_cta] the item that cut c + 1 goes through first
  int* any;                // whether any flag is set
  uint8_t* flags;          // [B·Hkv·2·pairs] row tiles to look through again
  float4* part;            // [2·n_cta][2][DH/4 + 1][128] pieces
};

// ---- items ------------------------------------------------------------------

// One slot's row tile: `rows` rows of tokens tok0.., at positions p0 .. p1, and
// the list positions it works on: [0, ia) and [ib, ic).
struct SlotRange {
  int tok0, rows, p0, p1, ia, ib, ic;
  __device__ __forceinline__ bool on(int x) const { return x < ia || (x >= ib && x < ic); }
  __device__ __forceinline__ int first_on(int t0, int t1) const {
    if (t0 < min(ia, t1)) return t0;
    const int f = max(t0, ib);
    return f < min(ic, t1) ? f : -1;
  }
  __device__ __forceinline__ int last_on(int t0, int t1) const {
    if (max(t0, ib) < min(ic, t1)) return min(ic, t1) - 1;
    return t0 < min(ia, t1) ? min(ia, t1) - 1 : -1;
  }
};
// A pair of row tiles: its key tiles (list position x is key tile x < ns ? x :
// x - ns + wl), cnt of them; keys from `end` on and in [hid0, hid1) are hidden
// from all its rows.
struct Item {
  SlotRange s0, s1;
  int ns, wl, cnt, end, hid0, hid1;
  __device__ __forceinline__ int tile(int x) const { return x < ns ? x : x - ns + wl; }
};
__device__ __forceinline__ SlotRange slot_range(const ManyArgs& m, const SeqRange& sr, int rt) {
  SlotRange s{0, 0, 0, -1, 0, 0, 0};
  s.tok0 = rt * m.tpt;
  const int toks = min(m.tpt, sr.nn - s.tok0);
  if (toks <= 0) return s;
  s.rows = toks * (kBM / m.tpt);
  s.p0 = sr.first + s.tok0;
  s.p1 = s.p0 + toks - 1;
  return s;
}
__device__ __forceinline__ void slot_list(SlotRange& s, const Item& it, const AttnArgs& a) {
  if (s.rows == 0 || s.p1 < 0) {
    s.ia = s.ib = s.ic = 0;
    return;
  }
  const int hi = s.p1 / kBN, lo = win_lo(s.p0, a.window) / kBN;
  const int sk = min((min(a.sinks, s.p1 + 1) + kBN - 1) / kBN, hi + 1);     // key tiles with sinks
  s.ia = sk <= it.ns ? sk : (sk > it.wl ? sk - it.wl + it.ns : it.ns);
  s.ib = lo - it.wl + it.ns;
  s.ic = hi - it.wl + it.ns + 1;
}
__device__ __forceinline__ Item make_item(const ManyArgs& m, const SeqRange& sr, int p) {
  const AttnArgs& a = m.a;
  Item it{};
  it.s0 = slot_range(m, sr, 2 * p);
  it.s1 = slot_range(m, sr, 2 * p + 1);
  const int last = it.s1.rows ? it.s1.p1 : it.s0.p1;
  if (it.s0.rows == 0 || last < 0) return it;
  it.hid1 = win_lo(it.s0.p0, a.window);
  it.hid0 = min(a.sinks, it.hid1);
  it.end = last + 1;
  it.wl = it.hid1 / kBN;
  it.ns = min((min(a.sinks, it.end) + kBN - 1) / kBN, it.wl);
  it.cnt = it.ns + last / kBN - it.wl + 1;
  slot_list(it.s0, it, a);
  slot_list(it.s1, it, a);
  return it;
}
// What an item costs on the line: its key tiles and one for its queries and
// output; nothing without rows.
__device__ __forceinline__ int item_cost(const ManyArgs& m, const SeqRange& sr, int p) {
  const Item it = make_item(m, sr, p);
  return it.s0.rows ? it.cnt + 1 : 0;
}

// Where line position x lies: sequence, KV head, pair and the item's start.
struct Place {
  int b, h, p;
  long long start;
};
__device__ __forceinline__ Place find_item(const ManyArgs& m, long long x) {
  Place r;
  int lo = 0, hi = m.a.c.B - 1;
  const int Hkv = m.a.c.Hkv;
  while (lo < hi) {                              // the last sequence that starts at or before x
    const int mid = (lo + hi + 1) >> 1;
    if (m.pre[(size_t)mid * m.pairs] * Hkv <= x) lo = mid; else hi = mid - 1;
  }
  r.b = lo;
  const long long* pb = m.pre + (size_t)lo * m.pairs;
  const long long per = pb[m.pairs] - pb[0];     // positive: x lies inside the line
  const long long off = x - pb[0] * Hkv;
  r.h = (int)(off / per);
  const long long in = off - r.h * per + pb[0];
  lo = 0, hi = m.pairs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pb[mid] <= in) lo = mid; else hi = mid - 1;
  }
  r.p = lo;
  r.start = pb[0] * Hkv + r.h * per + pb[lo] - pb[0];
  return r;
}
// How many parts the line has.  An item of s key tiles in t parts takes the time of
// s / t of them and of t pieces in the merge, so parts beyond some multiple of
// sqrt(s) per item only cost: 64 rows over one sequence of 64k with one KV head 121
// us without the limit, 57 with 1.3 sqrt(s), 58 with 1 and 64 with 2.
__device__ __forceinline__ int parts_of(const ManyArgs& m, long long total) {
  const float items = (float)m.a.c.B * m.a.c.Hkv * m.pairs;
  return 1 + (int)fminf((float)(m.n_cta - 1), kParts * sqrtf((float)total * items));
}
// Where part c begins.
__device__ __forceinline__ long long cut(int parts, long long total, int c) {
  return total * min(c, parts) / parts;
}
// The key tiles [t0, t1) of the item at [start, start + cnt + 1) in the part [x0, x1).
__device__ __forceinline__ int2 piece_of(long long start, int cnt, long long x0, long long x1) {
  const long long t0 = max(x0 - start, 1LL) - 1, t1 = min(x1 - start, (long long)cnt + 1) - 1;
  return make_int2((int)t0, (int)max(t0, t1));
}

// The pieces of a CTA, in order; each role walks them alike.  Only the first
// item is looked up on the line; the next one follows from the one before.
struct Pieces {
  const ManyArgs& m;
  long long x, x1;
  Place at;
  Item it;
  SeqRange sr;
  int t0, t1, where;          // where: -1 the whole item, else the piece's slot in the workspace
  bool any = false;
  __device__ Pieces(const ManyArgs& m_, long long a, long long b) : m(m_), x(a), x1(b) {}
  __device__ __forceinline__ void step() {
    if (!any) {
      any = true;
      at = find_item(m, x);
      sr = seq_range(m.a, at.b);
      it = make_item(m, sr, at.p);
      return;
    }
    at.start += it.cnt + 1;
    if (++at.p < m.pairs) {
      it = make_item(m, sr, at.p);
      if (it.s0.rows) return;
    }
    at.p = 0;
    if (++at.h == m.a.c.Hkv) {
      at.h = 0;
      do sr = seq_range(m.a, ++at.b); while (sr.nn == 0);      // the line goes on: there is one
    }
    it = make_item(m, sr, 0);
  }
  __device__ __forceinline__ bool next() {
    while (x < x1) {
      step();
      const int2 t = piece_of(at.start, it.cnt, x, x1);
      const bool begins = x == at.start;
      x = min(x1, at.start + it.cnt + 1);
      t0 = t.x;
      t1 = t.y;
      if (t0 == 0 && t1 == it.cnt && (it.cnt > 0 || begins)) {
        where = -1;
        return true;
      }
      if (t0 < t1) {
        where = 2 * (int)blockIdx.x + (begins ? 1 : 0);
        return true;
      }
    }
    return false;
  }
};

// A piece as the copying warp hands it to the other roles, through a ring in
// shared memory; `last` follows the last piece.
struct PieceDesc {
  int t0, t1, where, last, b, h, p;
  int ns, wl, end, hid0, hid1;
  // One row tile only: slot 0 takes the key tiles t0, t0 + 2, ..., slot 1 the
  // others (all of the list's are its), and slot 0 joins the two.
  int split;
  SlotRange s[2];
  __device__ __forceinline__ bool on(int g, int x) const { return split ? ((x - t0) & 1) == g : s[g].on(x); }
  __device__ __forceinline__ int first_on(int g) const {
    return split ? (t0 + g < t1 ? t0 + g : -1) : s[g].first_on(t0, t1);
  }
  __device__ __forceinline__ int last_on(int g) const {
    return split ? (t0 + g < t1 ? t1 - 1 - ((t1 - 1 - t0 - g) & 1) : -1) : s[g].last_on(t0, t1);
  }
  __device__ __forceinline__ int key(int x) const { return (x < ns ? x : x - ns + wl) * kBN; }
  // whether the tile at `key` holds rows that no row of the item sees
  __device__ __forceinline__ bool border(int key) const {
    return key + kBN > end || (key < hid1 && key + kBN > hid0);
  }
};
constexpr int kDescs = 4;

// pre[e] for e = (sequence, pair) in order, and the flags cleared; one CTA.
__global__ void __launch_bounds__(1024) k_many_plan(const ManyArgs m, int n_flag_words) {
  pdl_trigger();
  pdl_wait();
  __shared__ long long warp_sum_s[32];
  __shared__ long long carry_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < n_flag_words; i += 1024) reinterpret_cast<uint32_t*>(m.flags)[i] = 0u;
  if (tid == 0) {
    carry_s = 0;
    *m.any = 0;
  }
  __syncthreads();
  const int E = m.a.c.B * m.pairs;
  for (int e0 = 0; e0 < E; e0 += 1024) {
    const int e = e0 + tid;
    long long v = 0;
    if (e < E) {
      const int b = e / m.pairs;
      v = item_cost(m, seq_range(m.a, b), e - b * m.pairs);
    }
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sum_s[warp] = inc;
    __syncthreads();
    long long base = carry_s;
    for (int i = 0; i < warp; ++i) base += warp_sum_s[i];
    if (e < E) m.pre[e] = base + inc - v;
    if (e == E - 1) m.pre[E] = base + inc;
    __syncthreads();
    if (tid == 1023) carry_s = base + inc;
    __syncthreads();
  }
}

// ---- the kernel ---------------------------------------------------------------

// mbar_wait with all but the first attempt out of line: the loops of all roles run
// at once and have to share the instruction cache.
__device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  return mbar_wait(bar, parity, abort, err);
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  return mbar_try_wait(smem_u32(bar), parity) || wait_longer(bar, parity, abort, err);
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  const bool ok = wait_one(bar, parity, abort, err);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void tma_load_4d(const CUtensorMap* m, void* dst, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
template <bool E4>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t d;
  if constexpr (E4)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// Instruction descriptor of P·V, kind::f16 with fp16 (E4) or bf16 operands, fp32
// sums, V MN-major.
template <bool E4>
__host__ __device__ constexpr uint32_t idesc_pv(int M, int N) {
  return idesc_bf16(M, N, false, true) & ~(E4 ? (1u << 7 | 1u << 10) : 0u);
}
template <int DH, bool E4>
__global__ void __launch_bounds__((ManyCfg<DH, E4>::THREADS), 1)
    k_attn_many(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const ManyArgs m) {
  pdl_trigger();
  using C = ManyCfg<DH, E4>;
  const AttnArgs& a = m.a;
  int* err = a.c.err;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* q_ready = bars + 2;      // E4: the queries are fp16
  uint64_t* drain = bars + 3;
  uint64_t* k_full = bars + 4;       // [2]
  uint64_t* k_empty = bars + 6;
  uint64_t* v_full = bars + 8;
  uint64_t* v_empty = bars + 10;
  uint64_t* s_full = bars + 12;      // [slot]
  uint64_t* p_full = bars + 14;
  uint64_t* pv_done = bars + 16;
  uint64_t* o_full = bars + 18;
  uint64_t* raw_full = bars + 20;    // [kRaw]
  uint64_t* raw_empty = bars + 28;   // [kRaw]
  uint64_t* sc_full = bars + 36;     // [kScTiles]
  uint64_t* d_full = bars + 44;      // [kDescs]
  uint64_t* d_empty = bars + 48;     // [kDescs]
  uint64_t* fix_full = bars + 52;    // [2]: a border V tile has landed, its hidden rows not yet zeroed
  uint64_t* join_full = bars + 54;   // a split piece: slot 1 is through; slot 0 has read its output
  uint64_t* join_done = bars + 55;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 56);
  float2* ml_s = reinterpret_cast<float2*>(smem + C::OFF_JOIN);
  float* zs_s = reinterpret_cast<float*>(smem + C::OFF_JOIN + 1024);
  PieceDesc* descs = reinterpret_cast<PieceDesc*>(smem + C::OFF_DESC);
  static_assert(sizeof(PieceDesc) * kDescs <= 1024 && 56 * 8 + 8 <= 512, "layout");
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* sc = reinterpret_cast<float*>(smem + C::OFF_SC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(q_ready, 8);
    mbar_init(drain, 1);
    mbar_init(join_full, 4);
    mbar_init(join_done, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], E4 ? kBN / kChunk : 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&fix_full[i], 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 1);
    }
    for (int i = 0; i < kScTiles; ++i) mbar_init(&sc_full[i], 1);
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 9 + kVWarps<E4>);   // the MMA warp, eight softmax warps, those that see to V
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();                                   // the plan, and whatever wrote q and the cache
  const long long total = m.pre[(size_t)a.c.B * m.pairs] * a.c.Hkv;
  const int parts = parts_of(m, total);
  const long long x0 = cut(parts, total, blockIdx.x), x1 = cut(parts, total, blockIdx.x + 1);
  const int G = kBM / m.tpt;
  // The k-th piece for a role other than the copying one; false after the last
  // (or a wait that ran out).  done(k) hands the descriptor back.
  auto piece = [&](int k, PieceDesc*& d) -> bool {
    d = descs + k % kDescs;
    return wait_warp(&d_full[k % kDescs], (k / kDescs) & 1, abort_flag, err) && !d->last;
  };
  auto done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&d_empty[k % kDescs]);
  };

  if (warp == 8) {
    // ---------------- copies ----------------
    int nq = 0, nt = 0;                         // pieces with queries, key tiles
    int nk = 0, nv = 0;                         // K tiles and V tiles (E4: chunks) issued
    int n_fix[2] = {0, 0};                      // border V tiles of each stage; whether its last was one
    uint32_t fixed = 0;
    bool ok = true;
    Pieces pc(m, x0, x1);
    auto publish = [&](int k, bool last) -> bool {
      if (k >= kDescs && !wait_warp(&d_empty[k % kDescs], ((k / kDescs) & 1) ^ 1u, abort_flag, err)) return false;
      if (lane == 0) {
        PieceDesc& d = descs[k % kDescs];
        d.t0 = pc.t0;
        d.t1 = pc.t1;
        d.where = pc.where;
        d.last = last;
        d.b = pc.at.b;
        d.h = pc.at.h;
        d.p = pc.at.p;
        d.ns = pc.it.ns;
        d.wl = pc.it.wl;
        d.end = pc.it.end;
        d.hid0 = pc.it.hid0;
        d.hid1 = pc.it.hid1;
        d.split = pc.it.s1.rows == 0;
        d.s[0] = pc.it.s0;
        d.s[1] = d.split ? pc.it.s0 : pc.it.s1;
        mbar_arrive(&d_full[k % kDescs]);
      }
      __syncwarp();
      return true;
    };
    int np = 0;
    for (;; ++np) {
      const bool more = pc.next();
      if (!publish(np, !more)) {
        ok = false;
        break;
      }
      if (!more) break;
      if (pc.t0 == pc.t1) continue;             // rows without keys
      const Item& it = pc.it;
      if (nq > 0 && !wait_warp(q_empty, (nq - 1) & 1, abort_flag, err)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        const int slots = it.s1.rows ? 2 : 1;
        fence_proxy_async();                    // the queries were rewritten in place (E4)
        mbar_arrive_expect_tx(q_full, slots * C::Q_BYTES);
        for (int g = 0; g < slots; ++g)
#pragma unroll
          for (int blk = 0; blk < C::NB; ++blk)
            tma_load_4d(&tmQ, smem + g * C::Q_BYTES + blk * kBM * 128, q_full, blk * 64, pc.at.h * G,
                        g ? it.s1.tok0 : it.s0.tok0, pc.at.b);
      }
      __syncwarp();
      ++nq;
      // The page ids of a tile are read two tiles ahead, its scales one tile
      // ahead: lane i, box i of the tile (E4: run i of 16 keys).
      const int unit = E4 ? 16 : m.box;
      const bool mine = lane < kBN / unit;
      auto seen_at = [&](int key, int n) { return key < it.end && !(key >= it.hid0 && key + n <= it.hid1); };
      auto page_ahead = [&](int x) {
        if (x >= pc.t1 || !mine) return -1;
        const int key = it.tile(x) * kBN + lane * unit;
        return a.c.bt && seen_at(key, unit) ? a.c.bt[(size_t)pc.at.b * a.c.per + block_of(a.c, key)] : 0;
      };
      // the plane of a tile's keys (-1: not read), and the block scales
      auto plane_of = [&](int x, int page, float& ks, float& vs) {
        ks = vs = 1.f;
        if (x >= pc.t1 || !mine) return -1;
        const int key = it.tile(x) * kBN + lane * unit;
        if (!seen_at(key, unit)) return -1;
        int plane = pc.at.b * a.c.Hkv + pc.at.h;
        size_t si = (size_t)plane * a.c.per + (E4 ? block_of(a.c, key) : 0);
        if (a.c.bt) {
          if (page < 0 || page >= a.c.num_pages) {
            atomicOr(err, TB_DEVERR_BAD_PAGE);
            return a.c.num_pages * a.c.Hkv;     // outside the pool: the copies read zeros
          }
          plane = page * a.c.Hkv + pc.at.h;
          si = plane;
        }
        if constexpr (E4) {
          ks = a.c.ks[si];
          vs = a.c.vs[si];
        }
        return plane;
      };
      int page2 = page_ahead(pc.t0), plane1;
      float ks1, vs1;
      plane1 = plane_of(pc.t0, page2, ks1, vs1);
      page2 = page_ahead(pc.t0 + 1);
      for (int x = pc.t0; ok && x < pc.t1; ++x, ++nt) {
        const int st = nt & 1;
        const uint32_t ph = (nt >> 1) & 1;
        const int key = it.tile(x) * kBN + lane * unit;
        const int plane = plane1;
        const float ks = ks1, vs = vs1;
        plane1 = plane_of(x + 1, page2, ks1, vs1);
        page2 = page_ahead(x + 2);
        const bool want = plane >= 0;
        const int y = a.c.bt ? in_block(a.c, key) : key;
        // Boxes of `box` keys: lane i issues the box that its keys begin (E4: its
        // run of 16; a box is issued if any of its runs is wanted, from the page of
        // that run - all runs of a box lie in one page)
        auto lead_of = [&](int box, int& z) {
          const int per = E4 ? box / 16 : 1;
          const uint32_t any = __ballot_sync(0xffffffffu, want);
          const uint32_t runs = per >= 32 ? any : (any >> lane) & ((1u << per) - 1u);
          const int src = runs ? lane + __ffs(runs) - 1 : lane;
          z = __shfl_sync(0xffffffffu, plane, src & 31);
          return mine && lane % per == 0 && runs != 0;
        };
        int zk, zv = 0;
        const bool go_k = lead_of(m.box, zk);
        const bool go_v = E4 ? lead_of(m.vbox, zv) : go_k;
        const uint32_t loads = __ballot_sync(0xffffffffu, go_k), vloads = __ballot_sync(0xffffffffu, go_v);
        if constexpr (E4) {
          const int sl = nt % kScTiles;
          if (mine) reinterpret_cast<float2*>(sc)[sl * 8 + lane] = make_float2(ks, scale_exp(vs));
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[sl]);
        }
        if (!wait_warp(&k_empty[st], ph ^ 1u, abort_flag, err)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&k_full[st], (uint32_t)__popc(loads) * m.box * DH * (E4 ? 1 : 2));
        __syncwarp();
        if (go_k) {
          uint8_t* dst = smem + C::OFF_K + st * C::K_BYTES;
          if constexpr (E4) {
            tma_load_3d(&tmK, dst + lane * 16 * DH, &k_full[st], 0, y, zk);
          } else {
#pragma unroll
            for (int blk = 0; blk < C::NB; ++blk)
              tma_load_3d(&tmK, dst + blk * kBN * 128 + lane * unit * 128, &k_full[st], blk * 64, y, zk);
          }
        }
        ++nk;
        if constexpr (!E4) {
          if (!wait_warp(&v_empty[st], ph ^ 1u, abort_flag, err)) {
            ok = false;
            break;
          }
          // a border tile goes by way of the warp that zeroes its hidden rows
          const int k0 = it.tile(x) * kBN;
          const bool border = k0 + kBN > it.end || (k0 < it.hid1 && k0 + kBN > it.hid0);
          uint64_t* bar = border ? &fix_full[st] : &v_full[st];
          n_fix[st] += border;
          fixed = (fixed & ~(1u << st)) | (uint32_t)border << st;
          if (lane == 0) {
            fence_proxy_async();                // rows zeroed in place, before the copy
            mbar_arrive_expect_tx(bar, (uint32_t)__popc(loads) * m.box * DH * 2);
          }
          __syncwarp();
          if (go_k) {
#pragma unroll
            for (int blk = 0; blk < C::NB; ++blk)
              tma_load_3d(&tmV, smem + C::OFF_V + st * C::V_BYTES + blk * kBN * 128 + lane * unit * 128, bar,
                          blk * 64, y, zk);
          }
          ++nv;
        } else {
          for (int ch = 0; ch < kBN / kChunk; ++ch, ++nv) {
            const int rs = nv % kRaw;
            if (!wait_warp(&raw_empty[rs], ((nv / kRaw) & 1) ^ 1u, abort_flag, err)) {
              ok = false;
              break;
            }
            const uint32_t in = (vloads >> (2 * ch)) & 3u;       // runs 2ch, 2ch + 1 lead a box
            if (lane == 0) mbar_arrive_expect_tx(&raw_full[rs], (uint32_t)__popc(in) * m.vbox * DH);
            __syncwarp();
            if (go_v && (lane >> 1) == ch)
              tma_load_3d(&tmV, smem + C::OFF_RAW + rs * C::RAW + (lane & 1) * 16 * DH, &raw_full[rs], 0, y, zv);
            __syncwarp();
          }
        }
      }
      if (!ok) break;
    }
    // an item that begins here and goes on in the next CTA's part, for the merge
    if (lane == 0) {
      MergeRec rec{0, 0, 0, 0, 0};
      if (ok && pc.any && pc.at.start >= x0 && pc.at.start + pc.it.cnt + 1 > x1)
        rec = MergeRec{pc.at.b, pc.at.h, pc.at.p, 1, pc.at.start};
      m.rec[blockIdx.x] = rec;
    }
    // every copy issued must land before the CTA may exit
    __syncwarp();
    if (lane == 0) {
      volatile int no_abort = 0;
      if (nq > 0) mbar_wait(q_full, (nq - 1) & 1, &no_abort, err);
      for (int t = max(0, nk - 2); t < nk; ++t) mbar_wait(&k_full[t & 1], (t >> 1) & 1, &no_abort, err);
      if constexpr (E4) {
        for (int t = max(0, nv - kRaw); t < nv; ++t)
          mbar_wait(&raw_full[t % kRaw], (t / kRaw) & 1, &no_abort, err);
      } else {
        for (int t = max(0, nv - 2); t < nv; ++t) {
          const int st = t & 1;
          if ((fixed >> st) & 1)
            mbar_wait(&fix_full[st], (n_fix[st] - 1) & 1, &no_abort, err);
          else
            mbar_wait(&v_full[st], (t >> 1) & 1, &no_abort, err);
        }
      }
    }
  } else if (warp == 9) {
    // ---------------- MMA issue ----------------
    // by one thread, which shares its SM quarter with two softmax warps: every
    // instruction it spends between a wait and an MMA delays the tile
    if (lane == 0) {
      // the sign of a negative score scale goes into S (bit 13: A is negated)
      const uint32_t id_qk = (E4 ? idesc_e4m3(kBM, kBN) : idesc_bf16(kBM, kBN)) | (m.negate ? 1u << 13 : 0u);
      constexpr uint32_t id_pv = idesc_pv<E4>(kBM, DH);
      const uint32_t sQ = smem_u32(smem) + C::OFF_QT, sK = smem_u32(smem) + C::OFF_K, sV = smem_u32(smem) + C::OFF_V;
      auto kmajor = [](uint32_t addr) { return E4 && DH == 64 ? desc_kmajor_sw64(addr) : desc_kmajor_sw128(addr); };
      const uint64_t dq0 = kmajor(sQ), dq1 = kmajor(sQ + C::Q_BYTES);
      const uint64_t dk0 = kmajor(sK), dk1 = kmajor(sK + C::K_BYTES);
      const uint64_t dv0 = desc_mnmajor_sw128(sV, kBN * 128, 1024);
      const uint64_t dv1 = desc_mnmajor_sw128(sV + C::V_BYTES, kBN * 128, 1024);
      auto issue_s = [&](int g, int t, uint64_t qd) {
        const uint64_t kd = (t & 1) ? dk1 : dk0;
        if constexpr (E4) {
          // both terms of the queries, 32 dims (two 16-byte units) per MMA
#pragma unroll
          for (int i = 0; i < 2 * (DH / 32); ++i) {
            const int term = i / (DH / 32), kk = i % (DH / 32);
            mma_f8_ss(tmem + g * kBN, qd + term * (C::QT_BYTES >> 4) + 2 * kk, kd + 2 * kk, id_qk, i ? 1u : 0u);
          }
        } else {
          mma_tile_ss<DH / 16>(tmem + g * kBN, qd, kd, id_qk);
        }
        mma_commit(&s_full[g]);
      };
      auto issue_pv = [&](int g, int t, bool acc) {
        mma_tile_ts128(tmem + C::TMEM_O + g * DH, tmem + g * kBN, (t & 1) ? dv1 : dv0, id_pv, acc ? 1u : 0u);
        mma_commit(&pv_done[g]);
      };
      int kc = 0, nq = 0, c0 = 0, c1 = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!wait_one(&d_full[k % kDescs], (k / kDescs) & 1, abort_flag, err)) break;
        const PieceDesc pc = descs[k % kDescs];
        mbar_arrive(&d_empty[k % kDescs]);
        if (pc.last) break;
        if (pc.t0 == pc.t1) continue;
        const int nt = pc.t1 - pc.t0;
        const int f0 = pc.first_on(0), l0 = pc.last_on(0), f1 = pc.first_on(1), l1 = pc.last_on(1);
        bool on0 = pc.on(0, pc.t0), on1 = pc.on(1, pc.t0);
        const uint64_t dqs = pc.split ? dq0 : dq1;        // slot 1's queries
        if (!wait_one(E4 ? q_ready : q_full, nq & 1, abort_flag, err) ||
            !wait_one(&k_full[kc & 1], (kc >> 1) & 1, abort_flag, err))
          break;
        ++nq;
        tc_fence_after();
        if (on0) issue_s(0, kc, dq0);
        if (on1) issue_s(1, kc, dqs);
        mma_commit(&k_empty[kc & 1]);
        if (nt == 1) mma_commit(q_empty);
        for (int jj = 0; jj < nt; ++jj) {
          const int t = kc + jj, x = pc.t0 + jj;
          const bool next = jj + 1 < nt, on0n = next && pc.on(0, x + 1), on1n = next && pc.on(1, x + 1);
          if (!wait_one(&v_full[t & 1], (t >> 1) & 1, abort_flag, err)) {
            ok = false;
            break;
          }
          if (on0) {
            if (!wait_one(&p_full[0], c0 & 1, abort_flag, err)) {
              ok = false;
              break;
            }
            ++c0;
            tc_fence_after();
            issue_pv(0, t, x != f0);
            if (x == l0) mma_commit(&o_full[0]);
          }
          if (next) {
            if (!wait_one(&k_full[(t + 1) & 1], ((t + 1) >> 1) & 1, abort_flag, err)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (on0n) issue_s(0, t + 1, dq0);
          }
          if (on1) {
            if (!wait_one(&p_full[1], c1 & 1, abort_flag, err)) {
              ok = false;
              break;
            }
            ++c1;
            tc_fence_after();
            issue_pv(1, t, x != f1);
            if (x == l1) mma_commit(&o_full[1]);
          }
          if (next) {
            if (on1n) issue_s(1, t + 1, dqs);
            mma_commit(&k_empty[(t + 1) & 1]);
            if (jj + 2 == nt) mma_commit(q_empty);
          }
          mma_commit(&v_empty[t & 1]);
          on0 = on0n;
          on1 = on1n;
        }
        kc += nt;
      }
      mma_commit(drain);
      volatile int no_abort = 0;
      mbar_wait(drain, 0, &no_abort, err);
    }
  } else if (warp >= 10) {
    // ---------------- V: codes to fp16, chunk by chunk in turn (E4); else the hidden rows of border tiles ----------------
    if constexpr (E4) {
      const int me = warp - 10;
      int nt = 0;
      bool ok = true;
      PieceDesc* d;
      for (int k = 0; ok && piece(k, d); ++k) {
        const PieceDesc pc = *d;
        done(k);
        for (int x = pc.t0; ok && x < pc.t1; ++x, ++nt) {
          const int st = nt & 1;
          const int tile_key = pc.key(x);
#pragma unroll 1
          for (int ch = me; ch < kBN / kChunk; ch += kConv) {
            const int n = nt * (kBN / kChunk) + ch, rs = n % kRaw;     // running chunk
            if (!wait_warp(&v_empty[st], ((nt >> 1) & 1) ^ 1u, abort_flag, err) ||
                !wait_warp(&raw_full[rs], (n / kRaw) & 1, abort_flag, err)) {
              ok = false;
              break;
            }
            const uint32_t raw = smem_u32(smem) + C::OFF_RAW + rs * C::RAW;
            const uint32_t dst = smem_u32(smem) + C::OFF_V + st * C::V_BYTES;
            const int key0 = tile_key + ch * kChunk;
            const bool border = key0 + kChunk > pc.end || (key0 < pc.hid1 && key0 + kChunk > pc.hid0);
            // 16-byte pieces of 16 codes, PPR per row.  The four lanes of a half
            // quarter-warp take one half of a row, the next four the other half
            // of its neighbour, so that reads and writes spread over the banks.
            constexpr int PPR = DH / 16, RPS = 32 / PPR, STEPS = kChunk / RPS;
            int r0 = lane / PPR, pc0 = lane % PPR;
            if constexpr (PPR == 8) {
              const int r2 = lane >> 3, c = lane & 7;
              r0 = (r2 & ~1) + (c >> 2);
              pc0 = (c & 3) + 4 * ((r2 & 1) ^ (c >> 2));
            }
            constexpr int BATCH = 4;
#pragma unroll 1
            for (int i0 = 0; i0 < STEPS; i0 += BATCH) {
              uint4 w[BATCH];
#pragma unroll
              for (int i = 0; i < BATCH; ++i) w[i] = lds128(raw + ((i0 + i) * RPS + r0) * DH + pc0 * 16);
#pragma unroll
              for (int i = 0; i < BATCH; ++i) {
                const int row = (i0 + i) * RPS + r0;
                if (border) {
                  const int j = key0 + row;
                  if (j >= pc.end || (j >= pc.hid0 && j < pc.hid1)) w[i] = make_uint4(0u, 0u, 0u, 0u);
                }
                uint4 lo, hi;
                codes4(w[i].x, lo.x, lo.y);
                codes4(w[i].y, lo.z, lo.w);
                codes4(w[i].z, hi.x, hi.y);
                codes4(w[i].w, hi.z, hi.w);
                const int r = ch * kChunk + row, c = 2 * pc0;           // 16-byte piece of the fp16 row
                const uint32_t base = dst + (c >> 3) * kBN * 128 + r * 128;
                sts128(base + (((c ^ r) & 7) << 4), lo);
                sts128(base + ((((c + 1) ^ r) & 7) << 4), hi);
              }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&v_full[st]);
              mbar_arrive(&raw_empty[rs]);
            }
          }
        }
      }
    } else {
      int nt = 0, n_fix[2] = {0, 0};
      bool ok = true;
      PieceDesc* d;
      for (int k = 0; ok && piece(k, d); ++k) {
        const PieceDesc pc = *d;
        done(k);
        for (int x = pc.t0; x < pc.t1; ++x, ++nt) {
          const int key = pc.key(x), st = nt & 1;
          if (!pc.border(key)) continue;
          if (!wait_warp(&fix_full[st], n_fix[st] & 1, abort_flag, err)) {
            ok = false;
            break;
          }
          ++n_fix[st];
          const uint32_t vt = smem_u32(smem) + C::OFF_V + st * C::V_BYTES;
          for (int r = lane; r < kBN; r += 32) {
            const int j = key + r;
            if (j < pc.end && !(j >= pc.hid0 && j < pc.hid1)) continue;
#pragma unroll
            for (int i = 0; i < C::NB * 8; ++i)
              sts128(vt + (i >> 3) * kBN * 128 + r * 128 + (i & 7) * 16, make_uint4(0u, 0u, 0u, 0u));
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_full[st]);
        }
      }
    }
  } else {
    // ---------------- softmax: one query row per thread ----------------
    const int g = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t s_col = lane_base + g * kBN, o_col = lane_base + C::TMEM_O + g * DH;
    // (16-bit caches leave room for the whole wait in line, and a call costs registers)
    auto soft_wait = [](uint64_t* bar, uint32_t parity, volatile int* abort, int* e) {
      return E4 ? wait_warp(bar, parity, abort, e) : mbar_wait_warp(bar, parity, abort, e);
    };
    int c = 0, nt = 0, nq = 0, no = 0, nj = 0;  // this slot's tiles; key tiles, pieces with keys, outputs, joins
    bool ok = true;
    PieceDesc* d;
    for (int pk = 0; ok && piece(pk, d); ++pk) {
      const SlotRange& s_r = d->s[g];
      const int t0 = d->t0, t1 = d->t1;
      const int qp = r < s_r.rows ? s_r.p0 + r / G : -1;
      const int f_on = d->first_on(g), l_on = d->last_on(g);
      const bool split = d->split;
      float zs = fabsf(a.scale_log2);
      if constexpr (E4) {
        // this row of Q as two e4m3 terms, its largest element in [128, 256)
        if (t0 < t1) {
          if (!soft_wait(q_full, nq & 1, abort_flag, err)) {
            ok = false;
            break;
          }
          if (s_r.rows && !(split && g)) {
            const uint32_t qrow = smem_u32(smem) + g * C::Q_BYTES + r * 128;
            uint4 w[C::NB * 8];
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < C::NB * 8; ++i) {
              w[i] = lds128(qrow + (i >> 3) * kBM * 128 + (((i ^ r) & 7) << 4));
              const uint32_t* u = &w[i].x;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xffff0000u))));
            }
            const float fr = split_frame(amax);
            // Exact, but where the elements of a row, or the scale, are below 2^-90: held to 2^-102, so that the product
            // with a K scale (2^-24 at least) is a normal number.  With 0 the -inf of hidden
            // scores became NaN, and rows of zeros over blocks of zeros (a padded prompt's) were
            // all computed again key by key: 1024 of 8192 tokens 161 ms, now 0.14.  What is held
            // up are scores below 2^24 2^-102 2^60 = 2^-18.
            zs = fmaxf(zs / fr, 0x1p-102f);
            const uint32_t t1 = smem_u32(smem) + C::OFF_QT + g * C::Q_BYTES, t2 = t1 + C::QT_BYTES;
#pragma unroll
            for (int i = 0; i < DH / 16; ++i) { // 16 elements: one 16-byte piece of each term
              uint4 a1, a2;
              uint32_t *u1 = &a1.x, *u2 = &a2.x;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t* u = &w[2 * i + (j >> 1)].x + 2 * (j & 1);
                split4(u[0], u[1], fr, u1[j], u2[j]);
              }
              const uint32_t at = DH == 128 ? r * 128 + (((i ^ r) & 7) << 4) : r * 64 + (((i ^ (r >> 1)) & 3) << 4);
              sts128(t1 + at, a1);
              sts128(t2 + at, a2);
            }
            if (split) zs_s[r] = zs;            // slot 1 works on the same rows
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_ready);
        }
      }
      if (t0 < t1) ++nq;
      float m_used = -INFINITY, l = 0.f;
      const int wlo = win_lo(qp, a.window), p0m = s_r.p0 - (kBN - 1), w1 = win_lo(s_r.p1, a.window);
      const int ns = d->ns, shift = d->wl - ns, ia = s_r.ia, ib = s_r.ib, tn0 = nt - t0;
      // the slot's tiles: every list position but those in [ia, ib), or every second
      for (int x = f_on; x >= 0 && x <= l_on; x = split ? x + 2 : x + 1 >= ia && x + 1 < ib ? ib : x + 1) {
        const int tn = tn0 + x;                 // the CTA's running key tile
        if constexpr (E4) {
          if (!soft_wait(&sc_full[tn % kScTiles], (tn / kScTiles) & 1, abort_flag, err)) {
            ok = false;
            break;
          }
        }
        if (!soft_wait(&s_full[g], c & 1, abort_flag, err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if constexpr (E4) {
          if (split && g && x == f_on) zs = zs_s[r];
        }
        const int key = (x < ns ? x : x + shift) * kBN;
        const bool ahead = key > p0m, behind = key < w1 && key + kBN > a.sinks;
        // m_used (and with it l and O) follows the row's new maximum when that grew
        // by more than 2^kRescale; false when a wait ran out
        auto follow = [&](float mx) -> bool {
          const float m_new = fmaxf(m_used, mx);
          bool need = false;
          if (x == f_on)
            m_used = m_new;
          else
            need = m_new > m_used + kRescale;
          if (__any_sync(0xffffffffu, need)) {
            if (!soft_wait(&pv_done[g], (c - 1) & 1, abort_flag, err)) return false;
            tc_fence_after();
            const float factor = need ? ex2_approx(m_used - m_new) : 1.f;
#pragma unroll 1
            for (int cc = 0; cc < DH; cc += 8) {
              uint32_t u[8];
              tmem_ld8(o_col + cc, u);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * factor);
              tmem_st8(o_col + cc, u);
            }
            tmem_wait_st();
            if (need) {
              l *= factor;
              m_used = m_new;
            }
          }
          return true;
        };
        if (ahead || behind) {
          // A border tile: its hidden scores become -inf in tensor memory first, in a
          // short loop, so that the common path stays small (the instruction cache
          // holds the loops of all roles only just: with masks in line, or a second
          // copy for border tiles, all tiles ran 15 to 20% slower).
          const int lim = qp - key, wl = wlo - key, sl = a.sinks - key;
#pragma unroll 1
          for (int c0 = 0; c0 < kBN; c0 += 16) {
            uint32_t u[16];
            tmem_ld16(s_col + c0, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              asm volatile("" : "+r"(u[i]));
              const int cc = c0 + i;
              if (cc > lim || (cc < wl && cc >= sl)) u[i] = 0xff800000u;
            }
            tmem_st16(s_col + c0, u);
          }
          tmem_wait_st();
        }
        if constexpr (!E4) {
          float s[kBN];
#pragma unroll
          for (int cc = 0; cc < kBN; cc += 16) {
            uint32_t u[16];
            tmem_ld16(s_col + cc, u);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[cc + i] = __uint_as_float(u[i]);
          }
          tmem_wait_ld();
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = fmaxf(s[2 * i], s[2 * i + 1]);
#pragma unroll
            for (int cc = 8 + 2 * i; cc < kBN; cc += 8) v = fmax3(v, s[cc], s[cc + 1]);
            m4[i] = v;
          }
          if (!follow(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * zs)) {
            ok = false;
            break;
          }
          const float msub = m_used == -INFINITY ? 0.f : m_used;
          const float2 f2 = make_float2(zs, zs), n2 = make_float2(-msub, -msub);
          float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int cc = 0; cc < kBN; cc += 16) {
            uint32_t u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 arg = __ffma2_rn(make_float2(s[cc + 2 * i], s[cc + 2 * i + 1]), f2, n2);
              const float2 p = make_float2(ex2_approx(arg.x), ex2_approx(arg.y));
              sum2[i & 1] = __fadd2_rn(sum2[i & 1], p);
              u[i] = pack16<E4>(p.x, p.y);
            }
            tmem_st8(s_col + cc / 2, u);
          }
          const float2 s01 = __fadd2_rn(sum2[0], sum2[1]);
          l += s01.x + s01.y;
        } else {
          // 32 columns at a time, read twice (for the maximum, for the weights):
          // with the scales a whole row does not fit in registers
          const uint32_t scp = smem_u32(sc) + (tn % kScTiles) * 64;
          auto load = [&](uint32_t (&v)[32], int c0) {
            tmem_ld16(s_col + c0, *reinterpret_cast<uint32_t(*)[16]>(v));
            tmem_ld16(s_col + c0 + 16, *reinterpret_cast<uint32_t(*)[16]>(v + 16));
          };
          auto arrived = [](uint32_t (&v)[32]) {  // no use of v moves ahead of the wait
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));
          };
          float mx = -INFINITY;
          // (kv: score factor and exponent of V of the two runs)
          auto top = [&](uint32_t (&v)[32], const float4& kv) {
#pragma unroll
            for (int q = 0; q < 32; q += 16) {
              float v0 = fmaxf(__uint_as_float(v[q]), __uint_as_float(v[q + 1]));
              float v1 = fmaxf(__uint_as_float(v[q + 2]), __uint_as_float(v[q + 3]));
#pragma unroll
              for (int i = 4; i < 16; i += 4) {
                v0 = fmax3(v0, __uint_as_float(v[q + i]), __uint_as_float(v[q + i + 1]));
                v1 = fmax3(v1, __uint_as_float(v[q + i + 2]), __uint_as_float(v[q + i + 3]));
              }
              mx = fmaxf(mx, fmaf(fmaxf(v0, v1), zs * (q ? kv.z : kv.x), q ? kv.w : kv.y));
            }
          };
          uint32_t va[32], vb[32];
          load(va, 0);
          arrived(va);
#pragma unroll 1
          for (int c0 = 0; c0 < kBN; c0 += 64) {
            load(vb, c0 + 32);
            const float4 ka = lds_f4(scp + c0 / 2), kb = lds_f4(scp + c0 / 2 + 16);
            top(va, ka);
            arrived(vb);
            load(va, (c0 + 64) & (kBN - 1));    // the last time: the first columns again
            top(vb, kb);
            arrived(va);
          }
          if (!follow(mx)) {
            ok = false;
            break;
          }
          const float msub = m_used == -INFINITY ? 0.f : m_used;
          auto weights = [&](uint32_t (&v)[32], int c0, const float4& kv) {
#pragma unroll
            for (int q = 0; q < 32; q += 16) {
              const float f = zs * (q ? kv.z : kv.x), e = q ? kv.w : kv.y, nn = e - msub;
              const float2 f2 = make_float2(f, f), n2 = make_float2(nn, nn);
              float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
              uint32_t u[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 arg = __ffma2_rn(
                    make_float2(__uint_as_float(v[q + 2 * i]), __uint_as_float(v[q + 2 * i + 1])), f2, n2);
                const float2 p = make_float2(ex2_approx(arg.x), ex2_approx(arg.y));
                sum2[i & 1] = __fadd2_rn(sum2[i & 1], p);
                u[i] = pack16<E4>(p.x, p.y);
              }
              const float2 s01 = __fadd2_rn(sum2[0], sum2[1]);
              l = fmaf(s01.x + s01.y, __uint_as_float((uint32_t)(127 - (int)e) << 23), l);
              tmem_st8(s_col + (c0 + q) / 2, u);          // over columns read for the last time
            }
          };
#pragma unroll 1
          for (int c0 = 0; c0 < kBN; c0 += 64) {
            load(vb, c0 + 32);
            const float4 ka = lds_f4(scp + c0 / 2), kb = lds_f4(scp + c0 / 2 + 16);
            weights(va, c0, ka);
            arrived(vb);
            load(va, 64);                       // (the second time of no use)
            weights(vb, c0 + 32, kb);
            arrived(va);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[g]);
        ++c;
      }
      if (!ok) break;
      nt += t1 - t0;
      const int where = d->where, rows = s_r.rows;
      const size_t orow = ((size_t)d->b * a.n + s_r.tok0 + r / G) * a.H + d->h * G + r % G;
      const size_t flag = ((size_t)d->b * a.c.Hkv + d->h) * 2 * m.pairs + 2 * d->p + g;
      done(pk);
      if (rows == 0) continue;
      const bool valid = r < rows;
      if (f_on < 0 && !(split && t0 < t1)) {    // no tile of this piece
        if (split && g) continue;               // (slot 0 writes the zeros)
        if (where >= 0) {
          // (a sum below zero: no output follows)
          m.part[((size_t)(where * 2 + g) * (DH / 4 + 1)) * kBM + r] = make_float4(-INFINITY, -1.f, 0.f, 0.f);
        } else if (valid) {
          uint4* dst = reinterpret_cast<uint4*>((bf16*)a.o + orow * DH);
#pragma unroll
          for (int i = 0; i < DH / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      if (f_on >= 0) {
        if (!soft_wait(&o_full[g], no & 1, abort_flag, err)) {
          ok = false;
          break;
        }
        ++no;
        tc_fence_after();
      }
      float a0 = 1.f, a1 = 0.f;                 // factors of the slots' outputs
      const bool both = t0 + 1 < t1;            // split: slot 1 had a tile, its output is set
      if (split) {
        if (g) {
          // hand (max, sum) over, and keep the output until it has been read
          ml_s[r] = make_float2(m_used, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(join_full);
          if (!soft_wait(join_done, nj & 1, abort_flag, err)) {
            ok = false;
            break;
          }
          ++nj;
          continue;
        }
        if (!soft_wait(join_full, nj & 1, abort_flag, err)) {
          ok = false;
          break;
        }
        ++nj;
        tc_fence_after();
        const float2 ml = ml_s[r];
        const float mj = fmaxf(m_used, ml.x), base = mj == -INFINITY ? 0.f : mj;
        a0 = ex2_approx(m_used - base);
        a1 = ex2_approx(ml.x - base);
        l = l * a0 + ml.y * a1;
        m_used = mj;
      }
      // (a negative position sees no key; a sum of 0 elsewhere is that of scores of -inf, and no answer)
      const float inv = where >= 0 ? 1.f : qp < 0 ? 0.f : 1.0f / l;
      float4* piece_out = m.part + ((size_t)(max(where, 0) * 2 + g) * (DH / 4 + 1)) * kBM + r;
      bf16* dst = (bf16*)a.o + orow * DH;
      float probe = 0.f;                        // stays 0 while every output is finite
      if (where >= 0) piece_out[0] = make_float4(m_used, l, 0.f, 0.f);
#pragma unroll 1
      for (int cc = 0; cc < DH; cc += 16) {
        uint32_t u[16];
        tmem_ld16(o_col + cc, u);
        if (split) {
          uint32_t u1[16];
          tmem_ld16(o_col + DH + cc, u1);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            asm volatile("" : "+r"(u[i]), "+r"(u1[i]));
            const float v = __uint_as_float(u[i]) * a0;
            // (a factor of 0 too: scores of -inf or NaN leave no maximum, but count)
            u[i] = __float_as_uint(both ? fmaf(__uint_as_float(u1[i]), a1, v) : v);
          }
        } else {
          tmem_wait_ld();
        }
        if (where >= 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            piece_out[(size_t)(1 + cc / 4 + i) * kBM] =
                make_float4(__uint_as_float(u[4 * i]), __uint_as_float(u[4 * i + 1]), __uint_as_float(u[4 * i + 2]),
                            __uint_as_float(u[4 * i + 3]));
          continue;
        }
        uint4 wv[2];
        uint32_t* wp = &wv[0].x;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v0 = __uint_as_float(u[2 * i]) * inv, v1 = __uint_as_float(u[2 * i + 1]) * inv;
          probe = fmaf(v0, 0.f, fmaf(v1, 0.f, probe));
          wp[i] = pack16<false>(v0, v1);
        }
        if (valid) {
          *reinterpret_cast<uint4*>(dst + cc) = wv[0];
          *reinterpret_cast<uint4*>(dst + cc + 8) = wv[1];
        }
      }
      if (where < 0 && valid && !(probe == 0.f)) *m.any = m.flags[flag] = 1;
      tc_fence_before();
      if (split) {
        __syncwarp();
        if (lane == 0) mbar_arrive(join_done);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the items that cuts went through: CTA (c, slot, columns) the
// item that begins in part c and goes on, one thread per row; then computes again,
// one warp per row, every row whose result is not finite.
template <int DH>
__global__ void __launch_bounds__(128) k_many_merge(const ManyArgs m) {
  pdl_trigger();
  pdl_wait();
  const AttnArgs& a = m.a;
  const int G = kBM / m.tpt, r = threadIdx.x, lane = r & 31, warp = r >> 5;
  const int g = blockIdx.y, col = blockIdx.z * 32;
  // row `row` of the slot's tile, by this warp; columns [c0, c1) of it are written
  auto again = [&](int b, int h, int row, const SlotRange& s, const SeqRange& sr, int c0, int c1) {
    const int tok = s.tok0 + row / G;
    const size_t at = ((size_t)b * a.n + tok) * a.H + h * G + row % G;
    float out[DH / 32];
    attend_row<DH>(a, b, h, sr.first + tok, (const bf16*)a.q + at * DH, out);
#pragma unroll
    for (int u = 0; u < DH / 32; ++u) {
      const int e = lane * (DH / 32) + u;
      if (e >= c0 && e < c1) ((bf16*)a.o)[at * DH + e] = from_f<bf16>(out[u]);
    }
    __syncwarp();
  };
  __shared__ int list[kBM * 4];                     // workspace slots of the item's pieces, -1: none
  __shared__ int n_list, is_whole;
  const MergeRec rec = m.rec[blockIdx.x];
  if (rec.valid) {
    const long long total = m.pre[(size_t)a.c.B * m.pairs] * a.c.Hkv;
    const SeqRange sr = seq_range(a, rec.b);
    const Item it = make_item(m, sr, rec.p);
    const SlotRange s = g ? it.s1 : it.s0;
    const long long end = rec.start + it.cnt + 1;
    if (r == 0) n_list = is_whole = 0;
    __syncthreads();
    const int parts = parts_of(m, total);
    for (int k = blockIdx.x + r; k < parts; k += kBM) {
      const long long xk = cut(parts, total, k);
      if (xk >= end) break;
      const int2 t = piece_of(rec.start, it.cnt, max(xk, rec.start), cut(parts, total, k + 1));
      list[k - blockIdx.x] = t.x < t.y ? 2 * k + (xk <= rec.start ? 1 : 0) : -1;
      atomicMax(&n_list, k - (int)blockIdx.x + 1);
      if (t.x == 0 && t.y == it.cnt) is_whole = 1;  // one CTA holds all key tiles: written out
    }
    __syncthreads();
    if (s.rows && !is_whole) {
      auto at = [&](int w) { return m.part + ((size_t)(w * 2 + g) * (DH / 4 + 1)) * kBM + r; };
      float M = -INFINITY;
#pragma unroll 4
      for (int i = 0; i < n_list; ++i)
        if (list[i] >= 0) M = fmaxf(M, at(list[i])[0].x);
      const float base = M == -INFINITY ? 0.f : M;
      float l = 0.f;
      float4 acc[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int i = 0; i < n_list; ++i) {
        if (list[i] < 0) continue;
        const float4* p = at(list[i]);
        const float4 ml = p[0];
        if (ml.y < 0.f) continue;                   // no key tile of this slot in this piece: its O is unset
        const float wgt = ex2_approx(ml.x - base);
        l = fmaf(ml.y, wgt, l);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float4 v = p[(size_t)(1 + col / 4 + u) * kBM];
          acc[u].x = fmaf(v.x, wgt, acc[u].x);
          acc[u].y = fmaf(v.y, wgt, acc[u].y);
          acc[u].z = fmaf(v.z, wgt, acc[u].z);
          acc[u].w = fmaf(v.w, wgt, acc[u].w);
        }
      }
      const float inv = s.p0 + r / G < 0 ? 0.f : 1.0f / l;       // (as in the attention kernel)
      const bool valid = r < s.rows;
      bf16* dst = (bf16*)a.o + (((size_t)rec.b * a.n + s.tok0 + r / G) * a.H + rec.h * G + r % G) * DH + col;
      float probe = 0.f;
#pragma unroll
      for (int u = 0; u < 8; u += 2) {
        uint4 wv;
        uint32_t* wp = &wv.x;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float v0 = acc[u + j].x * inv, v1 = acc[u + j].y * inv, v2 = acc[u + j].z * inv, v3 = acc[u + j].w * inv;
          probe = fmaf(v0, 0.f, fmaf(v1, 0.f, fmaf(v2, 0.f, fmaf(v3, 0.f, probe))));
          wp[2 * j] = pack16<false>(v0, v1);
          wp[2 * j + 1] = pack16<false>(v2, v3);
        }
        if (valid) *reinterpret_cast<uint4*>(dst + 4 * u) = wv;
      }
      uint32_t bad = __ballot_sync(0xffffffffu, valid && !(probe == 0.f));
      while (bad) {
        const int who = __ffs(bad) - 1;
        bad &= bad - 1;
        again(rec.b, rec.h, warp * 32 + who, s, sr, col, col + 32);
      }
    }
  }
  // Row tiles that the attention kernel wrote out with a value that is not finite,
  // their rows dealt to all warps of the grid.
  if (!*m.any) return;
  const int tiles = a.c.B * a.c.Hkv * 2 * m.pairs;
  const int warps = (int)(gridDim.x * gridDim.y * gridDim.z) * 4;
  const int me = (int)((blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * 4 + warp;
  for (int i0 = 0; i0 < tiles; i0 += 128) {
    const int i = i0 + lane * 4;          // 4 flags per lane
    const uint32_t fl = i < tiles ? reinterpret_cast<const uint32_t*>(m.flags)[i >> 2] : 0u;
    for (uint32_t todo = __ballot_sync(0xffffffffu, fl != 0u); todo; todo &= todo - 1) {
      const int who = __ffs(todo) - 1;
      const uint32_t fw = __shfl_sync(0xffffffffu, fl, who);
      for (int u = 0; u < 4; ++u) {
        const int t = i0 + who * 4 + u;
        if (!((fw >> (8 * u)) & 255u) || t >= tiles) continue;
        const int rt = t % (2 * m.pairs), hk = t / (2 * m.pairs) % a.c.Hkv, b = t / (2 * m.pairs) / a.c.Hkv;
        const SeqRange sr = seq_range(a, b);
        const SlotRange s = slot_range(m, sr, rt);
        // row r of tile t belongs to warp (128 t + r) mod warps
        for (long long r = (me - (long long)t * kBM % warps + warps) % warps; r < s.rows; r += warps) {
          const int row = (int)r;
          const size_t at = ((size_t)b * a.n + s.tok0 + row / G) * a.H + hk * G + row % G;
          float probe = 0.f;
          for (int e = lane; e < DH; e += 32) probe = fmaf(to_f(((const bf16*)a.o)[at * DH + e]), 0.f, probe);
          if (__any_sync(0xffffffffu, !(probe == 0.f))) again(b, hk, row, s, sr, 0, DH);
        }
      }
    }
  }
}

struct ManyLayout {
  size_t pre, rec, flags, part, total;
  int pairs, flag_words;
};
ManyLayout layout_of(const AttnArgs& a) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  ManyLayout L{};
  const int G = a.H / a.c.Hkv, tpt = kBM / G;
  L.pairs = ((a.n + tpt - 1) / tpt + 1) / 2;
  const size_t flags = (size_t)a.c.B * a.c.Hkv * 2 * L.pairs;
  L.flag_words = (int)((flags + 3) / 4);
  L.pre = 0;
  L.rec = up(((size_t)a.c.B * L.pairs + 1) * 8);
  L.flags = L.rec + up((size_t)sm_count() * sizeof(MergeRec)) + 256;      // `any` in the 256 bytes before them
  L.part = L.flags + up((size_t)L.flag_words * 4);
  L.total = L.part + (size_t)2 * sm_count() * 2 * (a.c.dh / 4 + 1) * kBM * 16;
  return L;
}

cudaError_t tmap_q(CUtensorMap* t, const AttnArgs& a, int G) {
  return make_tmap_heads(t, a.q, a.c.B, a.n, a.H, a.c.dh, G, kBM / G);
}

template <int DH, bool E4>
cudaError_t run(const AttnArgs& a, void* ws, cudaStream_t s) {
  using C = ManyCfg<DH, E4>;
  const int G = a.H / a.c.Hkv;
  const ManyLayout L = layout_of(a);
  ManyArgs m;
  m.a = a;
  m.pairs = L.pairs;
  m.tpt = kBM / G;
  m.n_cta = sm_count();
  m.negate = a.scale_log2 < 0.f;
  m.pre = (long long*)ws;
  m.rec = (MergeRec*)((uint8_t*)ws + L.rec);
  m.flags = (uint8_t*)ws + L.flags;
  m.any = (int*)(m.flags - 256);
  m.part = (float4*)((uint8_t*)ws + L.part);
  m.box = kBN;
  m.vbox = kChunk;
  if (a.c.bt) {                                  // a box lies in one page (page_size is a multiple of 16)
    while (a.c.ps % m.box) m.box /= 2;
    while (a.c.ps % m.vbox) m.vbox /= 2;
  }
  CUtensorMap tq, tk, tv;
  cudaError_t e = tmap_q(&tq, a, G);
  if (e != cudaSuccess) return e;
  const uint64_t planes = a.c.bt ? (uint64_t)a.c.num_pages * a.c.Hkv : (uint64_t)a.c.B * a.c.Hkv;
  const uint64_t rows = a.c.bt ? (uint64_t)a.c.ps : (uint64_t)a.c.T;
  if constexpr (E4) {
    e = make_tmap_rows(&tk, 1, a.c.k, planes, rows, DH, DH, m.box);
    if (e == cudaSuccess) e = make_tmap_rows(&tv, 1, a.c.v, planes, rows, DH, DH, m.vbox, false);
  } else {
    e = make_tmap_rows(&tk, 2, a.c.k, planes, rows, DH, 64, m.box);
    if (e == cudaSuccess) e = make_tmap_rows(&tv, 2, a.c.v, planes, rows, DH, 64, m.box);
  }
  if (e != cudaSuccess) return e;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(k_attn_many<DH, E4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  e = launch_pdl(k_many_plan, dim3(1), dim3(1024), 0, s, m, L.flag_words);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_attn_many<DH, E4>, dim3(m.n_cta), dim3(C::THREADS), C::SMEM, s, tq, tk, tv, m);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_many_merge<DH>, dim3(m.n_cta, 2, DH / 32), dim3(kBM), 0, s, m);
}

}  // namespace

size_t cache_attn_many_workspace(const AttnArgs& a) { return a.c.B && a.n ? layout_of(a).total : 0; }

cudaError_t launch_cache_attn_many(const AttnArgs& a, void* ws, cudaStream_t s) {
  if (a.c.dtype == TB_E4M3) return a.c.dh == 128 ? run<128, true>(a, ws, s) : run<64, true>(a, ws, s);
  return a.c.dh == 128 ? run<128, false>(a, ws, s) : run<64, false>(a, ws, s);
}

}  // namespace tb
