// Attention of few query rows over a bf16 or e4m3 cache: the R = n·H/Hkv rows
// (tokens x query heads) that share a KV head, R up to kFewRows.
//
// Such a call reads every visible K and V row once and does 4·R operations per
// element, far below what the tensor cores could do in that time, so it is
// built to stream: each warp holds a ring of 8 KB stages that TMA fills, and the
// small products run as warp-level MMAs so that the instruction count per key
// stays low.
//
//   Work: the visible keys of a (sequence, KV head) are a list of 16-key runs
//   (sinks, then the window); the stages of all pairs form one line, cut into
//   equal parts, one per warp ("team"), so that ragged lengths cost no balance and
//   no counter or atomic orders anything.  Each part of a pair that a team covers
//   is a piece: its softmax state (max, sum, weighted sum of v) goes to the
//   workspace, and k_few_merge joins a pair's pieces in order.  Walking the
//   line, each new piece enters the next pair, the next team or both, so
//   team + pair numbers it without a table.
//   Lane 0 issues the copies; page ids and block scales are fetched 32 runs at a
//   time by the warp, so no copy waits for a table look-up.
//
//   Products (m16n8k16, fp32 sums): S[16 rows x 16 keys] = Q·Kᵀ, O[16 x dh] +=
//   P·V, P straight from S's accumulators.  Up to eight rows the rows are the
//   narrow side instead, Sᵀ[16 keys x 8] = K·Qᵀ, Oᵀ[dh x 8] += Vᵀ·Pᵀ with Pᵀ's
//   8 x 8 quarters transposed between lanes: half the MMAs and half the registers
//   for O (e4m3, 32 sequences of a 16k cache 96 -> 94 us, one of 64k 35 -> 33).
//   bf16: K by ldmatrix, V by ldmatrix.trans.  e4m3: the codes become fp16 exactly
//   (cvt.f16x2.e4m3x2).  ldmatrix on 16-bit units hands a lane four consecutive
//   dims of a key, which serve as the k pairs (2t, 2t+1) and (2t+8, 2t+9) in both
//   operands - a dot product does not care which; ldmatrix.trans hands it two keys
//   of two dims, which one byte permutation sorts into an even-dim and an odd-dim
//   fragment.
//   Over bf16 the weights are rounded to bf16 for their product with v, their sum is
//   not: the MMA takes one type for both operands, v's range does not fit fp16, and a
//   second product for the rest would double the work on V.  The exponentials are
//   ex2.approx (2^-22), far below either rounding.  Error against 64 bits of one token
//   over 32 sequences: 0.0023 of the output, 0.0017 of it the output's own rounding.
//   Queries enter as fp16 under a power of two per row that brings their
//   largest element into [0.5, 1).  (8-bit warp-level MMAs on the K codes, with the
//   queries split as for the tensor-memory kernel, ran slower: 108 against 100 us
//   for 32 sequences of a 16k cache; they are not native here.)
//   A V block's scale 2^e is never multiplied in: p' = 2^(z + e - m') carries
//   it, O = Σ p'·code, l = Σ p'·2^-e, and the running maximum is that of z + e,
//   so p' stays in fp16 whatever the scales.
//
// Measured (8 KV heads of 128, 4 query heads each, one token): 32 sequences,
// bf16, window 4096: 82.7 us, 0.88 of the copy bandwidth; 32 sequences of up to 16k
// over e4m3 95 us, 0.89; one of 64k over e4m3 30 us, 0.64, of which some 9 us are
// the two launches and their dependent reads (what a call of one short sequence
// takes).  7 tokens of 8 sequences, window 2048, e4m3: 27 us.
#include <math.h>

#include <algorithm>

#include "cache.cuh"
#include "gemm_tc.cuh"
#include "sm100_ptx.cuh"

namespace tb {
namespace {

using namespace ptx;

constexpr int kRun = 16;                      // keys per run: pages hold whole runs
constexpr uint32_t kStage = 8192;             // K then V bytes of one stage
constexpr int kMaxB = 1024;                   // sequences per launch
constexpr float kRescale = 8.f;               // rescale O only when the maximum grows by more than 2^8

// Warps of a CTA and stages per warp, by 16-row tiles MT of a warp (LO: up to
// eight rows).  What costs time beside the reads is the latency of a warp's own
// instructions, so a CTA has as many warps as the registers allow: with LO twelve
// (e4m3, 32 sequences of a 16k cache: 110 us with ten, 101 with eleven, 96 with
// twelve; thirteen would leave 128 registers, and spill: 162).  With two tiles the
// queries lie in shared memory, in the room of the third stage.
template <int MT, bool LO> struct FewShape {
  static constexpr int WARPS = LO ? 12 : 8;
  static constexpr int SLOTS = LO || MT == 2 ? 2 : 3;
};
constexpr int kStages = 24;

template <int DH, bool E4> struct FewCfg {
  static constexpr int ROW = E4 ? DH : 2 * DH;                    // bytes of a row
  static constexpr int RUNS = (int)(kStage / (2 * kRun * ROW));   // runs per stage
  static constexpr int BOXB = ROW < 128 ? ROW : 128;              // bytes of a box row
  static constexpr int NB = ROW / BOXB;                           // boxes per run
  static constexpr uint32_t BOX = kRun * BOXB;
  static constexpr uint32_t RUN = kRun * ROW;                     // bytes of a run (K or V)
  static constexpr uint32_t HALF = kStage / 2;
  static constexpr uint32_t OFF_Q = 16 * kStage;                  // MT = 2: 8 warps x [2][DH/16][32] fragments
  static constexpr uint32_t OFF_BAR = kStages * kStage;
  static constexpr uint32_t OFF_SC = OFF_BAR + kStages * 8;
  static constexpr uint32_t OFF_SEQ = OFF_SC + kStages * RUNS * 8;
  static constexpr size_t smem(int B) { return OFF_SEQ + (size_t)B * 16 + 16 + 1024; }
};

// Address of 16-byte piece `c` (of 16 bytes along the row) of row `r` of a run.
template <int DH, bool E4>
__device__ __forceinline__ uint32_t piece(uint32_t run, int r, int c) {
  using C = FewCfg<DH, E4>;
  if constexpr (C::BOXB == 128)
    return run + (c >> 3) * C::BOX + r * 128 + (((c ^ r) & 7) << 4);
  else
    return run + r * 64 + (((c ^ (r >> 1)) & 3) << 4);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <bool E4>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (E4)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit elements (a lane holds [g][2t, 2t + 1]) transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <bool E4>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t d;
  if constexpr (E4)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
struct FewArgs {
  AttnArgs a;
  int b0;                 // first sequence of this launch (a's tensors start at sequence 0)
  int B;                  // sequences of this launch
  int teams;
  int2* ends;             // [B·P] teams of a pair's first and last stage, for the merge
  float* part;            // [teams + B·P][rows][DH + 4]
  int R;                  // rows of a KV head: n·G
  int rows;               // rows per pair
  int tiles;              // pairs per KV head, 1 or 2, of `rows` rows each
  int P;                  // pairs of a sequence: Hkv·tiles
};

// Stages of a pair of sequence b.
__device__ __forceinline__ int stages_of(const AttnArgs& a, const SeqRange& s, int runs) {
  if (s.nn <= 0) return 0;
  return (key_runs(s.len, s.first, a.window, a.sinks, kRun).count + runs - 1) / runs;
}

// A walk along the line of stages: (sequence, pair, stage).
struct Walk {
  int b, p, st, n_st;
};

// pre[i] = Σ_{j < i} cnt[j] in place over smem ints, i <= n, by the whole CTA
// (pre has n + 1 entries; entry n holds the total).
__device__ __forceinline__ void scan_in_place(int* pre, int n, int* tmp) {
  const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, w = t >> 5;
  const int per = (n + nt - 1) / nt, i0 = min(t * per, n), i1 = min(i0 + per, n);
  int sum = 0;
  for (int i = i0; i < i1; ++i) sum += pre[i];
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) tmp[w] = inc;
  __syncthreads();
  int base = inc - sum;
  for (int i = 0; i < w; ++i) base += tmp[i];
  for (int i = i0; i < i1; ++i) {
    const int v = pre[i];
    pre[i] = base;
    base += v;
  }
  if (i1 == n && i0 < n) pre[n] = base;
  if (n == 0 && t == 0) pre[0] = 0;
  __syncthreads();
}

template <int DH, bool E4, int MT, bool LO>
__global__ void __launch_bounds__((FewShape<MT, LO>::WARPS * 32), 1)
    k_attn_few(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const FewArgs f) {
  pdl_trigger();
  pdl_wait();
  using C = FewCfg<DH, E4>;
  constexpr int kWarps = FewShape<MT, LO>::WARPS;
  constexpr int S = FewShape<MT, LO>::SLOTS;
  constexpr int NQ = LO ? 1 : 2;                // query rows of a lane and tile as operand: g, and g + 8
  constexpr int NR = LO ? 2 : MT * 2;           // rows of a lane as result: 2t and 2t + 1, or g and g + 8 of each tile
  constexpr int NE = LO ? 2 : 4;                // keys of a run in a lane's rows
  static_assert(MT == 1 || !LO, "half a tile stands alone");
  const AttnArgs& a = f.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  int* pre = reinterpret_cast<int*>(smem + C::OFF_SEQ);   // [B + 1] first stage of each sequence
  int* len_s = pre + f.B + 1;
  int* nn_s = len_s + f.B;
  int* st_s = nn_s + f.B;                                 // stages of a pair
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * S;
  float2* sc = reinterpret_cast<float2*>(smem + C::OFF_SC) + warp * S * C::RUNS;
  __shared__ int abort_word, tmp[kWarps];
  const int Hkv = a.c.Hkv, G = 1 << a.g_sh;

  for (int b = threadIdx.x; b < f.B; b += blockDim.x) {
    const SeqRange s = seq_range(a, f.b0 + b);
    len_s[b] = s.len;
    nn_s[b] = s.nn;
    st_s[b] = stages_of(a, s, C::RUNS);
    pre[b] = st_s[b] * f.P;
  }
  if (threadIdx.x == 0) {
    abort_word = 0;
    for (int i = 0; i < kWarps * S; ++i) mbar_init(reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + i, 1);
    fence_barrier_init();
  }
  __syncthreads();
  scan_in_place(pre, f.B, tmp);
  volatile int* abort_flag = &abort_word;
  const int total = pre[f.B];
  // Each team has a stage at least.  With s stages in a pair a call waits for s / t
  // of them and for t pieces in the merge, so teams beyond some multiple of sqrt(s)
  // per pair only cost: one sequence of 64k, one KV head, e4m3 21.8 us without the
  // limit, 16.5 with 16 sqrt(s) as with 12, 18.4 with 9.
  const int teams = min(total, 1 + (int)fminf((float)(f.teams - 1), 16.f * sqrtf((float)total * (float)(f.B * f.P))));
  const int team = warp * gridDim.x + blockIdx.x;
  const bool mine = team < teams;
  // [total·team / teams, total·(team + 1) / teams), in 32 bits (teams < 2^15)
  const unsigned each = mine ? (unsigned)total / (unsigned)teams : 0, rest = mine ? total - each * teams : 0;
  const int x0 = mine ? (int)(each * team + rest * team / teams) : 0;
  const int x1 = mine ? (int)(each * (team + 1) + rest * (team + 1) / teams) : 0;

  auto enter = [&](int x) {                     // the walk's state at stage x < total
    int lo = 0, hi = f.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= x) lo = mid; else hi = mid - 1;
    }
    Walk w;
    w.b = lo;                                   // the last with pre <= x: it has stages
    w.n_st = st_s[lo];
    w.p = (x - pre[lo]) / w.n_st;
    w.st = (x - pre[lo]) % w.n_st;
    return w;
  };
  auto next_pair = [&](Walk& w) {
    w.st = 0;
    if (++w.p < f.P) return;
    w.p = 0;
    do ++w.b; while (w.b < f.B && pre[w.b + 1] == pre[w.b]);
    if (w.b < f.B) w.n_st = st_s[w.b];
  };
  auto runs_of = [&](int b) { return key_runs(len_s[b], len_s[b] - nn_s[b], a.window, a.sinks, kRun); };

  // ---- producer state (all lanes alike) ----
  Walk pw{};
  KeyRuns pr{};
  int issued = x0, pbase = 0, ppage = 0;        // lane i: plane, and scales, of run pbase + i
  float pks = 1.f, pvs = 1.f;
  const uint64_t pol = policy_evict_first();
  if (x0 < x1) {
    pw = enter(x0);
    pr = runs_of(pw.b);
    pbase = -64;
  }
  uint8_t* ring = smem + (size_t)warp * S * kStage;
  auto produce = [&](int consumed) {
    while (issued < x1 && issued < consumed + S) {
      const int k = issued - x0, sl = k % S;
      const int r0 = pw.st * C::RUNS, nr = min(C::RUNS, pr.count - r0);
      if (r0 < pbase || r0 + nr > pbase + 32) {          // the next 32 runs of this pair
        pbase = r0;
        const int r = r0 + lane, h = pw.p >> (f.tiles - 1);
        if (r < pr.count) {
          const int key = run_index(pr, r) * kRun;
          long long si = 0;
          if (a.c.bt) {
            const int page = cache_page(a.c, f.b0 + pw.b, key);
            ppage = page < 0 ? -1 : page * Hkv + h;
            si = ppage;
          } else {
            ppage = (f.b0 + pw.b) * Hkv + h;
            si = (long long)ppage * a.c.per + block_of(a.c, key);
          }
          if constexpr (E4) {
            pks = ppage < 0 ? 1.f : a.c.ks[si];
            pvs = ppage < 0 ? 1.f : a.c.vs[si];
          }
        }
      }
      if constexpr (E4) {
        const int src = r0 - pbase + (lane < nr ? lane : 0);
        const float ks = __shfl_sync(0xffffffffu, pks, src), vs = __shfl_sync(0xffffffffu, pvs, src);
        if (lane < nr) sc[sl * C::RUNS + lane] = make_float2(ks, vs);
        __syncwarp();
      }
      if (lane == 0) {
        fence_proxy_async();                             // generic writes to the slot, before the copy
        mbar_arrive_expect_tx(&full[sl], (uint32_t)nr * 2 * C::RUN);
      }
      __syncwarp();
      for (int r = 0; r < nr; ++r) {
        const int key = run_index(pr, r0 + r) * kRun;
        const int plane = __shfl_sync(0xffffffffu, ppage, r0 + r - pbase);
        const int y = a.c.bt ? in_block(a.c, key) : key;
        const int z = plane < 0 ? a.c.num_pages * Hkv : plane;   // outside the pool: the copy reads zeros
        if (lane == 0) {
          uint8_t* dst = ring + sl * kStage + r * C::RUN;
#pragma unroll
          for (int nb = 0; nb < C::NB; ++nb) {
            constexpr int step = E4 ? C::BOXB : C::BOXB / 2;
            tma_load_3d_hint(&tmK, dst + nb * C::BOX, &full[sl], nb * step, y, z, pol);
            tma_load_3d_hint(&tmV, dst + C::HALF + nb * C::BOX, &full[sl], nb * step, y, z, pol);
          }
        }
      }
      ++issued;
      if (++pw.st == pw.n_st) {
        next_pair(pw);
        if (issued < x1) pr = runs_of(pw.b);
        pbase = -64;
      }
    }
  };

  // ---- consumer ----
  const int mi = lane >> 3;
  // Fragments of the queries: registers, or with two tiles shared memory
  uint32_t qa[MT == 1 ? DH / 16 : 1][2 * NQ];
  const uint32_t q_s = smem_u32(smem + C::OFF_Q) + (uint32_t)(warp * (2 * DH / 16) * 32 + lane) * 16;
  constexpr int NO = LO ? DH / 16 : DH / 8;
  float o[MT][NO][4];
  float m[NR], l[NR], zscale[NR];
  int qpos[NR];                                // position of the lane's rows; -1: none
  auto row_of = [&](int ri) { return LO ? 2 * t + ri : ri / 2 * 16 + g + 8 * (ri % 2); };
  Walk w{};
  KeyRuns kr{};
  int len = 0, first = 0, last = 0;
  bool ok = true;
  w = pw;
  bool fresh = true;
  for (int x = x0; x < x1; ++x) {
    produce(x);
    const int k = x - x0, sl = k % S;
    if (fresh) {                               // a new pair: its queries
      fresh = false;
      kr = runs_of(w.b);
      len = len_s[w.b];
      const int nn = nn_s[w.b];
      first = len - nn;
      last = len - 1;
      const int h = w.p >> (f.tiles - 1), row0 = (w.p & (f.tiles - 1)) * f.rows;
#pragma unroll
      for (int ri = 0; ri < NR; ++ri) {
        const int tok = (row0 + row_of(ri)) >> a.g_sh;
        qpos[ri] = tok < nn ? first + tok : -1;
        m[ri] = -INFINITY;
        l[ri] = 0.f;
        zscale[ri] = a.scale_log2;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t fr_[DH / 16][2 * NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const int row = row0 + mt * 16 + g + 8 * i, tok = row >> a.g_sh;
          const bool in = tok < nn;
          const bf16* q = (const bf16*)a.q +
                          (((size_t)(f.b0 + w.b) * a.n + (in ? tok : 0)) * a.H + h * G + (row & (G - 1))) * DH;
          if constexpr (!E4) {
#pragma unroll
            for (int p = 0; p < DH / 16; ++p) {
              fr_[p][i] = in ? *reinterpret_cast<const uint32_t*>(q + 16 * p + 2 * t) : 0u;
              fr_[p][NQ + i] = in ? *reinterpret_cast<const uint32_t*>(q + 16 * p + 8 + 2 * t) : 0u;
            }
          } else {
            float amax = 0.f;
            uint2 raw[DH / 16];
#pragma unroll
            for (int p = 0; p < DH / 16; ++p) {
              raw[p] = in ? *reinterpret_cast<const uint2*>(q + 16 * p + 4 * t) : make_uint2(0u, 0u);
              amax = fmaxf(fmaxf(amax, fmaxf(fabsf(__uint_as_float(raw[p].x << 16)), fabsf(__uint_as_float(raw[p].x & 0xffff0000u)))),
                           fmaxf(fabsf(__uint_as_float(raw[p].y << 16)), fabsf(__uint_as_float(raw[p].y & 0xffff0000u))));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const float fr = pow2_frame(amax), zs = a.scale_log2 / fr;         // exact
            if constexpr (LO) {                // (this lane's row g, wanted for rows 2t and 2t + 1)
              zscale[0] = __shfl_sync(0xffffffffu, zs, 8 * t);
              zscale[1] = __shfl_sync(0xffffffffu, zs, 8 * t + 4);
            } else {
              zscale[2 * mt + i] = zs;
            }
#pragma unroll
            for (int p = 0; p < DH / 16; ++p) {
              fr_[p][i] = pack<true>(__uint_as_float(raw[p].x << 16) * fr, __uint_as_float(raw[p].x & 0xffff0000u) * fr);
              fr_[p][NQ + i] = pack<true>(__uint_as_float(raw[p].y << 16) * fr, __uint_as_float(raw[p].y & 0xffff0000u) * fr);
            }
          }
        }
        if constexpr (MT == 1) {
#pragma unroll
          for (int p = 0; p < DH / 16; ++p)
#pragma unroll
            for (int j = 0; j < 2 * NQ; ++j) qa[p][j] = fr_[p][j];
        } else {
#pragma unroll
          for (int p = 0; p < DH / 16; ++p)
            sts128(q_s + (mt * (DH / 16) + p) * 512, make_uint4(fr_[p][0], fr_[p][1], fr_[p][NQ], fr_[p][2 * NQ - 1]));
        }
#pragma unroll
        for (int i = 0; i < NO; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[mt][i][j] = 0.f;
      }
    }
    if (!mbar_wait_warp(&full[sl], (k / S) & 1, abort_flag, a.c.err)) {
      ok = false;
      break;
    }
    const uint32_t kb0 = smem_u32(ring + sl * kStage), vb0 = kb0 + C::HALF;
    const int r0 = w.st * C::RUNS, nr = min(C::RUNS, kr.count - r0);
    // Scores of the stage's runs: zat(run, row, e) is key koff(e) of the run
    float z[C::RUNS][LO ? 1 : 2][MT][4];
    auto zat = [&](int r, int ri, int e) -> float& {
      return LO ? z[r][0][0][2 * e + ri] : z[r][LO ? 0 : e >> 1][ri / 2][2 * (ri % 2) + (e & 1)];
    };
    auto koff = [&](int e) { return LO ? 8 * e + g : 8 * (e >> 1) + 2 * t + (e & 1); };
#pragma unroll
    for (int r = 0; r < C::RUNS; ++r)
#pragma unroll
      for (int ri = 0; ri < NR; ++ri)
#pragma unroll
        for (int e = 0; e < NE; ++e) zat(r, ri, e) = 0.f;
    constexpr int PS = E4 ? 2 : 1;             // 16-dim slices per step: an ldmatrix holds that many
    auto step = [&](int r, int p, const uint32_t(&qf)[PS][MT][4]) {
      const uint32_t kb = kb0 + r * C::RUN;
      uint32_t b[4];
      if constexpr (!E4) {
        ldsm4(piece<DH, E4>(kb, 8 * (mi >> 1) + (lane & 7), 2 * p + (mi & 1)), b);
        if constexpr (LO) {
          mma<E4>(z[r][0][0], b[0], b[2], b[1], b[3], qf[0][0][0], qf[0][0][2]);
        } else {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma<E4>(z[r][0][mt], qf[0][mt][0], qf[0][mt][1], qf[0][mt][2], qf[0][mt][3], b[0], b[1]);
            mma<E4>(z[r][1][mt], qf[0][mt][0], qf[0][mt][1], qf[0][mt][2], qf[0][mt][3], b[2], b[3]);
          }
        }
      } else {
        ldsm4(piece<DH, E4>(kb, 8 * (mi & 1) + (lane & 7), p + (mi >> 1)), b);
#pragma unroll
        for (int u = 0; u < PS; ++u) {
          uint32_t lo[2], hi[2];               // keys 0..7, 8..15
          codes4(b[2 * u], lo[0], hi[0]);
          codes4(b[2 * u + 1], lo[1], hi[1]);
          if constexpr (LO) {
            mma<E4>(z[r][0][0], lo[0], lo[1], hi[0], hi[1], qf[u][0][0], qf[u][0][2]);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                mma<E4>(z[r][h][mt], qf[u][mt][0], qf[u][mt][1], qf[u][mt][2], qf[u][mt][3], lo[h], hi[h]);
          }
        }
      }
    };
    if constexpr (MT == 2) {
#pragma unroll
      for (int p = 0; p < DH / 16; p += PS) {  // a slice of the queries is loaded once for all runs
        uint32_t qf[PS][MT][4];
#pragma unroll
        for (int u = 0; u < PS; ++u)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 v = lds128(q_s + (mt * (DH / 16) + p + u) * 512);
            qf[u][mt][0] = v.x, qf[u][mt][1] = v.y, qf[u][mt][2] = v.z, qf[u][mt][3] = v.w;
          }
#pragma unroll
        for (int r = 0; r < C::RUNS; ++r) {
          if (r >= nr) break;
          step(r, p, qf);
        }
      }
    }
    // scaled to base 2, over e4m3 with log2 of the V scale added; hidden ones -inf
    float vsc[C::RUNS];                        // E4: the runs' V scales
#pragma unroll
    for (int r = 0; r < C::RUNS; ++r) {
      if (MT == 1 && r < nr) {
#pragma unroll
        for (int p = 0; p < DH / 16; p += PS) {
          uint32_t qf[PS][MT][4];
#pragma unroll
          for (int u = 0; u < PS; ++u) {
            const int pu = MT == 1 ? p + u : 0;
            qf[u][0][0] = qa[pu][0];
            qf[u][0][1] = qa[pu][NQ - 1];      // (LO: not used, nor [3])
            qf[u][0][2] = qa[pu][NQ];
            qf[u][0][3] = qa[pu][2 * NQ - 1];
          }
          step(r, p, qf);
        }
      }
      float ks = 1.f, ve = 0.f;
      vsc[r] = 1.f;
      if constexpr (E4) {
        if (r < nr) {
          const float2 v = lds_f2(smem_u32(sc + sl * C::RUNS + r));
          ks = v.x;
          ve = scale_exp(v.y);
          vsc[r] = v.y;
        }
      }
      const int key = run_index(kr, r0 + r) * kRun;
      // every row of the call sees the whole run?
      const bool all = r < nr && key + kRun - 1 <= first &&
                       (a.window == 0 || key >= win_lo(last, a.window) || key + kRun <= a.sinks);
#pragma unroll
      for (int ri = 0; ri < NR; ++ri) {
        const float zs = E4 ? zscale[ri] * ks : zscale[ri];
#pragma unroll
        for (int e = 0; e < NE; ++e) zat(r, ri, e) = E4 ? fmaf(zat(r, ri, e), zs, ve) : zat(r, ri, e) * zs;
        if (!all) {
          const int lo = win_lo(qpos[ri], a.window);
#pragma unroll
          for (int e = 0; e < NE; ++e) {
            const int kk = key + koff(e);
            const bool see = r < nr && kk <= qpos[ri] && (kk >= lo || kk < a.sinks);
            if (!see) zat(r, ri, e) = -INFINITY;
          }
        }
      }
      // v rows that no query of the call sees: 0·NaN is NaN inside an MMA
      if (r < nr) {
        const int hid1 = win_lo(first, a.window), hid0 = min(a.sinks, hid1);   // hidden: [hid0, hid1) and [len, ..)
        if (key + kRun > len || (key < hid1 && key + kRun > hid0)) {
          const uint32_t vr = vb0 + r * C::RUN;
          for (int i = lane; i < kRun * C::ROW / 16; i += 32) {
            const int nb = i / (kRun * C::BOXB / 16), row = i / (C::BOXB / 16) % kRun;
            const int kk = key + row;
            if (kk >= len || (kk >= hid0 && kk < hid1))
              sts128(vr + nb * C::BOX + row * C::BOXB + i % (C::BOXB / 16) * 16, make_uint4(0u, 0u, 0u, 0u));
          }
          __syncwarp();
        }
      }
    }
    // online softmax
#pragma unroll
    for (int ri = 0; ri < NR; ++ri) {
      float mx = -INFINITY;
#pragma unroll
      for (int r = 0; r < C::RUNS; ++r)
#pragma unroll
        for (int e = 0; e < NE; ++e) mx = fmaxf(mx, zat(r, ri, e));
#pragma unroll
      for (int d = LO ? 4 : 1; d < (LO ? 32 : 4); d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      if (mx > m[ri] + kRescale || (m[ri] == -INFINITY && mx > -INFINITY)) {
        const float fac = ex2_approx(m[ri] - mx);         // 0 from -inf
        l[ri] *= fac;
#pragma unroll
        for (int d = 0; d < NO; ++d) {
          o[LO ? 0 : ri / 2][d][LO ? ri : 2 * (ri % 2)] *= fac;
          o[LO ? 0 : ri / 2][d][LO ? 2 + ri : 2 * (ri % 2) + 1] *= fac;
        }
        m[ri] = mx;
      }
    }
#pragma unroll
    for (int r = 0; r < C::RUNS; ++r) {
      if (r >= nr) break;
      // P as an operand: rows by keys, or (LO) keys by rows, its 8 x 8 quarters transposed
      uint32_t pa[MT][4];
#pragma unroll
      for (int ri = 0; ri < NR; ++ri) {
        const float base = m[ri] == -INFINITY ? 0.f : m[ri];
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          zat(r, ri, e) = ex2_approx(zat(r, ri, e) - base);
          sum += zat(r, ri, e);
        }
        l[ri] = E4 ? fmaf(sum, scale_inv(vsc[r]), l[ri]) : l[ri] + sum;
      }
      if constexpr (LO) {
        pa[0][0] = transpose8(pack<E4>(zat(r, 0, 0), zat(r, 1, 0)));
        pa[0][1] = transpose8(pack<E4>(zat(r, 0, 1), zat(r, 1, 1)));
      } else {
#pragma unroll
        for (int ri = 0; ri < NR; ++ri) {
          pa[ri / 2][ri % 2] = pack<E4>(zat(r, ri, 0), zat(r, ri, 1));
          pa[ri / 2][2 + ri % 2] = pack<E4>(zat(r, ri, 2), zat(r, ri, 3));
        }
      }
      const uint32_t vb = vb0 + r * C::RUN;
      const int row = 8 * (mi & 1) + (lane & 7);
#pragma unroll
      for (int c = 0; c < (E4 ? DH / 16 : DH / 8); c += 2) {
        uint32_t b[4];
        ldsm4t(piece<DH, E4>(vb, row, c + (mi >> 1)), b);
        if constexpr (!E4) {
          if constexpr (LO) {                  // dims 8c + g, 8c + 8 + g
            mma<E4>(o[0][c / 2], b[0], b[2], b[1], b[3], pa[0][0], pa[0][1]);
          } else {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                mma<E4>(o[mt][LO ? 0 : c + u], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], b[2 * u], b[2 * u + 1]);
          }
        } else {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t e0, o0, e1, o1;           // even and odd dims; keys 0..7, 8..15
            codes4(__byte_perm(b[2 * u], 0, 0x3120), e0, o0);
            codes4(__byte_perm(b[2 * u + 1], 0, 0x3120), e1, o1);
            if constexpr (LO) {                // dims 16(c + u) + 2g, + 2g + 1
              mma<E4>(o[0][c + u], e0, o0, e1, o1, pa[0][0], pa[0][1]);
            } else {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma<E4>(o[mt][2 * (c + u)], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], e0, e1);
                mma<E4>(o[mt][2 * (c + u) + 1], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], o0, o1);
              }
            }
          }
        }
      }
    }
    __syncwarp();                              // the slot may be refilled
    const bool pair_ends = w.st + 1 == w.n_st;
    if (pair_ends || x + 1 == x1) {            // this piece's state
      int* e = reinterpret_cast<int*>(f.ends + w.b * f.P + w.p);
      if (lane == 0 && x - w.st >= x0) e[0] = team;
      if (lane == 0 && pair_ends) e[1] = team;
      const long long pc = (long long)team + (long long)w.b * f.P + w.p;
#pragma unroll
      for (int ri = 0; ri < NR; ++ri) {
        float ls = l[ri];
#pragma unroll
        for (int d = LO ? 4 : 1; d < (LO ? 32 : 4); d <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
        const int row = row_of(ri);
        if (row >= f.rows) continue;
        float* dst = f.part + (pc * f.rows + row) * (DH + 4);
        if constexpr (LO) {
#pragma unroll
          for (int c = 0; c < NO; ++c) {
            if constexpr (E4) {
              *reinterpret_cast<float2*>(dst + 4 + 16 * c + 2 * g) = make_float2(o[0][c][ri], o[0][c][2 + ri]);
            } else {
              dst[4 + 16 * c + g] = o[0][c][ri];
              dst[4 + 16 * c + 8 + g] = o[0][c][2 + ri];
            }
          }
        } else {
          const int mt = ri / 2, i = ri % 2;
          if constexpr (!E4) {
#pragma unroll
            for (int d = 0; d < DH / 8; ++d)
              *reinterpret_cast<float2*>(dst + 4 + 8 * d + 2 * t) =
                  make_float2(o[mt][LO ? 0 : d][2 * i], o[mt][LO ? 0 : d][2 * i + 1]);
          } else {
#pragma unroll
            for (int c = 0; c < DH / 16; ++c) {
              const int d = LO ? 0 : 2 * c;
              *reinterpret_cast<float4*>(dst + 4 + 16 * c + 4 * t) =
                  make_float4(o[mt][d][2 * i], o[mt][d + !LO][2 * i], o[mt][d][2 * i + 1], o[mt][d + !LO][2 * i + 1]);
            }
          }
        }
        if ((LO ? g : t) == 0) *reinterpret_cast<float2*>(dst) = make_float2(m[ri], ls);
      }
    }
    if (pair_ends) {
      next_pair(w);
      fresh = true;
    } else {
      ++w.st;
    }
  }
  // copies issued but not consumed (after a wait that ran out) must land first
  if (!ok && lane == 0) {
    volatile int no_abort = 0;
    for (int x = x0 > issued - S ? x0 : issued - S; x < issued; ++x)
      mbar_wait(&full[(x - x0) % S], ((x - x0) / S) & 1, &no_abort, a.c.err);
  }
}

// Joins the pieces of a row of a pair: o = Σ w_i O_i / Σ w_i l_i,
// w_i = 2^(m_i - M), in the order of the teams.  One warp per row, or with many
// pieces W, each a run of them, whose results are joined the same way (one
// sequence of 64k over e4m3: eight warps 33.1 us, 32 29.8; with one KV head 46.7
// and 21.8).  A lane holds DH/32 consecutive dims.  Latency counts here: eight
// pieces are loaded at a time, under a running maximum (a pass for the maximum
// before it would wait for memory twice).
template <int DH, int W>
__global__ void __launch_bounds__(W == 1 ? 256 : 32 * W) k_few_merge(const FewArgs f) {
  pdl_trigger();
  pdl_wait();
  constexpr int D = DH / 32;
  const AttnArgs& a = f.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = 1 << a.g_sh;
  const int row = W > 1 ? blockIdx.x : blockIdx.x * 8 + warp, h = blockIdx.y, b = blockIdx.z;
  const int tile = row >= f.rows, pair = h * f.tiles + tile;
  if (row >= f.R) return;
  const int2 ends = f.ends[b * f.P + pair];     // (unless the sequence is empty)
  const SeqRange sr = seq_range(a, f.b0 + b);
  const int tok = row >> a.g_sh, head = h * G + (row & (G - 1));
  if (tok >= sr.nn) return;
  const size_t at = (((size_t)(f.b0 + b) * a.n + tok) * a.H + head) * DH;
  float M = -INFINITY, L = 0.f, acc[D];
#pragma unroll
  for (int u = 0; u < D; ++u) acc[u] = 0.f;
  if (sr.len > 0) {
    // (held to the teams: after a wait that ran out they may not have been written)
    const int t0 = min(max(ends.x, 0), f.teams - 1), np = min(max(ends.y, t0), f.teams - 1) + 1 - t0;
    const float* p0 = f.part + ((t0 + (long long)b * f.P + pair) * f.rows + row - tile * f.rows) * (DH + 4);
    const size_t step = (size_t)f.rows * (DH + 4);
    const int i0 = W > 1 ? np * warp / W : 0, i1 = W > 1 ? np * (warp + 1) / W : np;
    constexpr int U = 8;                        // pieces in flight
    for (int i = i0; i < i1; i += U) {
      float2 ml[U];
      float v[U][D];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        ml[j] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int u = 0; u < D; ++u) v[j][u] = 0.f;
        if (i + j < i1) {
          const float* p = p0 + (i + j) * step;
          ml[j] = *reinterpret_cast<const float2*>(p);
          if constexpr (D == 4) {
            const float4 x = *reinterpret_cast<const float4*>(p + 4 + 4 * lane);
            v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(p + 4 + 2 * lane);
            v[j][0] = x.x, v[j][1] = x.y;
          }
        }
      }
      float mx = M;
#pragma unroll
      for (int j = 0; j < U; ++j) mx = fmaxf(mx, ml[j].x);
      const float base = mx == -INFINITY ? 0.f : mx, fac = ex2_approx(M - base);
      L *= fac;
#pragma unroll
      for (int u = 0; u < D; ++u) acc[u] *= fac;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const float w = ex2_approx(ml[j].x - base);
        L = fmaf(ml[j].y, w, L);
#pragma unroll
        for (int u = 0; u < D; ++u) acc[u] = fmaf(v[j][u], w, acc[u]);
      }
      M = mx;
    }
    if constexpr (W > 1) {
      __shared__ float m_s[W], l_s[W];
      __shared__ __align__(16) float acc_s[W][DH];
      if (lane == 0) {
        m_s[warp] = M;
        l_s[warp] = L;
      }
#pragma unroll
      for (int u = 0; u < D; ++u) acc_s[warp][lane * D + u] = acc[u];
      __syncthreads();
      if (warp > 0) return;
      const float m = lane < W ? m_s[lane] : -INFINITY;
      M = m;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float w = ex2_approx(m - (M == -INFINITY ? 0.f : M));
      L = lane < W ? w * l_s[lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
      for (int u = 0; u < D; ++u) acc[u] = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
        for (int u = 0; u < D; ++u) acc[u] = fmaf(acc_s[i][lane * D + u], wi, acc[u]);
      }
    }
  } else if (W > 1 && warp > 0) {
    return;
  }
  // (a negative position sees no key; a sum of 0 elsewhere is that of scores of -inf, and no answer)
  const float inv = sr.first + tok < 0 ? 0.f : 1.0f / L;
  float probe = 0.f;
#pragma unroll
  for (int u = 0; u < D; ++u) {
    acc[u] *= inv;
    probe = fmaf(acc[u], 0.f, probe);
  }
  if (__any_sync(0xffffffffu, !(probe == 0.f))) {        // not finite: see attend_row
    attend_row<DH>(a, f.b0 + b, h, sr.first + tok, (const bf16*)a.q + at, acc);
    __syncwarp();
  }
  bf16* out = (bf16*)a.o + at + lane * D;
  if constexpr (D == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(pack<false>(acc[0], acc[1]), pack<false>(acc[2], acc[3]));
  else
    *reinterpret_cast<uint32_t*>(out) = pack<false>(acc[0], acc[1]);
}

// How the rows of a KV head are dealt: pairs of `rows` rows, warps with `mt`
// tiles of 16.  From 17 rows on a warp holds two tiles, so that a key is read and
// converted once for both: 53 against 62 us over e4m3 (4 sequences of 16k, 32
// rows), 56 against 69 in bf16, 84 against 106 (32 of 4k, e4m3).  With little to
// read the tiles are pairs of their own, as twice the parts shorten the line more
// than the second read from L2 costs: 31 against 38 us (8 sequences, window 2048).
struct Deal {
  int mt, rows, tiles, warps;
};
Deal deal_of(const AttnArgs& a) {
  const int R = a.n * (a.H / a.c.Hkv);
  if (R <= 16) return {1, R, 1, R <= 8 ? FewShape<1, true>::WARPS : FewShape<1, false>::WARPS};
  const long long keys = a.window > 0 ? std::min<long long>(a.c.T, (long long)a.window + a.sinks + a.n) : a.c.T;
  if (keys * a.c.B * a.c.Hkv <= 1 << 18) return {1, 16, 2, FewShape<1, false>::WARPS};
  return {2, R, 1, FewShape<2, false>::WARPS};
}

// Sequences per launch: the line's stage numbers stay below 2^30 (one sequence
// alone does, see cache_attn_few_fits).
int batch_of(const AttnArgs& a, const Deal& d) {
  const long long per = (long long)a.c.Hkv * d.tiles * ((a.c.T + kRun - 1) / kRun + 1);
  return (int)std::min<long long>(std::min(a.c.B, kMaxB), std::max<long long>(1, (1LL << 30) / per));
}

size_t ends_bytes(const AttnArgs& a, const Deal& d) {
  return ((size_t)batch_of(a, d) * a.c.Hkv * d.tiles * 8 + 255) / 256 * 256;
}

template <int DH, bool E4, int MT, bool LO>
cudaError_t run(const AttnArgs& a, const Deal& d, void* ws, cudaStream_t s) {
  using C = FewCfg<DH, E4>;
  CUtensorMap tk, tv;
  const uint64_t planes = a.c.bt ? (uint64_t)a.c.num_pages * a.c.Hkv : (uint64_t)a.c.B * a.c.Hkv;
  const uint64_t rows = a.c.bt ? (uint64_t)a.c.ps : (uint64_t)a.c.T;
  const int es = E4 ? 1 : 2;
  cudaError_t e = make_tmap_rows(&tk, es, a.c.k, planes, rows, DH, C::BOXB / es, kRun);
  if (e != cudaSuccess) return e;
  e = make_tmap_rows(&tv, es, a.c.v, planes, rows, DH, C::BOXB / es, kRun);
  if (e != cudaSuccess) return e;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(k_attn_few<DH, E4, MT, LO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)C::smem(kMaxB));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  FewArgs f;
  f.a = a;
  f.R = a.n * (a.H / a.c.Hkv);
  f.rows = d.rows;
  f.tiles = d.tiles;
  f.P = a.c.Hkv * d.tiles;
  f.teams = sm_count() * d.warps;
  const int Bl = batch_of(a, d);
  f.ends = (int2*)ws;
  f.part = (float*)((uint8_t*)ws + ends_bytes(a, d));
  for (int b0 = 0; b0 < a.c.B; b0 += Bl) {
    f.b0 = b0;
    f.B = std::min(Bl, a.c.B - b0);
    e = launch_pdl(k_attn_few<DH, E4, MT, LO>, dim3(sm_count()), dim3(d.warps * 32), C::smem(f.B), s, tk, tv, f);
    if (e != cudaSuccess) return e;
    // warps per row by the pieces of a pair, at equal lengths
    const long long pairs = (long long)f.B * f.P;
    if (f.teams >= 64 * pairs)
      e = launch_pdl(k_few_merge<DH, 32>, dim3(f.R, a.c.Hkv, f.B), dim3(1024), 0, s, f);
    else if (f.teams >= 16 * pairs)
      e = launch_pdl(k_few_merge<DH, 8>, dim3(f.R, a.c.Hkv, f.B), dim3(256), 0, s, f);
    else
      e = launch_pdl(k_few_merge<DH, 1>, dim3((f.R + 7) / 8, a.c.Hkv, f.B), dim3(256), 0, s, f);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int DH, bool E4>
cudaError_t by_rows(const AttnArgs& a, void* ws, cudaStream_t s) {
  const Deal d = deal_of(a);
  if (d.mt == 2) return run<DH, E4, 2, false>(a, d, ws, s);
  return d.rows <= 8 ? run<DH, E4, 1, true>(a, d, ws, s) : run<DH, E4, 1, false>(a, d, ws, s);
}

}  // namespace

bool cache_attn_few_fits(const AttnArgs& a) {
  long long runs = a.c.T / kRun + 1;
  if (a.window > 0) runs = std::min(runs, ((long long)a.window + a.n) / kRun + a.sinks / kRun + 3);
  return runs * a.c.Hkv * deal_of(a).tiles <= 1LL << 30;
}

size_t cache_attn_few_workspace(const AttnArgs& a) {
  if (a.c.B == 0 || a.n == 0) return 0;
  const Deal d = deal_of(a);
  const long long pieces = (long long)sm_count() * d.warps + (long long)batch_of(a, d) * a.c.Hkv * d.tiles;
  return ends_bytes(a, d) + (size_t)pieces * d.rows * (a.c.dh + 4) * 4;
}

cudaError_t launch_cache_attn_few(const AttnArgs& a, void* ws, cudaStream_t s) {
  if (a.n * (a.H / a.c.Hkv) > kFewRows) return cudaErrorInvalidValue;
  if (a.c.dtype == TB_E4M3) return a.c.dh == 128 ? by_rows<128, true>(a, ws, s) : by_rows<64, true>(a, ws, s);
  return a.c.dh == 128 ? by_rows<128, false>(a, ws, s) : by_rows<64, false>(a, ws, s);
}

}  // namespace tb
