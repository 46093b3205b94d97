// Attention of few query rows over a bf16 or e4m3 cache: the R = n·H/Hkv rows
// (tokens x query heads) that share a KV head, R up to kFewRows.
//
// Such a call reads every visible K and V row once and does 4·R operations per
// element, far below what the tensor cores could do in that time, so it is
// built to stream: teams of warps hold rings of 8 KB stages that TMA fills, and
// the small products run as warp-level MMAs so that the instruction count per
// key stays low.
//
//   Work: the visible keys of a (sequence, KV head) are a list of 16-key runs
//   (sinks, then the window); the stages of all pairs form one line, cut into
//   equal parts, one per team, so that ragged lengths cost no balance and no
//   counter or atomic orders anything.  Each part of a pair that a team covers
//   is a piece: its softmax state (max, sum, weighted sum of v) goes to the
//   workspace, and k_few_merge joins a pair's pieces in order.  Walking the
//   line, each new piece enters the next pair, the next team or both, so
//   team + pair numbers it without a table.
//   A team is one warp for up to 16 rows, two for 32, sixteen rows each over the
//   same stages.  Lane 0 of its first warp issues the
//   copies; page ids and block scales are fetched 32 runs at a time by the
//   warp, so no copy waits for a table look-up.
//
//   Products (m16n8k16, fp32 sums): S[16 x 16 keys] = Q·Kᵀ, O[16 x dh] += P·V,
//   P straight from S's accumulators.  bf16: K by ldmatrix, V by
//   ldmatrix.trans.  e4m3: the codes become fp16 exactly (cvt.f16x2.e4m3x2).
//   ldmatrix on 16-bit units hands a lane four consecutive dims of a key, which
//   serve as the k pairs (2t, 2t+1) and (2t+8, 2t+9) in both operands - a dot
//   product does not care which; ldmatrix.trans hands it two keys of two dims,
//   which one byte permutation sorts into an even-dim and an odd-dim fragment.
//   Queries enter as fp16 under a power of two per row that brings their
//   largest element into [0.5, 1).  (8-bit warp-level MMAs on the K codes, with the
//   queries split as for the tensor-memory kernel, ran slower: 108 against 100 us
//   for 32 sequences of a 16k cache; they are not native here.)
//   A V block's scale 2^e is never multiplied in: p' = 2^(z + e - m') carries
//   it, O = Σ p'·code, l = Σ p'·2^-e, and the running maximum is that of z + e,
//   so p' stays in fp16 whatever the scales.
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

// Warps of a CTA and stages per warp, 24 stages in all.  The e4m3 form of up to
// eight rows spends more instructions per byte and fewer registers: twelve warps
// hide its latencies better than eight (PLACEHOLDER).
template <bool E4, bool LO> struct FewShape {
  static constexpr int WARPS = E4 && LO ? 12 : 8;
  static constexpr int SLOTS = E4 && LO ? 2 : 3;
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
  static constexpr uint32_t OFF_BAR = kStages * kStage;
  static constexpr uint32_t OFF_SC = OFF_BAR + 2 * kStages * 8;
  static constexpr uint32_t OFF_SEQ = OFF_SC + kStages * RUNS * 8;
  static constexpr size_t smem(int B) { return OFF_SEQ + (size_t)B * 12 + 16 + 1024; }
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
  int* pre;               // [B + 1] first stage of each sequence, left for the merge
  float* part;            // [teams + B·Hkv][R][DH + 4]
  int R;                  // rows per piece: n·G
};

// Stages of sequence b (per KV head).
__device__ __forceinline__ int stages_of(const AttnArgs& a, const SeqRange& s, int runs) {
  if (s.nn <= 0) return 0;
  return (key_runs(s.len, s.first, a.window, a.sinks, kRun).count + runs - 1) / runs;
}

// A walk along the line of stages: (sequence, KV head, stage).
struct Walk {
  int b, h, st, n_st;
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

template <int DH, bool E4, int TW, bool LO>
__global__ void __launch_bounds__((FewShape<E4, LO>::WARPS * 32), 1)
    k_attn_few(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const FewArgs f) {
  pdl_trigger();
  pdl_wait();
  using C = FewCfg<DH, E4>;
  constexpr int kWarps = FewShape<E4, LO>::WARPS;
  constexpr int S = FewShape<E4, LO>::SLOTS * TW;        // slots of a team
  constexpr int NR = LO ? 1 : 2;                // rows of a lane: g, and g + 8
  const AttnArgs& a = f.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int team_in = warp / TW, tw = warp % TW;
  int* pre = reinterpret_cast<int*>(smem + C::OFF_SEQ);   // [B + 1] first stage of each sequence
  int* len_s = pre + f.B + 1;
  int* nn_s = len_s + f.B;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + team_in * S;
  uint64_t* empty = full + kStages;
  float2* sc = reinterpret_cast<float2*>(smem + C::OFF_SC) + team_in * S * C::RUNS;
  __shared__ int abort_word, tmp[kWarps];
  const int Hkv = a.c.Hkv, G = a.H / Hkv;

  for (int b = threadIdx.x; b < f.B; b += blockDim.x) {
    const SeqRange s = seq_range(a, f.b0 + b);
    len_s[b] = s.len;
    nn_s[b] = s.nn;
    pre[b] = stages_of(a, s, C::RUNS) * Hkv;
  }
  if (threadIdx.x == 0) {
    abort_word = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + i, 1);
      mbar_init(reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + kStages + i, TW);
    }
    fence_barrier_init();
  }
  __syncthreads();
  scan_in_place(pre, f.B, tmp);
  volatile int* abort_flag = &abort_word;
  const int total = pre[f.B];
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= f.B; b += blockDim.x) f.pre[b] = pre[b];
  const int teams = min(f.teams, total);        // each of them has a stage at least
  const int team = team_in * gridDim.x + blockIdx.x;
  const bool mine = team < teams;
  const int x0 = mine ? (int)((long long)total * team / teams) : 0;
  const int x1 = mine ? (int)((long long)total * (team + 1) / teams) : 0;

  auto enter = [&](int x) {                     // the walk's state at stage x < total
    int lo = 0, hi = f.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= x) lo = mid; else hi = mid - 1;
    }
    Walk w;
    w.b = lo;                                   // the last with pre <= x: it has stages
    w.n_st = (pre[lo + 1] - pre[lo]) / Hkv;
    w.h = (x - pre[lo]) / w.n_st;
    w.st = (x - pre[lo]) % w.n_st;
    return w;
  };
  auto next_pair = [&](Walk& w) {
    w.st = 0;
    if (++w.h < Hkv) return;
    w.h = 0;
    do ++w.b; while (w.b < f.B && pre[w.b + 1] == pre[w.b]);
    if (w.b < f.B) w.n_st = (pre[w.b + 1] - pre[w.b]) / Hkv;
  };
  auto runs_of = [&](int b) { return key_runs(len_s[b], len_s[b] - nn_s[b], a.window, a.sinks, kRun); };

  // ---- producer state (the team's first warp, all lanes alike) ----
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
  uint8_t* ring = smem + (size_t)team_in * S * kStage;
  auto produce = [&](int consumed) -> bool {
    // (one slot of slack for the other warps of a team)
    while (issued < x1 && issued < consumed + S - (TW > 1 ? 1 : 0)) {
      const int k = issued - x0, sl = k % S;
      if constexpr (TW > 1) {
        if (k >= S && !mbar_wait_warp(&empty[sl], ((k / S) - 1) & 1, abort_flag, f.a.c.err)) return false;
      }
      const int r0 = pw.st * C::RUNS, nr = min(C::RUNS, pr.count - r0);
      if (r0 < pbase || r0 + nr > pbase + 32) {          // the next 32 runs of this pair
        pbase = r0;
        const int r = r0 + lane;
        if (r < pr.count) {
          const int key = run_index(pr, r) * kRun;
          long long si = 0;
          if (a.c.bt) {
            const int page = cache_page(a.c, f.b0 + pw.b, key);
            ppage = page < 0 ? -1 : page * Hkv + pw.h;
            si = ppage;
          } else {
            ppage = (f.b0 + pw.b) * Hkv + pw.h;
            si = (long long)ppage * a.c.per + key / a.c.ps;
          }
          if constexpr (E4) {
            pks = ppage < 0 ? 1.f : __ldg(a.c.ks + si);
            pvs = ppage < 0 ? 1.f : __ldg(a.c.vs + si);
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
        const int y = a.c.bt ? key % a.c.ps : key;
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
    return true;
  };

  // ---- consumer ----
  const int mi = lane >> 3;
  uint32_t qa[DH / 16][2 * NR];
  float o[DH / 8][4];                          // (with eight rows the upper half stays 0)
  float m[NR], l[NR], zscale[NR];
  int qpos[NR];                                // position of the lane's rows; -1: none
  Walk w{};
  KeyRuns kr{};
  int len = 0, first = 0, last = 0;
  bool ok = true;
  if (x0 < x1) w = enter(x0);
  bool fresh = true;
  for (int x = x0; x < x1; ++x) {
    if (tw == 0 && !produce(x)) {
      ok = false;
      break;
    }
    const int k = x - x0, sl = k % S;
    if (fresh) {                               // a new pair: its queries
      fresh = false;
      kr = runs_of(w.b);
      len = len_s[w.b];
      const int nn = nn_s[w.b];
      first = len - nn;
      last = len - 1;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int row = tw * 16 + g + 8 * i;
        const int tok = row / G;
        const bool in = tok < nn;
        qpos[i] = in ? first + tok : -1;
        const bf16* q = (const bf16*)a.q +
                        (((size_t)(f.b0 + w.b) * a.n + (in ? tok : 0)) * a.H + w.h * G + row % G) * DH;
        m[i] = -INFINITY;
        l[i] = 0.f;
        zscale[i] = a.scale_log2;
        if constexpr (!E4) {
#pragma unroll
          for (int p = 0; p < DH / 16; ++p) {
            qa[p][i] = in ? *reinterpret_cast<const uint32_t*>(q + 16 * p + 2 * t) : 0u;
            qa[p][NR + i] = in ? *reinterpret_cast<const uint32_t*>(q + 16 * p + 8 + 2 * t) : 0u;
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
          const float fr = pow2_frame(amax);
          zscale[i] = a.scale_log2 / fr;       // exact
#pragma unroll
          for (int p = 0; p < DH / 16; ++p) {
            qa[p][i] = pack<true>(__uint_as_float(raw[p].x << 16) * fr, __uint_as_float(raw[p].x & 0xffff0000u) * fr);
            qa[p][NR + i] = pack<true>(__uint_as_float(raw[p].y << 16) * fr, __uint_as_float(raw[p].y & 0xffff0000u) * fr);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < DH / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    }
    if (!mbar_wait_warp(&full[sl], (k / S) & 1, abort_flag, a.c.err)) {
      ok = false;
      break;
    }
    const uint32_t kb0 = smem_u32(ring + sl * kStage), vb0 = kb0 + C::HALF;
    const int r0 = w.st * C::RUNS, nr = min(C::RUNS, kr.count - r0);
    // Scores, scaled to base 2 (over e4m3 with log2 of the V scale added), of
    // the stage's runs: z[run][8-key tile][row i: keys 2t, 2t+1]
    float z[C::RUNS][2][2 * NR];
    float vsc[C::RUNS];                        // E4: the runs' V scales
#pragma unroll
    for (int r = 0; r < C::RUNS; ++r) {
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < nr) {
        const uint32_t kb = kb0 + r * C::RUN;
        if constexpr (!E4) {
          const int row = 8 * (mi >> 1) + (lane & 7);
#pragma unroll
          for (int p = 0; p < DH / 16; ++p) {
            uint32_t b[4];
            ldsm4(piece<DH, E4>(kb, row, 2 * p + (mi & 1)), b);
            mma<E4>(s0, qa[p][0], LO ? 0u : qa[p][NR - 1], qa[p][NR], LO ? 0u : qa[p][2 * NR - 1], b[0], b[1]);
            mma<E4>(s1, qa[p][0], LO ? 0u : qa[p][NR - 1], qa[p][NR], LO ? 0u : qa[p][2 * NR - 1], b[2], b[3]);
          }
        } else {
          const int row = 8 * (mi & 1) + (lane & 7);
#pragma unroll
          for (int p = 0; p < DH / 16; p += 2) {
            uint32_t b[4], lo, hi;
            ldsm4(piece<DH, E4>(kb, row, p + (mi >> 1)), b);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              codes4(b[2 * u], lo, hi);
              mma<E4>(s0, qa[p + u][0], LO ? 0u : qa[p + u][NR - 1], qa[p + u][NR], LO ? 0u : qa[p + u][2 * NR - 1], lo, hi);
              codes4(b[2 * u + 1], lo, hi);
              mma<E4>(s1, qa[p + u][0], LO ? 0u : qa[p + u][NR - 1], qa[p + u][NR], LO ? 0u : qa[p + u][2 * NR - 1], lo, hi);
            }
          }
        }
      }
      float ks = 1.f, ve = 0.f;
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
      for (int i = 0; i < NR; ++i) {
        const float zs = E4 ? zscale[i] * ks : zscale[i];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          z[r][0][2 * i + j] = E4 ? fmaf(s0[2 * i + j], zs, ve) : s0[2 * i + j] * zs;
          z[r][1][2 * i + j] = E4 ? fmaf(s1[2 * i + j], zs, ve) : s1[2 * i + j] * zs;
        }
        if (!all) {
          const int lo = win_lo(qpos[i], a.window);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int kk = key + 8 * h + 2 * t + j;
              const bool see = r < nr && kk <= qpos[i] && (kk >= lo || kk < a.sinks);
              if (!see) z[r][h][2 * i + j] = -INFINITY;
            }
        }
      }
      // v rows that no query of the call sees: 0·NaN is NaN inside an MMA
      if (r < nr) {
        const int hid0 = min(max(a.sinks, 0), win_lo(first, a.window));   // hidden: [hid0, win_lo(first)) and [len, ..)
        const int hid1 = win_lo(first, a.window);
        if (key + kRun > len || (key < hid1 && key + kRun > hid0)) {
          uint8_t* vr = ring + sl * kStage + C::HALF + r * C::RUN;
          for (int i = lane; i < kRun * C::ROW / 16; i += 32) {
            const int nb = i / (kRun * C::BOXB / 16), row = i / (C::BOXB / 16) % kRun;
            const int kk = key + row;
            if (kk >= len || (kk >= hid0 && kk < hid1))
              *reinterpret_cast<uint4*>(vr + nb * C::BOX + row * C::BOXB + i % (C::BOXB / 16) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
        }
      }
    }
    // online softmax
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int r = 0; r < C::RUNS; ++r)
        mx = fmaxf(mx, fmaxf(fmaxf(z[r][0][2 * i], z[r][0][2 * i + 1]), fmaxf(z[r][1][2 * i], z[r][1][2 * i + 1])));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (mx > m[i] + kRescale || (m[i] == -INFINITY && mx > -INFINITY)) {
        const float fac = ex2_approx(m[i] - mx);          // 0 from -inf
        l[i] *= fac;
#pragma unroll
        for (int d = 0; d < DH / 8; ++d) {
          o[d][2 * i] *= fac;
          o[d][2 * i + 1] *= fac;
        }
        m[i] = mx;
      }
    }
#pragma unroll
    for (int r = 0; r < C::RUNS; ++r) {
      if (r >= nr) break;
      uint32_t pa[2 * NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float base = m[i] == -INFINITY ? 0.f : m[i];
        const float p0 = ex2_approx(z[r][0][2 * i] - base), p1 = ex2_approx(z[r][0][2 * i + 1] - base);
        const float p2 = ex2_approx(z[r][1][2 * i] - base), p3 = ex2_approx(z[r][1][2 * i + 1] - base);
        const float sum = (p0 + p1) + (p2 + p3);
        if constexpr (E4) {
          l[i] = fmaf(sum, scale_inv(vsc[r]), l[i]);
        } else {
          l[i] += sum;
        }
        pa[i] = pack<E4>(p0, p1);
        pa[NR + i] = pack<E4>(p2, p3);
      }
      const uint32_t vb = vb0 + r * C::RUN;
      const int row = 8 * (mi & 1) + (lane & 7);
      if constexpr (!E4) {
#pragma unroll
        for (int dt = 0; dt < DH / 8; dt += 2) {
          uint32_t b[4];
          ldsm4t(piece<DH, E4>(vb, row, dt + (mi >> 1)), b);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            mma<E4>(o[dt + u], pa[0], LO ? 0u : pa[NR - 1], pa[NR], LO ? 0u : pa[2 * NR - 1], b[2 * u], b[2 * u + 1]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < DH / 16; c += 2) {
          uint32_t b[4];
          ldsm4t(piece<DH, E4>(vb, row, c + (mi >> 1)), b);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t e0, o0, e1, o1;           // even and odd dims; keys 0..7, 8..15
            codes4(__byte_perm(b[2 * u], 0, 0x3120), e0, o0);
            codes4(__byte_perm(b[2 * u + 1], 0, 0x3120), e1, o1);
            const int d = 2 * (c + u);
            mma<E4>(o[d], pa[0], LO ? 0u : pa[NR - 1], pa[NR], LO ? 0u : pa[2 * NR - 1], e0, e1);
            mma<E4>(o[d + 1], pa[0], LO ? 0u : pa[NR - 1], pa[NR], LO ? 0u : pa[2 * NR - 1], o0, o1);
          }
        }
      }
    }
    __syncwarp();                              // the slot may be refilled
    if constexpr (TW > 1) {
      if (lane == 0) mbar_arrive(&empty[sl]);
    }
    const bool pair_ends = w.st + 1 == w.n_st;
    if (pair_ends || x + 1 == x1) {            // this piece's state
      const long long pc = (long long)team + (long long)w.b * Hkv + w.h;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float ls = l[i];
        ls += __shfl_xor_sync(0xffffffffu, ls, 1);
        ls += __shfl_xor_sync(0xffffffffu, ls, 2);
        const int row = tw * 16 + g + 8 * i;
        if (row >= f.R) continue;
        float* dst = f.part + (pc * f.R + row) * (DH + 4);
        if constexpr (!E4) {
#pragma unroll
          for (int d = 0; d < DH / 8; ++d)
            *reinterpret_cast<float2*>(dst + 4 + 8 * d + 2 * t) = make_float2(o[d][2 * i], o[d][2 * i + 1]);
        } else {
#pragma unroll
          for (int c = 0; c < DH / 16; ++c)
            *reinterpret_cast<float4*>(dst + 4 + 16 * c + 4 * t) =
                make_float4(o[2 * c][2 * i], o[2 * c + 1][2 * i], o[2 * c][2 * i + 1], o[2 * c + 1][2 * i + 1]);
        }
        if (t == 0) *reinterpret_cast<float2*>(dst) = make_float2(m[i], ls);
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
  if (!ok && tw == 0 && lane == 0) {
    volatile int no_abort = 0;
    for (int x = x0 > issued - S ? x0 : issued - S; x < issued; ++x)
      mbar_wait(&full[(x - x0) % S], ((x - x0) / S) & 1, &no_abort, a.c.err);
  }
}

// Joins the pieces of a row of a (sequence, KV head): o = Σ w_i O_i / Σ w_i l_i,
// w_i = 2^(m_i - M), in the order of the teams.  One warp per row, or with many
// pieces (WIDE) eight warps, each a run of them, whose results are joined the same
// way.  A lane holds DH/32 consecutive dims.
template <int DH, bool WIDE>
__global__ void __launch_bounds__(256) k_few_merge(const FewArgs f) {
  pdl_trigger();
  pdl_wait();
  constexpr int D = DH / 32;
  const AttnArgs& a = f.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int Hkv = a.c.Hkv, G = a.H / Hkv;
  const int row = WIDE ? blockIdx.x : blockIdx.x * 8 + warp, h = blockIdx.y, b = blockIdx.z;
  const int total = f.pre[f.B], before = f.pre[b], n_st = (f.pre[b + 1] - before) / Hkv;
  const int nn = a.n_new ? min(max(a.n_new[f.b0 + b], 0), a.n) : a.n;
  const int tok = row / G, head = h * G + row % G;
  if (row >= f.R || tok >= nn) return;
  const size_t at = (((size_t)(f.b0 + b) * a.n + tok) * a.H + head) * DH;
  float M = -INFINITY, L = 0.f, acc[D];
#pragma unroll
  for (int u = 0; u < D; ++u) acc[u] = 0.f;
  if (n_st > 0) {                               // (no stages: no rows in the cache)
    // team t has stages [total·t / teams, total·(t+1) / teams): those of the pair's first and last stage
    const int teams = min(f.teams, total);
    const long long U0 = before + (long long)h * n_st, U1 = U0 + n_st;
    const int t0 = (int)(((U0 + 1) * teams + total - 1) / total) - 1;
    const int np = (int)((U1 * teams + total - 1) / total) - t0;
    const float* p0 = f.part + ((t0 + (long long)b * Hkv + h) * f.R + row) * (DH + 4);
    const size_t step = (size_t)f.R * (DH + 4);
    const int i0 = WIDE ? np * warp / 8 : 0, i1 = WIDE ? np * (warp + 1) / 8 : np;
    for (int i = i0 + lane; i < i1; i += 32) M = fmaxf(M, p0[i * step]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -INFINITY ? 0.f : M;
#pragma unroll 4
    for (int i = i0; i < i1; ++i) {
      const float2 ml = *reinterpret_cast<const float2*>(p0 + i * step);
      const float w = ex2_approx(ml.x - base);
      L = fmaf(ml.y, w, L);
      if constexpr (D == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p0 + i * step + 4 + 4 * lane);
        acc[0] = fmaf(v.x, w, acc[0]);
        acc[1] = fmaf(v.y, w, acc[1]);
        acc[2] = fmaf(v.z, w, acc[2]);
        acc[3] = fmaf(v.w, w, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(p0 + i * step + 4 + 2 * lane);
        acc[0] = fmaf(v.x, w, acc[0]);
        acc[1] = fmaf(v.y, w, acc[1]);
      }
    }
    if constexpr (WIDE) {
      __shared__ float m_s[8], l_s[8], acc_s[8][DH];
      if (lane == 0) {
        m_s[warp] = M;
        l_s[warp] = L;
      }
#pragma unroll
      for (int u = 0; u < D; ++u) acc_s[warp][lane * D + u] = acc[u];
      __syncthreads();
      if (warp > 0) return;
      M = m_s[lane & 7];
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float all = M == -INFINITY ? 0.f : M;
      L = 0.f;
#pragma unroll
      for (int u = 0; u < D; ++u) acc[u] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = ex2_approx(m_s[i] - all);
        L = fmaf(l_s[i], w, L);
#pragma unroll
        for (int u = 0; u < D; ++u) acc[u] = fmaf(acc_s[i][lane * D + u], w, acc[u]);
      }
    }
  } else if (WIDE && warp > 0) {
    return;
  }
  const float inv = L == 0.f ? 0.f : 1.0f / L;
  float probe = 0.f;
#pragma unroll
  for (int u = 0; u < D; ++u) {
    acc[u] *= inv;
    probe = fmaf(acc[u], 0.f, probe);
  }
  if (__any_sync(0xffffffffu, !(probe == 0.f))) {        // not finite: see attend_row
    const SeqRange sr = seq_range(a, f.b0 + b);
    attend_row<DH>(a, f.b0 + b, h, sr.first + tok, (const bf16*)a.q + at, acc);
    __syncwarp();
  }
  bf16* out = (bf16*)a.o + at + lane * D;
  if constexpr (D == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(pack<false>(acc[0], acc[1]), pack<false>(acc[2], acc[3]));
  else
    *reinterpret_cast<uint32_t*>(out) = pack<false>(acc[0], acc[1]);
}

constexpr size_t kPreBytes = (kMaxB + 1) * 4 / 256 * 256 + 256;
int team_warps(int R) { return R <= 16 ? 1 : 2; }

template <int DH, bool E4, int TW, bool LO>
cudaError_t run(const AttnArgs& a, void* ws, int Bl, cudaStream_t s) {
  using C = FewCfg<DH, E4>;
  CUtensorMap tk, tv;
  const uint64_t planes = a.c.bt ? (uint64_t)a.c.num_pages * a.c.Hkv : (uint64_t)a.c.B * a.c.Hkv;
  const uint64_t rows = a.c.bt ? (uint64_t)a.c.ps : (uint64_t)a.c.T;
  const int es = E4 ? 1 : 2;
  cudaError_t e = make_tmap_rows(&tk, es, a.c.k, planes, rows, DH, C::BOXB / es, kRun);
  if (e != cudaSuccess) return e;
  e = make_tmap_rows(&tv, es, a.c.v, planes, rows, DH, C::BOXB / es, kRun);
  if (e != cudaSuccess) return e;
  const size_t smem = C::smem(Bl);
  static size_t attr_set[64] = {0};             // raised only when a launch needs more than before
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || attr_set[dev] < smem) {
    e = cudaFuncSetAttribute(k_attn_few<DH, E4, TW, LO>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = smem;
  }
  FewArgs f;
  f.a = a;
  f.pre = (int*)ws;
  f.part = (float*)((uint8_t*)ws + kPreBytes);
  f.R = a.n * (a.H / a.c.Hkv);
  constexpr int warps = FewShape<E4, LO>::WARPS;
  f.teams = sm_count() * (warps / TW);
  for (int b0 = 0; b0 < a.c.B; b0 += Bl) {
    f.b0 = b0;
    f.B = std::min(Bl, a.c.B - b0);
    e = launch_pdl(k_attn_few<DH, E4, TW, LO>, dim3(sm_count()), dim3(warps * 32), smem, s, tk, tv, f);
    if (e != cudaSuccess) return e;
    // eight warps per row from 16 pieces of a pair on (at equal lengths)
    const int rows = f.R;
    if (f.teams >= 16 * f.B * a.c.Hkv)
      e = launch_pdl(k_few_merge<DH, true>, dim3(rows, a.c.Hkv, f.B), dim3(256), 0, s, f);
    else
      e = launch_pdl(k_few_merge<DH, false>, dim3((rows + 7) / 8, a.c.Hkv, f.B), dim3(256), 0, s, f);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int DH, bool E4>
cudaError_t by_rows(const AttnArgs& a, void* part, int Bl, cudaStream_t s) {
  const int R = a.n * (a.H / a.c.Hkv);
  if (R <= 8) return run<DH, E4, 1, true>(a, part, Bl, s);
  if (R <= 16) return run<DH, E4, 1, false>(a, part, Bl, s);
  if (R <= kFewRows) return run<DH, E4, 2, false>(a, part, Bl, s);
  return cudaErrorInvalidValue;
}

// Sequences per launch: the line's stage numbers stay below 2^30.
int batch_of(const AttnArgs& a) {
  const long long per = (long long)a.c.Hkv * ((a.c.T + kRun - 1) / kRun + 1);
  return (int)std::min<long long>(std::min(a.c.B, kMaxB), std::max<long long>(1, (1LL << 30) / per));
}

}  // namespace

size_t cache_attn_few_workspace(const AttnArgs& a) {
  const int R = a.n * (a.H / a.c.Hkv);
  if (a.c.B == 0 || R == 0) return 0;
  const int warps = R <= 8 && a.c.dtype == TB_E4M3 ? FewShape<true, true>::WARPS : FewShape<false, false>::WARPS;
  const long long pieces = (long long)sm_count() * (warps / team_warps(R)) + (long long)batch_of(a) * a.c.Hkv;
  return kPreBytes + (size_t)pieces * R * (a.c.dh + 4) * 4;
}

cudaError_t launch_cache_attn_few(const AttnArgs& a, void* ws, cudaStream_t s) {
  const int Bl = batch_of(a);
  if (a.c.dtype == TB_E4M3)
    return a.c.dh == 128 ? by_rows<128, true>(a, ws, Bl, s) : by_rows<64, true>(a, ws, Bl, s);
  return a.c.dh == 128 ? by_rows<128, false>(a, ws, Bl, s) : by_rows<64, false>(a, ws, Bl, s);
}

}  // namespace tb
