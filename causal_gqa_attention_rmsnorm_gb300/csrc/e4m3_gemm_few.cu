// Products of e4m3 rows with e4m3 weights, for few rows (and for any): C = X·Wᵀ, or
// SiLU(X·W1ᵀ) * (X·W3ᵀ), where every 128 columns of a row of X and every 128 x 128 of a
// W have a power-of-two scale.
//
//   C[m, n] = sum_b 2^(sx[m, b] + sw[n / 128, b]) · sum_{k in block b} x[m, k] w[n, k]
//
// The scales go into the tensor core's instruction (kind::mxf8f6f4, which takes one per
// 32 elements of K: the four instructions of a K block name the same byte), so no sum
// is touched on its way.  With few rows the product is bound by the weights' stream, so
// it is formed transposed, Cᵀ = W·Xᵀ: 128 weight rows are the instruction's M and the
// rows of X, padded to NT, its N.  The `splits` CTAs of a tile form a cluster, CTA rank
// r taking part r of the K blocks:
//   warp 0      TMA: a K block's weight tiles [128, 128] and row tile [NT, 128] into a
//               ring of stages (the first weights before the wait for the kernel
//               before, which they do not depend on);
//   warp 1      issues the instructions, K blocks in order, and hands a chunk of K back
//               after every kChunk scale sets;
//   warps 2..5  put the scales into tensor memory, four K blocks at a time, ahead of
//               the instructions; then take the sums: without a split straight to y;
//               with few rows of one matrix into the CTA of the cluster that finishes
//               the row, by asynchronous stores that count on its barrier, so that no
//               CTA waits for another's end; else to shared memory, where after a
//               cluster barrier each CTA adds its share of the rows up over the
//               cluster.  Always in rank order.
// Chunks: the tensor core's accumulation cuts sums off instead of rounding them, which
// shifts a sum of n instructions by up to n steps of fp32 (terms of one sign: 3 steps at 64
// instructions, 10 at 128, 64 at 448, 0.65 n at 32768).  A chunk is 64
// instructions (2048 of K); the chunks are added with rounding, in registers.  (A part of
// K of one chunk, the usual case, keeps no sums there.)
//
// Measured in a stream of calls: 1 x 128256 x 4096 77 us, 6.8 TB/s, as fast as memory is
// copied; 32 x 14336 x 4096 gated 21.5 us (5.5 TB/s), 32 x 4096 x 14336 12.9 (4.6), 1 x
// 6144 x 4096 6.0 (4.2): a call takes 3 to 4 us whatever it reads, of which 1 is the first
// row tile's and the scales' load, 0.2 each K block's instructions, 0.5 the partial sums'
// way.  (Partial sums read by the finishing CTA between two cluster barriers: 1 x 6144 x
// 4096 7.1, 32 x 4096 x 14336 13.4; pushed row by row, 4 bytes at a time: 6.1 and 13.9.)
// Tried: rings of 73 and 55 KB, which let three and four CTAs share an SM (13.7 and 15.3
// us for 13.5), one CTA per SM with a ring of 216 KB (13.6; 1 x 6144 x 4096 8.0), clusters
// of 3, 5 and 6 (7.8, 7.3 and 11.4 for 7.2: clusters of 6 do not all find a place at once).
#include "e4m3_epilogue.cuh"
#include "gemm_tc.cuh"
#include "sm100_ptx.cuh"

namespace tb {
namespace {

using namespace ptx;

constexpr int kSet = 4;          // K blocks per scale set: one exponent byte each in a word
constexpr int kChunk = 4;        // scale sets per chunk
constexpr int kSets = 8;         // scale sets held in tensor memory: two chunks

// NT rows of X; MATS 1 or 2 weight matrices; CPS CTAs per SM; ONE: a CTA's part of K is
// at most one chunk, whose sums go from tensor memory straight on.
template <int NT, int MATS, int CPS, bool ONE> struct FewCfg {
  static constexpr uint32_t W_BYTES = MATS * kBlk * kBlk;
  static constexpr uint32_t STAGE_BYTES = W_BYTES + NT * kBlk;
  // With few rows of one matrix the partial sums of a split go straight into the CTA that
  // adds them up, four rows of a column at a time; it has a place for them beside the ring
  // (up to 8 parts of 4 rows, or 4 of 8, 2 of 16).
  static constexpr bool PUSH = ONE && MATS == 1 && NT <= 32;
  static constexpr uint32_t INBOX = PUSH ? 32 * kBlk * 4 : 0;
  static constexpr uint32_t ROOM = (CPS == 2 ? 110 * 1024 : 220 * 1024) - INBOX;
  static constexpr int FIT = ROOM / STAGE_BYTES;
  static constexpr int STAGES = FIT > 12 ? 12 : FIT;
  static constexpr uint32_t OFF_INBOX = STAGES * STAGE_BYTES;
  static constexpr uint32_t OFF_BAR = OFF_INBOX + INBOX;
  static constexpr size_t SMEM = OFF_BAR + 512 + 1024;
  static constexpr uint32_t ACC = MATS * NT;                 // columns of one accumulator
  static constexpr uint32_t SET_COLS = 4 * MATS + 4;         // a word per weight row / 32 and row / 32
  static constexpr uint32_t SETS_AT = ONE ? ACC : 2 * ACC;
  static constexpr uint32_t NEED = SETS_AT + (ONE ? kChunk : kSets) * SET_COLS;
  static constexpr uint32_t TMEM_COLS = NEED <= 128 ? 128 : NEED <= 256 ? 256 : 512;
  static_assert(CPS * TMEM_COLS <= 512, "tensor memory of an SM");
  static_assert(2 * TMEM_COLS + kSkinnyMostTmem <= 512 || 2 * SMEM + kSkinnyLeastSmem + 3 * kSmemPerCta > kSmemOfSm,
                "a third CTA that waits for tensor memory");
  static_assert(CPS == 2 || SMEM + kSkinnyLeastSmem + 2 * kSmemPerCta > kSmemOfSm, "a second one");
  static_assert(STAGES >= 2 && (2 * STAGES + 2 * kSets + 7) * 8 + 8 <= 512, "barriers");
  static_assert(MATS * NT * kBlk * 4 <= OFF_INBOX, "the sums reuse the ring");
};

// Rows t, t + 4, ... below t1 of a tile by one warp, four columns to a lane: the sums of
// the S CTAs of the cluster added up in rank order and finished.  B rows at a time, so that
// S·B loads (of each matrix) are on their way together.  S 1: what lies in part_s is the
// gated result already, to become codes.
template <int NT, int MATS, int S, int B>
__device__ __forceinline__ void finish_rows(const GemmArgs& a, const float* part_s, int m0, int wt, int t, int t1, int lane) {
  const int col = wt * kBlk + 4 * lane;
  const uint32_t base = smem_u32(part_s) + 16u * lane;
  for (; t < t1; t += 4 * B) {
    float4 v[B], p[B][MATS][S];
    if constexpr (MATS == 1) {
      if (a.res && col < a.N)
        get4<B>(v, a.res, a.y_dtype, [&](int b) { return (size_t)(m0 + min(t + 4 * b, t1 - 1)) * a.N + col; });
      else
        for (int b = 0; b < B; ++b) v[b] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int tb = min(t + 4 * b, t1 - 1);         // (past the last: again, not stored)
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int r = 0; r < S; ++r) {
          const uint32_t at = base + (uint32_t)((m * NT + tb) * kBlk * 4);
          if constexpr (S == 1) p[b][m][r] = *reinterpret_cast<const float4*>(part_s + tb * kBlk + 4 * lane);
          else p[b][m][r] = ld_dsmem_f4(mapa_shared(at, (uint32_t)r));
        }
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const bool in = t + 4 * b < t1;
      const size_t at = (size_t)(m0 + t + 4 * b) * a.N + col;
      float4 u[MATS];
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        u[m] = p[b][m][0];
#pragma unroll
        for (int r = 1; r < S; ++r)
          u[m] = make_float4(u[m].x + p[b][m][r].x, u[m].y + p[b][m][r].y, u[m].z + p[b][m][r].z, u[m].w + p[b][m][r].w);
      }
      float4 y = u[0];
      if constexpr (MATS == 1) {
        y = make_float4(y.x + v[b].x, y.y + v[b].y, y.z + v[b].z, y.w + v[b].w);
      } else if constexpr (S > 1) {
        y = make_float4(gated(u[0].x, u[1].x), gated(u[0].y, u[1].y), gated(u[0].z, u[1].z), gated(u[0].w, u[1].w));
      }
      if (MATS == 1 || a.y_dtype != TB_E4M3) {
        if (in && col < a.N) put4(a.y, a.y_dtype, at, y);
        continue;
      }
      // (columns past N hold zeros: weight rows past N read as zeros)
      float top = fmaxf(fmaxf(finite_mag(y.x), finite_mag(y.y)), fmaxf(finite_mag(y.z), finite_mag(y.w)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = block_exponent(top);
      const float inv = pow2i(-e);
      if (in && col < a.N)
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.y) + at) =
            codes_of4(to_code(y.x, inv), to_code(y.y, inv), to_code(y.z, inv), to_code(y.w, inv));
      if (in && lane == 0)
        a.y_scale[(size_t)(m0 + t + 4 * b) * ((a.N + kBlk - 1) / kBlk) + wt] = (uint8_t)(e + 127);
    }
  }
}

// P rows of a column of y (`live`, at least one, of them exist), with the residual at `at` of
// res.  (Its loads depend on nothing, so that all are on their way together: 1024 x 2304 x
// 768 21.0 us by a branch for each, 10.0 so; 9.5 with the lines in L2 by then.)
template <typename T, int P>
__device__ __forceinline__ void put_column(T* y, const T* res, size_t at, int N, int live, float (&v)[P]) {
  if (res) {
    const T* r = res + at;
    T add[P];
#pragma unroll
    for (int k = 0; k < P; ++k) add[k] = r[(size_t)min(k, live - 1) * N];
#pragma unroll
    for (int k = 0; k < P; ++k) v[k] += to_f(add[k]);
  }
#pragma unroll
  for (int k = 0; k < P; ++k)
    if (k < live) y[(size_t)k * N] = from_f<T>(v[k]);
}

template <int NT, int MATS, int CPS, bool ONE>
__global__ void __launch_bounds__(192, CPS)
    k_e4m3_few(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmW3,
               const __grid_constant__ CUtensorMap tmX, GemmArgs a, int wtiles, int splits, int* err) {
  using C = FewCfg<NT, MATS, CPS, ONE>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* sfull = empty + STAGES;       // scale sets
  uint64_t* sempty = sfull + kSets;
  uint64_t* tfull = sempty + kSets;       // accumulators
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* inbox_full = drain + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(inbox_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* part_s = reinterpret_cast<float*>(smem);       // [MATS][NT][128] after the main loop
  float4* inbox = reinterpret_cast<float4*>(smem + C::OFF_INBOX);  // [splits][tpr / 4][128], four rows each

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();              // blockIdx.x % splits
  const int tile = (int)(blockIdx.x / splits);
  const int wt = tile % wtiles, m0 = tile / wtiles * NT;
  const int kblocks = (a.K + kBlk - 1) / kBlk;
  const int kb0 = (int)((long long)kblocks * rank / splits);
  const int nkb = (int)((long long)kblocks * (rank + 1) / splits) - kb0;   // >= 1: splits <= kblocks
  const int nsets = (nkb + kSet - 1) / kSet, nchunks = (nsets + kChunk - 1) / kChunk;
  const int rows = min(NT, a.M - m0);
  const bool push = C::PUSH && splits > 1;
  int tpr = (rows + splits - 1) / splits;               // rows each CTA of the cluster finishes
  if (push) tpr = (tpr + 3) & ~3;                       // (whole fours: some CTAs may have none)
  const int t0 = min(rows, rank * tpr), t1 = min(rows, t0 + tpr);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSets; ++s) {
      mbar_init(&sfull[s], 4);
      mbar_init(&sempty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 4);
    }
    mbar_init(drain, 1);
    mbar_init(inbox_full, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if (push && t1 > t0) mbar_arrive_expect_tx(inbox_full, (uint32_t)((splits - 1) * ((t1 - t0 + 3) / 4) * kBlk * 16));
    prefetch_tmap(&tmW);
    if (MATS == 2) prefetch_tmap(&tmW3);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
    pdl_trigger();                                // (only now: common.cuh)
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (waited for where the first partial sums leave: the other CTAs' barriers exist then)
  if (push) cluster_arrive();

  if (warp == 0) {
    // (the whole warp, its elected lane issuing)
    const uint32_t elected = elect_one();
    const uint64_t pol = policy_evict_first();
    const bool once = a.M <= NT;                // the weights are read once: they need not stay in L2
    const uint32_t ring = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
    const int wrow = wt * kBlk;
    bool dep = false;
    auto release = [&]() {
      pdl_wait();
      dep = true;
      const int held = nkb < STAGES ? nkb : STAGES;
#pragma unroll 1
      for (int h = 0; h < held; ++h)
        tma_load_3d_elected<1>(&tmX, ring + h * C::STAGE_BYTES + C::W_BYTES, full0 + h * 8, (kb0 + h) * kBlk, m0, 0, elected);
    };
    uint32_t st = 0, phase = 0;
    int j = 0;
#pragma unroll 1
    for (; j < nkb; ++j) {
      if (!__all_sync(0xffffffffu, mbar_try_wait(empty0 + st * 8, phase ^ 1u)) &&
          !mbar_wait_warp(&empty[st], phase ^ 1u, abort_flag, err))
        break;
      const uint32_t sw = ring + st * C::STAGE_BYTES, bar = full0 + st * 8;
      const int k = (kb0 + j) * kBlk;
      mbar_expect_elected(bar, C::STAGE_BYTES, elected);
      if (once) {
        tma_load_3d_elected<1>(&tmW, sw, bar, k, wrow, 0, pol, elected);
        if constexpr (MATS == 2) tma_load_3d_elected<1>(&tmW3, sw + kBlk * kBlk, bar, k, wrow, 0, pol, elected);
      } else {
        tma_load_3d_elected<1>(&tmW, sw, bar, k, wrow, 0, elected);
        if constexpr (MATS == 2) tma_load_3d_elected<1>(&tmW3, sw + kBlk * kBlk, bar, k, wrow, 0, elected);
      }
      if (dep) tma_load_3d_elected<1>(&tmX, sw + C::W_BYTES, bar, k, m0, 0, elected);
      else if (j + 1 == STAGES) release();
      if (++st == STAGES) st = 0, phase ^= 1u;
    }
    if (!dep) release();
    // every copy issued must land before the CTA may exit (earlier copies into the same
    // stages were consumed, hence complete)
    volatile int no_abort = 0;
    for (int t = j - STAGES < 0 ? 0 : j - STAGES; t < j; ++t)
      mbar_wait_warp(&full[t % STAGES], (t / STAGES) & 1, &no_abort, err);
  } else if (warp == 1) {
    // The whole warp walks the blocks; its elected lane issues (mma_mx_k128).
    const uint32_t elected = elect_one();
    const uint64_t desc = desc_kmajor_sw128(smem_u32(smem));
    const uint32_t desc_hi = (uint32_t)(desc >> 32), desc0 = (uint32_t)desc;
    const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    pdl_wait();                           // (the limit of its waits is for this kernel's work)
    for (int set = 0; ok && set < nsets; ++set) {
      const int chunk = set / kChunk, buf = chunk & 1;
      const bool first = set % kChunk == 0, last = set + 1 == nsets;
      if (first && !mbar_wait_warp(&tempty[buf], ((chunk >> 1) & 1) ^ 1u, abort_flag, err)) break;
      if (!mbar_wait_warp(&sfull[set % kSets], (set / kSets) & 1, abort_flag, err)) break;
      const uint32_t d = tmem + buf * C::ACC, sf = tmem + C::SETS_AT + (set % kSets) * C::SET_COLS;
#pragma unroll
      for (int b = 0; b < kSet; ++b) {
        if (set * kSet + b < nkb) {
          if (!__all_sync(0xffffffffu, mbar_try_wait(full0 + stage * 8, phase)) &&
              !(ok = mbar_wait_warp(&full[stage], phase, abort_flag, err)))
            break;
          tc_fence_after();
          const uint32_t w = desc0 + stage * (C::STAGE_BYTES >> 4), x = w + (C::W_BYTES >> 4);
#pragma unroll
          for (int m = 0; m < MATS; ++m)
            mma_mx_k128<1>(d + m * NT, w + m * (kBlk * kBlk >> 4), x, desc_hi, idesc_mx_e4m3(kBlk, NT, b), sf + 4 * m,
                           sf + 4 * MATS, !(first && b == 0), elected);
          mma_commit_elected(empty0 + stage * 8, elected);
          if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
      }
      mma_commit_elected(smem_u32(&sempty[set % kSets]), elected);
      if (ok && (last || (set + 1) % kChunk == 0)) mma_commit_elected(smem_u32(&tfull[buf]), elected);
    }
    // all of them must be done before tensor memory is released
    mma_commit_elected(smem_u32(drain), elected);
    volatile int no_abort = 0;
    mbar_wait_warp(drain, 0, &no_abort, err);
  } else {
    pdl_wait();
    const int quad = warp & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    // Scale set s: a word per row for its K blocks; the weights' is the same for all rows
    // of the tile.
    constexpr int XC = NT < 32 ? 1 : NT / 32;
    struct Words {
      uint32_t w[MATS], x[XC];
    };
    auto words = [&](int s) {
      const int kb = kb0 + s * kSet, n = min(kSet, kb0 + nkb - kb);
      Words v;
      v.w[0] = scale_word(a.w.scale + (size_t)wt * kblocks + kb, n);
      if constexpr (MATS == 2) v.w[1] = scale_word(a.w3.scale + (size_t)wt * kblocks + kb, n);
#pragma unroll
      for (int c = 0; c < XC; ++c) {
        const int m = m0 + c * 32 + lane;
        v.x[c] = m < a.M ? scale_word(a.x.scale + (size_t)m * kblocks + kb, n) : 0x7f7f7f7fu;
      }
      return v;
    };
    auto place = [&](int s, const Words& v) {
      const uint32_t at = tmem + lanes + C::SETS_AT + (s % kSets) * C::SET_COLS;
#pragma unroll
      for (int m = 0; m < MATS; ++m) tmem_st4(at + 4 * m, v.w[m], v.w[m], v.w[m], v.w[m]);
      tmem_st4(at + 4 * MATS, v.x[0], v.x[XC > 1 ? 1 : 0], v.x[XC > 2 ? 2 : 0], v.x[XC > 3 ? 3 : 0]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sfull[s % kSets]);
    };
    auto feed = [&](int s) {
      if (!mbar_wait_warp(&sempty[s % kSets], ((s / kSets) & 1) ^ 1u, abort_flag, err)) return false;
      const Words v = words(s);
      tc_fence_after();
      place(s, v);
      return true;
    };
    // Lane l of quarter q holds weight row 32 q + l, that is a column of y, of every row
    // of the tile: of `P` rows from `i` on, in u.  Without a split they are finished here,
    // and stored if nothing has to be known of the row's other columns; else all goes to
    // shared memory.  (The last chunk's sums come after every instruction, and so after
    // every read of the ring.)
    constexpr int P = 16;
    const int f = quad * 32 + lane, col = wt * kBlk + f;
    auto put = [&](int i, const float (&u)[MATS][P]) {
      if (push) {
#pragma unroll
        for (int k = 0; k < P; k += 4) {
          const int four = (i + k) / 4, owner = four * 4 / tpr;
          float4* to = inbox + (rank * (tpr / 4) + four - owner * (tpr / 4)) * kBlk + f;
          if (i + k >= rows) break;
          if (owner == rank) *to = make_float4(u[0][k], u[0][k + 1], u[0][k + 2], u[0][k + 3]);
          else
            st_async_f4(mapa_shared(smem_u32(to), (uint32_t)owner), u[0][k], u[0][k + 1], u[0][k + 2], u[0][k + 3],
                        mapa_shared(smem_u32(inbox_full), (uint32_t)owner));
        }
        return;
      }
      if (splits > 1) {
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
          for (int k = 0; k < P; ++k) part_s[(m * NT + i + k) * kBlk + f] = u[m][k];
        return;
      }
      float v[P];
#pragma unroll
      for (int k = 0; k < P; ++k) v[k] = MATS == 2 ? gated(u[0][k], u[MATS - 1][k]) : u[0][k];
      if (a.y_dtype == TB_E4M3) {
#pragma unroll
        for (int k = 0; k < P; ++k) part_s[(i + k) * kBlk + f] = v[k];
        return;
      }
      if (col >= a.N) return;
      const size_t at = (size_t)(m0 + i) * a.N + col;
      if (a.y_dtype == TB_F32)
        put_column(static_cast<float*>(a.y) + at, static_cast<const float*>(MATS == 1 ? a.res : nullptr), at, a.N, rows - i, v);
      else
        put_column(static_cast<bf16*>(a.y) + at, static_cast<const bf16*>(MATS == 1 ? a.res : nullptr), at, a.N, rows - i, v);
    };
    // the residual that this CTA adds comes into L2 meanwhile
    auto ahead = [&]() {
      const int t = t0 + (int)threadIdx.x - 64, c = wt * kBlk;
      const uint32_t e = a.y_dtype == TB_F32 ? 4 : 2;
      if (MATS == 1 && a.res && t < t1)
        prefetch_l2_bulk(static_cast<const uint8_t*>(a.res) + ((size_t)(m0 + t) * a.N + c) * e, (uint32_t)min(kBlk, a.N - c) * e);
    };
    if constexpr (ONE) {
      // all sets at once: one latency
      Words v[kChunk];
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (i < nsets) v[i] = words(i);
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (i < nsets) place(i, v[i]);
      ahead();
      const bool ok = mbar_wait_warp(tfull, 0, abort_flag, err);
      if (push) cluster_wait();
      if (ok) {
        tc_fence_after();
        // (a loop: code that runs once costs its way into the instruction cache)
#pragma unroll 1
        for (int i = 0; i < NT && i < rows; i += P) {
          float u[MATS][P];
#pragma unroll
          for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int k = 0; k < P; k += 16)
              tmem_ld16(tmem + lanes + m * NT + i + k, *reinterpret_cast<uint32_t(*)[16]>(&u[m][k]));
          tmem_wait_ld();
          put(i, u);
        }
      }
    } else {
      ahead();
      bool ok = true;
      int fed = 0;
      float acc[MATS][NT];
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][i] = 0.f;
      for (int c = 0; ok && c < nchunks; ++c) {
        // the sets of this chunk and of the next one: those they replace belong to the
        // chunk before, whose sums are in registers already
        for (const int upto = min(nsets, (c + 2) * kChunk); ok && fed < upto; ++fed) ok = feed(fed);
        if (!ok || !(ok = mbar_wait_warp(&tfull[c & 1], (c >> 1) & 1, abort_flag, err))) break;
        tc_fence_after();
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
          for (int i = 0; i < NT; i += 16) {
            uint32_t u[16];
            tmem_ld16(tmem + lanes + (c & 1) * C::ACC + m * NT + i, u);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[m][i + k] += __uint_as_float(u[k]);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[c & 1]);
      }
      if (ok) {
#pragma unroll
        for (int i = 0; i < NT; i += P) {
          if (i >= rows) break;
          float u[MATS][P];
#pragma unroll
          for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int k = 0; k < P; ++k) u[m][k] = acc[m][i + k];
          put(i, u);
        }
      }
    }
  }

  if (push) {
    if (warp < 2) {
      cluster_wait();
    } else if (t1 > t0 && mbar_wait_cluster_warp(inbox_full, 0, abort_flag, err)) {
      // a column of the tile per thread, which has put this CTA's own share there itself
      const int f = (warp & 3) * 32 + lane, col = wt * kBlk + f;
      if (col < a.N) {
        for (int t = t0; t < t1; t += 4) {
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          for (int r = 0; r < splits; ++r) {          // in rank order
            const float4 p = inbox[(r * (tpr / 4) + (t - t0) / 4) * kBlk + f];
            v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
          }
          const size_t at = (size_t)(m0 + t) * a.N + col;
          if (a.y_dtype == TB_F32)
            put_column(static_cast<float*>(a.y) + at, static_cast<const float*>(a.res), at, a.N, t1 - t, v);
          else
            put_column(static_cast<bf16*>(a.y) + at, static_cast<const bf16*>(a.res), at, a.N, t1 - t, v);
        }
      }
    }
  } else {
    // the sums of every CTA of the cluster are in shared memory
    tc_fence_before();
    __syncwarp();
    if (splits > 1) cluster_sync();
    else __syncthreads();

    if (warp >= 2) {
      const int t = t0 + warp - 2;
      if (splits == 8) finish_rows<NT, MATS, 8, 1>(a, part_s, m0, wt, t, t1, lane);
      else if (splits == 4) finish_rows<NT, MATS, 4, 2>(a, part_s, m0, wt, t, t1, lane);
      else if (splits == 2) finish_rows<NT, MATS, 2, 2>(a, part_s, m0, wt, t, t1, lane);
      else if (MATS == 2 && a.y_dtype == TB_E4M3) finish_rows<NT, MATS, 1, 2>(a, part_s, m0, wt, t, t1, lane);
    }
  }

  // no CTA leaves (and frees its shared memory) while another still reads it
  tc_fence_before();
  __syncwarp();
  if (splits > 1 && !push) cluster_sync();
  else __syncthreads();
  // (what was pushed has all arrived; a CTA that gave up stays until the others are gone)
  if (push && *abort_flag) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int NT, int MATS, int CPS, bool ONE> cudaError_t launch(const GemmArgs& a, int wtiles, int sp, cudaStream_t s) {
  using C = FewCfg<NT, MATS, CPS, ONE>;
  CUtensorMap tw, tw3, tx;
  cudaError_t e = make_tmap_rows(&tw, 1, a.w.codes, 1, (uint64_t)a.N, (uint64_t)a.K, kBlk, kBlk);
  if (e != cudaSuccess) return e;
  tw3 = tw;
  if (MATS == 2 && (e = make_tmap_rows(&tw3, 1, a.w3.codes, 1, (uint64_t)a.N, (uint64_t)a.K, kBlk, kBlk)) != cudaSuccess)
    return e;
  e = make_tmap_rows(&tx, 1, a.x.codes, 1, (uint64_t)a.M, (uint64_t)a.K, kBlk, NT);
  if (e != cudaSuccess) return e;
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    e = cudaFuncSetAttribute(k_e4m3_few<NT, MATS, CPS, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  const long long ctas = (long long)wtiles * ((a.M + NT - 1) / NT) * sp;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = sp;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = sp > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_e4m3_few<NT, MATS, CPS, ONE>, tw, tw3, tx, a, wtiles, sp, device_error_word());
}

// CPS: CTAs per SM of the form with several chunks (the one with one chunk has two; gated
// tiles of 64 rows are for long sums, and for them alone).
template <int NT, int MATS, int CPS> cudaError_t go(const GemmArgs& a, cudaStream_t s) {
  const int wtiles = (a.N + kBlk - 1) / kBlk, kblocks = (a.K + kBlk - 1) / kBlk;
  const long long tiles = (long long)wtiles * ((a.M + NT - 1) / NT);
  auto split = [&](int cps) {
    const long long slots = (long long)cps * sm_count();
    return tiles > slots ? 1 : skinny_split_count((int)tiles, kblocks, (int)slots);
  };
  if constexpr (MATS == 1 || NT < 64) {
    const int two = split(2);
    if ((kblocks + two - 1) / two <= kSet * kChunk) return launch<NT, MATS, 2, true>(a, wtiles, two, s);
  }
  return launch<NT, MATS, CPS, false>(a, wtiles, split(CPS), s);
}

}  // namespace

// Rows of X per tile for M rows, or 0 where k_e4m3_many is the better one, -1 with a CTA
// to a tile.
//
// Short K (up to 2048): a call is its fixed cost, which grows with the tile, so the smallest
// tile whose tiles are all resident at once, two CTAs per SM; the largest, and gated ones,
// only up to 128 rows, where half of k_e4m3_many's tile is empty, or for `light` results
// (fp32 without a residual; gated ones not to codes); then 256 x 256 tiles.  Long K: the first tile whose tiles are
// resident twice over, that is with K split in two or more; then 256 x 256 tiles.  (64 rows
// of one matrix: one split less.)  Up to 128 rows, where the second CTA of a pair would have
// none, a CTA to a tile once there are more tiles than pairs, which then are fewer rounds.
// Measured, us, by rows per tile, and k_e4m3_many:
//                                32     64    128   many
//   K 768, N 2304:    512 rows   5.4    5.6    7.2    7.0      1024:  9.8   6.5   8.1   7.2
//        1371: 14.3  10.6   8.6   7.9   (to fp32: 14.8  11.3   9.3   9.4; residual: - - 14.6  12.4)
//   K 1024, N 32768:  128       21.9   14.7   10.6   12.3
//   K 1536, N 2304:   512        6.8    8.0    9.4    8.7      1371: 18.8  13.6  10.1   9.6
//        (to fp32: 18.9  13.8  10.0  11.1)
//   K 4096, N 4096:   256       11.8   10.7   12.1   14.4       512: 22.4  14.3  14.0  14.5
//   K 4096, N 14336:  128       24.5   17.0   15.9   17.1       256: 36.9  28.9  30.4  17.4
//   K 14336, N 4096:  256       30.2   22.4   19.9   35.4       512: 59.4  36.3  31.8  35.8
//   gated, K 768, F 2048:    128   6.8   9.8    -    7.2        256:  7.7   9.9    -   7.2
//        (to bf16: 128  5.7   7.2    -    7.0        333:  6.8   7.9    -   7.0)
//   gated, K 1536, F 4096:   128   9.5  12.0    -    9.5        192: 10.5  12.5    -   9.5
//   gated, K 2048, F 11008:   96  14.5  19.7    -   17.1
//   gated, K 4096, F 2048:   256  13.1  14.4    -   14.5        333: 18.2  17.6    -  14.7
//   gated, K 4096, F 14336:   64  29.1  25.2    -   27.1, a CTA to a tile 23.9
//                            128  52.3  43.8    -   27.9                  23.7
//   gated, K 4096, F 11008:  128  38.8  39.3    -   27.4                  21.0
//   K 768, N 50304:          128    -   19.5  18.7  14.1                  12.9
int e4m3_few_tile(int M, int N, int K, int mats, bool light, int sms) {
  const long long wtiles = ((long long)N + kBlk - 1) / kBlk, slots = 2LL * sms;
  auto fits = [&](int nt, int times) { return wtiles * (((long long)M + nt - 1) / nt) * times <= slots; };
  if (M <= 16) return 16;
  if (M <= 32) return 32;
  if (K <= 2048) {
    if ((mats == 1 || light || M <= 128) && fits(32, 1)) return 32;
    if (mats == 1 && fits(64, 1)) return 64;
    if (mats == 1 && (light || M <= 128) && fits(128, 1)) return 128;
  } else if (mats == 1) {
    if (fits(64, 2)) return 64;
    if (M > 64 && fits(128, 2)) return 128;
  } else if (fits(32, 2)) {
    return 32;
  }
  if (M <= 64 && mats == 1) return 64;
  const long long tiles = mats == 1 ? (wtiles + 1) / 2 : wtiles;        // 256 x 256
  return M <= 128 && 2 * tiles > sms ? -1 : 0;
}

cudaError_t launch_gemm_e4m3_few(const GemmArgs& a, int tile, cudaStream_t s) {
  switch (tile) {
    case 16: return go<16, 1, 2>(a, s);
    case 32: return go<32, 1, 2>(a, s);
    case 64: return go<64, 1, 2>(a, s);
    default: return go<128, 1, 1>(a, s);
  }
}
cudaError_t launch_gated_e4m3_few(const GemmArgs& a, int tile, cudaStream_t s) {
  switch (tile) {
    case 16: return go<16, 2, 2>(a, s);
    case 32: return go<32, 2, 2>(a, s);
    default: return go<64, 2, 1>(a, s);
  }
}

}  // namespace tb
