// The products of e4m3_gemm_few.cu for many rows: 256 x 256 tiles on CTA pairs, or, for up to
// 128 rows, 128 x 256 on single CTAs.
//
// The clusters of two CTAs walk the tiles (persistent).  A CTA stages its own 128 rows
// of X and 128 rows of W per K block of 128 (32 KB, six stages); the even CTA issues
// M = 256 instructions that read B from both CTAs' shared memory.  In the gated product
// one CTA stages rows of W1 and the other the same rows of W3, so that half of the
// accumulator's columns are gates and half what they gate: one tile is one block of 128
// columns of the result.  Accumulator 0 has the gates first and accumulator 1 last.
// Or (CG 1) each CTA has tiles of its own, of 128 rows: all 256 rows of W, four stages.
//   warp 0      TMA;
//   warp 1      issues the instructions (even CTA), or tells that CTA of scales (odd CTA);
//   warps 2..9  epilogue, half a row of the tile per lane;
//   warps 10..13  put the scales of four K blocks at a time into shared memory, from where
//               the issuing warp has them copied to tensor memory.
// Tensor memory holds two accumulators of 256 columns and two scale sets of 12, which
// is more than its 512 columns: accumulator 0 takes columns 0..255, accumulator 1
// columns 224..479, and the 32 columns that they share are read first when a tile is
// finished; the next tile's instructions wait for that (and not for the rest).
//
// Measured in short graphs of calls: 16384 x 4096 x 14336 with the residual 535-565 us
// (3400-3590 TFLOP/s, 0.88-0.93 of twice cuBLAS's bf16 rate), gated 8192 x 14336 x 4096 500-515
// us (3740-3850); the power limit sets both (over seconds 646 and 595 us, 2980 and 3240 at 1.4
// to 1.6 GHz).  Short K: 16384 x 768 x 768 12.7-14.0 us, 16384 x 2304 x 768 27.3, gated 8192 x
// 2048 x 768 21.4-22.4 (a tile's instructions take 3100 cycles there, its change 1200; without SiLU, stores and the exponents' exchange 19.8).
// What short K gained: scales through shared memory and the issuing warp's copies, where
// they had been stored to tensor memory by warps that first waited for a set's last
// instruction (17.6 -> 13.2 us, gated 31.5 -> 27); eight epilogue warps for four (gated
// 16384 x 2048 x 768 to fp32 59 -> 53 us); both for the smallest calls (gated 256 x 2048 x 768
// 8.7 -> 7.3).  Single CTAs: gated 128 x 14336 x 4096 29.1 -> 24.7, whose 112 tiles are one
// round of 152 CTAs and two of 76 pairs.
// Tried: operands in a branch on the lane instead of a converged warp (650 us for 569 at
// that time); three more sets of scales by sharing 64 columns (672 for 650: the division
// by five sat in the issuing warp); clusters of two pairs that multicast X (557 for 551:
// a quarter less traffic from L2, but only 144 SMs hold clusters of four).
#include <algorithm>

#include "e4m3_epilogue.cuh"
#include "gemm_tc.cuh"
#include "sm100_ptx.cuh"

namespace tb {
namespace {

using namespace ptx;

constexpr int kSet = 4;          // K blocks per scale set
constexpr int kRowsCta = 128;    // rows of X per CTA

// CG: CTAs that share a tile.
template <int CG> struct ManyCfg {
  static constexpr int STAGES = CG == 2 ? 6 : 4;
  static constexpr uint32_t A_BYTES = kRowsCta * kBlk, B_BYTES = (256 / CG) * kBlk, STAGE_BYTES = A_BYTES + B_BYTES;
  // two pieces of 32 rows x 64 bytes of y for each epilogue warp
  static constexpr uint32_t OFF_EPI = STAGES * STAGE_BYTES, PIECE = 32 * 64;
  // scale sets: a word of four scales for each of the CTA's rows of X, row 32 c + l at 16 l + 4 c,
  // and eight rows of 16 bytes of the one word of either half of W
  static constexpr uint32_t OFF_SF = OFF_EPI + 8 * 2 * PIECE, SF_W = 512, SF_BYTES = 768;
  static constexpr uint32_t OFF_EXP = OFF_SF + 2 * SF_BYTES, OFF_BAR = OFF_EXP + 512;
  static constexpr size_t SMEM = OFF_BAR + 384;
  static constexpr uint32_t ACC1 = 224, SETS_AT = 480, SET_COLS = 16;
  static constexpr int THREADS = 448;
};

// Tile -> (row unit of 256, column tile): column tiles fastest, or in groups of
// `group` row units, rows fastest inside a group.
__device__ __forceinline__ void place(int tile, int m_units, int n_tiles, int group, int& mu, int& nt) {
  if (group <= 0) {
    mu = tile / n_tiles;
    nt = tile - mu * n_tiles;
    return;
  }
  const int per = group * n_tiles, g = tile / per, first = g * group, gm = min(group, m_units - first);
  const int local = tile - g * per;
  nt = local / gm;
  mu = first + local - nt * gm;
}

// ESIZE: bytes of an element of y.
template <int CG, bool GATED, int ESIZE>
__global__ void __launch_bounds__(ManyCfg<CG>::THREADS, 1)
    k_e4m3_many(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                const __grid_constant__ CUtensorMap tmW3, const __grid_constant__ CUtensorMap tmY,
                const __grid_constant__ CUtensorMap tmRes, GemmArgs a, int m_units, int n_tiles, int group, int stream, int* err) {
  using C = ManyCfg<CG>;
  constexpr int STAGES = C::STAGES;
  constexpr int COLS = GATED ? 128 : 256;               // columns of y per tile
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {                         // (every CTA alike; the tiles' swizzle needs it)
    if (threadIdx.x == 0) atomicOr(err, TB_DEVERR_TIMEOUT);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* sfull = empty + STAGES;                     // scale sets
  uint64_t* sempty = sfull + 2;                         // ... copied to tensor memory
  uint64_t* sdone = sempty + 2;                         // ... and used there
  uint64_t* tfull = sdone + 2;                         // accumulators
  uint64_t* tempty = tfull + 2;
  uint64_t* shared_free = tempty + 2;                   // the columns both accumulators use
  uint64_t* rfull = shared_free + 1;                    // residual pieces, two for each epilogue warp
  uint64_t* efull = rfull + 16;                         // exponents of both halves of 32 rows
  uint64_t* drain = efull + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * STAGES + 32) * 8 + 8 <= 384, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = m_units * n_tiles;
  const int kblocks = (a.K + kBlk - 1) / kBlk, nsets = (kblocks + kSet - 1) / kSet;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;
  const int tile0 = CG == 2 ? (int)cluster_id_x() : (int)blockIdx.x, tstep = CG == 2 ? (int)nclusters_x() : (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], CG == 2 && rank == 0 ? 5 : 4);   // this CTA's four warps, and the odd CTA's warp 1
      mbar_init(&sempty[s], 1);
      mbar_init(&sdone[s], 1);
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 8 * CG);  // eight epilogue warps
    }
    mbar_init(shared_free, 4 * CG);
    for (int i = 0; i < 16; ++i) mbar_init(&rfull[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&efull[i], 2);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmW);
    if (GATED) prefetch_tmap(&tmW3);
    prefetch_tmap(&tmY);
  }
  // both CTAs' barriers exist before either CTA's copies or commits reach them
  __syncthreads();
  if (CG == 2) cluster_sync();
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
    pdl_trigger();                        // (only now: common.cuh)
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto commit = [](uint32_t bar, uint32_t elected) {
    if constexpr (CG == 2) mma_commit_pair_elected(bar, elected);
    else mma_commit_elected(bar, elected);
  };

  if (warp == 0) {
    // (the whole warp, its elected lane issuing)
    pdl_wait();
    const uint32_t elected = elect_one();
    const uint64_t first = policy_evict_first();
    const uint32_t ring = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
    const uint32_t even0 = CG == 2 ? mapa_shared(full0, 0) : full0;    // a pair's bytes complete on its even CTA's barriers
    uint32_t stage = 0, phase = 0;
    int issued = 0;
    uint32_t acc = 0;
    bool ok = true;
    for (int tile = tile0; ok && tile < tiles; tile += tstep, acc ^= 1) {
      // the first 128 rows of B, of a pair those of this CTA; the others of a single CTA
      const CUtensorMap *tw = GATED && rank != acc ? &tmW3 : &tmW, *tw2 = GATED && !acc ? &tmW3 : &tmW;
      int mu, nt;
      place(tile, m_units, n_tiles, group, mu, nt);
      const int xrow = (mu * CG + (int)rank) * kRowsCta;      // a block past M reads zeros
      const int wrow = GATED ? nt * 128 : nt * 256 + (int)rank * 128;
#pragma unroll 1
      for (int kb = 0; kb < kblocks; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_try_wait(empty0 + stage * 8, phase ^ 1u)) &&
            !(ok = mbar_wait_warp(&empty[stage], phase ^ 1u, abort_flag, err)))
          break;
        const uint32_t sa = ring + stage * C::STAGE_BYTES, bar = even0 + stage * 8;
        if (rank == 0) mbar_expect_elected(full0 + stage * 8, CG * C::STAGE_BYTES, elected);
        if (stream) tma_load_3d_elected<CG>(&tmX, sa, bar, kb * kBlk, xrow, 0, first, elected);
        else tma_load_3d_elected<CG>(&tmX, sa, bar, kb * kBlk, xrow, 0, elected);
        tma_load_3d_elected<CG>(tw, sa + C::A_BYTES, bar, kb * kBlk, wrow, 0, elected);
        if constexpr (CG == 1)
          tma_load_3d_elected<CG>(tw2, sa + C::A_BYTES + 128 * kBlk, bar, kb * kBlk, GATED ? wrow : wrow + 128, 0, elected);
        if (issued < STAGES) ++issued;
        if (++stage == STAGES) stage = 0, phase ^= 1u;
      }
    }
    // every copy must have landed before the CTA may exit (the odd CTA waits for the even
    // one at the cluster barrier)
    if (rank == 0) {
      volatile int no_abort = 0;
      for (int i = 0; i < issued; ++i) {
        if (stage == 0) stage = STAGES, phase ^= 1u;
        --stage;
        mbar_wait_warp(&full[stage], phase, &no_abort, err);
      }
    }
  } else if (warp == 1) {
    // The whole warp walks the blocks; its elected lane issues (mma_mx_k128).
    pdl_wait();                           // (the limit of its waits is for this kernel's work)
    if (rank == 0) {
      const uint32_t elected = elect_one();
      const uint64_t desc = desc_kmajor_sw128(smem_u32(smem));
      const uint32_t desc_hi = (uint32_t)(desc >> 32), desc0 = (uint32_t)desc;
      constexpr uint32_t NEXT = C::STAGE_BYTES >> 4;      // in a descriptor's address field
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      uint32_t stage = 0, phase = 0, set = 0;             // set: scale sets used so far
      int local = 0;
      bool ok = true;
      for (int tile = tile0; ok && tile < tiles; tile += tstep, ++local) {
        const int acc = local & 1;
        if (!mbar_wait_warp(&tempty[acc], ((local >> 1) & 1) ^ 1u, abort_flag, err)) break;
        const uint32_t d = tmem + acc * C::ACC1;
        for (int kb = 0; ok && kb < kblocks; kb += kSet, ++set) {
          const uint32_t sb = set & 1, sf = tmem + C::SETS_AT + sb * C::SET_COLS;
          if (!(ok = mbar_wait_cluster_warp(&sfull[sb], (set >> 1) & 1, abort_flag, err))) break;
          // the place in tensor memory: free when the set before the last is done, while the last
          // one's instructions run
          if (!(ok = mbar_wait_warp(&sdone[sb], ((set >> 1) & 1) ^ 1u, abort_flag, err))) break;
          const uint32_t at = smem_u32(smem) + C::OFF_SF + sb * C::SF_BYTES;
          tmem_copy_elected<CG>(sf, desc_rows16(at, 128), elected);
          tmem_copy_elected<CG>(sf + 4, desc_rows16(at + C::SF_W, 0), elected);
          tmem_copy_elected<CG>(sf + 8, desc_rows16(at + C::SF_W + 128, 0), elected);
          commit(smem_u32(&sempty[sb]), elected);
          // (after the scales: the tile before holds the shared columns up a little longer)
          if (kb == 0 && local && !(ok = mbar_wait_warp(shared_free, (local - 1) & 1, abort_flag, err))) break;
#pragma unroll
          for (int b = 0; b < kSet; ++b) {
            if (kb + b < kblocks) {
              if (!__all_sync(0xffffffffu, mbar_try_wait(full0 + stage * 8, phase)) &&
                  !(ok = mbar_wait_warp(&full[stage], phase, abort_flag, err)))
                break;
              tc_fence_after();
              const uint32_t lo = desc0 + stage * NEXT;
              mma_mx_k128<CG>(d, lo, lo + (C::A_BYTES >> 4), desc_hi, idesc_mx_e4m3(CG * kRowsCta, 256, b), sf, sf + 4,
                           kb + b != 0, elected);
              commit(empty0 + stage * 8, elected);      // frees the stage in both CTAs
              if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
          }
          commit(smem_u32(&sdone[sb]), elected);
        }
        if (ok) commit(smem_u32(&tfull[acc]), elected);
      }
      // all of them must be done before tensor memory is released
      commit(smem_u32(drain), elected);
      volatile int no_abort = 0;
      mbar_wait_warp(drain, 0, &no_abort, err);
    } else {
      // The issuing warp has this CTA's scales copied too, from this CTA's shared memory: what
      // the scale warps wrote and this one has seen is released to it at cluster scope.  (By
      // the scale warps themselves, who have loads on their way: 16384 x 768 x 768 16.7 us
      // for 13.2.)
      const uint32_t even[2] = {mapa_shared(smem_u32(&sfull[0]), 0), mapa_shared(smem_u32(&sfull[1]), 0)};
      bool ok = true;
      int set = 0;
      for (int tile = tile0; ok && tile < tiles; tile += tstep) {
        for (int s = 0; s < nsets; ++s, ++set) {
          if (!(ok = mbar_wait_warp(&sfull[set & 1], (set >> 1) & 1, abort_flag, err))) break;
          if (lane == 0) mbar_arrive_release_cluster(even[set & 1]);
        }
      }
    }
  } else if (warp >= 10) {
    // Scales: a word for a row of X per lane, and of two warps one for a half of W.  Those of
    // set s + 1 are requested before the wait for set s's place.
    pdl_wait();
    const int c = warp & 3;
    uint8_t* put = smem + C::OFF_SF;
    const int nb = (a.N + kBlk - 1) / kBlk;
    int set = 0;
    int tile = tile0, s = 0, acc = 0;
    uint32_t x = 0, w = 0;
    auto load = [&]() {
      int mu, nt;
      place(tile, m_units, n_tiles, group, mu, nt);
      const int kb = s * kSet, n = min(kSet, kblocks - kb);
      const int m = (mu * CG + (int)rank) * kRowsCta + c * 32 + lane, b = GATED ? nt : 2 * nt + c;
      x = m < a.M ? scale_word(a.x.scale + (size_t)m * kblocks + kb, n) : 0x7f7f7f7fu;
      if (c < 2) w = b < nb ? scale_word((GATED && c != acc ? a.w3.scale : a.w.scale) + (size_t)b * kblocks + kb, n) : 0x7f7f7f7fu;
    };
    bool more = tile < tiles;
    if (more) load();
    for (; more; ++set) {
      if (!mbar_wait_warp(&sempty[set & 1], ((set >> 1) & 1) ^ 1u, abort_flag, err)) break;
      uint8_t* to = put + (set & 1) * C::SF_BYTES;
      *reinterpret_cast<uint32_t*>(to + 16 * lane + 4 * c) = x;
      if (c < 2) *reinterpret_cast<uint32_t*>(to + C::SF_W + 128 * c + 4 * lane) = w;
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sfull[set & 1]);
      if (++s == nsets) s = 0, tile += tstep, acc ^= 1;
      more = tile < tiles;
      if (more) load();
    }
  } else {
    // Epilogue: a lane has half a row of the tile, a warp 32 of those.  A piece of 64 bytes
    // of each goes through shared memory (64-byte swizzle) to a TMA store, which drops what
    // lies past M or N; the next piece's residual is on its way into the other buffer
    // meanwhile, the next tile's first one before its sums are there.
    pdl_wait();
    const int quad = warp & 3, w = warp - 2, half = w >> 2;
    uint8_t* buf = smem + C::OFF_EPI + w * 2 * C::PIECE;
    const uint32_t tempty_cl[2] = {mapa_shared(smem_u32(&tempty[0]), 0), mapa_shared(smem_u32(&tempty[1]), 0)};
    const uint32_t shared_cl = mapa_shared(smem_u32(shared_free), 0);
    constexpr int CHUNKS = COLS / 64, PER = ESIZE == 4 ? 2 : 1;      // of 32 columns; pieces of one
    constexpr int wide = 64 / ESIZE, pieces = ESIZE == 1 ? 1 : CHUNKS * PER;
    const bool res = !GATED && a.res;
    // The half's chunk k in accumulator `acc`, the one with the shared columns first: the last
    // of accumulator 0, the first of accumulator 1; and the first column of its piece i.
    auto chunk_of = [&](int k, int acc) { return acc || !half ? k : (k == 0 ? CHUNKS - 1 : k - 1); };
    auto piece_at = [&](int i, int acc) { return ESIZE == 1 ? 0 : chunk_of(i / PER, acc) * 32 + i % PER * wide; };
    // first row and column of the warp's part of a tile
    auto corner = [&](int tile) {
      int mu, nt;
      place(tile, m_units, n_tiles, group, mu, nt);
      return make_int2((mu * CG + (int)rank) * kRowsCta + quad * 32, nt * COLS + half * (COLS / 2));
    };
    uint32_t n = 0, rphase = 0;        // pieces so far; bit b: the parity of buffer b's next residual
    auto request = [&](int row, int col, uint32_t b) {
      if (row >= a.M || col >= a.N || lane != 0) return;
      mbar_arrive_expect_tx(&rfull[w * 2 + b], C::PIECE);
      if (stream) tma_load_3d_hint(&tmRes, buf + b * C::PIECE, &rfull[w * 2 + b], col * ESIZE, row, 0, policy_evict_first());
      else tma_load_3d(&tmRes, buf + b * C::PIECE, &rfull[w * 2 + b], col * ESIZE, row, 0);
    };
    int2 at = corner(tile0), next = at;
    if (res) request(at.x, at.y + piece_at(0, 0), 0);
    bool ok = true;
    int local = 0;
    for (int tile = tile0; ok && tile < tiles; tile += tstep, ++local, at = next) {
      const int acc = local & 1;
      if (!(ok = mbar_wait_warp(&tfull[acc], (local >> 1) & 1, abort_flag, err))) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + acc * C::ACC1 + half * (COLS / 2);
      // Chunk k: 32 columns of this lane's row, finished but for the residual.
      auto take = [&](int k, bool free_all, float (&v)[32]) {
        const uint32_t from = taddr + chunk_of(k, acc) * 32;
        const bool free_shared = k == 0 && half != acc;
        uint32_t r[32], u[32];
        // what the gates gate, which is what lies in the shared columns, before the gates: gated
        // 8192 x 2048 x 768 25.5 us together, 24.3 so
        if constexpr (GATED) tmem_ld32(from + (acc ? 0 : 128), u);
        else tmem_ld32(from, r);
        if (free_shared) {
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(shared_cl);
        }
        if constexpr (GATED) tmem_ld32(from + (acc ? 128 : 0), r);
        tmem_wait_ld();
        if (free_all) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty_cl[acc]);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j)
          v[j] = !GATED ? __uint_as_float(r[j])
                 : ESIZE == 4 ? gated(__uint_as_float(r[j]), __uint_as_float(u[j]))
                              : gated_short(__uint_as_float(r[j]), __uint_as_float(u[j]));
      };
      const int row = at.x;
      uint8_t* mine = nullptr;           // this lane's row of the current piece
      // its 16-byte part p lies at p ^ (row / 2 % 4)
      auto part = [&](int p) { return reinterpret_cast<uint4*>(mine + ((p ^ (lane >> 1 & 3)) << 4)); };
      // Piece i, into a buffer that its last store has left and that holds the residual.
      auto open = [&](int i) {
        const uint32_t b = n & 1;
        mine = buf + b * C::PIECE + lane * 64;
        if (!res) {
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          return;
        }
        // (the next piece's is requested once the store before this one has left its buffer)
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        if (i + 1 == pieces) request(next.x, next.y + piece_at(0, acc ^ 1), b ^ 1);
        else request(row, at.y + piece_at(i + 1, acc), b ^ 1);
        if (row < a.M && at.y + piece_at(i, acc) < a.N) {
          ok = mbar_wait_warp(&rfull[w * 2 + b], rphase >> b & 1, abort_flag, err);
          rphase ^= 1u << b;
        }
      };
      auto close = [&](int i) {
        const int col = at.y + piece_at(i, acc);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          if (row < a.M && col < a.N) {
            if (stream) tma_store_3d_hint(&tmY, buf + (n & 1) * C::PIECE, col * ESIZE, row, 0, policy_evict_first());
            else tma_store_3d(&tmY, buf + (n & 1) * C::PIECE, col * ESIZE, row, 0);
          }
          bulk_commit();
        }
        ++n;
      };
      // All loops here stay loops: unrolled, their code was fetched anew for each tile
      // (gated 16384 x 768 x 768 33.6 us, 26.0 so with four warps).  The chunk that reaches
      // into the shared columns comes first, and addresses after it.
      if constexpr (ESIZE == 1) {
        // The values go back to tensor memory, into those of their columns that no other tile
        // uses, until the row's scale is known; the two warps of a row exchange exponents.
        const uint32_t keep = taddr + (acc ? 128 : 0);
        float top = 0.f;
#pragma unroll 1
        for (int q = 0; q < CHUNKS; ++q) {
          float v[32];
          take(q, false, v);
#pragma unroll
          for (int j = 0; j < 32; j += 2) top = fmax3(top, fabsf(v[j]), fabsf(v[j + 1]));
          tmem_st32(keep + chunk_of(q, acc) * 32, *reinterpret_cast<const uint32_t(*)[32]>(v));
        }
        next = tile + tstep < tiles ? corner(tile + tstep) : make_int2(a.M, 0);
        tmem_wait_st();
        const bool wild = top == INFINITY;           // an infinity: told from values one by one
        if (wild) top = 0.f;
        if (__any_sync(0xffffffffu, wild)) {
#pragma unroll 1
          for (int q = 0; q < CHUNKS; ++q) {
            uint32_t r[32];
            tmem_ld32(keep + q * 32, r);
            tmem_wait_ld();
            if (wild) {
#pragma unroll
              for (int j = 0; j < 32; ++j) top = fmaxf(top, finite_mag(__uint_as_float(r[j])));
            }
          }
        }
        // [accumulator][half][row]: a warp is here again two tiles later, past the other's
        // arrival of the tile between, which follows that one's reading
        volatile int8_t* exps = reinterpret_cast<volatile int8_t*>(smem + C::OFF_EXP) + acc * 256;
        const int half_e = block_exponent(top);
        exps[half * 128 + quad * 32 + lane] = (int8_t)half_e;
        __syncwarp();
        if (lane == 0) mbar_arrive(&efull[quad]);
        if (!(ok = mbar_wait_warp(&efull[quad], local & 1, abort_flag, err))) break;
        const int e = max(half_e, (int)exps[(half ^ 1) * 128 + quad * 32 + lane]);
        const float inv = pow2i(-e);
        open(0);
#pragma unroll 1
        for (int q = 0; q < CHUNKS; ++q) {
          uint32_t r[32], k[8];
          tmem_ld32(keep + q * 32, r);
          tmem_wait_ld();
          if (q == CHUNKS - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty_cl[acc]);
          }
          if (wild) {
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(to_code(__uint_as_float(r[j]), 1.f));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            k[j] = codes_of4(__uint_as_float(r[4 * j]) * inv, __uint_as_float(r[4 * j + 1]) * inv,
                             __uint_as_float(r[4 * j + 2]) * inv, __uint_as_float(r[4 * j + 3]) * inv);
          *part(2 * q) = make_uint4(k[0], k[1], k[2], k[3]);
          *part(2 * q + 1) = make_uint4(k[4], k[5], k[6], k[7]);
        }
        if (!half && row + lane < a.M) a.y_scale[(size_t)(row + lane) * n_tiles + at.y / 128] = (uint8_t)(e + 127);
        close(0);
      } else {
#pragma unroll 1
        for (int k = 0; ok && k < CHUNKS; ++k) {
          float v[32];
          take(k, k + 1 == CHUNKS, v);
          if (k == 0) next = tile + tstep < tiles ? corner(tile + tstep) : make_int2(a.M, 0);
#pragma unroll
          for (int h = 0; h < PER; ++h) {
            open(k * PER + h);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              uint4* to = part(p);
              if constexpr (ESIZE == 4) {
                const float* f = v + 16 * h + 4 * p;
                float4 t = make_float4(f[0], f[1], f[2], f[3]);
                if (res) {
                  const float4 r = *reinterpret_cast<const float4*>(to);
                  t = make_float4(t.x + r.x, t.y + r.y, t.z + r.z, t.w + r.w);
                }
                *reinterpret_cast<float4*>(to) = t;
              } else {
                float* f = v + 8 * p;
                if (res) {
                  const uint4 r = *to;
                  const uint32_t* rr = &r.x;
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    f[2 * j] += __uint_as_float(rr[j] << 16);
                    f[2 * j + 1] += __uint_as_float(rr[j] & 0xffff0000u);
                  }
                }
                uint4 o;
                uint32_t* oo = &o.x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
                  oo[j] = *reinterpret_cast<const uint32_t*>(&t);
                }
                *to = o;
              }
            }
            close(k * PER + h);
          }
        }
      }
    }
    // a residual that was requested lands before the CTA ends, whatever became of its sums
    if (!ok && res) {
      volatile int no_abort = 0;
      for (uint32_t b = 0; b < 2; ++b) mbar_wait(&rfull[w * 2 + b], rphase >> b & 1, &no_abort, err);
    }
    if (lane == 0) bulk_wait_all();
  }

  // Every instruction of the pair is done (the issuer waited on its drain) before
  // either CTA releases the pair's tensor memory.
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

template <int CG, bool GATED, int ESIZE> cudaError_t go(const GemmArgs& a, cudaStream_t s) {
  using C = ManyCfg<CG>;
  CUtensorMap tx, tw, tw3, ty, tr;
  cudaError_t e = make_tmap_rows(&tx, 1, a.x.codes, 1, (uint64_t)a.M, (uint64_t)a.K, kBlk, kRowsCta);
  if (e != cudaSuccess) return e;
  e = make_tmap_rows(&tw, 1, a.w.codes, 1, (uint64_t)a.N, (uint64_t)a.K, kBlk, 128);
  if (e != cudaSuccess) return e;
  tw3 = tw;
  if (GATED && (e = make_tmap_rows(&tw3, 1, a.w3.codes, 1, (uint64_t)a.N, (uint64_t)a.K, kBlk, 128)) != cudaSuccess)
    return e;
  // y and the residual by bytes: a piece is 64 of each of 32 rows
  const uint64_t row_bytes = (uint64_t)a.N * ESIZE;
  if ((e = make_tmap_rows(&ty, 1, a.y, 1, (uint64_t)a.M, row_bytes, 64, 32)) != cudaSuccess) return e;
  tr = ty;
  if (a.res && (e = make_tmap_rows(&tr, 1, a.res, 1, (uint64_t)a.M, row_bytes, 64, 32)) != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  static int clusters[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!clusters[dev]) {
    e = cudaFuncSetAttribute(k_e4m3_many<CG, GATED, ESIZE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    int n = 0;
    cfg.gridDim = dim3(CG * (sm_count() / CG));
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, k_e4m3_many<CG, GATED, ESIZE>, &cfg);
    if (e != cudaSuccess) return e;
    if (n <= 0) return cudaErrorNotSupported;
    clusters[dev] = n;
  }
  const int m_units = (int)((a.M + 1LL * CG * kRowsCta - 1) / (CG * kRowsCta));
  const int n_tiles = GATED ? (a.N + 127) / 128 : (a.N + 255) / 256;
  const long long tiles = (long long)m_units * n_tiles;
  if (tiles > 0x7fffffffLL / 2) return cudaErrorInvalidValue;
  // Weights beyond what L2 keeps, short rows: groups of 32 row units, so that a weight
  // tile is read once per group.  (Groups of 4, 8, 16 and 64 units for 16384 x 4096 x 14336,
  // which has none, 566, 561, 566 and 641 us for 564; for gated 8192 x 14336 x 4096 566, 548,
  // 540 and 534 for 533.)  Off and on, us: gated 8192 x 14336 x 4096 605 and 520, 16384 x 14336 x
  // 4096 620 and 597, gated 4096 x 14336 x 6144 508 and 425, 8192 x 14336 x 8192 718 and 580, 8192 x
  // 8192 x 8192 361 and 371, 8192 x 8192 x 14336 630 and 620; after seconds of load 16384 x 4096 x
  // 14336 627 and 671, so that long rows go without (though gated 4096 x 14336 x 10240 822 and 665).
  const size_t w_bytes = (size_t)a.N * a.K * (GATED ? 2 : 1);
  const int group = a.K <= 8192 && w_bytes > (size_t(48) << 20) && m_units > 1 ? std::min(m_units, 32) : 0;
  // Column tiles fastest and all of a row unit resident at once, y too large to stay in L2
  // for its reader: X, the residual and y pass through once and need not push the weights
  // out (16384 x 4096 x 14336 with the residual 539 -> 533 us, after seconds of load 632 ->
  // 619; X alone changes nothing.  In groups, where X is read again, 602 -> 711).
  const int stream = group == 0 && n_tiles <= clusters[dev] && (size_t)a.M * a.N * ESIZE > (size_t(64) << 20);
  cfg.gridDim = dim3(CG * (unsigned)std::min<long long>(tiles, clusters[dev]));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_e4m3_many<CG, GATED, ESIZE>, tx, tw, tw3, ty, tr, a, m_units, n_tiles, group, stream, device_error_word());
}

}  // namespace

cudaError_t launch_gemm_e4m3_many(const GemmArgs& a, bool one, cudaStream_t s) {
  if (one) return a.y_dtype == TB_F32 ? go<1, false, 4>(a, s) : go<1, false, 2>(a, s);
  return a.y_dtype == TB_F32 ? go<2, false, 4>(a, s) : go<2, false, 2>(a, s);
}
cudaError_t launch_gated_e4m3_many(const GemmArgs& a, bool one, cudaStream_t s) {
  if (one) return a.y_dtype == TB_E4M3 ? go<1, true, 1>(a, s) : a.y_dtype == TB_F32 ? go<1, true, 4>(a, s) : go<1, true, 2>(a, s);
  return a.y_dtype == TB_E4M3 ? go<2, true, 1>(a, s) : a.y_dtype == TB_F32 ? go<2, true, 4>(a, s) : go<2, true, 2>(a, s);
}

}  // namespace tb
