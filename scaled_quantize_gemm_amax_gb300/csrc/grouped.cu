// grouped.cu -- products of FP8 matrices grouped by expert, on the 5th-generation tensor cores.
//
//   rows   C[r, n]    = sum_k deq(A)[r, k] deq(B_e)[n, k]       for the rows r of expert e's segment
//   depth  C[e][m, n] = sum over r in e's segment of deq(A)[m, r] deq(B)[n, r]
// Segments are [offsets[e], offsets[e + 1]), multiples of 128 rows known on the device only: every
// CTA reads the offsets, sums up the experts' tiles and walks the tiles of all experts as one list,
// so a call is one launch and the host never waits for a routing.
//
// Per-tensor scales multiply the accumulator in the epilogue; MXFP8's are applied by the tensor
// core (kind::mxf8f6f4.block_scale).  Accumulation is binary32 in TMEM.
//
// Structure of a CTA, as the ungrouped product's: warp 0 fetches tiles by TMA into a ring of
// stages, warp 1 issues the MMAs, with MXFP8 a further warp copies scale factors into TMEM, eight
// warps drain the accumulator.  Every wait is bounded (ptx.cuh).
#include <atomic>
#include <cstring>

#include "gemm_util.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8q {

namespace {

using namespace gemm_util;

constexpr int kRows = 128;             // rows of A that a CTA holds, and of a segment's granularity
constexpr int kDepth = 128;            // K of a stage
constexpr int kUmmaDepth = 32;         // K of one MMA of 8-bit operands
constexpr int kEpi = 8;                // epilogue warps
constexpr uint32_t kTmemAll = 512;

// PAIR: two CTAs share a 256 x 256 tile (cta_group::2), each with its 128 rows of A and half of B's.
// Otherwise one CTA a 128 x BN tile.
template <int KIND, bool PAIR, int BN>
struct GroupedLayout {
  static constexpr bool MX = KIND == kMx;
  static constexpr int S = 5;   // stages
  static constexpr int ACC = MX && BN == 256 ? 1 : 2;   // accumulators; a wide MX one leaves TMEM for one and the scale factors
  static constexpr uint32_t A_BYTES = kRows * kDepth, B_BYTES = (PAIR ? BN / 2 : BN) * kDepth;
  static constexpr uint32_t STAGE = A_BYTES + B_BYTES;
  static constexpr int B_ATOMS = BN / 128;
  static constexpr uint32_t SF = MX ? 512 * (1 + B_ATOMS) : 0;
  static constexpr uint32_t OFF_SF = S * STAGE;
  static constexpr uint32_t OFF_STG = (OFF_SF + S * SF + 1023) & ~1023u;   // a 4 KB box an epilogue warp
  static constexpr uint32_t OFF_FULL = OFF_STG + kEpi * 4096, OFF_EMPTY = OFF_FULL + 8 * S, OFF_SFR = OFF_EMPTY + 8 * S;
  static constexpr uint32_t OFF_TFULL = OFF_SFR + 8 * S, OFF_TEMPTY = OFF_TFULL + 16, OFF_FINAL = OFF_TEMPTY + 16;
  static constexpr uint32_t OFF_TMEM = OFF_FINAL + 8, OFF_ABORT = OFF_TMEM + 4;
  static constexpr uint32_t OFF_TABLE = OFF_ABORT + 8;   // offsets [E + 1], first tiles [E + 1]
  static constexpr uint32_t FIXED = OFF_TABLE + 1024;    // + alignment slack
  static constexpr uint32_t TX = (PAIR ? 2 : 1) * (STAGE + SF);   // bytes that complete a stage
  static constexpr uint32_t SF_COL = BN * ACC;           // first TMEM column of the scale factors
  static constexpr uint32_t SF_COLS = 4 + 4 * B_ATOMS;   // of a stage
  static_assert(SF_COL + (MX ? S * SF_COLS : 0) <= kTmemAll, "TMEM");
};
constexpr uint32_t table_bytes(int n_experts) { return 8u * static_cast<uint32_t>(n_experts + 1); }
static_assert(GroupedLayout<kTensor, true, 256>::FIXED + table_bytes(kMaxExperts) <= 232448, "shared memory");
static_assert(GroupedLayout<kMx, true, 256>::FIXED + table_bytes(kMaxExperts) <= 232448, "shared memory");

// warps: producer, MMA issuer, kEpi epilogue warps, and with MXFP8 the scale factors' copier
template <int KIND>
constexpr int grouped_threads() { return 32 * (2 + kEpi + (KIND == kMx ? 1 : 0)); }

// One tile of the list.
struct Tile {
  int e;             // expert
  int a_row, a_kb;   // this CTA's first row of A, and the first 128-deep block
  int b_row, b_kb;   // the tile's first row of B and its first block
  int nkb;           // blocks
  int c_row, c_col;  // this CTA's first row of C, the tile's first column
  bool held;         // whether this CTA's rows belong to the expert (of the last half tile, the second CTA's do not)
};

template <int KIND, bool PAIR, int BN>
__global__ void __launch_bounds__(grouped_threads<KIND>(), 1)
    k_grouped(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const __grid_constant__ CUtensorMap tm_sfa, const __grid_constant__ CUtensorMap tm_sfb,
              const __grid_constant__ CUtensorMap tm_c, const GroupedParams p) {
  using L = GroupedLayout<KIND, PAIR, BN>;
  constexpr bool MX = L::MX;
  constexpr int S = L::S, ACC = L::ACC, TM = PAIR ? 2 * kRows : kRows;
  constexpr int kCopier = 2 + kEpi;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - smem_u32(smem_raw));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(base_ptr + L::OFF_ABORT);
  int* const offs = reinterpret_cast<int*>(base_ptr + L::OFF_TABLE);
  int* const first = offs + p.n_experts + 1;   // the experts' first tiles
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int unit = static_cast<int>(blockIdx.x) / (PAIR ? 2 : 1), units = static_cast<int>(gridDim.x) / (PAIR ? 2 : 1);
  const int tiles_n = (p.N + BN - 1) / BN;
  const bool depth = p.depth != 0;

  if (threadIdx.x == 0) {
    if (p.loads) {
      prefetch_tmap(&tm_a);
      prefetch_tmap(&tm_b);
    }
    for (int s = 0; s < S; ++s) {
      mbar_init(base + L::OFF_FULL + 8 * s, 1);
      mbar_init(base + L::OFF_EMPTY + 8 * s, 1);
      mbar_init(base + L::OFF_SFR + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(base + L::OFF_TFULL + 8 * a, 1);
      mbar_init(base + L::OFF_TEMPTY + 8 * a, PAIR ? 2 * kEpi : kEpi);
    }
    mbar_init(base + L::OFF_FINAL, MX ? 2 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(base + L::OFF_TMEM, kTmemAll);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(base + L::OFF_TMEM, kTmemAll);
      tmem_relinquish();
    }
  }
  pdl_wait();   // the offsets may come from the previous kernel in the stream
  if (warp == 2) {
    // The offsets checked and the experts' tiles summed up, 32 experts at a time.  Offsets that
    // are not ascending multiples of 128 within the capacity make the list empty.
    bool good = true;
    int sum = 0;
    for (int e0 = 0; e0 <= p.n_experts; e0 += 32) {
      const int e = e0 + lane;
      const int64_t lo = e <= p.n_experts ? p.offsets[e] : 0, hi = e < p.n_experts ? p.offsets[e + 1] : lo;
      const bool fine = lo >= 0 && lo <= hi && hi <= p.capacity && lo % kRows == 0 && hi % kRows == 0;
      good = __all_sync(0xFFFFFFFFu, fine) && good;
      int n = e < p.n_experts && fine ? (depth ? (p.M + TM - 1) / TM : static_cast<int>((hi - lo + TM - 1) / TM)) * tiles_n : 0;
      int before = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += v;
      }
      if (e <= p.n_experts) {
        offs[e] = static_cast<int>(lo);
        first[e] = sum + before - n;
      }
      sum += __shfl_sync(0xFFFFFFFFu, before, 31);
    }
    if (!good) {
      for (int e = lane; e <= p.n_experts; e += 32) first[e] = 0;
      if (lane == 0 && blockIdx.x == 0) atomicOr(p.err, kErrBadState);
      if (lane == 0) offs[p.n_experts] = static_cast<int>(p.capacity);   // no rows behind the last segment either
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();   // the peer's barriers are initialised before anyone signals them
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base_ptr + L::OFF_TMEM);
  const int ntiles = first[p.n_experts];

  // Tile t; `e` moves on from the expert of the tile before.
  auto tile_at = [&](int t, int& e) -> Tile {
    while (t >= first[e + 1]) ++e;
    const int lo = offs[e], rows = offs[e + 1] - lo, tiles_m = depth ? (p.M + TM - 1) / TM : (rows + TM - 1) / TM;
    int tm, tn;
    tile_coords<16>(t - first[e], tiles_m, tiles_n, tm, tn);
    const int row = tm * TM + static_cast<int>(rank) * kRows;
    Tile w;
    w.e = e;
    w.held = row < (depth ? p.M : rows);
    const int from = w.held ? row : row - kRows;   // rows that are not the expert's: the peer's once more, from L2
    w.c_col = tn * BN;
    if (depth) {
      w.a_row = from;
      w.a_kb = w.b_kb = lo / kDepth;
      w.nkb = rows / kDepth;
      w.b_row = tn * BN;
      w.c_row = e * p.M + row;
    } else {
      w.a_row = lo + from;
      w.a_kb = 0;
      w.nkb = p.K / kDepth;
      w.b_kb = p.b_cols ? e * w.nkb : 0;
      w.b_row = (p.b_cols ? 0 : e * p.N) + tn * BN;
      w.c_row = lo + row;
    }
    return w;
  };

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------ producer
    int issued = 0, stage = 0, e = 0;
    uint32_t phase = 0;
    bool ok = true;
    // atoms of a scale array's row of 128 rows
    const int a_atoms = p.a_cols / kDepth, b_atoms = p.b_cols_all / kDepth, b_last = p.b_rows_all / kRows - 1;
    for (int t = unit; t < ntiles && ok; t += units) {
      const Tile w = tile_at(t, e);
      for (int kb = 0; kb < w.nkb; ++kb) {
        if (!mbar_wait(base + L::OFF_EMPTY + 8 * stage, phase ^ 1u, p.err, kErrTimeoutStage, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t full = base + L::OFF_FULL + 8 * stage, sig = PAIR ? mapa_shared(full, 0) : full;
        const uint32_t sa = base + stage * L::STAGE, sf = base + L::OFF_SF + stage * L::SF;
        const int ak = w.a_kb + kb, bk = w.b_kb + kb;
        if (leader) mbar_arrive_expect_tx(full, L::TX);
        if (PAIR) {
          tma_load_2d_pair(sa, &tm_a, ak * kDepth, w.a_row, sig);
          tma_load_2d_pair(sa + L::A_BYTES, &tm_b, bk * kDepth, w.b_row + static_cast<int>(rank) * (BN / 2), sig);
        } else {
          tma_load_2d(sa, &tm_a, ak * kDepth, w.a_row, sig);
          tma_load_2d(sa + L::A_BYTES, &tm_b, bk * kDepth, w.b_row, sig);
        }
        if (MX) {
          const int atom_a = w.a_row / kRows * a_atoms + ak;
          if (PAIR) tma_load_2d_pair(sf, &tm_sfa, 0, 2 * atom_a, sig);
          else tma_load_2d(sf, &tm_sfa, 0, 2 * atom_a, sig);
#pragma unroll
          for (int h = 0; h < L::B_ATOMS; ++h) {
            // a tile that hangs over B's last row takes its last atoms (those columns are not stored)
            const int atom_b = min(w.b_row / kRows + h, b_last) * b_atoms + bk;
            if (PAIR) tma_load_2d_pair(sf + 512 + 512 * h, &tm_sfb, 0, 2 * atom_b, sig);
            else tma_load_2d(sf + 512 + 512 * h, &tm_sfb, 0, 2 * atom_b, sig);
          }
        }
        ++issued;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // this CTA's loads land before it exits: awaited through the stages' release by the MMAs that
    // follow them (a pair's land on the leader's barrier)
    for (int s = 0; s < S; ++s) {
      const int n = issued / S + (s < issued % S ? 1 : 0);
      if (n == 0) continue;
      if (PAIR)
        mbar_wait(base + L::OFF_EMPTY + 8 * s, static_cast<uint32_t>(n - 1) & 1u, p.err, kErrTimeoutStage, abort_flag);
      else
        mbar_wait(base + L::OFF_FULL + 8 * s, static_cast<uint32_t>(n - 1) & 1u, p.err, kErrTimeoutTmaLoad, nullptr);
    }
  } else if ((warp == 1 || (MX && warp == kCopier)) && lane == 0 && !leader) {
    // ------------------------------------------------ the peer issues no MMAs: it waits for the leader's last
    mbar_wait(base + L::OFF_FINAL, 0, p.err, kErrTimeoutMma, abort_flag);
  } else if (MX && warp == kCopier && lane == 0) {
    // ------------------------------------------------ scale factors into TMEM (leader)
    int stage = 0, e = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = unit; t < ntiles && ok; t += units) {
      const Tile w = tile_at(t, e);
      for (int kb = 0; kb < w.nkb; ++kb) {
        if (!mbar_wait(base + L::OFF_FULL + 8 * stage, phase, p.err, kErrTimeoutTmaLoad, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the stage's columns were last read by MMAs that finished before the stage was refilled
        const uint32_t sf = base + L::OFF_SF + stage * L::SF, col = tmem + L::SF_COL + static_cast<uint32_t>(stage) * L::SF_COLS;
#pragma unroll
        for (int h = 0; h <= L::B_ATOMS; ++h) {
          if (PAIR) tc_cp_32x128b_warpx4_pair(col + 4 * h, sdesc_rows16(sf + 512 * h));
          else tc_cp_32x128b_warpx4(col + 4 * h, sdesc_rows16(sf + 512 * h));
        }
        if (PAIR) tc_commit_pair_mc(base + L::OFF_SFR + 8 * stage, 1);
        else tc_commit(base + L::OFF_SFR + 8 * stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (PAIR) tc_commit_pair_mc(base + L::OFF_FINAL, 3);
    else tc_commit(base + L::OFF_FINAL);
    mbar_wait(base + L::OFF_FINAL, 0, p.err, kErrTimeoutMma, nullptr);
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------ MMA issuer (leader)
    const uint32_t shape = (static_cast<uint32_t>(p.e5m2_a) << 7) | (static_cast<uint32_t>(p.e5m2_b) << 10) |
                           (static_cast<uint32_t>(BN >> 3) << 17) | (static_cast<uint32_t>(TM >> 4) << 24);
    const uint32_t idesc = shape | (MX ? 1u << 23 : 1u << 4);
    auto commit = [&](uint32_t bar) {
      if (PAIR) tc_commit_pair_mc(bar, 3);
      else tc_commit(bar);
    };
    int stage = 0, e = 0;
    uint32_t phase = 0, acc_it = 0;
    bool ok = true;
    for (int t = unit; t < ntiles && ok; t += units) {
      const Tile w = tile_at(t, e);
      if (w.nkb == 0) continue;   // the epilogue stores 0 without an accumulator
      const uint32_t a = acc_it % ACC, parity = ((acc_it / ACC) & 1u) ^ 1u;
      const uint32_t bar = base + L::OFF_TEMPTY + 8 * a;
      if (!(PAIR ? mbar_wait_cluster(bar, parity, p.err, kErrTimeoutMma, abort_flag)
                 : mbar_wait(bar, parity, p.err, kErrTimeoutMma, abort_flag)))
        break;
      tc_fence_after();
      const uint32_t d = tmem + a * BN;
      for (int kb = 0; kb < w.nkb; ++kb) {
        // MXFP8: the copier's signal stands for the stage's data too
        if (!mbar_wait(base + (MX ? L::OFF_SFR : L::OFF_FULL) + 8 * stage, phase, p.err, kErrTimeoutTmaLoad, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sa = base + stage * L::STAGE, sb = sa + L::A_BYTES;
        const uint32_t sfa = tmem + L::SF_COL + static_cast<uint32_t>(stage) * L::SF_COLS, sfb = sfa + 4;
#pragma unroll
        for (int k = 0; k < kDepth / kUmmaDepth; ++k) {
          const uint64_t da = sdesc_k_sw128(sa + k * kUmmaDepth), db = sdesc_k_sw128(sb + k * kUmmaDepth);
          const uint32_t more = (kb | k) != 0 ? 1u : 0u;
          if (MX) {
            const uint32_t id = idesc | (static_cast<uint32_t>(k) << 4) | (static_cast<uint32_t>(k) << 29);
            if (PAIR) tc_mma_mxf8f6f4_pair(d, da, db, id, sfa, sfb, more);
            else tc_mma_mxf8f6f4(d, da, db, id, sfa, sfb, more);
          } else {
            if (PAIR) tc_mma_f8f6f4_pair(d, da, db, idesc, more);
            else tc_mma_f8f6f4(d, da, db, idesc, more);
          }
        }
        commit(base + L::OFF_EMPTY + 8 * stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      commit(base + L::OFF_TFULL + 8 * a);
      ++acc_it;
    }
    // every MMA has finished before TMEM is released (in both CTAs of a pair)
    commit(base + L::OFF_FINAL);
    mbar_wait(base + L::OFF_FINAL, 0, p.err, kErrTimeoutMma, nullptr);
  } else if (warp >= 2 && warp < 2 + kEpi) {
    // ------------------------------------------------ epilogue
    constexpr int COLS = BN / (kEpi / 4), CH = COLS / 32;   // a thread's columns, in chunks of 32
    const int q = warp & 3, h = (warp - 2) >> 2;             // TMEM lane quarter and column half of this warp
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const uint32_t stg = base + L::OFF_STG + static_cast<uint32_t>(warp - 2) * 4096u;
    const bool fp32 = p.out_fp32 != 0;
    // This warp's 32 rows x 128 bytes at a time staged in its swizzled box for one TMA store; bf16
    // chunks go out in pairs.
    auto store_chunk = [&](const float (&v)[32], int c, int col, int row) {
      if (fp32 || (c & 1) == 0) {
        if (lane == 0) bulk_wait_read<0>();   // the box's previous store has read it
        __syncwarp();
      }
      const uint32_t rowb = stg + static_cast<uint32_t>(lane) * 128u;
      if (fp32) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          sts128(rowb + ((static_cast<uint32_t>(k) ^ (lane & 7u)) << 4), __float_as_uint(v[4 * k]),
                 __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3]));
      } else {
        const uint32_t k0 = (c & 1) * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          sts128(rowb + (((k0 + k) ^ (lane & 7u)) << 4), pack_bf16(v[8 * k], v[8 * k + 1]),
                 pack_bf16(v[8 * k + 2], v[8 * k + 3]), pack_bf16(v[8 * k + 4], v[8 * k + 5]),
                 pack_bf16(v[8 * k + 6], v[8 * k + 7]));
      }
      if (fp32 || (c & 1) == 1) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tm_c, stg, fp32 ? col + 32 * c : col + 32 * (c - 1), row);
          bulk_commit();
        }
      }
    };
    uint32_t acc_it = 0;
    int e = 0;
    for (int t = unit; t < ntiles; t += units) {
      const Tile w = tile_at(t, e);
      const int col = w.c_col + h * COLS, row = w.c_row + 32 * q;
      uint32_t r[CH][32];
      if (w.nkb > 0) {
        const uint32_t a = acc_it % ACC;
        // warp-uniform decision: the TMEM loads that follow are .sync.aligned
        if (!__all_sync(0xFFFFFFFFu,
                        mbar_wait(base + L::OFF_TFULL + 8 * a, (acc_it / ACC) & 1u, p.err, kErrTimeoutMma, abort_flag)))
          break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < CH; ++c) tc_ld_32x32b_x32(lane_base + a * BN + h * COLS + 32 * c, r[c]);
#pragma unroll
        for (int c = 0; c < CH; ++c) tc_wait_ld(r[c]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {   // the accumulator goes back before its values are stored
          const uint32_t bar = base + L::OFF_TEMPTY + 8 * a;
          if (PAIR && !leader) mbar_arrive_remote(mapa_shared(bar, 0));
          else mbar_arrive(bar);
        }
        ++acc_it;
      } else {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) r[c][j] = 0u;
      }
      if (!w.held) continue;
      float scale = 1.0f;
      if (!MX && w.nkb > 0) scale = __fmul_rn(*p.sa, p.sb[p.sb_step * w.e]);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (col + 32 * (c & ~1) >= p.N) break;   // N is a multiple of 128, a pair of chunks inside or outside
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = MX ? __uint_as_float(r[c][j]) : __fmul_rn(__uint_as_float(r[c][j]), scale);
        store_chunk(v, c, col, row);
      }
    }
    if (p.zero_tail && !depth) {
      // rows behind the last segment
      const int64_t row_bytes = static_cast<int64_t>(p.N) * (fp32 ? 4 : 2), total = p.capacity * row_bytes;
      const int64_t step = static_cast<int64_t>(gridDim.x) * (32 * kEpi) * 16;
      for (int64_t at = offs[p.n_experts] * row_bytes + (static_cast<int64_t>(blockIdx.x) * (32 * kEpi) + threadIdx.x - 64) * 16;
           at < total; at += step)
        FP8Q_GUARD(at, 16, total, p.err) { stg128(static_cast<uint8_t*>(p.c) + at, 0u, 0u, 0u, 0u); }
    }
    if (lane == 0) bulk_wait_all<0>();   // this warp's stores have finished
  }

  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();   // no CTA leaves while its peer may still signal its barriers
  if (warp == 1) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem, kTmemAll);
    else tmem_dealloc(tmem, kTmemAll);
  }
}

template <int KIND, bool PAIR, int BN>
cudaError_t run_grouped(const GroupedParams& p, const GroupedMaps& m, int64_t tiles, int num_sms, cudaStream_t s) {
  using L = GroupedLayout<KIND, PAIR, BN>;
  auto kern = k_grouped<KIND, PAIR, BN>;
  static std::atomic<bool> attr_done[kMaxDevices] = {};
  cudaError_t e = ensure_smem_limit(kern, static_cast<int>(L::FIXED + table_bytes(kMaxExperts)), attr_done);
  if (e != cudaSuccess) return e;
  const size_t smem = L::FIXED + table_bytes(p.n_experts);
  int64_t units = num_sms;
  if (PAIR) {
    // resident pairs, queried once per device
    static std::atomic<int> resident[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (resident[dev].load(std::memory_order_relaxed) == 0) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(static_cast<unsigned>(num_sms / 2 * 2));
      cfg.blockDim = dim3(grouped_threads<KIND>());
      cfg.dynamicSmemBytes = L::FIXED + table_bytes(kMaxExperts);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) n = num_sms / 2;
      resident[dev].store(n < num_sms / 2 ? n : num_sms / 2, std::memory_order_relaxed);
    }
    units = resident[dev].load(std::memory_order_relaxed);
  }
  if (tiles < units) units = tiles;
  if (units < 1) units = 1;
  return launch_pdl(kern, dim3(static_cast<unsigned>(units * (PAIR ? 2 : 1))), dim3(grouped_threads<KIND>()), smem, s, PAIR ? 2 : 1,
                    m.a, m.b, m.sfa, m.sfb, m.c, p);
}

// the most tiles that a call can have, whatever its offsets are
int64_t most_tiles(const GroupedParams& p, int tile_rows, int tile_cols) {
  const int64_t tn = (p.N + tile_cols - 1) / tile_cols;
  if (p.depth) return static_cast<int64_t>(p.n_experts) * ((p.M + tile_rows - 1) / tile_rows) * tn;
  const int64_t blocks = p.capacity / kRows, used = p.n_experts < blocks ? p.n_experts : blocks;
  const int64_t per = tile_rows / kRows;
  return (blocks + used * (per - 1)) / per * tn;
}

}  // namespace

// CTA pairs halve what the tensor core reads of B from shared memory; with fewer than two tiles a pair
// the smaller tiles spread the work over more SMs (one token at 2 experts, 4096 -> 11008: 28.9 us
// against 33.3; 8192 tokens: 747 against 537).
int grouped_tile(const GroupedParams& p, int num_sms) { return most_tiles(p, 2 * kRows, 256) < num_sms ? 128 : 256; }

cudaError_t launch_grouped(const GroupedParams& p, const GroupedMaps& m, int tile, int num_sms, cudaStream_t s) {
  const bool mx = p.kind == kMx;
  if (tile == 256) {
    const int64_t tiles = most_tiles(p, 2 * kRows, 256);
    return mx ? run_grouped<kMx, true, 256>(p, m, tiles, num_sms, s) : run_grouped<kTensor, true, 256>(p, m, tiles, num_sms, s);
  }
  const int64_t tiles = most_tiles(p, kRows, tile);
  return mx ? run_grouped<kMx, false, 128>(p, m, tiles, num_sms, s) : run_grouped<kTensor, false, 128>(p, m, tiles, num_sms, s);
}

}  // namespace fp8q
