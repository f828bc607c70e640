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
// Structure of a CTA: two warps fetch A's and B's blocks by TMA into a ring of stages, one issues the
// MMAs, with MXFP8 a further one copies scale factors into TMEM, eight drain the accumulator.  The four work
// as converged warps with uniform operands: a 128-deep block issued by single lanes of a branch took 510 cycles, so
// 405 (128 rows, per-tensor; its four MMAs 256 to 550), and 64 experts of few rows 163 us, so 145.  Every wait is bounded (ptx.cuh).
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

// ------------------------------------------------------------------ the list of tiles
// The offsets checked and the experts' tiles summed up by one warp, 32 experts at a time: offs
// [E + 1] the offsets, first [E + 1] the experts' first tiles.  Offsets that are not ascending
// multiples of 128 within the capacity make the list empty.
__device__ __forceinline__ void list_tiles(const GroupedParams& p, int tile_rows, int tiles_n, int* offs, int* first, int lane) {
  bool good = true;
  int sum = 0;
  for (int e0 = 0; e0 <= p.n_experts; e0 += 32) {
    const int e = e0 + lane;
    const int64_t lo = e <= p.n_experts ? p.offsets[e] : 0, hi = e < p.n_experts ? p.offsets[e + 1] : lo;
    const bool fine = lo >= 0 && lo <= hi && hi <= p.capacity && lo % kRows == 0 && hi % kRows == 0;
    good = __all_sync(0xFFFFFFFFu, fine) && good;
    const int64_t rows = p.depth ? p.M : hi - lo;
    const int n = e < p.n_experts && fine ? static_cast<int>((rows + tile_rows - 1) / tile_rows) * tiles_n : 0;
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (e <= p.n_experts) {
      offs[e] = static_cast<int>(lo);
      first[e] = sum + upto - n;
    }
    sum += __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  if (!good) {
    __syncwarp();
    for (int e = lane; e <= p.n_experts; e += 32) first[e] = 0;
    if (lane == 0) {
      offs[0] = 0;   // no rows in front of the first segment and behind the last either
      offs[p.n_experts] = static_cast<int>(p.capacity);
      if (blockIdx.x == 0) atomicOr(p.err, kErrBadState);
    }
  }
}

// One tile of the list.
struct Tile {
  int e;             // expert
  int a_row, a_kb;   // this CTA's first row of A, and the first 128-deep block
  int b_row, b_kb;   // the tile's first row of B and its first block
  int nkb;           // blocks
  int c_row, c_col;  // this CTA's first row of C, the tile's first column
  bool held;         // whether this CTA's rows belong to the expert
  bool half;         // a pair's tile has 128 rows only: 64 a CTA (HALVES), or those of the first CTA alone
};

// Tile t for CTA `rank` of its unit; `e` moves on from the expert of the tile before.
template <int TILE_ROWS, bool HALVES>
__device__ __forceinline__ Tile tile_of(const GroupedParams& p, const int* offs, const int* first, int tile_cols, int tiles_n, int rank,
                                        int t, int& e) {
  while (t >= first[e + 1]) ++e;
  const int lo = offs[e], seg = offs[e + 1] - lo, rows = p.depth ? p.M : seg;
  int tm, tn;
  tile_coords<16>(t - first[e], (rows + TILE_ROWS - 1) / TILE_ROWS, tiles_n, tm, tn);
  Tile w;
  w.half = TILE_ROWS > kRows && tm * TILE_ROWS + kRows >= rows;
  const int row = tm * TILE_ROWS + rank * (HALVES && w.half ? kRows / 2 : kRows);
  w.e = e;
  w.held = row < rows;
  w.c_col = tn * tile_cols;
  if (p.depth) {
    w.a_row = row;
    w.a_kb = w.b_kb = lo / kDepth;
    w.nkb = seg / kDepth;
    w.b_row = w.c_col;
    w.c_row = e * p.M + row;
  } else {
    w.a_row = lo + row;
    w.a_kb = 0;
    w.nkb = p.K / kDepth;
    w.b_kb = p.b_cols ? e * w.nkb : 0;
    w.b_row = (p.b_cols ? 0 : e * p.N) + w.c_col;
    w.c_row = lo + row;
  }
  // in the place of rows that are not the expert's, rows behind A's last: TMA makes them zeros without reading, and
  // zeros cost the tensor core little power
  if (!w.held) w.a_row = p.a_rows;
  return w;
}

// Rows [from, to) of C set to 0, by the 32 * kEpi epilogue threads of every CTA.
__device__ __forceinline__ void zero_rows(const GroupedParams& p, int64_t from, int64_t to, int thread) {
  const int64_t row_bytes = static_cast<int64_t>(p.N) * (p.out_fp32 ? 4 : 2), end = to * row_bytes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (32 * kEpi) * 16;
  for (int64_t at = from * row_bytes + (static_cast<int64_t>(blockIdx.x) * (32 * kEpi) + thread) * 16; at < end; at += step)
    FP8Q_GUARD(at, 16, p.capacity * row_bytes, p.err) { stg128(static_cast<uint8_t*>(p.c) + at, 0u, 0u, 0u, 0u); }
}
// The rows outside the segments, as p.zero_tail asks.
__device__ __forceinline__ void zero_outside(const GroupedParams& p, const int* offs, int thread) {
  const int lo = offs[0], hi = offs[p.n_experts];
  if (p.zero_tail > 0 && hi < p.capacity) zero_rows(p, hi, p.capacity, thread);
  if (p.zero_tail > 1 && lo > 0) zero_rows(p, 0, lo, thread);
}

__host__ __device__ constexpr uint32_t table_bytes(int n_experts) { return 8u * static_cast<uint32_t>(n_experts + 1); }   // offs, first
constexpr uint32_t kSmem = 232448;

// warps: B's producer, MMA issuer, kEpi epilogue warps, A's producer, and with MXFP8 the scale factors' copier
template <int KIND>
constexpr int grouped_threads() { return 32 * (3 + kEpi + (KIND == kMx ? 1 : 0)); }
constexpr int kFetchA = 2 + kEpi, kCopier = 3 + kEpi;

// ------------------------------------------------------------------ many rows: CTA pairs
// Two CTAs share a 256 x 256 tile (cta_group::2), each with its 128 rows of A and half of B's.  Tiles go round the pairs in
// the order of the list, 16 of an expert's row tiles walking its columns together.
// Bound by the tensor core: 8 x 2176 rows, 4096 -> 11008, MXFP8 477 us (3290 TFLOP/s, 0.87 of twice the measured BF16
// rate), per-tensor 450 (3490); a pair's 128-deep block takes 560 to 620 cycles
// with all pairs at work, 490 alone.  64 experts of 256 rows, 2048 -> 4096, per-tensor 109 us (0.96 of HBM).
// An expert whose rows are an odd number of 128s has a last tile of 128: per-tensor one of 64 rows a CTA (64 experts, 4096 ->
// 2048, of 384 rows 151 us, with 256 rows, of which half are zeros, 161; of 256 and 384 in turn 128 and 133); MXFP8's scale
// factors come by atoms of 128 rows, and its tile keeps 256, zeros in the place of those that are not the expert's.
constexpr int kPairCols = 256;
// S stages: 6 with per-tensor scales and up to 200 experts (their table of segments shares the memory), else 5.  (8192
// tokens at 2 of 8 experts 452 -> 443 us, 64 experts of 256 rows 112 -> 110.6; with 4 stages 478 and 121.)
constexpr int kSixStageExperts = 200;
template <int KIND, int S>
struct PairLayout {
  static constexpr bool MX = KIND == kMx;
  static constexpr int ACC = MX ? 1 : 2; // accumulators; MXFP8's scale factors leave TMEM for one
  static constexpr uint32_t A_BYTES = kRows * kDepth, B_BYTES = kPairCols / 2 * kDepth, STAGE = A_BYTES + B_BYTES;
  static constexpr int B_ATOMS = kPairCols / 128;
  static constexpr uint32_t SF = MX ? 512 * (1 + B_ATOMS) : 0;
  static constexpr uint32_t OFF_SF = S * STAGE;
  static constexpr uint32_t OFF_STG = (OFF_SF + S * SF + 1023) & ~1023u;   // a 4 KB box an epilogue warp
  static constexpr uint32_t OFF_FULL = OFF_STG + kEpi * 4096, OFF_EMPTY = OFF_FULL + 8 * S, OFF_SFR = OFF_EMPTY + 8 * S;
  static constexpr uint32_t OFF_TFULL = OFF_SFR + 8 * S, OFF_TEMPTY = OFF_TFULL + 16, OFF_FINAL = OFF_TEMPTY + 16;
  static constexpr uint32_t OFF_TMEM = OFF_FINAL + 8, OFF_ABORT = OFF_TMEM + 4, OFF_TABLE = OFF_ABORT + 4;
  static constexpr uint32_t FIXED = OFF_TABLE + 1024;    // + alignment slack
  static constexpr uint32_t TX = 2 * (STAGE + SF);       // bytes of both CTAs that complete a stage
  static constexpr uint32_t TX_HALF = TX - (MX ? 0 : A_BYTES);   // of a tile of 128 rows
  static constexpr uint32_t SF_COL = kPairCols * ACC;    // first TMEM column of the scale factors
  static constexpr uint32_t SF_COLS = 4 + 4 * B_ATOMS;   // of a stage
  static_assert(SF_COL + (MX ? S * SF_COLS : 0) <= kTmemAll, "TMEM");

};

template <int KIND, int S>
__global__ void __launch_bounds__(grouped_threads<KIND>(), 1)
    k_grouped(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const __grid_constant__ CUtensorMap tm_sfa, const __grid_constant__ CUtensorMap tm_sfb,
              const __grid_constant__ CUtensorMap tm_c, const GroupedParams p) {
  using L = PairLayout<KIND, S>;
  constexpr bool MX = L::MX;
  constexpr int ACC = L::ACC, TM = 2 * kRows, BN = kPairCols;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - smem_u32(smem_raw));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(base_ptr + L::OFF_ABORT);
  int* const offs = reinterpret_cast<int*>(base_ptr + L::OFF_TABLE);
  int* const first = offs + p.n_experts + 1;   // the experts' first tiles
  const int warp = warp_uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint32_t rank = warp_uniform(cluster_ctarank());
  const bool leader = rank == 0;
  const int unit = static_cast<int>(blockIdx.x) / 2, units = static_cast<int>(gridDim.x) / 2;
  const int tiles_n = (p.N + BN - 1) / BN;

  if (threadIdx.x == 0) {
    if (p.loads) {
      prefetch_tmap(&tm_a);
      prefetch_tmap(&tm_b);
      prefetch_tmap(&tm_sfa);
    }
    for (int s = 0; s < S; ++s) {
      mbar_init(base + L::OFF_FULL + 8 * s, 1);
      mbar_init(base + L::OFF_EMPTY + 8 * s, 1);
      mbar_init(base + L::OFF_SFR + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(base + L::OFF_TFULL + 8 * a, 1);
      mbar_init(base + L::OFF_TEMPTY + 8 * a, 2 * kEpi);
    }
    mbar_init(base + L::OFF_FINAL, MX ? 2 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(base + L::OFF_TMEM, kTmemAll);
    tmem_relinquish_pair();
  }
  pdl_wait();   // the offsets may come from the previous kernel in the stream
  if (warp == 2) list_tiles(p, TM, tiles_n, offs, first, lane);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the peer's barriers are initialised before anyone signals them
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = warp_uniform(*reinterpret_cast<volatile uint32_t*>(base_ptr + L::OFF_TMEM));
  const int ntiles = warp_uniform(first[p.n_experts]);

  auto tile_at = [&](int t, int& e) { return tile_of<TM, !MX>(p, offs, first, BN, tiles_n, static_cast<int>(rank), t, e); };

  if (warp == 0 || warp == kFetchA) {
    // ------------------------------------------------ producers (whole warps): B, and A, each with its scale factors
    const bool fetch_b = warp == 0;
    int issued = 0, stage = 0, e = 0;
    uint32_t phase = 0;
    bool ok = true;
    // atoms of a scale array's row of 128 rows
    const int a_atoms = p.a_cols / kDepth, b_atoms = p.b_cols_all / kDepth, b_last = p.b_rows_all / kRows - 1;
    for (int t = unit; t < ntiles && ok; t += units) {
      const Tile w = tile_at(t, e);
      const int nkb = warp_uniform(w.nkb), a_row = warp_uniform(w.a_row), b_row = warp_uniform(w.b_row);
      int x = warp_uniform(fetch_b ? w.b_kb : w.a_kb) * kDepth;
      int atom = warp_uniform(2 * (fetch_b ? b_row / kRows * b_atoms + w.b_kb : a_row / kRows * a_atoms + w.a_kb));
      // a tile that hangs over B's last row takes its last atoms twice (those columns are not stored)
      const int second = b_row / kRows < b_last ? 2 * b_atoms : 0;
      const uint32_t tx = warp_uniform(w.half ? L::TX_HALF : L::TX);
      const CUtensorMap* const map_a = !MX && w.half ? &tm_sfa : &tm_a;
      for (int kb = 0; kb < nkb; ++kb) {
        ok = warp_uniform(mbar_wait(base + L::OFF_EMPTY + 8 * stage, phase ^ 1u, p.err, kErrTimeoutStage, abort_flag));
        if (!ok) break;
        const uint32_t full = base + L::OFF_FULL + 8 * stage, sig = mapa_shared(full, 0);
        const uint32_t sa = base + stage * L::STAGE, sf = base + L::OFF_SF + stage * L::SF;
        if (fetch_b) {
          if (leader) mbar_arrive_expect_tx_warp(full, tx);
          tma_load_2d_pair_warp(sa + L::A_BYTES, &tm_b, x, b_row + static_cast<int>(rank) * (BN / 2), sig);
          if (MX) {
            tma_load_2d_pair_warp(sf + 512, &tm_sfb, 0, atom, sig);
            tma_load_2d_pair_warp(sf + 1024, &tm_sfb, 0, atom + second, sig);
          }
        } else {
          tma_load_2d_pair_warp(sa, map_a, x, a_row, sig);
          if (MX) tma_load_2d_pair_warp(sf, &tm_sfa, 0, atom, sig);
        }
        x += kDepth;
        atom += 2;
        ++issued;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // this CTA's loads land before it exits: awaited through the stages' release by the MMAs that
    // follow them (they land on the leader's barrier)
    for (int s = 0; s < S; ++s) {
      const int n = issued / S + (s < issued % S ? 1 : 0);
      if (n > 0) mbar_wait(base + L::OFF_EMPTY + 8 * s, static_cast<uint32_t>(n - 1) & 1u, p.err, kErrTimeoutStage, abort_flag);
    }
  } else if ((warp == 1 || (MX && warp == kCopier)) && !leader) {
    // ------------------------------------------------ the peer issues no MMAs: it waits for the leader's last
    if (lane == 0) mbar_wait(base + L::OFF_FINAL, 0, p.err, kErrTimeoutMma, abort_flag);
  } else if (MX && warp == kCopier) {
    // ------------------------------------------------ scale factors into TMEM (leader; the whole warp)
    int stage = 0, e = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = unit; t < ntiles && ok; t += units) {
      const int nkb = warp_uniform(tile_at(t, e).nkb);
      for (int kb = 0; kb < nkb; ++kb) {
        ok = warp_uniform(mbar_wait(base + L::OFF_FULL + 8 * stage, phase, p.err, kErrTimeoutTmaLoad, abort_flag));
        if (!ok) break;
        tc_fence_after();
        // the stage's columns were last read by MMAs that finished before the stage was refilled
        const uint32_t sf = base + L::OFF_SF + stage * L::SF, col = tmem + L::SF_COL + static_cast<uint32_t>(stage) * L::SF_COLS;
#pragma unroll
        for (int h = 0; h <= L::B_ATOMS; ++h) tc_cp_32x128b_warpx4_pair_warp(col + 4 * h, sdesc_rows16(sf + 512 * h));
        tc_commit_pair_mc_warp(base + L::OFF_SFR + 8 * stage, 1);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    tc_commit_pair_mc_warp(base + L::OFF_FINAL, 3);
    mbar_wait(base + L::OFF_FINAL, 0, p.err, kErrTimeoutMma, nullptr);
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (leader; the whole warp)
    const uint32_t shape = (static_cast<uint32_t>(p.e5m2_a) << 7) | (static_cast<uint32_t>(p.e5m2_b) << 10) |
                           (static_cast<uint32_t>(BN >> 3) << 17) | (static_cast<uint32_t>(TM >> 4) << 24);
    const uint32_t full_tile = shape | (MX ? 1u << 23 : 1u << 4);
    auto commit = [&](uint32_t bar) { tc_commit_pair_mc_warp(bar, 3); };
    int stage = 0, e = 0;
    uint32_t phase = 0, acc_it = 0;
    bool ok = true;
    for (int t = unit; t < ntiles && ok; t += units) {
      const Tile w = tile_at(t, e);
      const int nkb = warp_uniform(w.nkb);
      if (nkb == 0) continue;   // the epilogue stores 0 without an accumulator
      const uint32_t idesc = warp_uniform(full_tile - (!MX && w.half ? static_cast<uint32_t>(kRows >> 4) << 24 : 0u));
      const uint32_t a = acc_it % ACC, parity = ((acc_it / ACC) & 1u) ^ 1u;
      ok = warp_uniform(mbar_wait_cluster(base + L::OFF_TEMPTY + 8 * a, parity, p.err, kErrTimeoutMma, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + a * BN;
      for (int kb = 0; kb < nkb; ++kb) {
        // MXFP8: the copier's signal stands for the stage's data too
        ok = warp_uniform(
            mbar_wait(base + (MX ? L::OFF_SFR : L::OFF_FULL) + 8 * stage, phase, p.err, kErrTimeoutTmaLoad, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = base + stage * L::STAGE, sb = sa + L::A_BYTES;
        const uint32_t sfa = tmem + L::SF_COL + static_cast<uint32_t>(stage) * L::SF_COLS, sfb = sfa + 4;
#pragma unroll
        for (int k = 0; k < kDepth / kUmmaDepth; ++k) {
          const uint64_t da = sdesc_k_sw128(sa + k * kUmmaDepth), db = sdesc_k_sw128(sb + k * kUmmaDepth);
          const uint32_t more = (kb | k) != 0 ? 1u : 0u;
          if (MX) {
            const uint32_t id = idesc | (static_cast<uint32_t>(k) << 4) | (static_cast<uint32_t>(k) << 29);
            tc_mma_mxf8f6f4_pair_warp(d, da, db, id, sfa, sfb, more);
          } else {
            tc_mma_f8f6f4_pair_warp(d, da, db, idesc, more);
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
      // of 64 rows a CTA, TMEM has the first 128 columns in its lanes 0..63 and the others in 64..127
      const bool half = !MX && w.half;
      const int col = half ? w.c_col + (q >> 1) * (BN / 2) + h * (COLS / 2) : w.c_col + h * COLS;
      const int row = w.c_row + 32 * (half ? q & 1 : q), chunks = half ? CH / 2 : CH;
      const uint32_t from = lane_base + static_cast<uint32_t>(h * (half ? COLS / 2 : COLS));
      if (w.nkb > 0) {
        // warp-uniform decision: the TMEM loads that follow are .sync.aligned
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(base + L::OFF_TFULL + 8 * (acc_it % ACC), (acc_it / ACC) & 1u, p.err, kErrTimeoutMma,
                                               abort_flag)))
          break;
        tc_fence_after();
      }
      // A lone accumulator goes back before its values are stored, so all of them wait in registers;
      // one of two can take its time and the registers of half of them.
      constexpr int HOLD = ACC == 1 ? CH : CH / 2;
      float scale = 1.0f;
      if (!MX && w.nkb > 0) scale = __fmul_rn(*p.sa, p.sb[p.sb_step * w.e]);
#pragma unroll
      for (int c0 = 0; c0 < CH; c0 += HOLD) {
        uint32_t r[HOLD][32];
        if (w.nkb > 0) {
          const uint32_t a = acc_it % ACC;
#pragma unroll
          for (int c = 0; c < HOLD; ++c) tc_ld_32x32b_x32(from + a * BN + 32 * (c0 + c), r[c]);
#pragma unroll
          for (int c = 0; c < HOLD; ++c) tc_wait_ld(r[c]);
          if (c0 + HOLD == CH) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              const uint32_t bar = base + L::OFF_TEMPTY + 8 * a;
              if (!leader) mbar_arrive_remote(mapa_shared(bar, 0));
              else mbar_arrive(bar);
            }
            ++acc_it;
          }
        } else {
#pragma unroll
          for (int c = 0; c < HOLD; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) r[c][j] = 0u;
        }
        if (!w.held) continue;
#pragma unroll
        for (int c = 0; c < HOLD; ++c) {
          // N is a multiple of 128, a pair of chunks inside or outside
          if (c0 + c >= chunks || col + 32 * ((c0 + c) & ~1) >= p.N) break;
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = MX ? __uint_as_float(r[c][j]) : __fmul_rn(__uint_as_float(r[c][j]), scale);
          store_chunk(v, c0 + c, col, row);
        }
      }
    }
    zero_outside(p, offs, static_cast<int>(threadIdx.x) - 64);
    if (lane == 0) bulk_wait_all<0>();   // this warp's stores have finished
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();   // no CTA leaves while its peer may still signal its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemAll);
  }
}

// ------------------------------------------------------------------ few rows: one CTA a tile
// With few tiles the product is bound by streaming the experts' weights once, by every SM (one token at 2 of 8
// experts, 4096 -> 11008, MXFP8 20.7 us, 4.7 TB/s; 8 x 128 rows 67, 5.8 TB/s; 4 us are launch, first loads and the way out):
// a CTA takes a 128 x width tile, and the host picks the width for which the tiles divide evenly: a multiple of 32, with MXFP8 of
// 64, since a tile's scale factors then start at an even column of TMEM.
//
// What the stream of weights needs is bytes on their way (13 MB over all SMs), so B's blocks have a ring of
// their own, as deep as shared memory allows, and A's, which every tile reads from L2, a short one.  Each has a warp that
// fetches it; both complete the barrier of B's stage.
struct FewLayout {
  static constexpr uint32_t A_BYTES = kRows * kDepth;
  static constexpr int MAX_SB = 8;                       // blocks of B's ring at most
  static constexpr uint32_t SF_BYTES = 3 * 512;          // A's atom and up to two of B's, of a block
  static constexpr uint32_t OFF_FULL = 0, OFF_EMPTY = OFF_FULL + 8 * MAX_SB, OFF_SFR = OFF_EMPTY + 8 * MAX_SB;
  static constexpr uint32_t OFF_TFULL = OFF_SFR + 8 * MAX_SB, OFF_TEMPTY = OFF_TFULL + 16, OFF_FINAL = OFF_TEMPTY + 16;
  static constexpr uint32_t OFF_TMEM = OFF_FINAL + 8, OFF_ABORT = OFF_TMEM + 4, OFF_TABLE = OFF_ABORT + 4;
  static constexpr uint32_t SF_COL = 384, SF_COLS = 12;  // TMEM with MXFP8: accumulators below, scale factors from there on
  static_assert(SF_COL + MAX_SB * SF_COLS <= kTmemAll, "TMEM");
  __host__ __device__ static constexpr int accumulators(bool mx, int width) { return 2 * width <= static_cast<int>(mx ? SF_COL : kTmemAll) ? 2 : 1; }

  // Where the rest lies: scale factors, a box of 32 x 32 elements an epilogue warp, A's ring, B's ring.
  int width, sa, sb;
  uint32_t sf, stg, a, b, total;
  FewLayout(int width_, bool mx, bool fp32, int n_experts) : width(width_) {
    auto up = [](uint32_t v) { return (v + 1023) & ~1023u; };
    const uint32_t block = static_cast<uint32_t>(width) * kDepth + (mx ? SF_BYTES : 0), box = kEpi * (fp32 ? 4096 : 2048);
    sf = up(OFF_TABLE + table_bytes(n_experts));
    const uint32_t room = kSmem - 1024 - sf - box - 1024;   // alignment of the base and behind the scale factors
    // B's ring as deep as leaves A's at most one block less (with three of A's, tiles narrower than 192 columns wait for A:
    // 8 x 128 rows, 11008 columns, tiles of 128, 83 us instead of 72)
    sb = MAX_SB;
    while (sb > 4 && room < sb * block + (sb - 1) * A_BYTES) --sb;
    sa = static_cast<int>((room - sb * block) / A_BYTES);
    if (sa > sb) sa = sb;
    stg = up(sf + (mx ? static_cast<uint32_t>(sb) * SF_BYTES : 0));
    a = stg + box;
    b = a + static_cast<uint32_t>(sa) * A_BYTES;
    total = b + static_cast<uint32_t>(sb * width) * kDepth + 1024;
  }
};

template <int KIND>
__global__ void __launch_bounds__(grouped_threads<KIND>(), 1)
    k_grouped_few(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                  const __grid_constant__ CUtensorMap tm_sfa, const __grid_constant__ CUtensorMap tm_sfb,
                  const __grid_constant__ CUtensorMap tm_c, const GroupedParams p, const FewLayout l) {
  using L = FewLayout;
  constexpr bool MX = KIND == kMx;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - smem_u32(smem_raw));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(base_ptr + L::OFF_ABORT);
  int* const offs = reinterpret_cast<int*>(base_ptr + L::OFF_TABLE);
  int* const first = offs + p.n_experts + 1;
  const int width = l.width, S = l.sb, SA = l.sa;
  const uint32_t b_bytes = static_cast<uint32_t>(width) * kDepth;
  const int warp = warp_uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int unit = static_cast<int>(blockIdx.x), units = static_cast<int>(gridDim.x);
  const int tiles_n = (p.N + width - 1) / width, ACC = L::accumulators(MX, width);

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
      mbar_init(base + L::OFF_TEMPTY + 8 * a, kEpi);
    }
    mbar_init(base + L::OFF_FINAL, MX ? 2 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(base + L::OFF_TMEM, kTmemAll);
    tmem_relinquish();
  }
  pdl_wait();   // the offsets may come from the previous kernel in the stream
  if (warp == 2) list_tiles(p, kRows, tiles_n, offs, first, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = warp_uniform(*reinterpret_cast<volatile uint32_t*>(base_ptr + L::OFF_TMEM));
  const int ntiles = warp_uniform(first[p.n_experts]);
  auto tile_at = [&](int t, int& e) { return tile_of<kRows, false>(p, offs, first, width, tiles_n, 0, t, e); };
  auto next = [&](int& stage, uint32_t& phase) {
    if (++stage == S) {
      stage = 0;
      phase ^= 1u;
    }
  };

  if (warp == 0) {
    // ------------------------------------------------ B and its scale factors (the whole warp)
    int uses = 0, stage = 0, e = 0;
    uint32_t phase = 0;
    bool ok = true;
    const int b_atoms = p.b_cols_all / kDepth, b_last = p.b_rows_all / kRows - 1;
    for (int t = unit; t < ntiles && ok; t += units) {
      const Tile w = tile_at(t, e);
      const int nkb = warp_uniform(w.nkb), b_row = warp_uniform(w.b_row);
      // atoms of B's scales: 128 rows each, from the one that holds the tile's first row; past B's last row its last atoms
      // (those columns are not stored)
      const bool two = b_row % kRows + width > kRows;
      int atom = warp_uniform(2 * (b_row / kRows * b_atoms + w.b_kb)), x = warp_uniform(w.b_kb) * kDepth;
      const int second = b_row / kRows < b_last ? 2 * b_atoms : 0;
      const uint32_t tx = L::A_BYTES + b_bytes + (MX ? (two ? 1536u : 1024u) : 0u);
      for (int kb = 0; kb < nkb; ++kb) {
        ok = warp_uniform(mbar_wait(base + L::OFF_EMPTY + 8 * stage, phase ^ 1u, p.err, kErrTimeoutStage, abort_flag));
        if (!ok) break;
        const uint32_t full = base + L::OFF_FULL + 8 * stage, sf = base + l.sf + static_cast<uint32_t>(stage) * L::SF_BYTES;
        mbar_arrive_expect_tx_warp(full, tx);
        tma_load_2d_warp(base + l.b + static_cast<uint32_t>(stage) * b_bytes, &tm_b, x, b_row, full);
        if (MX) {
          tma_load_2d_warp(sf + 512, &tm_sfb, 0, atom, full);
          if (two) tma_load_2d_warp(sf + 1024, &tm_sfb, 0, atom + second, full);
        }
        x += kDepth;
        atom += 2;
        ++uses;
        next(stage, phase);
      }
    }
    // the loads land before the CTA exits, A's of the same blocks too
    for (int s = 0; s < S; ++s) {
      const int n = uses / S + (s < uses % S ? 1 : 0);
      if (n > 0) mbar_wait(base + L::OFF_FULL + 8 * s, static_cast<uint32_t>(n - 1) & 1u, p.err, kErrTimeoutTmaLoad, nullptr);
    }
  } else if (warp == kFetchA) {
    // ------------------------------------------------ A and its scale factors (the whole warp)
    int stage = 0, slot = 0, old = 0, fill = 0, e = 0;   // old: the stage of the block whose MMAs make room
    uint32_t phase = 0, old_phase = 0;
    bool ok = true;
    const int a_atoms = p.a_cols / kDepth;
    for (int t = unit; t < ntiles && ok; t += units) {
      const Tile w = tile_at(t, e);
      const int nkb = warp_uniform(w.nkb), a_row = warp_uniform(w.a_row);
      int atom = warp_uniform(2 * (a_row / kRows * a_atoms + w.a_kb)), x = warp_uniform(w.a_kb) * kDepth;
      for (int kb = 0; kb < nkb; ++kb) {
        if (fill < SA) {
          ++fill;
        } else {
          ok = warp_uniform(mbar_wait(base + L::OFF_EMPTY + 8 * old, old_phase, p.err, kErrTimeoutStage, abort_flag));
          if (!ok) break;
          next(old, old_phase);
        }
        const uint32_t full = base + L::OFF_FULL + 8 * stage;
        tma_load_2d_warp(base + l.a + static_cast<uint32_t>(slot) * L::A_BYTES, &tm_a, x, a_row, full);
        if (MX) tma_load_2d_warp(base + l.sf + static_cast<uint32_t>(stage) * L::SF_BYTES, &tm_sfa, 0, atom, full);
        x += kDepth;
        atom += 2;
        slot = slot + 1 == SA ? 0 : slot + 1;
        next(stage, phase);
      }
    }
  } else if (MX && warp == kCopier) {
    // ------------------------------------------------ scale factors into TMEM (the whole warp)
    int stage = 0, e = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = unit; t < ntiles && ok; t += units) {
      const Tile w = tile_at(t, e);
      const int n_atoms = warp_uniform((w.b_row % kRows + width + kRows - 1) / kRows), nkb = warp_uniform(w.nkb);
      for (int kb = 0; kb < nkb; ++kb) {
        ok = warp_uniform(mbar_wait(base + L::OFF_FULL + 8 * stage, phase, p.err, kErrTimeoutTmaLoad, abort_flag));
        if (!ok) break;
        tc_fence_after();
        // the stage's columns were last read by MMAs that finished before the stage was refilled
        const uint32_t sf = base + l.sf + static_cast<uint32_t>(stage) * L::SF_BYTES;
        const uint32_t col = tmem + L::SF_COL + static_cast<uint32_t>(stage) * L::SF_COLS;
        for (int h = 0; h <= n_atoms; ++h) tc_cp_32x128b_warpx4_warp(col + 4 * h, sdesc_rows16(sf + 512 * h));
        tc_commit_warp(base + L::OFF_SFR + 8 * stage);
        next(stage, phase);
      }
    }
    tc_commit_warp(base + L::OFF_FINAL);
    mbar_wait(base + L::OFF_FINAL, 0, p.err, kErrTimeoutMma, nullptr);
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (the whole warp)
    const uint32_t idesc = (static_cast<uint32_t>(p.e5m2_a) << 7) | (static_cast<uint32_t>(p.e5m2_b) << 10) |
                           (static_cast<uint32_t>(width >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24) |
                           (MX ? 1u << 23 : 1u << 4);
    int stage = 0, slot_a = 0, e = 0;
    uint32_t phase = 0, acc_it = 0;
    bool ok = true;
    for (int t = unit; t < ntiles && ok; t += units) {
      const Tile w = tile_at(t, e);
      const int nkb = warp_uniform(w.nkb);
      if (nkb == 0) continue;   // the epilogue stores 0 without an accumulator
      // B's first row may be the middle one of its first atom: 32 rows are one column of scale factors
      const uint32_t sfb_col = warp_uniform(4u + static_cast<uint32_t>(w.b_row % kRows / 32));
      const uint32_t a = ACC == 2 ? acc_it & 1u : 0u, use = ACC == 2 ? acc_it >> 1 : acc_it;
      ok = warp_uniform(mbar_wait(base + L::OFF_TEMPTY + 8 * a, (use & 1u) ^ 1u, p.err, kErrTimeoutMma, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + a * static_cast<uint32_t>(width);
      for (int kb = 0; kb < nkb; ++kb) {
        // MXFP8: the copier's signal stands for the stage's data too
        ok = warp_uniform(
            mbar_wait(base + (MX ? L::OFF_SFR : L::OFF_FULL) + 8 * stage, phase, p.err, kErrTimeoutTmaLoad, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = base + l.a + static_cast<uint32_t>(slot_a) * L::A_BYTES, sb = base + l.b + static_cast<uint32_t>(stage) * b_bytes;
        const uint32_t sfa = tmem + L::SF_COL + static_cast<uint32_t>(stage) * L::SF_COLS, sfb = sfa + sfb_col;
#pragma unroll
        for (int k = 0; k < kDepth / kUmmaDepth; ++k) {
          const uint64_t da = sdesc_k_sw128(sa + k * kUmmaDepth), db = sdesc_k_sw128(sb + k * kUmmaDepth);
          const uint32_t more = (kb | k) != 0 ? 1u : 0u;
          if (MX)
            tc_mma_mxf8f6f4_warp(d, da, db, idesc | (static_cast<uint32_t>(k) << 4) | (static_cast<uint32_t>(k) << 29), sfa, sfb, more);
          else
            tc_mma_f8f6f4_warp(d, da, db, idesc, more);
        }
        tc_commit_warp(base + L::OFF_EMPTY + 8 * stage);
        slot_a = slot_a + 1 == SA ? 0 : slot_a + 1;
        next(stage, phase);
      }
      if (!ok) break;
      tc_commit_warp(base + L::OFF_TFULL + 8 * a);
      ++acc_it;
    }
    tc_commit_warp(base + L::OFF_FINAL);   // every MMA has finished before TMEM is released
    mbar_wait(base + L::OFF_FINAL, 0, p.err, kErrTimeoutMma, nullptr);
  } else if (warp >= 2 && warp < 2 + kEpi) {
    // ------------------------------------------------ epilogue
    const int q = warp & 3, h = (warp - 2) >> 2;   // TMEM lane quarter; chunks h, h + 2, ... of 32 columns
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const bool fp32 = p.out_fp32 != 0;
    const uint32_t stg = base + l.stg + static_cast<uint32_t>(warp - 2) * (fp32 ? 4096u : 2048u);
    uint32_t acc_it = 0;
    int e = 0;
    for (int t = unit; t < ntiles; t += units) {
      const Tile w = tile_at(t, e);
      const uint32_t a = ACC == 2 ? acc_it & 1u : 0u, use = ACC == 2 ? acc_it >> 1 : acc_it;
      const int chunks = min(width, p.N - w.c_col) / 32;   // N and the width are multiples of 32
      float scale = 1.0f;
      if (w.nkb > 0) {
        if (!MX) scale = __fmul_rn(*p.sa, p.sb[p.sb_step * w.e]);
        // warp-uniform decision: the TMEM loads that follow are .sync.aligned
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(base + L::OFF_TFULL + 8 * a, use & 1u, p.err, kErrTimeoutMma, abort_flag))) break;
        tc_fence_after();
      }
      for (int c = h; c < chunks; c += 2) {
        uint32_t r[32];
        if (w.nkb > 0) {
          tc_ld_32x32b_x32(lane_base + a * static_cast<uint32_t>(width) + 32 * c, r);
          tc_wait_ld(r);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0u;
        }
        // this warp's 32 rows x 32 columns staged for one TMA store, rows of 64 (bf16) or 128 bytes, swizzled as wide (plain
        // rows meet in the same banks: 109 experts of at most 128 rows, gradients of 128 x 1920 in binary32, 40.4 us, so 22.7)
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = MX ? __uint_as_float(r[j]) : __fmul_rn(__uint_as_float(r[j]), scale);
        if (lane == 0) bulk_wait_read<0>();   // the box's previous store has read it
        __syncwarp();
        if (fp32) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            sts128(stg + static_cast<uint32_t>(lane) * 128u + ((static_cast<uint32_t>(k) ^ (lane & 7u)) << 4), __float_as_uint(v[4 * k]),
                   __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3]));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            sts128(stg + static_cast<uint32_t>(lane) * 64u + ((static_cast<uint32_t>(k) ^ ((lane >> 1) & 3u)) << 4),
                   pack_bf16(v[8 * k], v[8 * k + 1]), pack_bf16(v[8 * k + 2], v[8 * k + 3]), pack_bf16(v[8 * k + 4], v[8 * k + 5]),
                   pack_bf16(v[8 * k + 6], v[8 * k + 7]));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tm_c, stg, w.c_col + 32 * c, w.c_row + 32 * q);
          bulk_commit();
        }
      }
      if (w.nkb > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(base + L::OFF_TEMPTY + 8 * a);
        ++acc_it;
      }
    }
    zero_outside(p, offs, static_cast<int>(threadIdx.x) - 64);
    if (lane == 0) bulk_wait_all<0>();   // this warp's stores have finished
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemAll);
  }
}

// ------------------------------------------------------------------ launches
template <int KIND, int S>
cudaError_t run_pairs(const GroupedParams& p, const GroupedMaps& m, int64_t tiles, int num_sms, cudaStream_t s) {
  using L = PairLayout<KIND, S>;
  constexpr int kMostSmem = static_cast<int>(L::FIXED + table_bytes(S == 6 ? kSixStageExperts : kMaxExperts));
  static_assert(kMostSmem <= static_cast<int>(kSmem), "shared memory");
  auto kern = k_grouped<KIND, S>;
  static std::atomic<bool> attr_done[kMaxDevices] = {};
  cudaError_t e = ensure_smem_limit(kern, kMostSmem, attr_done);
  if (e != cudaSuccess) return e;
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
    cfg.dynamicSmemBytes = kMostSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) n = num_sms / 2;
    resident[dev].store(n < num_sms / 2 ? n : num_sms / 2, std::memory_order_relaxed);
  }
  int64_t pairs = resident[dev].load(std::memory_order_relaxed);
  if (tiles < pairs) pairs = tiles < 1 ? 1 : tiles;
  return launch_pdl(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(grouped_threads<KIND>()), L::FIXED + table_bytes(p.n_experts), s,
                    2, m.a, m.b, m.sfa, m.sfb, m.c, p);
}

template <int KIND>
cudaError_t run_few(const GroupedParams& p, const GroupedMaps& m, int width, int64_t tiles, int num_sms, cudaStream_t s) {
  auto kern = k_grouped_few<KIND>;
  static std::atomic<bool> attr_done[kMaxDevices] = {};
  const cudaError_t e = ensure_smem_limit(kern, static_cast<int>(kSmem), attr_done);
  if (e != cudaSuccess) return e;
  const FewLayout l(width, KIND == kMx, p.out_fp32 != 0, p.n_experts);
  const int64_t units = tiles < num_sms ? (tiles < 1 ? 1 : tiles) : num_sms;
  return launch_pdl(kern, dim3(static_cast<unsigned>(units)), dim3(grouped_threads<KIND>()), l.total, s, 1, m.a, m.b, m.sfa, m.sfb, m.c, p,
                    l);
}

// the most tiles that a call can have, whatever its offsets are
int64_t most_tiles(const GroupedParams& p, int tile_rows, int tile_cols) {
  const int64_t tn = (p.N + tile_cols - 1) / tile_cols;
  if (p.depth) return static_cast<int64_t>(p.n_experts) * ((p.M + tile_rows - 1) / tile_rows) * tn;
  const int64_t blocks = p.capacity / kRows, used = p.n_experts < blocks ? p.n_experts : blocks;
  const int64_t per = tile_rows / kRows;
  return (blocks + used * (per - 1)) / per * tn;
}

// The tile width of a call: 0 for CTA pairs, else that of one CTA's 128-row tiles: what takes the fewest cycles a
// 128-deep block, rounds of tiles times a tile's.  A pair's tile is bound by its four MMAs (~175 each); a tile of
// one CTA by what it fetches, A's 128 rows and its width of B's at 48 bytes a cycle, and where TMEM holds one
// accumulator, by a seventh more.  One segment of 128 rows each (us, pairs | one CTA at the rule's width and at 128;
// MXFP8, K = 4096): 2 x 11008 columns 32.5 | 20.7, 25.3; 8 x 11008 73 | 66, 65; 16 x 4096 63 | 53, 53.  Pairs by the rule (us,
// pairs | one CTA at the best width): 16 segments of 256, 4096 columns 62 | 64; one of 1024 16.2 | 17.1; 64 of 128 to 384,
// K = 2048, 127 | 126; three of 384, all odd where the rule expects half of them to be, 27.8 | 18.9.
int grouped_width(const GroupedParams& p, int num_sms) {
  int64_t blocks, pairs;   // tiles of 128 and of 256 rows, for each of tile columns
  if (p.depth) {
    blocks = static_cast<int64_t>(p.n_experts) * (p.M / kRows);
    pairs = static_cast<int64_t>(p.n_experts) * ((p.M / kRows + 1) / 2);
  } else {
    // the capacity has room for 127 rows of padding an expert, of which half are expected; so are as many odd
    // segments as even ones (what they are is known on the device only)
    const int64_t room = p.capacity / kRows, used = p.n_experts < room ? p.n_experts : room;
    blocks = room - (room - used < used / 2 ? room - used : used / 2);
    pairs = (blocks + used / 2) / 2 > used ? (blocks + used / 2) / 2 : used;
  }
  auto rounds = [&](int64_t tiles, int cols, int units) { return (tiles * ((p.N + cols - 1) / cols) + units - 1) / units; };
  const bool mx = p.kind == kMx;
  int best = 0;
  int64_t least = rounds(pairs, kPairCols, num_sms < 2 ? 1 : num_sms / 2) * 700;
  const int step = mx ? 64 : 32;
  for (int width = step; width <= 256; width += step) {
    const int64_t n = rounds(blocks, width, num_sms);
    int64_t cost = n * (width + kRows) * 8 / 3;
    if (n > 1 && FewLayout::accumulators(mx, width) == 1) cost += cost / 7;
    if (cost < least) {
      least = cost;
      best = width;
    }
  }
  return best;
}

}  // namespace

GroupedPlan grouped_plan(const GroupedParams& p, int num_sms) {
  GroupedPlan g{};
  const bool mx = p.kind == kMx;
  g.width = grouped_width(p, num_sms);
  if (g.width == 0) {
    g.stages = !mx && p.n_experts <= kSixStageExperts ? 6 : 5;
    g.accumulators = mx ? PairLayout<kMx, 5>::ACC : PairLayout<kTensor, 5>::ACC;
  } else {
    g.stages = FewLayout(g.width, mx, p.out_fp32 != 0, p.n_experts).sb;
    g.accumulators = FewLayout::accumulators(mx, g.width);
  }
  return g;
}

cudaError_t launch_grouped(const GroupedParams& p, const GroupedMaps& m, const GroupedPlan& g, int num_sms, cudaStream_t s) {
  const bool mx = p.kind == kMx;
  const int width = g.width;
  if (width == 0) {
    const int64_t tiles = most_tiles(p, 2 * kRows, kPairCols);
    if (mx) return run_pairs<kMx, 5>(p, m, tiles, num_sms, s);
    return g.stages == 6 ? run_pairs<kTensor, 6>(p, m, tiles, num_sms, s) : run_pairs<kTensor, 5>(p, m, tiles, num_sms, s);
  }
  const int64_t tiles = most_tiles(p, kRows, width);
  return mx ? run_few<kMx>(p, m, width, tiles, num_sms, s) : run_few<kTensor>(p, m, width, tiles, num_sms, s);
}

}  // namespace fp8q
