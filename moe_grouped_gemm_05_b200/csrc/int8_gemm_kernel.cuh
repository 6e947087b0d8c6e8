// Warp-specialised, persistent int8 GEMM for sm_100a, dense and M-grouped:
//
//   D[m,n] = sa[m] * sb[n] * sum_k A[m,k] B[n,k]      (BF16 or FP32 out)
//
// A and B are int8, K-contiguous; sa is one FP32 scale per row of A (token),
// sb one per row of B (output channel).  tcgen05.mma kind::i8 sums the
// products exactly in int32 in tensor memory (the host keeps 128 * 128 * K
// below 2^31), so the only roundings are those of the epilogue: the sum to
// FP32, the two products with the scales, and BF16.
//
// Unlike the block-scaled FP8 kernel there are no scales to bring into tensor
// memory: two accumulators of 256 columns fill it, and the issuing thread has
// nothing to do but four MMAs and a commit for every 128 of K.  Roles (one
// CTA per SM, persistent over output tiles):
//   issuer     (warp 0, the TMEM owner) one thread issues the MMAs (of the
//              pair's first CTA)
//   producer   (warp 1) TMA loads of A/B K-blocks into a STAGES-deep ring
//   epilogue   (eight warps) tcgen05.ld, scaling, swizzled staging + TMA store of
//              fully valid 32-row slices, predicated stores for the others
// CTAS = 2: a cluster of two CTAs computes a 256 x BN tile (cta_group::2), each
// loading its own 128 rows of A and half of B's.  No load is multicast.
// A K that is no multiple of 128 ends in a block that the TMA fills with zeros.
//
// Measured (BF16 out): 4096x7168x2048 45.6 us, 2.64 POPS; 82% of the busiest
// SM's cycles are MMAs, the rest set-up, first load, last epilogue and teardown.
// Contiguous, 8 experts, 32768 rows, 4096x7168: 600 us before the power cap sets
// in (3.2 POPS), 735 us under it.  Masked, 16 experts of up to 256 rows,
// 7168x2048: 53 us, 5 rounds of 128x256 tiles.
//
// PIPES = 2 (few rows): a narrow tile's K loop is bound by its issuing thread
// (some 60 cycles an instruction, 380 a K block against 128 of the tensor core
// on 64 columns), so two issuers (warps 0, 1) and two producers (warps 2, 3)
// take half of K each, with half of the ring and an accumulator of their own,
// which the epilogue adds: integers, so the sum is the same.  64x7168x2048: 5.5 us
// against 7.5 with one pipeline; 64x4096x7168 12.5 against 18.6.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "fp8_gemm_kernel.cuh"
#include "int8_ptx.cuh"
#include "ptx.cuh"

namespace dg {

// An issuer and a producer for each pipeline, and eight epilogue warps.
template <int PIPES>
constexpr int kInt8Threads = 32 * (8 + 2 * PIPES);

struct Int8Args : GemmArgs {
  const float* sa;  // [G][rows] (masked) or [rows]
  const float* sb;  // [G][N]
};

template <int BN, int STAGES, int MODE, int CTAS, int PIPES>
struct Int8Layout {
  static_assert(PIPES == 1 || (PIPES == 2 && CTAS == 1 && STAGES % 2 == 0), "two pipelines run on one CTA");
  static constexpr int kTileM = 128 * CTAS;
  static constexpr int kBRows = BN / CTAS;
  static constexpr int kABytes = 128 * kBK;
  static constexpr int kBBytes = kBRows * kBK;
  static constexpr int kEpiBuf = 32 * 32 * 2;  // 32 rows x 32 BF16 (or x 16 FP32)
  static constexpr int kAccStride = BN;
  static constexpr int kTmemCols = 512;
  static constexpr int kOffB = STAGES * kABytes;
  static constexpr int kOffEpi = kOffB + STAGES * kBBytes;
  static constexpr int kMine = BN / 64;  // 32-column chunks of an epilogue warp
  static constexpr int kOffScale = kOffEpi + 8 * kEpiBuf;  // B's scales of each epilogue warp's chunks
  static constexpr int kOffBar = kOffScale + 8 * kMine * 32 * 4;
  static constexpr int kNumBars = 2 * STAGES + 2 * 2 + PIPES;
  static constexpr int kOffMisc = kOffBar + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kOffGroups = kOffMisc + 16;
  static constexpr int kGroupsBytes = MODE == MODE_MASKED                   ? (2 * kMaxMaskedGroups + 1) * 4
                                      : (MODE == MODE_CONTIG && CTAS == 2) ? (kMaxContigBlocks + 1) * 4
                                                                           : 0;
  static constexpr int kSmemBytes = kOffGroups + kGroupsBytes + 1024;
  static_assert(kSmemBytes <= kMaxSmem, "shared-memory budget exceeded");
  static_assert(BN % 64 == 0 && BN <= 256 && 2 * kAccStride <= kTmemCols, "two accumulators fit in tensor memory");
  static_assert(kOffEpi % 1024 == 0 && kBBytes % 1024 == 0, "swizzle atoms are 1024-byte aligned");
};

// tile_of; in the masked layout with an expert's tiles counted without leaving int
// for counts next to 2^31 (FP8 rows of so many do not fit in memory, 16-byte ones do).
template <int MODE, int TILE_M>
__device__ __forceinline__ Tile int8_tile_of(int t, const GemmArgs& p, const int* prefix, const int* counts) {
  if constexpr (MODE != MODE_MASKED) {
    return tile_of<MODE, TILE_M>(t, p, prefix, counts);
  } else {
    Tile tl;
    tl.g = 0;
    while (prefix[tl.g + 1] <= t) ++tl.g;
    const int local = t - prefix[tl.g];
    const int blocks = static_cast<int>((static_cast<uint32_t>(counts[tl.g]) + TILE_M - 1) / TILE_M);
    tl.n_blk = local / blocks;
    tl.m_blk = local - tl.n_blk * blocks;
    tl.row0 = tl.m_blk * TILE_M;
    return tl;
  }
}

// One warp: the masked layout's valid rows per expert and running sum of tiles.
template <int TILE_M>
__device__ __forceinline__ void masked_tile_prefix(const GemmArgs& p, int* prefix, int* counts, int lane) {
  // counts[g] = clamp(masked_m[g], 0, M_max); prefix = running sum of tiles
  int run = 0;
  for (int base = 0; base < p.G; base += 32) {
    const int g = base + lane;
    int tiles = 0;
    if (g < p.G) {
      int mg = __ldg(&p.masked_m[g]);
      if (mg < 0 || mg > p.rows) {
        if (blockIdx.x == 0) atomicOr(&g_dg_error, 0x4);
        mg = mg < 0 ? 0 : p.rows;
      }
      counts[g] = mg;
      tiles = static_cast<int>((static_cast<uint32_t>(mg) + TILE_M - 1) / TILE_M) * p.num_n_blocks;
    }
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (g < p.G) prefix[g + 1] = run + incl;
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) prefix[0] = 0;
}

// One warp: the contiguous layout's pair table (count, then first blocks).
__device__ __forceinline__ void contig_pair_table(const GemmArgs& p, int* prefix, int lane) {
  // Pair table: block b (128 rows, expert = that of its first row) starts a
  // pair when it lies an even number of blocks into its run of equal
  // experts; blocks with an index outside [0, G) start none.  The experts
  // of all blocks are loaded at once (at most 32 per lane), then scanned.
  const int nb = p.rows / 128;
  int ev[kMaxContigBlocks / 32];
#pragma unroll
  for (int i = 0; i < kMaxContigBlocks / 32; ++i) {
    const int b = 32 * i + lane;
    ev[i] = b < nb ? __ldg(&p.m_indices[b * 128]) : -1;
  }
  int count = 0, run_start = 0, prev_e = -2;
#pragma unroll
  for (int i = 0; i < kMaxContigBlocks / 32; ++i) {
    if (32 * i >= nb) break;
    const int b = 32 * i + lane;
    const int e = ev[i];
    if (b < nb && (e < -1 || e >= p.G) && blockIdx.x == 0) atomicOr(&g_dg_error, 0x2);
    int e_prev = __shfl_up_sync(0xffffffffu, e, 1);
    if (lane == 0) e_prev = prev_e;
    // start of the run holding block b: the last block <= b where the expert changes
    int rs = (b < nb && (b == 0 || e != e_prev)) ? b : -1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, rs, o);
      if (lane >= o) rs = max(rs, v);
    }
    if (rs < 0) rs = run_start;
    const bool starts = b < nb && e >= 0 && e < p.G && ((b - rs) & 1) == 0;
    const uint32_t bal = __ballot_sync(0xffffffffu, starts);
    if (starts) prefix[1 + count + __popc(bal & ((1u << lane) - 1u))] = b;
    count += __popc(bal);
    run_start = __shfl_sync(0xffffffffu, rs, 31);
    prev_e = __shfl_sync(0xffffffffu, e, 31);
  }
  if (lane == 0) prefix[0] = count;
}

template <int BN, int STAGES, int MODE, int CTAS, bool OUT_F32, int PIPES>
__global__ void __launch_bounds__(kInt8Threads<PIPES>, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_d, const Int8Args p) {
  using L = Int8Layout<BN, STAGES, MODE, CTAS, PIPES>;
  constexpr bool kPair = CTAS == 2;
  constexpr int kRing = STAGES / PIPES;  // stages of a pipeline
  constexpr int kEpi0 = 2 * PIPES;       // first epilogue warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* empty_bar = full_bar + STAGES;
  uint64_t* tmem_full = full_bar + 2 * STAGES;
  uint64_t* tmem_empty = tmem_full + 2;
  uint64_t* final_bar = tmem_full + 4;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  uint32_t* peer_loads = reinterpret_cast<uint32_t*>(smem + L::kOffMisc + 8);  // written by the pair's second CTA
  // pairs: the issuer has waited for every load of both CTAs (written in both by the first)
  volatile uint32_t* all_landed = reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc + 12);
  int* prefix = reinterpret_cast<int*>(smem + L::kOffGroups);
  int* counts = prefix + kMaxMaskedGroups + 1;
  uint32_t it = 0;  // loads issued (producer warp)

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const bool is_issuer = warp < PIPES, is_producer = warp >= PIPES && warp < kEpi0;
  const int pipe = PIPES == 2 ? warp & 1 : 0;  // of an issuer or a producer
  // the pipeline's K blocks and stages
  const int all_kb = (p.K + kBK - 1) / kBK;
  const int half_kb = (all_kb + 1) / 2;
  const int kb_lo = PIPES == 2 && pipe == 1 ? half_kb : 0;
  const int kb_hi = PIPES == 2 && pipe == 0 ? half_kb : all_kb;
  const int s_lo = pipe * kRing;
  const uint32_t rank = kPair ? cluster_cta_rank() : 0;
  const int unit0 = kPair ? static_cast<int>(blockIdx.x / 2) : static_cast<int>(blockIdx.x);
  const int units = kPair ? static_cast<int>(gridDim.x / 2) : static_cast<int>(gridDim.x);

  // ---------------------------------------------------------------- set-up
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], CTAS);
      mbar_init(&empty_bar[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tmem_full[i], 1);
      mbar_init(&tmem_empty[i], 8 * CTAS);
    }
    for (int i = 0; i < PIPES; ++i) mbar_init(&final_bar[i], 1);
    *abort_flag = 0;
    *all_landed = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_a);
    prefetch_tensormap(&tm_b);
    prefetch_tensormap(&tm_d);
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc<CTAS>(tmem_holder, L::kTmemCols);
    tmem_relinquish<CTAS>();
  }
  grid_dep_wait();
  grid_dep_launch();
  if (MODE == MODE_MASKED && warp == kEpi0) masked_tile_prefix<L::kTileM>(p, prefix, counts, lane);
  if (MODE == MODE_CONTIG && kPair && warp == kEpi0) contig_pair_table(p, prefix, lane);
  tc_fence_before();
  if constexpr (kPair) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int ntiles = total_tiles<MODE, CTAS>(p, prefix);

  if (is_producer) {
    // ============================================================ producer
    const uint32_t full0 = kPair ? mapa_shared(smem_u32(full_bar), 0) : smem_u32(full_bar);
    bool ok = true;
    for (int t = unit0; t < ntiles && ok; t += units) {
      const Tile tl = int8_tile_of<MODE, L::kTileM>(t, p, prefix, counts);
      int grp_a = 0, grp_b = 0;
      if (MODE == MODE_CONTIG) {
        grp_b = contig_expert<CTAS>(tl, p);
        if (grp_b < 0) continue;
      } else if (MODE == MODE_MASKED) {
        grp_a = grp_b = tl.g;
      }
      const int m_base = tl.row0 + 128 * static_cast<int>(rank);
      const int n0 = tl.n_blk * BN;
      // each CTA of a pair holds half of the tile's MMA width of B
      const int b_row = n0 + static_cast<int>(rank) * (tile_mma_n<BN, CTAS, 0>(n0, p.N) / CTAS);
      for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
        const uint32_t s = s_lo + it % kRing;
        ok = wait_phase<false>(&empty_bar[s], ((it / kRing) & 1) ^ 1, abort_flag, p.wait_limit_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          uint8_t* a_dst = smem + s * L::kABytes;
          uint8_t* b_dst = smem + L::kOffB + s * L::kBBytes;
          if constexpr (kPair) {
            tma_load_3d_pair(a_dst, &tm_a, full0 + 8 * s, kb * kBK, m_base, grp_a);
            tma_load_3d_pair(b_dst, &tm_b, full0 + 8 * s, kb * kBK, b_row, grp_b);
            mbar_arrive_expect_tx_cluster(full0 + 8 * s, L::kABytes + L::kBBytes);
          } else {
            tma_load_3d(a_dst, &tm_a, &full_bar[s], kb * kBK, m_base, grp_a);
            tma_load_3d(b_dst, &tm_b, &full_bar[s], kb * kBK, b_row, grp_b);
            mbar_arrive_expect_tx(&full_bar[s], L::kABytes + L::kBBytes);
          }
        }
      }
    }
    // Every load must land before its CTA exits: alone, the last loads of the
    // ring are waited for here; in a pair all loads signal the first CTA, which
    // drains both after the cluster barrier of the teardown.
    if constexpr (!kPair) {
      if (lane == 0) {
        for (uint32_t i = it > kRing ? it - kRing : 0; i < it; ++i)
          wait_phase_drain(&full_bar[s_lo + i % kRing], (i / kRing) & 1);
      }
    } else if (lane == 0) {
      // The commits that free a stage arrive in both CTAs, and the last ones are
      // waited for by no load: they must have arrived before the CTA exits.
      for (uint32_t i = it > kRing ? it - kRing : 0; i < it && ok; ++i)
        ok = wait_phase<false>(&empty_bar[i % kRing], (i / kRing) & 1, abort_flag, p.wait_limit_ns);
      if (rank == 1) st_shared_cluster_u32(mapa_shared(smem_u32(peer_loads), 0), it);
    }
    __syncwarp();
  } else if (is_issuer) {
    // ============================================================ MMA issuer
    if ((!kPair || rank == 0) && lane == 0) {
      const uint64_t a0 = make_smem_desc(smem_u32(smem + s_lo * L::kABytes), 16, 1024, 2);
      const uint64_t b0 = make_smem_desc(smem_u32(smem + L::kOffB + s_lo * L::kBBytes), 16, 1024, 2);
      const uint32_t full_base = smem_u32(full_bar + s_lo), empty_base = smem_u32(empty_bar + s_lo);
      uint32_t s = 0, phase = 0, own = 0;
      bool ok = true;
      const bool ragged_n = p.N % BN != 0;
      for (int t = unit0; t < ntiles && ok; t += units) {
        int mma_n = BN;
        if (MODE == MODE_CONTIG || ragged_n) {
          const Tile tl = int8_tile_of<MODE, L::kTileM>(t, p, prefix, counts);
          if (MODE == MODE_CONTIG && contig_expert<CTAS>(tl, p) < 0) continue;
          mma_n = tile_mma_n<BN, CTAS, 0>(tl.n_blk * BN, p.N);
        }
        const uint32_t idesc = make_idesc_i8(L::kTileM, mma_n);
        // one pipeline alternates the accumulators, two have one each
        const uint32_t acc = PIPES == 2 ? pipe : own & 1, use = PIPES == 2 ? own : own >> 1;
        ++own;
        if (!mbar_try_wait(&tmem_empty[acc], (use & 1) ^ 1))
          ok = wait_phase<false>(&tmem_empty[acc], (use & 1) ^ 1, abort_flag, p.wait_limit_ns);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * L::kAccStride;
        // An instruction of the tensor core costs this thread some 60 cycles to
        // issue, a K block 300 of the 512 that it takes on 256 columns: so the
        // rest is kept short, and the next block's barrier is looked at between
        // the MMAs of this one.
        uint32_t accumulate = 0;
        bool ready = mbar_test_wait_addr(full_base + 8 * s, phase);
        for (int kb = kb_lo; kb < kb_hi; ++kb) {
          if (!ready && !mbar_try_wait_addr(full_base + 8 * s, phase)) {
            ok = wait_phase<false>(&full_bar[s_lo + s], phase, abort_flag, p.wait_limit_ns);
            if (!ok) break;
          }
          const uint64_t a = a0 + s * (L::kABytes >> 4), b = b0 + s * (L::kBBytes >> 4);
          const uint32_t done = empty_base + 8 * s;
          mma_i8<CTAS>(d_tmem, a, b, idesc, accumulate);
          mma_i8<CTAS>(d_tmem, a + 2, b + 2, idesc, 1u);
          if (++s == kRing) {
            s = 0;
            phase ^= 1;
          }
          ready = mbar_test_wait_addr(full_base + 8 * s, phase);
          mma_i8<CTAS>(d_tmem, a + 4, b + 4, idesc, 1u);
          mma_i8<CTAS>(d_tmem, a + 6, b + 6, idesc, 1u);
          accumulate = 1;
          if constexpr (kPair) tc_commit_pair_addr(done);
          else tc_commit_addr<1>(done);
        }
        if (!ok) break;
        if constexpr (kPair) tc_commit_pair(&tmem_full[acc]);
        else tc_commit<1>(&tmem_full[acc]);
      }
      // all MMAs issued here complete before TMEM is freed
      tc_commit<CTAS>(&final_bar[pipe]);
      wait_phase_drain(&final_bar[pipe], 0);
      if constexpr (kPair) {
        if (ok) {
          const uint32_t at = smem_u32(const_cast<uint32_t*>(all_landed));
          st_shared_cluster_u32(mapa_shared(at, 0), 1);
          st_shared_cluster_u32(mapa_shared(at, 1), 1);
        }
      }
    }
    __syncwarp();
  } else {
    // ============================================================ epilogue
    // Two warps per TMEM lane quarter, one on the even, one on the odd
    // 32-column chunks; the next chunk's tcgen05.ld is in flight while the
    // current one is scaled and stored.
    const int q = warp % 4;
    const int epi = warp - kEpi0;
    const int half = epi >> 2;
    uint8_t* buf = smem + L::kOffEpi + epi * L::kEpiBuf;
    const uint32_t empty0 = kPair ? mapa_shared(smem_u32(tmem_empty), 0) : smem_u32(tmem_empty);
    float* sbuf = reinterpret_cast<float*>(smem + L::kOffScale) + epi * L::kMine * 32;
    constexpr int kMine = L::kMine;
    uint32_t own = 0;
    for (int t = unit0; t < ntiles; t += units) {
      const Tile tl = int8_tile_of<MODE, L::kTileM>(t, p, prefix, counts);
      int expert = 0, own_e = 0;
      if (MODE == MODE_CONTIG) {
        const int own_blk = tl.row0 / 128 + static_cast<int>(rank);  // a pair's blocks may differ in expert
        own_e = own_blk < p.rows / 128 ? __ldg(&p.m_indices[own_blk * 128]) : -1;
        if ((own_e < -1 || own_e >= p.G) && warp == kEpi0 && lane == 0 && tl.n_blk == 0) atomicOr(&g_dg_error, 0x2);
        expert = contig_expert<CTAS>(tl, p);
        if (expert < 0) continue;
      } else if (MODE == MODE_MASKED) {
        expert = tl.g;
      }
      const uint32_t acc = PIPES == 2 ? 0 : own & 1, use = PIPES == 2 ? own : own >> 1;
      ++own;
      const int row0 = tl.row0 + 128 * static_cast<int>(rank) + 32 * q;  // the warp's first row
      const int m = row0 + lane;
      bool valid;
      if (MODE == MODE_DENSE) {
        valid = m < p.rows;
      } else if (MODE == MODE_CONTIG) {
        const int idx = m < p.rows ? __ldg(&p.m_indices[m]) : -1;
        valid = own_e == expert && idx == expert;
        if (own_e == expert && idx != expert && idx != -1 && tl.n_blk == 0 && half == 0)
          atomicOr(&g_dg_error, (idx >= 0 && idx < p.G) ? 0x8 : 0x2);
      } else {
        valid = m < counts[tl.g];
      }
      const bool all_valid = __all_sync(0xffffffffu, valid);
      const bool any_valid = __any_sync(0xffffffffu, valid);
      const int n0 = tl.n_blk * BN;
      const int zd = MODE == MODE_MASKED ? tl.g : 0;
      const size_t row_g = static_cast<size_t>(zd) * p.rows + m;
      const float sa = valid ? __ldg(p.sa + row_g) : 0.0f;
      // B's scales of the warp's chunks come in while the tile is computed (once every
      // lane has read those of the tile before)
      __syncwarp();
      const float* sb = p.sb + static_cast<size_t>(expert) * p.N;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int col = n0 + 32 * (half + 2 * i) + lane;
        sbuf[32 * i + lane] = col < p.N ? __ldg(sb + col) : 0.0f;
      }
      __syncwarp();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * L::kAccStride;

      bool ok = wait_phase<false>(&tmem_full[acc], use & 1, abort_flag, p.wait_limit_ns);
      if (PIPES == 2 && ok) ok = wait_phase<false>(&tmem_full[1], use & 1, abort_flag, p.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();

      // 16 columns of 64 bytes a row (FP32), or 32 columns (BF16), by TMA or by each lane for its row
      auto store64 = [&](const uint4 (&w)[4], int col, void* d_row, int per16) {
        if (all_valid) {
          if (lane == 0) bulk_wait_group_read<0>();  // the previous store has read the buffer
          __syncwarp();
          uint8_t* rowp = buf + lane * 64;
#pragma unroll
          for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(rowp + (i ^ ((lane >> 1) & 3)) * 16) = w[i];
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tm_d, buf, col, row0, zd);
            bulk_commit_group();
          }
        } else if (valid) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (col + per16 * i < p.N) static_cast<uint4*>(d_row)[i] = w[i];
        }
      };
      auto finish = [&](uint32_t (&r)[32], int col0, const float* scales) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 b = reinterpret_cast<const float4*>(scales)[i];
          r[4 * i] = __float_as_uint(__int2float_rn(static_cast<int>(r[4 * i])) * sa * b.x);
          r[4 * i + 1] = __float_as_uint(__int2float_rn(static_cast<int>(r[4 * i + 1])) * sa * b.y);
          r[4 * i + 2] = __float_as_uint(__int2float_rn(static_cast<int>(r[4 * i + 2])) * sa * b.z);
          r[4 * i + 3] = __float_as_uint(__int2float_rn(static_cast<int>(r[4 * i + 3])) * sa * b.w);
        }
        uint4 w[4];
        if constexpr (OUT_F32) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = col0 + 16 * h;
            if (col >= p.N) break;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = make_uint4(r[16 * h + 4 * i], r[16 * h + 4 * i + 1], r[16 * h + 4 * i + 2], r[16 * h + 4 * i + 3]);
            store64(w, col, p.d32 + row_g * p.N + col, 4);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[8 * i + 2 * j]),
                                                             __uint_as_float(r[8 * i + 2 * j + 1]));
              h[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
            w[i] = make_uint4(h[0], h[1], h[2], h[3]);
          }
          store64(w, col0, p.d + row_g * p.N + col0, 8);
        }
      };

      // The accumulator is handed back as soon as its last chunk has been read.
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair) mbar_arrive_remote(empty0 + 8 * acc);
          else mbar_arrive(&tmem_empty[acc]);
          if (PIPES == 2) mbar_arrive(&tmem_empty[1]);
        }
      };
      const int mine = any_valid ? min(kMine, max(0, ((min(p.N - n0, BN) + 31) / 32 - half + 1) / 2)) : 0;
      if (mine == 0) {
        release();
        continue;
      }
      uint32_t r[2][32];
      tmem_ld_32x32b_x32(t_row + 32 * half, r[0]);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        if (i >= mine) break;
        const int c = half + 2 * i;
        if (i + 1 < mine) tmem_ld_32x32b_x32(t_row + 32 * (c + 2), r[(i + 1) & 1]);
        if constexpr (PIPES == 2) {  // the other half of K
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(t_row + L::kAccStride + 32 * c + 16 * h, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) r[i & 1][16 * h + j] += o[j];
          }
        }
        if (i + 1 == mine) release();
        finish(r[i & 1], n0 + 32 * c, sbuf + 32 * i);
        if (i + 1 < mine) tmem_wait_ld();
      }
    }
    // the staging buffers must have been read before the CTA exits
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  if constexpr (kPair) {
    // Both CTAs have stopped issuing.  What crosses from one to the other must be
    // there before the other exits: loads (the issuer waited for them, or all_landed
    // is not set), commits (the producers and the epilogues waited for them),
    // accumulators handed back and the two words below (the barrier releases them;
    // a relaxed one, with waits for the last accumulators, measured 0.2 us slower on
    // 1000x7168x2048 and the same on larger shapes).
    cluster_sync();
    if (!*all_landed) {
      if (rank == 0 && is_producer && lane == 0) {
        // A CTA that gave up before issuing load j never arrives: arrive in its
        // place, then wait for the loads that were issued.
        const uint32_t it1 = *reinterpret_cast<volatile uint32_t*>(peer_loads);
        const uint32_t hi = it > it1 ? it : it1;
        for (uint32_t j = hi > STAGES ? hi - STAGES : 0; j < hi; ++j) {
          uint64_t* b = &full_bar[j % STAGES];
          if (j >= it) mbar_arrive(b);
          if (j >= it1) mbar_arrive(b);
          wait_phase_drain(b, (j / STAGES) & 1);
        }
      }
      __syncwarp();
      cluster_sync();
    }
  } else {
    __syncthreads();
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc<CTAS>(tmem_base, L::kTmemCols);
  }
}

}  // namespace dg
