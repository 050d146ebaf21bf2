// gemm_bf16.cu -- grouped GEMMs on bf16 operands (forward, dgrad, wgrad), on tcgen05, CTA pairs.
//
//   forward  Y[t,n]    = sum_k X[t,k]  W[e,n,k]      (t a row of expert e)
//   dgrad    dX[t,k]   = sum_n dY[t,n] W[e,n,k]
//   wgrad    dW[e,n,k] = sum_{t of e} dY[t,n] X[t,k]
//
// The layers that stay in bf16, and what the low-precision products are compared with ("Scaling and Optimizing
// Frontier Model Training", "MXFP8 expert kernels").  Operands are read as they lie in memory: W is K-major for the
// forward and MN-major for dgrad, wgrad's operands are MN-major, so nothing is transposed, padded or copied.
// Products and sums are kept in fp32 in tensor memory over the whole contraction, in steps of 16 in order, and rounded
// once: there is no split, so a row's result depends neither on other rows nor on which form below runs.  But each step
// of the MMA cuts its sum towards zero, which adds up: relative error of dW over 4096, 20000 and 65536 rows of an expert 5e-6, 2e-5 and
// 8e-5 (4% of half a bf16 step).  fp32 shows that: there wgrad hands over a sum every 16 stages (1024 rows), and the
// epilogue's warps add those up in registers, rounded to nearest: 8e-7, 8e-7 and 9e-7 (65536 rows, one expert of 4096 x 7168: 1.99 ms,
// bf16 in one sum 1.93).  bf16 shows it past 65536 rows of an expert, where
// it does the same every 1024 stages (sums of one sign over 2^25 rows 4% too small in one; the forward's and dgrad's
// contractions end at 65536).
//
// What bounds them.  A stage of 64 of the contraction takes a pair's M = 256, N = 256 MMAs 512 cycles; the 48 KB that
// they read of an SM's shared memory and the 32 KB that the copies write there take 640 at 128 bytes a cycle, and 620 are
// measured (without the copies the MMAs run at their rate).  65536 x 4096 x 7168, one expert: forward 1.95 ms,
// 1.98 PFLOP/s, dgrad 1.96, wgrad 1.92; 32 experts of 2048 rows of 7168 x 2048: 0.99, 0.99 and 0.99 ms.  Kept up for
// seconds, the power cap sets 1.61 PFLOP/s.  Tiles are 256 x 256 a pair, two accumulators in tensor memory, a ring of six
// 32 KB stages.  12 warps a CTA:
//   warp 0      producer: A and B by TMA, completing on the leader's barriers;
//   warp 1      allocates tensor memory; in the leader issues the MMAs, a commit a stage frees it in both CTAs, one a tile
//               hands the accumulator to both epilogues;
//   warp 2      wgrad: experts that end within the tensor's first 64 rows;
//   warps 4-11  epilogue: 32 rows x 128 columns each, while the next tile's MMAs run.
//
// wgrad's contraction runs over the rows of one expert, and the block of 64 rows at an expert's end reaches into the
// next expert's.  Those must read as zeros in both operands (0 times a NaN of another expert would be NaN).  The operands' maps
// are of all windows of 64 rows: a block is a window, and the last one, which starts inside the window that ends with the
// expert, has nothing behind it, where the map fills in zeros.  Its MMAs stop at the K = 16 step that holds the end.
// An end within the tensor's first 64 rows has no such window: there warp 2 of each CTA copies the block and writes the zeros (at
// most 15 rows), and the leader's completes the stage.  Zeros written for every expert, or last blocks in copies of 8 rows and
// of one, hold up each tile by 1 us: 500 rows of each of 32 experts of 7168 x 2048 442 and 396 us, by windows 318.
#include <algorithm>

#include "gemm_tiles.cuh"

namespace fme {

namespace {

constexpr int kThreadsBf = 384;
constexpr int kEpiWarp0 = 4;
constexpr int kStageK = 64;  // bf16 of the contraction in a stage: one 128-byte swizzle row
constexpr int kStageBytesBf = kABytes + kBBytes;
constexpr int kMaxStagesBf = 6;
constexpr int kOutBlockBytes = 32 * 128;  // a warp's staging block: 32 rows of 128 bytes
constexpr int kSumStages32 = 16, kSumStages16 = 1024;  // wgrad: stages of a sum in tensor memory, for fp32 and for bf16 dW
constexpr int kHalfMnBytes = kStageK * 128;  // 64 M or N values (128 bytes) of an MN-major stage

enum class KindBf { kFwd, kDgrad, kWgrad };

struct SharedBf {
  uint64_t full[kMaxStagesBf];
  uint64_t freed[kMaxStagesBf];  // the stage's MMAs are done (own CTA)
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint64_t peer_fills_bar;
  uint64_t early_go[kMaxStagesBf];    // wgrad, blocks for warp 2: the stage is free,
  uint64_t early_peer[kMaxStagesBf];  // the peer's half is there (the leader's),
  uint64_t early_full;                // the copies have landed
  uint32_t peer_fills;
  uint32_t peer_early;  // a bit a stage: the peer's latest fill is such a block
  uint32_t tmem_base;
  int abort_flag;
  int ok_flag;
};

// Instruction descriptor: fp32 accumulator (bit 4), bf16 operands (bits 7 and 10), the operands'
// major-ness (bits 15, 16: 1 = MN-major), N / 8 and M / 16.
constexpr uint32_t idesc_bf16(bool a_mn, bool b_mn, uint32_t m, uint32_t n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((n >> 3) << 17) |
         ((m >> 4) << 24);
}

// One stage (64 of the contraction): four K = 16 steps, M = 256 over the pair, and the commit that frees the stage in
// both CTAs.  kA, kB: distance of the steps in the operands' descriptors (16-byte units).
template <uint32_t kA, uint32_t kB>
__device__ __forceinline__ void mma_stage_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate, uint64_t *freed) {
  asm volatile(
      "{\n\t.reg .pred z, o;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.u32 z, %8, 0;\n\tsetp.eq.u32 o, 0, 0;\n\t"
      "add.s64 a1, %1, %5;\n\tadd.s64 a2, %1, 2 * %5;\n\tadd.s64 a3, %1, 3 * %5;\n\t"
      "add.s64 b1, %2, %6;\n\tadd.s64 b2, %2, 2 * %6;\n\tadd.s64 b3, %2, 3 * %6;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, z;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, o;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, o;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, o;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%4], %7;\n\t"
      "}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(smem_u32(freed)), "n"(kA), "n"(kB), "h"(static_cast<uint16_t>(3)),
      "r"(accumulate)
      : "memory");
}

// The same of fewer steps.
template <uint32_t kA, uint32_t kB>
__device__ __forceinline__ void mma_steps_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate, uint64_t *freed, int steps) {
  for (int j = 0; j < steps; ++j)
    asm volatile(
        "{\n\t.reg .pred z;\n\tsetp.ne.u32 z, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, z;\n\t}" ::"r"(d_tmem),
        "l"(a_desc + j * kA), "l"(b_desc + j * kB), "r"(idesc), "r"(accumulate || j > 0 ? 1u : 0u)
        : "memory");
  pair::commit_both(freed);
}

struct TileBf {
  int32_t e;
  int32_t nk;          // stages of the contraction
  int32_t row0;        // this CTA's first output row: of all rows (fwd, dgrad) or of the expert's (wgrad)
  int32_t rows_valid;  // of its 128
  int32_t col0;        // first output column of the tile
  int32_t p0, p1;      // wgrad: the expert's rows, the contraction
};

// Tiles and their counts are in 32 bits (checked on the host).
template <KindBf K>
__device__ __forceinline__ TileBf tile_bf(const LaunchBf16 &p, const Tables &s, uint32_t t, int rank) {
  TileBf tl;
  const uint32_t nb = (static_cast<uint32_t>(p.n) + kBN - 1) / kBN;
  if constexpr (K == KindBf::kWgrad) {
    const uint32_t mb = (static_cast<uint32_t>(p.m) + kPairM - 1) / kPairM;
    const uint32_t per = mb * nb;
    const uint32_t order = t / per;
    const uint32_t rem = t - order * per;
    tl.e = s.aux[order];
    tl.p0 = s.off[tl.e];
    tl.p1 = s.off[tl.e + 1];
    // Row by row of the expert's tiles.  Where its operands do not fit in L2 (64 MB as the border) the tiles worked on at
    // a time read each operand again from memory, the less the nearer they are to a square: bands of 8 tiles' height
    // then, column by column (65536 rows, one expert of 4096 x 7168: 2.19 -> 2.05 ms; 512 rows of each of 32 experts 0.63
    // with bands, 0.61 without).
    uint32_t row, col;
    if (static_cast<int64_t>(tl.p1 - tl.p0) * (p.m + p.n) > (int64_t(64) << 19)) {
      const uint32_t band = rem / (8 * nb), in = rem - band * 8 * nb, high = min(8u, mb - 8 * band);
      col = in / high;
      row = 8 * band + in - col * high;
    } else {
      row = rem / nb;
      col = rem - row * nb;
    }
    tl.nk = (tl.p1 - tl.p0 + kStageK - 1) / kStageK;
    tl.row0 = static_cast<int32_t>(row * kPairM + rank * kBM);
    tl.rows_valid = min(kBM, static_cast<int32_t>(p.m) - tl.row0);
    tl.col0 = static_cast<int32_t>(col * kBN);
  } else {
    const uint32_t g = t / nb;
    tl.col0 = static_cast<int32_t>((t - g * nb) * kBN);
    tl.e = find_group(s.aux, p.num_experts, g);
    const int32_t first = (static_cast<int32_t>(g) - s.aux[tl.e]) * kPairM + rank * kBM;
    tl.row0 = s.off[tl.e] + first;
    tl.rows_valid = min(kBM, s.off[tl.e + 1] - s.off[tl.e] - first);
    tl.nk = static_cast<int32_t>((p.k + kStageK - 1) / kStageK);
    tl.p0 = tl.p1 = 0;
  }
  return tl;
}

// 32 lanes x 8 columns, and the wait for them.
__device__ __forceinline__ void tmem_ld_32x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// A staged block (32 rows of 128 bytes, swizzled) to columns `col` on, by plain stores; with kAdd added to what is there
// (one unfused add an element, all reads before the first write: they are in flight together).  Past the output's edge
// nothing is written.
template <typename T, bool kAdd>
__device__ __forceinline__ void store_rows(T *y, int64_t ld, int64_t row0, int64_t col, int rows_valid, const uint8_t *blk,
                                           int lane) {
  constexpr int kPer = 16 / sizeof(T);
  const int j = lane & 7;
  col += kPer * j;
  if (col >= ld) return;
  T *base = y + row0 * ld + col;
  float4 old[8];
  if (kAdd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      old[i] = r < rows_valid ? *reinterpret_cast<const float4 *>(base + r * ld) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    float4 v = *reinterpret_cast<const float4 *>(blk + r * 128 + 16 * (j ^ (r & 7)));
    if (kAdd)
      v = make_float4(__fadd_rn(old[i].x, v.x), __fadd_rn(old[i].y, v.y), __fadd_rn(old[i].z, v.z),
                      __fadd_rn(old[i].w, v.w));
    if (r < rows_valid) *reinterpret_cast<float4 *>(base + r * ld) = v;
  }
}

// kSum: wgrad in sums of so many stages, a power of two (kSumStages32 into fp32, kSumStages16 into bf16); 0: in one.
template <KindBf K, int kSum>
__global__ void __launch_bounds__(kThreadsBf, 1) gemm_bf16_kernel(const __grid_constant__ LaunchBf16 p) {
  constexpr bool kAmn = K == KindBf::kWgrad;
  constexpr bool kBmn = K != KindBf::kFwd;
  __shared__ SharedBf s;
  extern __shared__ uint8_t dyn_smem[];
  const uint32_t S = p.stages;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  uint8_t *smem_a = smem;
  uint8_t *smem_b = smem_a + S * kABytes;
  uint8_t *smem_out = smem + S * kStageBytesBf;
  int32_t *gmem = reinterpret_cast<int32_t *>(smem_out + 8 * kOutBlockBytes);
  const Tables tab{gmem, gmem + (p.num_experts + 1)};

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(pair::cta_rank());
  const uint32_t pair_id = blockIdx.x >> 1;
  const uint32_t pairs = gridDim.x >> 1;

  if (threadIdx.x == 32) {
    for (uint32_t i = 0; i < S; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.freed[i], 1);
      mbar_init(&s.early_go[i], 1);
      mbar_init(&s.early_peer[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], kAccEmptyArrivals);
    }
    mbar_init(&s.drain, 1);
    mbar_init(&s.peer_fills_bar, 1);
    s.abort_flag = 0;
    mbar_init(&s.early_full, 1);
    s.peer_early = 0;
    fence_barrier_init();
    fence_proxy_async_shared();
    prefetch_tensormap(&p.map_a);
    prefetch_tensormap(&p.map_b);
  }
  if (warp == 1) {
    __syncwarp();
    pair::tmem_alloc(&s.tmem_base, kTmemCols);
    pair::tmem_relinquish();
  }
  start_next_kernel();  // its CTAs find room as these end
  wait_for_previous_kernel();
  // ---- tables (both CTAs of a pair see the same offsets and take the same way out)
  if (warp == 0) {
    const int32_t total = scan_groups(p.offsets, p.num_experts, p.rows, kPairM,
                                      [&](int g, int32_t lo, int32_t, int32_t first) {
                                        tab.off[g] = lo;
                                        if (K != KindBf::kWgrad) tab.aux[g] = first;
                                      });
    if (lane == 0) {
      tab.off[p.num_experts] = static_cast<int32_t>(p.rows);
      if (K != KindBf::kWgrad) tab.aux[p.num_experts] = total;
      s.ok_flag = total >= 0;
    }
  }
  if constexpr (K == KindBf::kWgrad) {  // experts by decreasing work
    __syncthreads();
    if (s.ok_flag) {
      for (int e = threadIdx.x; e < p.num_experts; e += kThreadsBf) {
        const int32_t w = tab.off[e + 1] - tab.off[e];
        int order = 0;
        for (int f = 0; f < p.num_experts; ++f) {
          const int32_t wf = tab.off[f + 1] - tab.off[f];
          order += (wf > w) || (wf == w && f < e);
        }
        tab.aux[order] = e;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  pair::cluster_sync();  // both CTAs' barriers exist before any copy or arrive crosses the pair
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  volatile int *abort_flag = &s.abort_flag;
  // A pair's tile of each round: one of every `pairs`.  wgrad's come with decreasing work, and every other round is
  // walked backwards, so that a pair with a long tile gets a short one next.
  auto tile_at = [&](uint32_t round) {
    return round * pairs + (K == KindBf::kWgrad && (round & 1) ? pairs - 1 - pair_id : pair_id);
  };
  const uint32_t nb = static_cast<uint32_t>((p.n + kBN - 1) / kBN);
  // malformed offsets: no tile, straight to the end
  if (!s.ok_flag && blockIdx.x == 0 && threadIdx.x == 0) report(p.status, kDevBadOffsets);
  const uint32_t total =
      !s.ok_flag ? 0
                 : (K == KindBf::kWgrad ? p.num_experts * static_cast<uint32_t>((p.m + kPairM - 1) / kPairM)
                                        : tab.aux[p.num_experts]) *
                       nb;

  if (warp < kEpiWarp0) {
    if (warp == 0) {
      if (lane == 0) {
        // ---------------------------------------------------------------- producer
        uint32_t stage = 0, phase = 1, filled = 0;
        uint32_t early = 0;  // a bit a stage: its latest fill is warp 2's
        bool stop = false;
        for (uint32_t round = 0, t; (t = tile_at(round)) < total && !stop; ++round) {
          const TileBf tl = tile_bf<K>(p, tab, t, rank);
          const int32_t bcol = tl.col0 + rank * kHalfN;
          for (int i = 0; i < tl.nk; ++i) {
            if (!mbar_wait<true>(&s.freed[stage], phase, abort_flag, p.status)) {
              stop = true;
              break;
            }
            if (K == KindBf::kWgrad && tl.p1 < kStageK) {
              mbar_arrive(&s.early_go[stage]);
              early |= 1u << stage;
            } else {
              if (rank == 0) mbar_arrive_expect_tx(&s.full[stage], 2 * kStageBytesBf);
              const uint32_t bar = pair::map_to_rank(&s.full[stage], 0);
              uint8_t *a = smem_a + stage * kABytes, *b = smem_b + stage * kBBytes;
              const int32_t k0 = i * kStageK;
              if constexpr (K == KindBf::kWgrad) {
                // the window of 64 rows that starts here or ends with the expert
                const int32_t window = min(tl.p0 + k0, tl.p1 - kStageK), from = tl.p0 + k0 - window;
                if (p.wide_a) {
                  tma_load_4d_pair(a, &p.map_a, bar, 0, from, tl.row0 / 64, window);
                } else {
                  tma_load_3d_pair(a, &p.map_a, bar, tl.row0, from, window);
                  tma_load_3d_pair(a + kHalfMnBytes, &p.map_a, bar, tl.row0 + 64, from, window);
                }
                if (p.wide_b) {
                  tma_load_4d_pair(b, &p.map_b, bar, 0, from, bcol / 64, window);
                } else {
                  tma_load_3d_pair(b, &p.map_b, bar, bcol, from, window);
                  tma_load_3d_pair(b + kHalfMnBytes, &p.map_b, bar, bcol + 64, from, window);
                }
              } else {
                pair::tma_load_2d(a, &p.map_a, bar, k0, tl.row0);
                if constexpr (K == KindBf::kFwd) {
                  tma_load_3d_pair(b, &p.map_b, bar, k0, bcol, tl.e);
                } else if (p.wide_b) {
                  tma_load_4d_pair(b, &p.map_b, bar, 0, k0, bcol / 64, tl.e);
                } else {
                  tma_load_3d_pair(b, &p.map_b, bar, bcol, k0, tl.e);
                  tma_load_3d_pair(b + kHalfMnBytes, &p.map_b, bar, bcol + 64, k0, tl.e);
                }
              }
              early &= ~(1u << stage);
            }
            ++filled;
            if (++stage == S) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        if (rank != 0) pair::st_remote_u32(pair::map_to_rank(&s.peer_early, 0), early);  // seen with the fills
        const uint32_t peer = exchange_fills(rank, filled, &s.peer_fills, &s.peer_fills_bar, p.status);
        if (rank == 0)
          drain_pair_ring(s.full, S, filled, peer, kStageBytesBf, early, *static_cast<volatile uint32_t *>(&s.peer_early));
      }
    } else if (K == KindBf::kWgrad && warp == 2) {
      // ------------------------------------------------ blocks that end within the first 64 rows (a tile's only one)
      uint32_t stage = 0, seen = 0, landed = 0;  // seen: a bit a stage, the parity of its early_go and early_peer
      for (uint32_t round = 0, t; (t = tile_at(round)) < total; ++round) {
        const TileBf tl = tile_bf<K>(p, tab, t, rank);
        const uint32_t at = stage;
        stage = (stage + tl.nk) % S;
        if (tl.nk == 0 || tl.p1 >= kStageK) continue;
        const uint32_t parity = (seen >> at) & 1;
        seen ^= 1u << at;
        if (warp_any(!mbar_wait<true>(&s.early_go[at], parity, abort_flag, p.status))) break;
        uint8_t *a = smem_a + at * kABytes, *b = smem_b + at * kBBytes;
        if (lane == 0) {
          mbar_arrive_expect_tx(&s.early_full, kStageBytesBf);
          const uint32_t bar = pair::map_to_rank(&s.early_full, rank);
          const int32_t bcol = tl.col0 + rank * kHalfN;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            pair::tma_load_2d(a + half * kHalfMnBytes, &p.early_a, bar, tl.row0 + 64 * half, tl.p0);
            pair::tma_load_2d(b + half * kHalfMnBytes, &p.early_b, bar, bcol + 64 * half, tl.p0);
          }
        }
        __syncwarp();
        if (warp_any(!mbar_wait<true>(&s.early_full, landed, abort_flag, p.status))) {
          mbar_drain(&s.early_full, landed);
          break;
        }
        landed ^= 1;
        const int32_t rows = tl.p1 - tl.p0;
        a += rows * 128;
        b += rows * 128;
        for (int i = lane; i < (15 - (rows + 15) % 16) * 8; i += 32)  // 16 bytes of each half of A and B; the swizzle stays in a row
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            *reinterpret_cast<uint4 *>(a + half * kHalfMnBytes + 16 * i) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(b + half * kHalfMnBytes + 16 * i) = make_uint4(0, 0, 0, 0);
          }
        fence_proxy_async_shared();
        __syncwarp();
        if (rank != 0) {
          if (lane == 0) pair::arrive_remote_release(pair::map_to_rank(&s.early_peer[at], 0));
        } else {
          if (warp_any(!pair::wait_acquire_cluster(&s.early_peer[at], parity, kWaitLimitNs))) {
            *abort_flag = 1;
            report(p.status, kDevTimeout);
            break;
          }
          if (lane == 0) mbar_arrive(&s.full[at]);
        }
        __syncwarp();
      }
    } else if (warp == 1) {
      if (rank == 0) {
        // ------------------------------------------- MMA issuer (leader, whole warp)
        constexpr uint32_t idesc = idesc_bf16(kAmn, kBmn, 256, 256);
        const uint64_t a_desc = desc_sw128(smem_u32(smem_a), kAmn, kHalfMnBytes);
        const uint64_t b_desc = desc_sw128(smem_u32(smem_b), kBmn, kHalfMnBytes);
        uint32_t stage = 0, phase = 0, tiles = 0;
        bool stop = false;
        for (uint32_t round = 0, t; (t = tile_at(round)) < total && !stop; ++round) {
          const TileBf tl = tile_bf<K>(p, tab, t, 0);
          const int nk = tl.nk;
          if (nk == 0) continue;  // an expert without rows: the epilogue writes zeros
          const int left = K == KindBf::kWgrad ? (tl.p1 - tl.p0) % kStageK : 0;
          uint32_t b = 0;
          for (int i = 0; i < nk && !stop; ++i) {
            const int in = kSum ? i % (kSum ? kSum : 1) : i;  // the stage's place in its sum
            if (in == 0) {
              b = tiles & 1;
              stop = warp_any(!mbar_wait(&s.acc_empty[b], ((tiles >> 1) & 1) ^ 1, abort_flag, p.status));
              if (stop) break;
              ++tiles;
            }
            stop = warp_any(!mbar_wait(&s.full[stage], phase, abort_flag, p.status));
            if (stop) break;
            tc_fence_after();
            // 16 of K: 32 bytes along a K-major row, 16 rows of an MN-major tile
            if (elect_one()) {
              constexpr uint32_t kA = (kAmn ? 2048 : 32) / 16, kB = (kBmn ? 2048 : 32) / 16;
              const uint64_t a = a_desc + stage * (kABytes / 16), bd = b_desc + stage * (kBBytes / 16);
              if (left != 0 && i == nk - 1)
                mma_steps_pair<kA, kB>(tmem + b * kBN, a, bd, idesc, in > 0, &s.freed[stage], (left + 15) / 16);
              else
                mma_stage_pair<kA, kB>(tmem + b * kBN, a, bd, idesc, in > 0, &s.freed[stage]);
              if (i == nk - 1 || (kSum && in == kSum - 1)) pair::commit_both(&s.acc_full[b]);
            }
            __syncwarp();
            if (++stage == S) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        __syncwarp();
        if (elect_one()) {
          pair::commit_local(&s.drain);
          mbar_drain(&s.drain, 0);
        }
        __syncwarp();
      }
    }
  } else {
    // ----------------------------------------------------------------- epilogue
    const int ew = warp - kEpiWarp0;
    const int q = warp & 3;    // tensor-memory lane quarter
    const int half = ew >> 2;  // column half of the tile
    // from its 32-bit address: the compiler then keeps no 64-bit pointers through wgrad's sums, which have no registers to spare
    uint8_t *blk = static_cast<uint8_t *>(__cvta_shared_to_generic(smem_u32(smem_out) + ew * kOutBlockBytes));
    const uint32_t leader_empty[2] = {pair::map_to_rank(&s.acc_empty[0], 0), pair::map_to_rank(&s.acc_empty[1], 0)};
    const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * 128;
    const int xs = lane & 7;  // the 128-byte swizzle of this lane's row
    uint32_t tiles = 0;
    bool stop = false;
    for (uint32_t round = 0, t; (t = tile_at(round)) < total && !stop; ++round) {
      const TileBf tl = tile_bf<K>(p, tab, t, rank);
      const int c0 = tl.col0 + half * 128;
      const int warp_rows = tl.rows_valid - 32 * q;
      const bool wanted = warp_rows > 0 && c0 < p.n;
      const bool empty = K == KindBf::kWgrad && tl.nk == 0;
      if (K == KindBf::kWgrad && p.accumulate && !empty && wanted) {
        // what the sums are added to is on its way into L2 while the MMAs run
        const float *at = static_cast<const float *>(p.y) + (static_cast<int64_t>(tl.e) * p.m + tl.row0 + 32 * q + lane) * p.n + c0;
        if (lane < warp_rows)
          for (int c = 0; c < 128 && c0 + c < p.n; c += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + c));
      }
      uint32_t b = 0;
      auto next_sum = [&] {
        b = tiles & 1;
        stop = warp_any(!mbar_wait(&s.acc_full[b], (tiles >> 1) & 1, abort_flag, p.status));
        tc_fence_after();
        ++tiles;
      };
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) pair::arrive_remote_relaxed(leader_empty[b]);
      };
      const int64_t out_row = (K == KindBf::kWgrad ? tl.e * p.m : int64_t(0)) + tl.row0 + 32 * q;
      uint4 *row = reinterpret_cast<uint4 *>(blk + lane * 128);
      auto pack = [](const uint32_t *v) {  // 8 values
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
          w[i] = *reinterpret_cast<const uint32_t *>(&x);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
      };
      if constexpr (K == KindBf::kWgrad) {
        const bool add = kSum != kSumStages16 && p.accumulate, fp32 = kSum ? kSum == kSumStages32 : p.out_fp32;
        // Columns 32 c on; blocks of 32 fp32 or 64 bf16 leave by plain stores (32 experts of 2048 rows, 7168 x 2048: 1.00 ms, 1.02
        // by bulk stores, fp32 1.07 and 1.09).
        auto put = [&](const uint32_t(&v)[32], int c) {
          if (fp32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) row[j ^ xs] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) row[(4 * (c & 1) + j) ^ xs] = pack(v + 8 * j);
            if ((c & 1) == 0) return;
          }
          __syncwarp();
          float *y = static_cast<float *>(p.y);
          if (add)
            store_rows<float, true>(y, p.n, out_row, c0 + 32 * c, warp_rows, blk, lane);
          else if (fp32)
            store_rows<float, false>(y, p.n, out_row, c0 + 32 * c, warp_rows, blk, lane);
          else
            store_rows<__nv_bfloat16, false>(static_cast<__nv_bfloat16 *>(p.y), p.n, out_row, c0 + 32 * (c - 1), warp_rows, blk, lane);
          __syncwarp();
        };
        if (kSum && tl.nk > kSum) {
          float tot[128];
#pragma unroll
          for (int j = 0; j < 128; ++j) tot[j] = 0.0f;
          for (int done = 0; done < tl.nk; done += kSum) {
            next_sum();
            if (stop) break;
            if (wanted) {
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                uint32_t v[8];
                tmem_ld_32x8(tq + b * kBN + 8 * c, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) tot[8 * c + j] += __uint_as_float(v[j]);
              }
            }
            release();
          }
          if (stop) break;
          if (!wanted) continue;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(tot[32 * c + j]);
            put(v, c);
          }
        } else {
          if (!empty) {
            next_sum();
            if (stop) break;
            if (!wanted) release();
          }
          if (!wanted || (empty && add)) continue;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t v[2][32];
            if (!empty) {
              tmem_ld_32x32(tq + b * kBN + 64 * c, v[0]);
              tmem_ld_32x32(tq + b * kBN + 64 * c + 32, v[1]);
              tmem_wait_ld_for(v[0]);
              tmem_wait_ld_for(v[1]);
              if (c == 1) release();  // registers hold the data
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[0][j] = v[1][j] = 0;
            }
            put(v[0], 2 * c);
            put(v[1], 2 * c + 1);
          }
        }
      } else {
        next_sum();
        if (stop) break;
        if (!wanted) {
          release();
          continue;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t v[2][32];
          tmem_ld_32x32(tq + b * kBN + 64 * c, v[0]);
          tmem_ld_32x32(tq + b * kBN + 64 * c + 32, v[1]);
          tmem_wait_ld_for(v[0]);
          tmem_wait_ld_for(v[1]);
          if (c == 1) release();  // registers hold the data
          const int col = c0 + 64 * c;
          if (col >= p.n) break;
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) row[j ^ xs] = pack(&v[j >> 2][8 * (j & 3)]);
          // A whole block leaves by a bulk store (0.5% faster than by plain ones); rows cut by the expert's end or columns by
          // the output's by plain ones.
          const bool bulk = warp_rows >= 32 && col + 64 <= p.n;
          if (bulk) fence_proxy_async_shared();
          __syncwarp();
          if (bulk) {
            if (lane == 0) {
              tma_store_2d(&p.map_y, col, static_cast<int32_t>(out_row), blk);
              bulk_commit();
            }
          } else {
            store_rows<__nv_bfloat16, false>(static_cast<__nv_bfloat16 *>(p.y), p.n, out_row, col, warp_rows, blk, lane);
            __syncwarp();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  __syncwarp();
  pair::cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    pair::tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------- forward, few rows an expert --
// The same sums with the operands exchanged: an item is 128 rows of W_e (the MMA's M; or 64 or 32, below) and up to 64
// of the expert's tokens (its N, in steps of 16), one CTA an item.  With few tokens the time is that of
// reading the weights once, and 256-row token tiles would leave all but a few rows of the MMAs
// empty and put the weights on half as many SMs.  A sum's steps over k are those of the tiles above, in the same
// order: a row's bits are the same in both forms.
//   warp 0 producer of W, warp 1 MMA issuer, warps 2-5 epilogue (thread = row of W), warp 6 producer of the tokens.
// A stage holds 128 of k, as two halves of 64: what bounds a CTA that has an SM to itself is the producers' and the
// issuer's way around their loops (4096 x 7168, one expert with one row, 32 CTAs: 28.1 us with 64 of k in nine stages, 24.8
// with 128 in four, 23.0 with a producer of its own for the tokens; with 64 rows 41, 39 and 28).  8 of 32 experts with a
// row each, 256 items: 72.5 us, 6.5 TB/s of weights; all 32 experts 270 us.
// With few items of 128 rows most SMs would have none.  Up to 32 tokens in all an item may have 64 rows of W and a stage 256 of
// k, up to 16 tokens 32 rows and 512: the stage's bytes are the same, kHalves blocks of 64 of k behind one another.  The
// MMA's M stays 128: behind an item's rows it reads what lies there, and those rows of the accumulator are not read.  The one
// expert with one row above: 16.6 us.
constexpr int kFewTokens = 64;
constexpr int kFewStages = 4;
constexpr int kFewThreads = 224;
constexpr int kFewTokenWarp = 6;
constexpr int kFewABytes = 2 * kABytes;
constexpr int kFewBBytes = 2 * kFewTokens * 128;
constexpr int kFewStageBytes = kFewABytes + kFewBBytes;
constexpr uint32_t kFewTmemCols = 2 * kFewTokens;

struct SharedFew {
  uint64_t full[kFewStages];    // W's copies
  uint64_t full_b[kFewStages];  // the tokens' copies
  uint64_t freed[kFewStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int ok_flag;
};

// 64 of the contraction: four K = 16 steps on one CTA (M = 128), both operands K-major.
__device__ __forceinline__ void mma_half_own(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred z, o;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.u32 z, %4, 0;\n\tsetp.eq.u32 o, 0, 0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, z;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, o;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, o;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, o;\n\t"
      "}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_own(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

struct ItemFew {
  int32_t e;
  int32_t row0;    // first token row
  int32_t tokens;  // 1 .. 64
  int32_t n0;      // first row of W_e = output column
};
template <int kRows>
__device__ __forceinline__ ItemFew item_few(const LaunchBf16 &p, const Tables &s, uint32_t t) {
  const uint32_t nb = (static_cast<uint32_t>(p.n) + kRows - 1) / kRows;
  const uint32_t g = t / nb;
  ItemFew it;
  it.n0 = static_cast<int32_t>((t - g * nb) * kRows);
  it.e = find_group(s.aux, p.num_experts, g);
  const int32_t first = (static_cast<int32_t>(g) - s.aux[it.e]) * kFewTokens;
  it.row0 = s.off[it.e] + first;
  it.tokens = min(kFewTokens, s.off[it.e + 1] - s.off[it.e] - first);
  return it;
}

template <int kHalves>
__global__ void __launch_bounds__(kFewThreads, 1) gemm_bf16_few_kernel(const __grid_constant__ LaunchBf16 p) {
  constexpr int kRows = 2 * kBM / kHalves;                // of W an item
  constexpr int kHalfA = kFewABytes / kHalves, kHalfB = kFewBBytes / kHalves;
  __shared__ SharedFew s;
  extern __shared__ uint8_t dyn_smem[];
  constexpr uint32_t S = kFewStages;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  uint8_t *smem_a = smem;
  uint8_t *smem_b = smem_a + S * kFewABytes;
  int32_t *gmem = reinterpret_cast<int32_t *>(smem + S * kFewStageBytes);
  const Tables tab{gmem, gmem + (p.num_experts + 1)};
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem_base)),
                 "r"(kFewTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (threadIdx.x == 64) {
    for (uint32_t i = 0; i < S; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.full_b[i], 1);
      mbar_init(&s.freed[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], 4);
    }
    mbar_init(&s.drain, 1);
    s.abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_shared();
    prefetch_tensormap(&p.map_a);
    prefetch_tensormap(&p.map_b);
  }
  start_next_kernel();
  wait_for_previous_kernel();
  if (warp == 0) {
    const int32_t total = scan_groups(p.offsets, p.num_experts, p.rows, kFewTokens,
                                      [&](int g, int32_t lo, int32_t, int32_t first) {
                                        tab.off[g] = lo;
                                        tab.aux[g] = first;
                                      });
    if (lane == 0) {
      tab.off[p.num_experts] = static_cast<int32_t>(p.rows);
      tab.aux[p.num_experts] = total;
      s.ok_flag = total >= 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  volatile int *abort_flag = &s.abort_flag;
  const int halves = static_cast<int>((p.k + kStageK - 1) / kStageK);
  const uint32_t nb = static_cast<uint32_t>((p.n + kRows - 1) / kRows);
  // malformed offsets: no item, straight to the end
  const uint32_t total = s.ok_flag ? static_cast<uint32_t>(tab.aux[p.num_experts]) * nb : 0;
  if (!s.ok_flag && blockIdx.x == 0 && threadIdx.x == 0) report(p.status, kDevBadOffsets);

  // every copy of a producer has landed before the CTA can exit
  auto drain = [](uint64_t *bars, uint32_t filled) {
    for (uint32_t j = 0; j < S && j < filled; ++j) {
      const uint32_t f = j + S * ((filled - 1 - j) / S);
      mbar_drain(&bars[j], (f / S) & 1);
    }
  };
  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------- producer of W
      uint32_t stage = 0, phase = 1, filled = 0;
      bool stop = false;
      for (uint32_t t = blockIdx.x; t < total && !stop; t += gridDim.x) {
        const ItemFew it = item_few<kRows>(p, tab, t);
        for (int i = 0; i < halves; i += kHalves) {
          if (!mbar_wait<true>(&s.freed[stage], phase, abort_flag, p.status)) {
            stop = true;
            break;
          }
          uint8_t *a = smem_a + stage * kFewABytes;
          mbar_arrive_expect_tx(&s.full[stage], min(kHalves, halves - i) * kHalfA);
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            if (i + h < halves) tma_load_3d_own(a + h * kHalfA, &p.map_a, &s.full[stage], (i + h) * kStageK, it.n0, it.e);
          ++filled;
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      drain(s.full, filled);
    }
  } else if (warp == kFewTokenWarp) {
    if (lane == 0) {
      // ---------------------------------------------- producer of the tokens
      uint32_t stage = 0, phase = 1, filled = 0;
      bool stop = false;
      for (uint32_t t = blockIdx.x; t < total && !stop; t += gridDim.x) {
        const ItemFew it = item_few<kRows>(p, tab, t);
        const uint32_t bytes = ((it.tokens + 15) >> 4) * 16 * 128;  // of a half
        for (int i = 0; i < halves; i += kHalves) {
          if (!mbar_wait<true>(&s.freed[stage], phase, abort_flag, p.status)) {
            stop = true;
            break;
          }
          uint8_t *b = smem_b + stage * kFewBBytes;
          mbar_arrive_expect_tx(&s.full_b[stage], min(kHalves, halves - i) * bytes);
          for (int j = 0; j < it.tokens; j += 16)
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              if (i + h < halves)
                tma_load_2d_own(b + h * kHalfB + j * 128, &p.map_b, &s.full_b[stage], (i + h) * kStageK, it.row0 + j);
          ++filled;
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      drain(s.full_b, filled);
    }
  } else if (warp == 1) {
    // -------------------------------------------------- MMA issuer (whole warp)
    const uint64_t a_desc = desc_sw128(smem_u32(smem_a), false), b_desc = desc_sw128(smem_u32(smem_b), false);
    uint32_t stage = 0, phase = 0, items = 0;
    bool stop = false;
    for (uint32_t t = blockIdx.x; t < total && !stop; t += gridDim.x, ++items) {
      const uint32_t cols = (item_few<kRows>(p, tab, t).tokens + 15) & ~15;
      const uint32_t idesc = idesc_bf16(false, false, 128, cols);
      const uint32_t b = items & 1;
      stop = warp_any(!mbar_wait(&s.acc_empty[b], ((items >> 1) & 1) ^ 1, abort_flag, p.status));
      for (int i = 0; i < halves && !stop; i += kHalves) {
        stop = warp_any(!mbar_wait(&s.full[stage], phase, abort_flag, p.status) ||
                        !mbar_wait(&s.full_b[stage], phase, abort_flag, p.status));
        if (stop) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ad = a_desc + stage * (kFewABytes / 16), bd = b_desc + stage * (kFewBBytes / 16);
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            if (i + h < halves)
              mma_half_own(tmem + b * kFewTokens, ad + h * (kHalfA / 16), bd + h * (kHalfB / 16), idesc, i + h > 0);
          commit_own(&s.freed[stage]);
          if (i + kHalves >= halves) commit_own(&s.acc_full[b]);
        }
        __syncwarp();
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    __syncwarp();
    if (elect_one()) {
      commit_own(&s.drain);
      mbar_drain(&s.drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;  // tensor-memory lane quarter
    const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t items = 0;
    bool stop = false;
    for (uint32_t t = blockIdx.x; t < total && !stop; t += gridDim.x, ++items) {
      const ItemFew it = item_few<kRows>(p, tab, t);
      const uint32_t b = items & 1;
      stop = warp_any(!mbar_wait(&s.acc_full[b], (items >> 1) & 1, abort_flag, p.status));
      if (stop) break;
      tc_fence_after();
      const int64_t col = it.n0 + q * 32 + lane;
      __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y) + static_cast<int64_t>(it.row0) * p.n + col;
#pragma unroll
      for (int c = 0; c < kFewTokens / 16; ++c) {
        if (16 * c < it.tokens && q * 32 < kRows) {
          uint32_t v[16];
          tmem_ld_32x16(tq + b * kFewTokens + 16 * c, v);
          tmem_wait_ld_for(v);
          if (col < p.n) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (16 * c + j < it.tokens) y[(16 * c + j) * p.n] = __float2bfloat16_rn(__uint_as_float(v[j]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.acc_empty[b]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kFewTmemCols) : "memory");
}

template <KindBf K, int kSum = 0>
cudaError_t launch_bf(LaunchBf16 a) {
  auto kernel = gemm_bf16_kernel<K, kSum>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_shared(reinterpret_cast<const void *>(kernel), allowed);
  if (err != cudaSuccess) return err;
  const int rest = 1024 + 8 * kOutBlockBytes + 8 * (a.num_experts + 1);
  // as many stages as fit beside the expert tables
  a.stages = std::min<int64_t>(kMaxStagesBf, (kGemmSmemLimit - rest) / kStageBytesBf);
  const int64_t nb = (a.n + kBN - 1) / kBN;
  const int64_t bound = K == KindBf::kWgrad ? a.num_experts * ((a.m + kPairM - 1) / kPairM) * nb
                                            : (a.m / kPairM + std::min<int64_t>(a.num_experts, a.m)) * nb;
  int64_t pairs = a.num_sms / 2;
  if (bound < pairs) pairs = bound;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(kThreadsBf, 1, 1);
  cfg.dynamicSmemBytes = rest + a.stages * kStageBytesBf;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int kHalves>
cudaError_t launch_few(const LaunchBf16 &a) {
  const int smem = 1024 + kFewStages * kFewStageBytes + 8 * (a.num_experts + 1);
  auto kernel = gemm_bf16_few_kernel<kHalves>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_shared(reinterpret_cast<const void *>(kernel), allowed);
  if (err != cudaSuccess) return err;
  constexpr int kRows = 2 * kBM / kHalves;
  const int64_t items = bf16_few_tiles(a.m, a.num_experts) * ((a.n + kRows - 1) / kRows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(a.num_sms, items)), 1, 1);
  cfg.blockDim = dim3(kFewThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_bf16_fwd(const LaunchBf16 &a) {
  switch (a.few_halves) {
    case 2: return launch_few<2>(a);
    case 4: return launch_few<4>(a);
    case 8: return launch_few<8>(a);
    default: return launch_bf<KindBf::kFwd>(a);
  }
}
cudaError_t launch_bf16_dgrad(const LaunchBf16 &a) { return launch_bf<KindBf::kDgrad>(a); }
cudaError_t launch_bf16_wgrad(const LaunchBf16 &a) {
  if (a.rows <= (a.out_fp32 ? kSumStages32 : kSumStages16) * kStageK) return launch_bf<KindBf::kWgrad>(a);
  return a.out_fp32 ? launch_bf<KindBf::kWgrad, kSumStages32>(a) : launch_bf<KindBf::kWgrad, kSumStages16>(a);
}

}  // namespace fme
