// gemm_block128.cu -- grouped GEMMs on FP8 operands with an fp32 scale per block of
// 128 along the contraction (forward, dgrad, wgrad), on tcgen05, CTA pairs.
//
//   forward  Y[t,n]    = sum_b sx[b,t]  sw[e,n/128,b]  sum_{k in b} qx[t,k]  qw[e,n,k]
//   dgrad    dX[t,k]   = sum_b sdy[b,t] sw[e,b,k/128]  sum_{n in b} qdy[t,n] qw[e,n,k]
//   wgrad    dW[e,n,k] = sum_b sdy[b,n] sx[b,k]        sum_{t in b} qdy[t,n] qx[t,k]
//
// The tensor core sums the 128 products of a block in tensor memory (four K = 32
// kind::f8f6f4 MMAs from zero); the scales are no powers of two, so each block's
// partial sum is multiplied by its scale and added to fp32 sums in registers, while the
// next block's MMAs fill the other of two accumulators (2 x 256 of tensor memory's 512
// columns; there are no block scales to keep there).  wgrad's scale differs for every
// output element: one multiply more each.
//
// What bounds them.  A pair's M = 256, N = 256, K = 128 block takes 632 cycles of MMAs
// alone: their operands are 80 KB a block and SM, 625 cycles at shared memory's 128 bytes
// a cycle.  With the sums it takes about 850: the scales' reads and the barriers go
// through the same shared memory and the accumulator is held while it is read out.
// 65536 x 4096 x 7168, one expert: 1.34 ms, 2.88 PFLOP/s; dgrad 65536 x 7168 x 2048, 32 experts of
// 2048 rows: 0.74 ms, 2.59 PFLOP/s; wgrad of the same: 1.17 ms, 1.64 PFLOP/s (about 1290 cycles a block,
// the epilogue's: without its sums and products 800), to fp32 1.28 ms, added into fp32 3.14 ms (the epilogue's
// reads of dW follow one another; one expert 1.04 and 1.09 ms).
//
// One set of weight codes serves both directions: blocks are 128 x 128, and dgrad reads
// the same [n x k] codes as an MN-major operand (its contraction runs down the rows).
// wgrad reads both token-major operands MN-major, so no quantizer transposes anything.
//
// Tiles are 256 x 256 a pair, walked round-robin (see gemm_common.cuh); every ragged edge
// is cut by the tensor maps (zero fill) and the stores, so n and k only have to be
// multiples of 16.  No split over the contraction: a row's result does not depend on the
// other rows.  12 warps a CTA:
//   warp 0      TMA producer: A and B into a ring of 32 KB stages, completing on the leader's
//               barriers; the epilogue frees a stage when it sees the block's MMAs done;
//   warp 1      allocates tensor memory; in the leader one thread issues the MMAs, a commit per
//               block hands the accumulator to both CTAs' epilogues;
//   warps 2-3   bring the blocks' scales into shared memory, in turn (loads by the epilogue
//               threads themselves, a few blocks ahead in registers, kept them waiting on the loads:
//               2.09 -> 1.48 ms for 65536 x 4096 x 7168).  Four blocks' together where a row's scale is one
//               product a block, for fewer accesses (1.42 -> 1.36 ms);
//   warps 4-11  epilogue: 32 rows x 128 columns each, sums in 128 registers a thread.  Forward, dgrad: a
//               thread has a row, so a block needs one scale.  wgrad: a thread has four rows and 32 columns,
//               so 36 scales serve its 128 sums (one row: 129 scales, 256 reads of 16 bytes a block and SM:
//               1.18 -> 1.02 ms for 65536 x 7168 x 2048).
#include <algorithm>

#include "block128.cuh"
#include "gemm_common.cuh"

namespace fme {

namespace {

constexpr int kThreads128 = 384;
constexpr int kEpiWarp0 = 4;
constexpr int kStageBytes128 = kABytes + kBBytes;
constexpr int kStages128 = 4;
constexpr int kOutBlocks = 2;                // staging blocks a warp: its 32 x 128 bf16 outputs of a tile
constexpr int kOutBlockBytes = 32 * 128;
constexpr int kScaleWarp0 = 2;                // and 3
constexpr int kScaleSlots = 4;                // slots of blocks' scales in shared memory
constexpr int kScaleGroup = 4;                // blocks of a slot (forward, dgrad); wgrad's holds one
constexpr int kScaleSlotFloats = kScaleGroup * 2 * 128;  // forward, dgrad: [column half][row][block]
constexpr int kColSet = 36;                              // wgrad: a lane's 32 column scales, spread over the banks
constexpr int kScaleSlotFloatsW = 128 + 2 * 4 * kColSet;  // wgrad: rows, then [column half][lane % 4][column]
constexpr int kStageOut = 8 * kOutBlocks * kOutBlockBytes + kScaleSlots * kScaleSlotFloats * 4;

enum class Kind128 { kFwd, kDgrad, kWgrad };

struct Shared128 {
  uint64_t full[kStages128];
  uint64_t freed[kStages128];  // the stage's MMAs are done (own CTA)
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t sc_full[kScaleSlots];
  uint64_t sc_empty[kScaleSlots];
  uint64_t drain;
  uint64_t peer_fills_bar;
  uint32_t peer_fills;
  uint32_t tmem_base;
  int abort_flag;
  int ok_flag;
};

// One block of 128 of the contraction: D = A B^T over four K = 32 steps, E4M3 x E4M3 -> fp32,
// M = 256 over the pair, then a commit to the barrier at the same shared address in both CTAs.
// kA, kB: distance of the steps in the operands' descriptors (16-byte units).  One asm statement,
// issued by one elected lane of a converged warp: as single MMAs under `lane == 0` the issuing
// thread itself took about 900 cycles a block, more than the MMAs.
template <uint32_t kA, uint32_t kB>
__device__ __forceinline__ void mma_block(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred z, o;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.u32 z, 0, 0;\n\tsetp.eq.u32 o, 0, 0;\n\t"
      "add.s64 a1, %1, %5;\n\tadd.s64 a2, %1, 2 * %5;\n\tadd.s64 a3, %1, 3 * %5;\n\t"
      "add.s64 b1, %2, %6;\n\tadd.s64 b2, %2, 2 * %6;\n\tadd.s64 b3, %2, 3 * %6;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, z;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a1, b1, %3, o;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a2, b2, %3, o;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a3, b3, %3, o;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%4], %7;\n\t"
      "}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(smem_u32(bar)), "n"(kA), "n"(kB), "h"(static_cast<uint16_t>(3))
      : "memory");
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// Warps that work as one (epilogue, scales) give up as one, so that no lane is left waiting at a
// warp-wide instruction: a lane whose wait ran out goes on with the others, every later wait of the CTA
// ends at once, and the warp leaves at the next vote, before it writes the tile.  What it adds until then
// is garbage, and so may be what the pair's other warps add; but it frees no stage any more, so the producers'
// fills stay within a ring of those consumed, as the drain at the end assumes.  The vote is once for a few
// blocks: one at every wait cost 2.5% (65536 x 4096 x 7168: 1.36 -> 1.40 ms).
constexpr int kVoteBlocks = 8;
__device__ __forceinline__ bool warp_any(bool stop) { return __any_sync(0xFFFFFFFFu, stop); }

// Instruction descriptor: fp32 accumulator (bit 4), E4M3 operands (0), the operands'
// major-ness (bits 15, 16: 1 = MN-major), N / 8 and M / 16.
constexpr uint32_t idesc_f8(bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((256u >> 3) << 17) | ((256u >> 4) << 24);
}

// Shared-memory descriptor of a 128-byte-swizzled tile.  K-major: rows of 128 bytes of K,
// 8-row atoms 1024 bytes apart.  MN-major: rows of 128 M or N values, one row for each k,
// 8-k atoms 1024 bytes apart (a CTA's 128 values are one atom wide, so the other stride
// is not used and holds the same value).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, bool mn) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFF) >> 4);
  d |= static_cast<uint64_t>((mn ? 1024 : 16) >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, uint32_t bar_cluster_addr,
                                                 int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// tcgen05.wait::ld that the 32 loaded registers depend on, so that no use of them can be
// moved before it.
__device__ __forceinline__ void tmem_wait_ld_for(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void tmem_wait_ld_for(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15])::"memory");
}

// 16 lanes x 32 columns: of each 8 columns a thread gets those at 2 (lane % 4) and the next, of rows
// lane / 4 and lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Expert tables in shared memory: first row and first 256-row block of each expert (forward,
// dgrad), or padded offsets and experts by decreasing work (wgrad).
struct Tables {
  int32_t *off;
  int32_t *aux;
};

struct Tile128 {
  int32_t e;
  int32_t nk;          // contraction blocks
  int32_t row0;        // this CTA's first output row: of all rows (fwd, dgrad) or of the expert's (wgrad)
  int32_t rows_valid;  // of its 128
  int32_t col0;        // first output column of the tile
  int32_t p0;          // wgrad: first padded position
};

// Tiles and their counts are in 32 bits (checked on the host).
template <Kind128 K>
__device__ __forceinline__ Tile128 tile128(const LaunchBlock128 &p, const Tables &s, uint32_t t, int rank) {
  Tile128 tl;
  const uint32_t nb = (static_cast<uint32_t>(p.n) + kBN - 1) / kBN;
  if constexpr (K == Kind128::kWgrad) {
    const uint32_t per = (static_cast<uint32_t>(p.m) + kPairM - 1) / kPairM * nb;
    const uint32_t order = t / per;
    const uint32_t rem = t - order * per;
    const uint32_t row = rem / nb;
    tl.e = s.aux[order];
    tl.p0 = s.off[tl.e];
    tl.nk = (s.off[tl.e + 1] - tl.p0) >> 7;
    tl.row0 = static_cast<int32_t>(row * kPairM + rank * kBM);
    tl.rows_valid = min(kBM, static_cast<int32_t>(p.m) - tl.row0);
    tl.col0 = static_cast<int32_t>((rem - row * nb) * kBN);
  } else {
    const uint32_t g = t / nb;
    tl.col0 = static_cast<int32_t>((t - g * nb) * kBN);
    tl.e = find_group(s.aux, p.num_experts, g);
    const int32_t first = (static_cast<int32_t>(g) - s.aux[tl.e]) * kPairM + rank * kBM;
    tl.row0 = s.off[tl.e] + first;
    tl.rows_valid = min(kBM, s.off[tl.e + 1] - s.off[tl.e] - first);
    tl.nk = static_cast<int32_t>((p.k + 127) >> 7);
    tl.p0 = 0;
  }
  return tl;
}

// 32 rows x 32 columns of sums to global memory.  `ld` output columns a row; columns at or
// past `cols_left` and rows at or past `rows_valid` are not written.
__device__ __forceinline__ void store_block_cut(__nv_bfloat16 *dst, int64_t ld, int rows_valid, int cols_left,
                                                uint8_t *stage, int lane, const uint32_t (&packed)[16]) {
  uint8_t *row = stage + lane * 64;
  const int x = (lane >> 1) & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4 *>(row + 16 * (j ^ x)) =
        make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
  __syncwarp();
  const int j = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    const uint4 v = *reinterpret_cast<const uint4 *>(stage + r * 64 + 16 * (j ^ ((r >> 1) & 3)));
    if (r < rows_valid && 8 * j < cols_left) *reinterpret_cast<uint4 *>(dst + r * ld + 8 * j) = v;
  }
  __syncwarp();
}

// wgrad: a staged block (32 rows of 128 bytes, swizzled) to columns `col` on, by plain stores; with
// p.accumulate added to dW (one unfused add an element).  Past the output's edge nothing is written.
__device__ __forceinline__ void store_staged(const LaunchBlock128 &p, bool fp32, int64_t out_row, int64_t col,
                                             int rows_valid, const uint8_t *blk, int lane) {
  const int j = lane & 7;
  col += (fp32 ? 4 : 8) * j;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    float4 v = *reinterpret_cast<const float4 *>(blk + r * 128 + 16 * (j ^ (r & 7)));
    if (r < rows_valid && col < p.n) {
      const int64_t at = (out_row + r) * p.n + col;
      float4 *to = fp32 ? reinterpret_cast<float4 *>(static_cast<float *>(p.y) + at)
                        : reinterpret_cast<float4 *>(static_cast<__nv_bfloat16 *>(p.y) + at);
      if (fp32 && p.accumulate) {
        const float4 b = *to;
        v = make_float4(__fadd_rn(b.x, v.x), __fadd_rn(b.y, v.y), __fadd_rn(b.z, v.z), __fadd_rn(b.w, v.w));
      }
      *to = v;
    }
  }
}

template <Kind128 K>
__global__ void __launch_bounds__(kThreads128, 1) gemm_block128_kernel(const __grid_constant__ LaunchBlock128 p) {
  constexpr bool kAmn = K == Kind128::kWgrad;
  constexpr bool kBmn = K != Kind128::kFwd;
  __shared__ Shared128 s;
  extern __shared__ uint8_t dyn_smem[];
  constexpr int S = kStages128;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  uint8_t *smem_a = smem;
  uint8_t *smem_b = smem_a + S * kABytes;
  uint8_t *smem_out = smem + S * kStageBytes128;
  float *scales = reinterpret_cast<float *>(smem_out + 8 * kOutBlocks * kOutBlockBytes);
  int32_t *gmem = reinterpret_cast<int32_t *>(smem_out + kStageOut);
  const Tables tab{gmem, gmem + (p.num_experts + 1)};

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(pair::cta_rank());
  const uint32_t pair_id = blockIdx.x >> 1;
  const uint32_t pairs = gridDim.x >> 1;

  if (threadIdx.x == 32) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.freed[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], kAccEmptyArrivals);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(&s.sc_full[i], 1);
      mbar_init(&s.sc_empty[i], 8);
    }
    mbar_init(&s.drain, 1);
    mbar_init(&s.peer_fills_bar, 1);
    s.abort_flag = 0;
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
  if constexpr (K == Kind128::kWgrad) {
    if (warp == 0) {
      bool ok = true;
      for (int e = lane; e <= p.num_experts; e += 32) {
        const int32_t v = p.offsets[e];
        const int32_t before = e ? p.offsets[e - 1] : 0;
        if ((e == 0 && v != 0) || v < before || (v & 127) != 0 || v > p.positions) ok = false;
        tab.off[e] = v;
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (lane == 0) s.ok_flag = ok;
    }
    __syncthreads();
    if (s.ok_flag) {
      for (int e = threadIdx.x; e < p.num_experts; e += kThreads128) {
        const int32_t w = tab.off[e + 1] - tab.off[e];
        int order = 0;
        for (int f = 0; f < p.num_experts; ++f) {
          const int32_t wf = tab.off[f + 1] - tab.off[f];
          order += (wf > w) || (wf == w && f < e);
        }
        tab.aux[order] = e;
      }
    }
  } else if (warp == 0) {
    const int32_t total = scan_groups(p.offsets, p.num_experts, p.m, kPairM,
                                      [&](int g, int32_t lo, int32_t, int32_t first) {
                                        tab.off[g] = lo;
                                        tab.aux[g] = first;
                                      });
    if (lane == 0) {
      tab.off[p.num_experts] = static_cast<int32_t>(p.m);
      tab.aux[p.num_experts] = total;
      s.ok_flag = total >= 0;
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
  // walked backwards, so that a pair with a long tile gets a short one next (1999 rows, 8 experts of
  // 1040 x 1392: 22 -> 20 us).
  auto tile_at = [&](uint32_t round) {
    return round * pairs + (K == Kind128::kWgrad && (round & 1) ? pairs - 1 - pair_id : pair_id);
  };
  const uint32_t nb = static_cast<uint32_t>((p.n + kBN - 1) / kBN);
  // malformed offsets: no tile, straight to the end
  if (!s.ok_flag && blockIdx.x == 0 && threadIdx.x == 0) report(p.status, kDevBadOffsets);
  const uint32_t total =
      !s.ok_flag ? 0
                 : (K == Kind128::kWgrad ? p.num_experts * static_cast<uint32_t>((p.m + kPairM - 1) / kPairM)
                                         : tab.aux[p.num_experts]) *
                       nb;

  if (warp < kEpiWarp0) {
    // 128 threads x 56 + 256 x 224 registers = the launch's 384 x 168
    regs_dec<56>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- producer
      uint32_t stage = 0, filled = 0;
      bool stop = false;
      for (uint32_t round = 0, t; (t = tile_at(round)) < total && !stop; ++round) {
        const Tile128 tl = tile128<K>(p, tab, t, rank);
        for (int i = 0; i < tl.nk; ++i) {
          if (!mbar_wait<true>(&s.freed[stage], ((filled / S) & 1) ^ 1, abort_flag, p.status)) {
            stop = true;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&s.full[stage], 2 * kStageBytes128);
          const uint32_t bar = pair::map_to_rank(&s.full[stage], 0);
          uint8_t *a = smem_a + stage * kABytes, *b = smem_b + stage * kBBytes;
          const int32_t bcol = tl.col0 + rank * kHalfN;
          if constexpr (K == Kind128::kWgrad) {
            pair::tma_load_2d(a, &p.map_a, bar, tl.row0, tl.p0 + i * 128);
            pair::tma_load_2d(b, &p.map_b, bar, bcol, tl.p0 + i * 128);
          } else {
            pair::tma_load_2d(a, &p.map_a, bar, i * 128, tl.row0);
            if constexpr (K == Kind128::kFwd)
              tma_load_3d_pair(b, &p.map_b, bar, i * 128, bcol, tl.e);
            else
              tma_load_3d_pair(b, &p.map_b, bar, bcol, i * 128, tl.e);
          }
          ++filled;
          if (++stage == S) stage = 0;
        }
      }
      const uint32_t peer = exchange_fills(rank, filled, &s.peer_fills, &s.peer_fills_bar, p.status);
      if (rank == 0) drain_pair_ring(s.full, S, filled, peer, kStageBytes128);
    } else if (warp == 1 && rank == 0) {
      // ------------------------------------------- MMA issuer (leader, whole warp)
      constexpr uint32_t idesc = idesc_f8(kAmn, kBmn);
      const uint64_t a_desc = desc_sw128(smem_u32(smem_a), kAmn), b_desc = desc_sw128(smem_u32(smem_b), kBmn);
      uint32_t stage = 0, phase = 0, fill = 0;
      bool stop = false;
      for (uint32_t round = 0, t; (t = tile_at(round)) < total && !stop; ++round) {
        const int nk = tile128<K>(p, tab, t, 0).nk;
        for (int i = 0; i < nk; ++i) {
          const uint32_t b = fill & 1;
          if (!mbar_wait(&s.full[stage], phase, abort_flag, p.status) ||
              !mbar_wait(&s.acc_empty[b], ((fill >> 1) & 1) ^ 1, abort_flag, p.status)) {
            stop = true;
          }
          stop = __any_sync(0xFFFFFFFFu, stop);
          if (stop) break;
          tc_fence_after();
          // 32 of K: 32 bytes along a K-major row, 32 rows of an MN-major tile
          if (elect_one())
            mma_block<(kAmn ? 4096 : 32) / 16, (kBmn ? 4096 : 32) / 16>(
                tmem + b * kBN, a_desc + stage * (kABytes / 16), b_desc + stage * (kBBytes / 16), idesc, &s.acc_full[b]);
          __syncwarp();
          ++fill;
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
    } else if (warp >= kScaleWarp0) {
      // ------------------------------------------------------------------ scales
      // Forward, dgrad: slot[half][row][block] = scale of the row times that of the weight block of the
      // column half, four blocks a slot.  wgrad: slot[row], then the tile's 256 column scales, one block
      // a slot.  Each of the two warps takes every other slot.
      uint32_t g = 0;
      bool stop = false;
      const int64_t kb_count = (p.k + 127) >> 7;
      const int64_t nb128 = (p.n + 127) >> 7;
      for (uint32_t round = 0, t; (t = tile_at(round)) < total && !stop; ++round) {
        const Tile128 tl = tile128<K>(p, tab, t, rank);
        if constexpr (K == Kind128::kWgrad) {
          const float *a = p.a_scale + (tl.p0 >> 7) * p.m + tl.row0;
          for (int i = 0; i < tl.nk; ++i, ++g) {
            if ((g & 1) != (warp & 1)) continue;
            const uint32_t slot = g % kScaleSlots;
            float *dst = scales + slot * kScaleSlotFloatsW;
            float ra[4], cb[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = lane + 32 * j;
              ra[j] = r < tl.rows_valid ? a[i * p.m + r] : 0.0f;
            }
            const float *b = p.b_scale + ((tl.p0 >> 7) + i) * p.n + tl.col0;
#pragma unroll
            for (int j = 0; j < 8; ++j) cb[j] = tl.col0 + lane + 32 * j < p.n ? b[lane + 32 * j] : 0.0f;
            stop = warp_any(!mbar_wait<true>(&s.sc_empty[slot], ((g / kScaleSlots) & 1) ^ 1, abort_flag, p.status));
            if (stop) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[32 * j + 4 * (lane & 7) + (lane >> 3)] = ra[j];
#pragma unroll
            for (int j = 0; j < 8; ++j)  // column lane + 32 (j % 4) of half j / 4
              dst[128 + ((j >> 2) * 4 + ((lane >> 1) & 3)) * kColSet + 8 * (j & 3) + 2 * (lane >> 3) + (lane & 1)] = cb[j];
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.sc_full[slot]);
          }
        } else {
          const float *a = p.a_scale + tl.row0;
          for (int i0 = 0; i0 < tl.nk; i0 += kScaleGroup, ++g) {
            if ((g & 1) != (warp & 1)) continue;
            const uint32_t slot = g % kScaleSlots;
            float4 *dst = reinterpret_cast<float4 *>(scales + slot * kScaleSlotFloats);
            float ra[4][kScaleGroup], cb[2][kScaleGroup];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = lane + 32 * j;
#pragma unroll
              for (int u = 0; u < kScaleGroup; ++u)
                ra[j][u] = r < tl.rows_valid && i0 + u < tl.nk ? a[(i0 + u) * p.m + r] : 0.0f;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int64_t c = (tl.col0 >> 7) + h;
#pragma unroll
              for (int u = 0; u < kScaleGroup; ++u) {
                const int64_t i = i0 + u;
                const int64_t at = K == Kind128::kFwd ? (tl.e * nb128 + c) * kb_count + i : (tl.e * kb_count + i) * nb128 + c;
                cb[h][u] = c < nb128 && i < tl.nk ? p.b_scale[at] : 0.0f;
              }
            }
            stop = warp_any(!mbar_wait<true>(&s.sc_empty[slot], ((g / kScaleSlots) & 1) ^ 1, abort_flag, p.status));
            if (stop) break;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                dst[h * 128 + lane + 32 * j] =
                    make_float4(ra[j][0] * cb[h][0], ra[j][1] * cb[h][1], ra[j][2] * cb[h][2], ra[j][3] * cb[h][3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.sc_full[slot]);
          }
        }
      }
    }
  } else {
    // ----------------------------------------------------------------- epilogue
    regs_inc<224>();
    const int ew = warp - kEpiWarp0;
    const int q = warp & 3;         // tensor-memory lane quarter
    const int half = ew >> 2;       // column half of the tile
    const int r = q * 32 + lane;    // row of the CTA's 128
    uint8_t *stage_blks = smem_out + ew * kOutBlocks * kOutBlockBytes;
    const uint32_t leader_empty[2] = {pair::map_to_rank(&s.acc_empty[0], 0), pair::map_to_rank(&s.acc_empty[1], 0)};
    const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * 128;
    uint32_t g = 0, sg = 0;  // blocks and scale groups so far
    bool stop = false;
    Tile128 next{};
    if (pair_id < total) next = tile128<K>(p, tab, pair_id, rank);
    for (uint32_t round = 0, t; (t = tile_at(round)) < total && !stop; ++round) {
      const Tile128 tl = next;
      if (tile_at(round + 1) < total) next = tile128<K>(p, tab, tile_at(round + 1), rank);  // while the MMAs of this one run
      const int c0 = tl.col0 + half * 128;
      const bool in_cols = c0 < p.n;
      float2 acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
      // Forward, dgrad: the block's four chunks of 32 columns, loaded while the one before is summed, the accumulator
      // released as soon as the last is in registers.
      auto sum_block = [&](uint32_t b, auto add) {
        const uint32_t tb = tq + b * kBN;
        uint32_t va[32], vb[32];
        tmem_ld_32x32(tb, va);
        tmem_wait_ld_for(va);
        tmem_ld_32x32(tb + 32, vb);
        add(0, va);
        tmem_wait_ld_for(vb);
        tmem_ld_32x32(tb + 64, va);
        add(1, vb);
        tmem_wait_ld_for(va);
        tmem_ld_32x32(tb + 96, vb);
        add(2, va);
        tmem_wait_ld_for(vb);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) pair::arrive_remote_relaxed(leader_empty[b]);
        add(3, vb);
      };
      if constexpr (K == Kind128::kWgrad) {
#pragma unroll 1
        for (int i = 0; i < tl.nk; ++i) {
          const uint32_t b = g & 1;
          const uint32_t slot = g % kScaleSlots;
          if (!mbar_wait(&s.sc_full[slot], (g / kScaleSlots) & 1, abort_flag, p.status)) stop = true;
          const float *sc = scales + slot * kScaleSlotFloatsW;
          const float4 rs = *reinterpret_cast<const float4 *>(sc + 32 * q + 4 * (lane >> 2));
          const float2 rf[4] = {make_float2(rs.x, rs.x), make_float2(rs.y, rs.y), make_float2(rs.z, rs.z),
                                make_float2(rs.w, rs.w)};
          const float4 *cs = reinterpret_cast<const float4 *>(sc + 128 + (half * 4 + (lane & 3)) * kColSet);
          if (!mbar_wait(&s.acc_full[b], (g >> 1) & 1, abort_flag, p.status)) stop = true;
          if (i % kVoteBlocks == kVoteBlocks - 1 && warp_any(stop)) {
            stop = true;
            break;
          }
          // the block's MMAs are done: its operands' stage is free
          if (ew == 0 && lane == 0 && !stop) mbar_arrive(&s.freed[g % S]);
          tc_fence_after();
          // Chunks of 16 rows x 32 columns, the two row halves of the columns in turn.
          float4 cv[2];
          const uint32_t tb = tq + b * kBN;
          auto at = [&](int c) { return tb + (static_cast<uint32_t>((c & 1) * 16) << 16) + (c >> 1) * 32; };
          auto add = [&](int c, const uint32_t(&d)[16]) {
            if ((c & 1) == 0) cv[0] = cs[c], cv[1] = cs[c + 1];
            float2 f[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                f[u][j] = __fmul2_rn(j & 1 ? make_float2(cv[j / 2].z, cv[j / 2].w) : make_float2(cv[j / 2].x, cv[j / 2].y),
                                     rf[2 * (c & 1) + u]);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float2 &to = acc[32 * (c & 1) + 16 * u + (c >> 1) * 4 + j];
                to = __ffma2_rn(f[u][j], make_float2(__uint_as_float(d[4 * j + 2 * u]), __uint_as_float(d[4 * j + 2 * u + 1])), to);
              }
          };
          uint32_t va[16], vb[16];
          tmem_ld_16x256b(at(0), va);
          tmem_wait_ld_for(va);
#pragma unroll
          for (int c = 0; c < 8; c += 2) {
            tmem_ld_16x256b(at(c + 1), vb);
            add(c, va);
            tmem_wait_ld_for(vb);
            if (c < 6) {
              tmem_ld_16x256b(at(c + 2), va);
            } else {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) pair::arrive_remote_relaxed(leader_empty[b]);
            }
            add(c + 1, vb);
            if (c < 6) tmem_wait_ld_for(va);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.sc_empty[slot]);
          ++g;
        }
      } else {
#pragma unroll 1
        for (int i0 = 0; i0 < tl.nk; i0 += kScaleGroup, ++sg) {
          const uint32_t slot = sg % kScaleSlots;
          if (!mbar_wait(&s.sc_full[slot], (sg / kScaleSlots) & 1, abort_flag, p.status)) stop = true;
          stop = warp_any(stop);
          if (stop) break;
          const float4 f4 = reinterpret_cast<const float4 *>(scales + slot * kScaleSlotFloats)[half * 128 + r];
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.sc_empty[slot]);
#pragma unroll
          for (int u = 0; u < kScaleGroup; ++u) {
            if (i0 + u >= tl.nk) continue;
            const uint32_t b = g & 1;
            const float v = u == 0 ? f4.x : u == 1 ? f4.y : u == 2 ? f4.z : f4.w;
            const float2 f = make_float2(v, v);
            if (!mbar_wait(&s.acc_full[b], (g >> 1) & 1, abort_flag, p.status)) stop = true;
            if (ew == 0 && lane == 0 && !stop) mbar_arrive(&s.freed[g % S]);
            tc_fence_after();
            auto add = [&](int c, const uint32_t(&d)[32]) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float2 x = make_float2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1]));
                acc[16 * c + j] = __ffma2_rn(x, f, acc[16 * c + j]);
              }
            };
            sum_block(b, add);
            ++g;
          }
        }
      }
      stop = warp_any(stop);
      if (stop) break;
      // ---- the tile's sums out
      const int warp_rows = tl.rows_valid - 32 * q;
      if (warp_rows <= 0 || !in_cols) continue;
      const int64_t out_row = (K == Kind128::kWgrad ? tl.e * p.m : int64_t(0)) + tl.row0 + 32 * q;
      // 4 KB blocks of 32 rows x 64 bf16 or 32 fp32 columns in the warp's staging area.  A whole
      // one leaves by a bulk store: two blocks are written, made visible and stored together (one
      // wait, one fence, two stores: issuing a store takes a few hundred cycles next to the loads); one
      // cut by the output's edge, and sums added to dW, by plain stores.
      const int xs = lane & 7;  // the 128-byte swizzle of this lane's row
      auto await_staging = [&] {
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
      };
      if constexpr (K == Kind128::kWgrad) {
        const bool fp32 = p.out_fp32;
        if (fp32 && tl.nk == 0 && p.accumulate) continue;
        const int fr = lane >> 2, fc = lane & 3;  // rows fr + 8 i, columns 2 fc and the next of each 8
#pragma unroll
        for (int half_tile = 0; half_tile < 2; ++half_tile) {
          if (!fp32 && half_tile == 1) break;
          const int wide = fp32 ? 32 : 64;
          const int base = c0 + half_tile * 64;
          if (base >= p.n) break;
          const int whole = (fp32 && p.accumulate) || warp_rows < 32 ? 0 : min(2, (static_cast<int>(p.n) - base) / wide);
          await_staging();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint8_t *row = stage_blks + (fr + 8 * i) * 128;
            if (fp32) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float2 *>(row + (j >> 2) * kOutBlockBytes + 16 * ((2 * (j & 3) + (fc >> 1)) ^ fr) +
                                            8 * (fc & 1)) = acc[16 * i + 8 * half_tile + j];
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                *reinterpret_cast<__nv_bfloat162 *>(row + (j >> 3) * kOutBlockBytes + 16 * ((j & 7) ^ fr) + 4 * fc) =
                    __floats2bfloat162_rn(acc[16 * i + j].x, acc[16 * i + j].y);
            }
          }
          if (whole > 0) fence_proxy_async_shared();
          __syncwarp();
          if (whole > 0 && lane == 0) {
            for (int c = 0; c < whole; ++c)
              tma_store_2d(&p.map_y, base + wide * c, static_cast<int32_t>(out_row), stage_blks + c * kOutBlockBytes);
            bulk_commit();
          }
          for (int c = whole; c < 2; ++c)
            store_staged(p, fp32, out_row, base + wide * c, warp_rows, stage_blks + c * kOutBlockBytes, lane);
        }
      } else {
        const int whole = warp_rows < 32 ? 0 : min(2, (static_cast<int>(p.n) - c0) / 64);
        await_staging();
        if (whole > 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint4 *row = reinterpret_cast<uint4 *>(stage_blks + c * kOutBlockBytes + lane * 128);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(acc[32 * c + 4 * j + i].x, acc[32 * c + 4 * j + i].y);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
              }
              row[j ^ xs] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            for (int c = 0; c < whole; ++c)
              tma_store_2d(&p.map_y, c0 + 64 * c, static_cast<int32_t>(out_row), stage_blks + c * kOutBlockBytes);
            bulk_commit();
          }
        }
        if (whole < 2 && c0 + 64 * whole < p.n) {
          await_staging();
          const int done = c0 + 64 * whole;  // columns before it are stored
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int col = c0 + 32 * c;
            if (col < done || col >= p.n) continue;
            uint32_t packed[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(acc[16 * c + j].x, acc[16 * c + j].y);
              packed[j] = *reinterpret_cast<const uint32_t *>(&h);
            }
            store_block_cut(static_cast<__nv_bfloat16 *>(p.y) + out_row * p.n + col, p.n, warp_rows,
                            static_cast<int>(p.n) - col, stage_blks, lane, packed);
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
// The same sums with the operands exchanged: an item is 128 rows of W_e (the MMA's M) and up to 64
// of the expert's tokens (its N, in steps of 16), one CTA an item.  With few tokens the time is that
// of reading the weights once, and 256-row token tiles would leave all but a few rows of the MMAs
// empty and put the weights on half as many SMs.  Each block's 16 KB of codes go through a ring of
// eight stages; the sums of up to four blocks are in tensor memory; thread = row of W, its
// tokens' sums in registers, scaled by sx[b,t] sw[e,n/128,b] exactly as above, in the same order of
// b: a row's bits are the same in both forms.
//   warp 0 producer, warp 1 MMA issuer, warps 2-3 scales (two blocks each in turn), warps 4-7 epilogue.
constexpr int kFewTokens = 64;
constexpr int kFewStages = 8;
constexpr int kFewAccs = 4;
constexpr int kFewSlots = 8;
constexpr int kFewThreads = 256;
constexpr int kFewBBytes = kFewTokens * kStageKBytes;
constexpr int kFewStageBytes = kABytes + kFewBBytes;
constexpr uint32_t kFewTmemCols = kFewAccs * kFewTokens;

struct SharedFew {
  uint64_t full[kFewStages];
  uint64_t freed[kFewStages];
  uint64_t acc_full[kFewAccs];
  uint64_t acc_empty[kFewAccs];
  uint64_t sc_full[kFewSlots];
  uint64_t sc_empty[kFewSlots];
  uint64_t drain;
  alignas(16) float scales[kFewSlots][kFewTokens];  // read as float4
  uint32_t tmem_base;
  int abort_flag;
  int ok_flag;
};

__device__ __forceinline__ void tma_load_2d_own(void *dst, const CUtensorMap *map, uint64_t *bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_own(void *dst, const CUtensorMap *map, uint64_t *bar, int32_t x, int32_t y,
                                                int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// One block on one CTA (M = 128), both operands K-major, and its commit.
__device__ __forceinline__ void mma_block_own(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred z, o;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.u32 z, 0, 0;\n\tsetp.eq.u32 o, 0, 0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, z;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, o;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, o;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, o;\n\t"
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
      "}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(smem_u32(bar))
      : "memory");
}

// 32 lanes x 16 columns, and the wait for them.
__device__ __forceinline__ void tmem_ld_32x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
struct ItemFew {
  int32_t e;
  int32_t row0;    // first token row
  int32_t tokens;  // 1 .. 64
  int32_t n0;      // first row of W_e = output column
};
__device__ __forceinline__ ItemFew item_few(const LaunchBlock128 &p, const Tables &s, int64_t t) {
  const int64_t nb = (p.n + kBM - 1) / kBM;
  const int64_t g = t / nb;
  ItemFew it;
  it.n0 = static_cast<int32_t>((t - g * nb) * kBM);
  it.e = find_group(s.aux, p.num_experts, g);
  const int32_t first = static_cast<int32_t>(g - s.aux[it.e]) * kFewTokens;
  it.row0 = s.off[it.e] + first;
  it.tokens = min(kFewTokens, s.off[it.e + 1] - s.off[it.e] - first);
  return it;
}

__global__ void __launch_bounds__(kFewThreads, 1) gemm_block128_few_kernel(const __grid_constant__ LaunchBlock128 p) {
  __shared__ SharedFew s;
  extern __shared__ uint8_t dyn_smem[];
  constexpr int S = kFewStages;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  uint8_t *smem_a = smem;
  uint8_t *smem_b = smem_a + S * kABytes;
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
    for (int i = 0; i < S; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.freed[i], 1);
    }
    for (int i = 0; i < kFewAccs; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], 4);
    }
    for (int i = 0; i < kFewSlots; ++i) {
      mbar_init(&s.sc_full[i], 1);
      mbar_init(&s.sc_empty[i], 4);
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
    const int32_t total = scan_groups(p.offsets, p.num_experts, p.m, kFewTokens,
                                      [&](int g, int32_t lo, int32_t, int32_t first) {
                                        tab.off[g] = lo;
                                        tab.aux[g] = first;
                                      });
    if (lane == 0) {
      tab.off[p.num_experts] = static_cast<int32_t>(p.m);
      tab.aux[p.num_experts] = total;
      s.ok_flag = total >= 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  volatile int *abort_flag = &s.abort_flag;
  const int nk = static_cast<int>((p.k + 127) >> 7);
  const int64_t nb = (p.n + kBM - 1) / kBM;
  // malformed offsets: no item, straight to the end
  const int64_t total = s.ok_flag ? static_cast<int64_t>(tab.aux[p.num_experts]) * nb : 0;
  if (!s.ok_flag && blockIdx.x == 0 && threadIdx.x == 0) report(p.status, kDevBadOffsets);

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------------------- producer
      uint32_t stage = 0, filled = 0;
      bool stop = false;
      for (int64_t t = blockIdx.x; t < total && !stop; t += gridDim.x) {
        const ItemFew it = item_few(p, tab, t);
        const int groups = (it.tokens + 15) >> 4;
        for (int i = 0; i < nk; ++i) {
          if (!mbar_wait<true>(&s.freed[stage], ((filled / S) & 1) ^ 1, abort_flag, p.status)) {
            stop = true;
            break;
          }
          mbar_arrive_expect_tx(&s.full[stage], kABytes + groups * 16 * kStageKBytes);
          tma_load_3d_own(smem_a + stage * kABytes, &p.map_a, &s.full[stage], i * 128, it.n0, it.e);
          for (int j = 0; j < groups; ++j)
            tma_load_2d_own(smem_b + stage * kFewBBytes + j * 16 * kStageKBytes, &p.map_b, &s.full[stage], i * 128,
                            it.row0 + 16 * j);
          ++filled;
          if (++stage == S) stage = 0;
        }
      }
      // every copy has landed before the CTA can exit
      for (uint32_t j = 0; j < S && j < filled; ++j) {
        const uint32_t f = j + S * ((filled - 1 - j) / S);
        mbar_drain(&s.full[j], (f / S) & 1);
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------- MMA issuer (whole warp)
    const uint64_t a_desc = desc_sw128(smem_u32(smem_a), false), b_desc = desc_sw128(smem_u32(smem_b), false);
    uint32_t stage = 0, phase = 0, fill = 0;
    bool stop = false;
    for (int64_t t = blockIdx.x; t < total && !stop; t += gridDim.x) {
      const uint32_t cols = (item_few(p, tab, t).tokens + 15) & ~15;
      const uint32_t idesc = (1u << 4) | ((cols >> 3) << 17) | ((128u >> 4) << 24);
      for (int i = 0; i < nk; ++i) {
        const uint32_t b = fill % kFewAccs;
        if (!mbar_wait(&s.full[stage], phase, abort_flag, p.status) ||
            !mbar_wait(&s.acc_empty[b], ((fill / kFewAccs) & 1) ^ 1, abort_flag, p.status))
          stop = true;
        stop = __any_sync(0xFFFFFFFFu, stop);
        if (stop) break;
        tc_fence_after();
        if (elect_one())
          mma_block_own(tmem + b * kFewTokens, a_desc + stage * (kABytes / 16), b_desc + stage * (kFewBBytes / 16), idesc,
                        &s.acc_full[b]);
        __syncwarp();
        ++fill;
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    __syncwarp();
    if (elect_one()) {
      asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                       smem_u32(&s.drain))
                   : "memory");
      mbar_drain(&s.drain, 0);
    }
    __syncwarp();
  } else if (warp < kEpiWarp0) {
    // -------------------------------------------------------------------- scales
    const int which = warp - kScaleWarp0;  // of every four blocks, this warp's first is 2 * which
    uint32_t g = 0;                        // blocks of earlier items
    bool stop = false;
    for (int64_t t = blockIdx.x; t < total && !stop; t += gridDim.x, g += nk) {
      const ItemFew it = item_few(p, tab, t);
      const float *a = p.a_scale + it.row0;
      const float *b = p.b_scale + (it.e * nb + (it.n0 >> 7)) * nk;
      for (int i0 = 2 * which; i0 < nk && !stop; i0 += 4) {
        float v[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = i0 + u;
          const float w = i < nk ? b[i] : 0.0f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int tok = lane + 32 * h;
            v[u][h] = i < nk && tok < it.tokens ? a[i * p.m + tok] * w : 0.0f;
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (i0 + u >= nk) break;
          const uint32_t q = g + i0 + u, slot = q % kFewSlots;
          stop = warp_any(!mbar_wait<true>(&s.sc_empty[slot], ((q / kFewSlots) & 1) ^ 1, abort_flag, p.status));
          if (stop) break;
          s.scales[slot][lane] = v[u][0];
          s.scales[slot][lane + 32] = v[u][1];
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.sc_full[slot]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t g = 0;
    bool stop = false;
    for (int64_t t = blockIdx.x; t < total && !stop; t += gridDim.x) {
      const ItemFew it = item_few(p, tab, t);
      float acc[kFewTokens];
#pragma unroll
      for (int j = 0; j < kFewTokens; ++j) acc[j] = 0.0f;
#pragma unroll 1
      for (int i = 0; i < nk; ++i, ++g) {
        const uint32_t b = g % kFewAccs, slot = g % kFewSlots;
        if (!mbar_wait(&s.sc_full[slot], (g / kFewSlots) & 1, abort_flag, p.status) ||
            !mbar_wait(&s.acc_full[b], (g / kFewAccs) & 1, abort_flag, p.status))
          stop = true;
        if (i % kVoteBlocks == kVoteBlocks - 1 && warp_any(stop)) {
          stop = true;
          break;
        }
        if (warp == kEpiWarp0 && lane == 0 && !stop) mbar_arrive(&s.freed[g % S]);  // the block's MMAs are done
        tc_fence_after();
        const float4 *f = reinterpret_cast<const float4 *>(s.scales[slot]);
#pragma unroll
        for (int c = 0; c < kFewTokens / 16; ++c) {
          if (16 * c < it.tokens) {
            uint32_t v[16];
            tmem_ld_32x16(tq + b * kFewTokens + 16 * c, v);
            tmem_wait_ld_for(v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 w = f[4 * c + j];
              acc[16 * c + 4 * j] = __fmaf_rn(__uint_as_float(v[4 * j]), w.x, acc[16 * c + 4 * j]);
              acc[16 * c + 4 * j + 1] = __fmaf_rn(__uint_as_float(v[4 * j + 1]), w.y, acc[16 * c + 4 * j + 1]);
              acc[16 * c + 4 * j + 2] = __fmaf_rn(__uint_as_float(v[4 * j + 2]), w.z, acc[16 * c + 4 * j + 2]);
              acc[16 * c + 4 * j + 3] = __fmaf_rn(__uint_as_float(v[4 * j + 3]), w.w, acc[16 * c + 4 * j + 3]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s.acc_empty[b]);
          mbar_arrive(&s.sc_empty[slot]);
        }
      }
      stop = warp_any(stop);
      if (stop) break;
      const int64_t col = it.n0 + q * 32 + lane;
      if (col < p.n) {
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y) + static_cast<int64_t>(it.row0) * p.n + col;
#pragma unroll
        for (int j = 0; j < kFewTokens; ++j)
          if (j < it.tokens) y[j * p.n] = __float2bfloat16_rn(acc[j]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kFewTmemCols) : "memory");
}

template <Kind128 K>
cudaError_t launch128(const LaunchBlock128 &a) {
  const int smem = 1024 + kStages128 * kStageBytes128 + kStageOut + 8 * (a.num_experts + 1);
  auto kernel = gemm_block128_kernel<K>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_shared(reinterpret_cast<const void *>(kernel), allowed);
  if (err != cudaSuccess) return err;
  const int64_t nb = (a.n + kBN - 1) / kBN;
  const int64_t bound = K == Kind128::kWgrad ? a.num_experts * ((a.m + kPairM - 1) / kPairM) * nb
                                             : (a.m / kPairM + std::min<int64_t>(a.num_experts, a.m)) * nb;
  int64_t pairs = a.num_sms / 2;
  if (bound < pairs) pairs = bound;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(kThreads128, 1, 1);
  cfg.dynamicSmemBytes = smem;
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

cudaError_t launch_few(const LaunchBlock128 &a) {
  const int smem = 1024 + kFewStages * kFewStageBytes + 8 * (a.num_experts + 1);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_shared(reinterpret_cast<const void *>(gemm_block128_few_kernel), allowed);
  if (err != cudaSuccess) return err;
  const int64_t items = (a.m / kFewTokens + std::min<int64_t>(a.num_experts, a.m)) * ((a.n + kBM - 1) / kBM);
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
  return cudaLaunchKernelEx(&cfg, gemm_block128_few_kernel, a);
}

}  // namespace

cudaError_t launch_block128_fwd(const LaunchBlock128 &a) {
  return block128_few_rows(a.m, a.num_experts) ? launch_few(a) : launch128<Kind128::kFwd>(a);
}
cudaError_t launch_block128_dgrad(const LaunchBlock128 &a) { return launch128<Kind128::kDgrad>(a); }
cudaError_t launch_block128_wgrad(const LaunchBlock128 &a) { return launch128<Kind128::kWgrad>(a); }

}  // namespace fme
