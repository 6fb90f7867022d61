// mx_b128_gemm.cu -- products of E4M3 operands with one fp32 scale per block of 128 along the
// contraction, on the 5th-generation tensor cores:
//   C[i][j] = sum_kb sa[kb, i] sb[kb, j] sum_{k in block kb} a[i][k] b[j][k],
// dense, by expert (rows of A by offsets, one B per expert), and by expert for weight gradients
// (the contraction runs over each expert's own rows).
//
// One step is one scale block: operand P (128 tensor-memory lanes per CTA) and operand Q (up to 256
// accumulator columns), 128 code bytes of each row, loaded by the tensor-memory accelerator into a
// ring of 128-byte swizzled stages; four tcgen05.mma kind::f8f6f4 (K = 32) give the block's sums in
// an accumulator; eight warps read it and add it, times its scales, to fp32 sums in registers. The
// scales cannot wait until the end because they change with every block, so each block of a 128 x 256
// tile costs 32768 fp32 FMAs and a trip through registers beside its MMAs (512 cycles at the tensor
// cores' rate): that trip, not the MMAs, is what the kernel is built around.
//   * Two accumulators of 256 columns fill tensor memory, so a step cannot be shorter than half of
//     (MMA + signal + read + signal). A step's stage is full when its operands have landed AND its
//     accumulator has been read (one barrier for both); the reads come before the sums.
//   * The warp that multiplies runs converged and issues a step in one statement with every operand
//     in uniform registers (issue_step): issued from a lone lane's branch it took 400 to 600 cycles.
//   * Scales come through shared memory from a warp of their own, a group of four steps ahead.
//   * fp32 sums are packed pairs: half the instructions beside the warp that issues the MMAs.
//
// Four shapes of the same kernel:
//   rows      P = A (rows' scales), Q = B (blocks' scales), CTA pairs, 256 x 256 tiles: large dense
//             products and experts with many rows. A pair (cta_group::2) shares one tile, each CTA
//             holding 128 lanes and half of Q: per step 32 KB into an SM instead of 48, which alone
//             bound 128 x 256 tiles. 8192^3: 343 us (14 rounds of tiles, each 64 steps of 0.34 us and 2.3 us
//             more); run for seconds on end, under the power cap, 390.
//   columns   the same with a scale per column as well (weight gradients): the accumulator is read
//             in fragments (4 rows x 32 columns per thread), which needs a quarter of the column
//             scales' reads that a row per thread does (those would take 1024 cycles a step).
//   narrow    the rows shape in 128 x 128 tiles on single CTAs, with four accumulators: experts with
//             few rows, whose weights bound the product. Of A only the sixteens of rows that exist are
//             loaded, and only the warps that hold some read the accumulator. A row for each of 128
//             experts of 1024 x 2048 takes 46 us (5.8 TB/s of weights), 128 for each of 152 68 us.
//   swapped   P = B (weights), Q = A (tokens), for few tokens in dense products: a tile has as many
//             columns as it has tokens (a multiple of 16, at run time), so a step costs its weights.
//             The contraction is split over the CTAs of a cluster, whose parts are added in rank
//             order through distributed shared memory. 1 x 8192 x 8192: 16.1 us with the weights from
//             memory (4.2 TB/s), 13.3 with them in L2.
//
// Every mbarrier wait is bounded (KernelArgs::wait_limit_ns); a role whose wait ran out sets the
// device error word and stops; loads and MMAs in flight are waited for (2 s) before the CTA frees its
// tensor memory and exits.
#include <atomic>
#include <utility>

#include "mx_device.cuh"
#include "mx_expert.h"
#include "mx_launch.h"
#include "mx_tcgen05.cuh"

namespace mxq {

namespace {

using namespace tc;

constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s: drains, whatever the limit

constexpr int kLanes = 128;      // rows of P in a CTA
constexpr int kColumns = 256;    // columns of half of tensor memory: of an accumulator, or of a batch
constexpr int kStepBytes = 128;  // one scale block of the contraction per step
constexpr int kPromoWarps = 8;
constexpr int kThreads = 128 + 32 * kPromoWarps;
constexpr uint32_t kTmemCols = 2 * kColumns;
constexpr int kMaxStages = 12;
// scales travel and are released by groups of steps
constexpr int kScaleGroup = 4, kScaleGroups = 4, kScaleSlots = kScaleGroup * kScaleGroups;
constexpr int kMaxExperts = 1024;
constexpr int kMaxSplit = 8;

// CTAS: CTAs that share a tile. SWAP: P is B (weights), C is written [column][lane]. P_ROWS, Q_ROWS:
// the operand has a scale per row (else one per block of 128 rows).
template <int CTAS_, int MODE_, bool SWAP_, bool P_ROWS_, bool Q_ROWS_, bool F32_>
struct Config {
  static constexpr int CTAS = CTAS_, MODE = MODE_;
  static constexpr bool kSwap = SWAP_, kPRows = P_ROWS_, kQRows = Q_ROWS_, kF32 = F32_;
  static constexpr bool kNarrow = CTAS_ == 1 && !SWAP_;
  static constexpr int kPTile = kLanes * CTAS;
  // columns of a tile (swapped: at most), accumulators of that many in tensor memory (swapped: two
  // batches)
  static constexpr int kTileCols = SWAP_ || kNarrow ? 128 : 256;
  static constexpr int kBufs = kNarrow ? 4 : 2;
  // most columns of a promoting warp, and the registers of the two halves of the block
  static constexpr int kWarpCols = kTileCols / 2;
  static constexpr int kOtherRegs = kWarpCols == 64 ? 88 : 40;
  static constexpr int kPromoRegs = kWarpCols == 64 ? 208 : 232;
  static_assert(kOtherRegs * 128 + kPromoRegs * 256 <= 168 * kThreads, "the launch's registers");
  // floats of a scale slot: one per lane / column (rows form) or one per block of 128
  static constexpr int kPScales = P_ROWS_ ? kLanes : 4, kQScales = Q_ROWS_ ? kTileCols : 4;
  static constexpr int kSlotFloats = kPScales + kQScales;
  // ring of stages: four or five of fixed size, or (swapped) as many as the call's tile size leaves
  // room for
  static constexpr int kFixedStageBytes = (kLanes + kTileCols / CTAS_) * kStepBytes;
  static constexpr int kStages = kNarrow ? 5 : 4;
  static constexpr int kRingBytes = SWAP_ ? 172 * 1024 : kStages * kFixedStageBytes;
  // staging of the output, per promoting warp: one or two boxes of 32 rows x 128 bytes for tensor-map
  // stores, or (swapped) 32 tokens x 32 bf16 in rows of 80 bytes
  static constexpr int kBoxes = kNarrow ? 1 : 2;
  static constexpr int kStagingBytes = SWAP_ ? 32 * 80 : kBoxes * 4096;
};

template <typename C>
constexpr int smem_bytes() {
  return 1024 + C::kRingBytes + kPromoWarps * C::kStagingBytes + kScaleSlots * C::kSlotFloats * 4 +
         (2 * kMaxStages + 6 + 2 * kScaleGroups + 1) * 8 + 16 +
         (C::MODE != kB128Dense ? 2 * (kMaxExperts + 1) * 4 : 0);
}

struct Divisor {
  int d;
  uint32_t magic;
};

struct KernelArgs {
  const float* p_scales;
  const float* q_scales;
  void* c;
  const int64_t* offsets;
  unsigned int* err;
  unsigned long long wait_limit_ns;
  int64_t p_rows, q_rows;        // rows of P and Q: of one expert's matrix, or of the whole of A
  int64_t p_pitch, q_pitch;      // rows form: floats per scale row; blocks form: per block row
  int64_t b_estride;             // blocks form: floats of one expert's B
  int64_t ldc;                   // elements per row of C
  int64_t rows_total;            // rows the offsets may name
  int64_t blocks_total;          // wgrad: 128-row blocks of the padded operands
  int E;
  int nk;                        // steps of the contraction (dense, grouped)
  int p_tiles, q_tiles;          // tiles of the operands (grouped: of the weights only)
  int row_min, row_max;          // grouped: experts with this many rows are this launch's
  Divisor run, per;              // eight rows of tiles; all tiles of one expert (wgrad)
  int q_even;                    // swapped: columns of a tile, the tokens spread evenly
  int stages, stage_bytes;       // swapped
  int batch, stride;             // swapped: accumulators (steps) handed over together, 2 or 4, and
                                 // the columns from one to the next
  int split;                     // swapped, dense: CTAs of a cluster along the contraction
};

struct Tile {
  int p_row, q_row;          // first rows in the tensor maps
  int p_valid, q_valid;      // rows of the tile that exist (p_valid <= 0: none of this CTA's)
  int n;                     // columns computed (swapped: a multiple of 16)
  int e;
  int k0;                    // first byte along the contraction
  int nk;                    // steps
  int64_t p_scale, q_scale;  // first scale: rows form [kb][row], blocks form [row / 128][kb]
  int64_t c;                 // element of C at (lane 0, column 0) (swapped)
  int c_row, c_col;          // the same in C's tensor map (not swapped)
};

// ------------------------------------------------------------------------------------------
// instructions
// ------------------------------------------------------------------------------------------

// The MMAs of one step (K = 128 in four of 32, the first overwriting the accumulator) and the
// commits that free the operands' stage and (if asked) hand the accumulator over, issued by one elected
// lane of a converged warp. One statement with every operand computed outside: in a branch of the elected
// lane the descriptors went through vector registers and a step took 400 to 600 cycles to issue.
// Of a pair the commits arrive at the same barriers of both CTAs. (Every register counts in the warps
// that gave theirs up: a few bytes of spills in the multiplying warp's loop cost half of the speed,
// hence no condition where none is needed.)
template <int CTAS>
__device__ __forceinline__ void issue_step(uint32_t d, uint64_t p, uint64_t q, uint32_t idesc,
                                           uint32_t empty, uint32_t acc_full, bool hand_over) {
  if constexpr (CTAS == 1) {
    asm volatile(
        "{\n\t.reg .pred e, on, off, h;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\tsetp.ne.b32 off, 0, 0;\n\tsetp.eq.b32 on, 0, 0;\n\t"
        "setp.ne.and.b32 h, %12, 0, e;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %5, %9, off;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %2, %6, %9, on;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %3, %7, %9, on;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %4, %8, %9, on;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%10];\n\t"
        "@h tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%11];\n\t"
        "}" ::"r"(d),
        "l"(p), "l"(p + 2), "l"(p + 4), "l"(p + 6), "l"(q), "l"(q + 2), "l"(q + 4), "l"(q + 6),
        "r"(idesc), "r"(empty), "r"(acc_full), "r"((uint32_t)hand_over)
        : "memory");
  } else {  // always hands over
    asm volatile(
        "{\n\t.reg .pred e, on, off;\n\t.reg .b16 both;\n\tmov.b16 both, 3;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\tsetp.ne.b32 off, 0, 0;\n\tsetp.eq.b32 on, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %5, %9, off;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %2, %6, %9, on;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %3, %7, %9, on;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %4, %8, %9, on;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%10], both;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%11], both;\n\t"
        "}" ::"r"(d),
        "l"(p), "l"(p + 2), "l"(p + 4), "l"(p + 6), "l"(q), "l"(q + 2), "l"(q + 4), "l"(q + 6),
        "r"(idesc), "r"(empty), "r"(acc_full)
        : "memory");
  }
}
// Instruction descriptor, kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), A and B E4M3 (bits 7-9
// and 10-12 = 0), both K-major, N >> 3 at bits 17-22, M >> 4 at bits 24-28.
__device__ __forceinline__ uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The cluster's rank, barrier and addresses.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {  // the same address there
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Box load of a pair: into this CTA, completion counted on the first CTA's barrier.
__device__ __forceinline__ void tma_load_box_pair(uint32_t dst, const void* map, int x, int y,
                                                  uint32_t first_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(first_bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_box_3d(const void* map, int x, int y, int z, uint32_t src) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z), "r"(src)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t slot_addr, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot_addr),
               "r"(ncols));
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols));
}
__device__ __forceinline__ void commit_pair(uint32_t bar) {  // to this CTA only
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}

// Reads of the accumulator: issue, wait and the joining of neighbouring columns into 64-bit pairs are
// one statement. Written apart, ptxas was free to place the pairs' halves in registers that are no
// pairs and to move them for every packed FMA, which it did or not depending on unrelated code (342
// against 477 us at 8192^3).
// 64 fp32 columns of this thread's lane.
__device__ __forceinline__ void read_row(uint32_t taddr, uint64_t (&v)[32]) {
  asm volatile(
      "{\n\t.reg .b32 r<64>;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "r0, r1, r2, r3, r4, r5, r6, r7, r8, r9, r10, r11, r12, r13, r14, r15, "
      "r16, r17, r18, r19, r20, r21, r22, r23, r24, r25, r26, r27, r28, r29, r30, r31, "
      "r32, r33, r34, r35, r36, r37, r38, r39, r40, r41, r42, r43, r44, r45, r46, r47, "
      "r48, r49, r50, r51, r52, r53, r54, r55, r56, r57, r58, r59, r60, r61, r62, r63}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "mov.b64 %0, {r0, r1};\n\tmov.b64 %1, {r2, r3};\n\tmov.b64 %2, {r4, r5};\n\t"
      "mov.b64 %3, {r6, r7};\n\tmov.b64 %4, {r8, r9};\n\tmov.b64 %5, {r10, r11};\n\t"
      "mov.b64 %6, {r12, r13};\n\tmov.b64 %7, {r14, r15};\n\tmov.b64 %8, {r16, r17};\n\t"
      "mov.b64 %9, {r18, r19};\n\tmov.b64 %10, {r20, r21};\n\tmov.b64 %11, {r22, r23};\n\t"
      "mov.b64 %12, {r24, r25};\n\tmov.b64 %13, {r26, r27};\n\tmov.b64 %14, {r28, r29};\n\t"
      "mov.b64 %15, {r30, r31};\n\tmov.b64 %16, {r32, r33};\n\tmov.b64 %17, {r34, r35};\n\t"
      "mov.b64 %18, {r36, r37};\n\tmov.b64 %19, {r38, r39};\n\tmov.b64 %20, {r40, r41};\n\t"
      "mov.b64 %21, {r42, r43};\n\tmov.b64 %22, {r44, r45};\n\tmov.b64 %23, {r46, r47};\n\t"
      "mov.b64 %24, {r48, r49};\n\tmov.b64 %25, {r50, r51};\n\tmov.b64 %26, {r52, r53};\n\t"
      "mov.b64 %27, {r54, r55};\n\tmov.b64 %28, {r56, r57};\n\tmov.b64 %29, {r58, r59};\n\t"
      "mov.b64 %30, {r60, r61};\n\tmov.b64 %31, {r62, r63};\n\t"
      "}"
      : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]),
        "=l"(v[6]), "=l"(v[7]), "=l"(v[8]), "=l"(v[9]), "=l"(v[10]), "=l"(v[11]),
        "=l"(v[12]), "=l"(v[13]), "=l"(v[14]), "=l"(v[15]), "=l"(v[16]), "=l"(v[17]),
        "=l"(v[18]), "=l"(v[19]), "=l"(v[20]), "=l"(v[21]), "=l"(v[22]), "=l"(v[23]),
        "=l"(v[24]), "=l"(v[25]), "=l"(v[26]), "=l"(v[27]), "=l"(v[28]), "=l"(v[29]),
        "=l"(v[30]), "=l"(v[31])
      : "r"(taddr)
      : "memory");
}
// 32 lanes x 32 columns in fragments: v[8 h + 2 g + i] of lane l is the columns 8 g + 2 (l % 4) +
// {0, 1} of row 16 h + 8 i + l / 4.
__device__ __forceinline__ void read_fragments(uint32_t taddr, uint64_t (&v)[16]) {
  asm volatile(
      "{\n\t.reg .b32 r<32>;\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {r0, r1, r2, r3, r4, r5, r6, r7, "
      "r8, r9, r10, r11, r12, r13, r14, r15}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {r16, r17, r18, r19, r20, r21, r22, r23, "
      "r24, r25, r26, r27, r28, r29, r30, r31}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "mov.b64 %0, {r0, r1};\n\tmov.b64 %1, {r2, r3};\n\tmov.b64 %2, {r4, r5};\n\t"
      "mov.b64 %3, {r6, r7};\n\tmov.b64 %4, {r8, r9};\n\tmov.b64 %5, {r10, r11};\n\t"
      "mov.b64 %6, {r12, r13};\n\tmov.b64 %7, {r14, r15};\n\tmov.b64 %8, {r16, r17};\n\t"
      "mov.b64 %9, {r18, r19};\n\tmov.b64 %10, {r20, r21};\n\tmov.b64 %11, {r22, r23};\n\t"
      "mov.b64 %12, {r24, r25};\n\tmov.b64 %13, {r26, r27};\n\tmov.b64 %14, {r28, r29};\n\t"
      "mov.b64 %15, {r30, r31};\n\t"
      "}"
      : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]),
        "=l"(v[6]), "=l"(v[7]), "=l"(v[8]), "=l"(v[9]), "=l"(v[10]), "=l"(v[11]),
        "=l"(v[12]), "=l"(v[13]), "=l"(v[14]), "=l"(v[15])
      : "r"(taddr), "r"(taddr + (16u << 16))
      : "memory");
}
// 32 lanes x 64 columns in fragments: v[16 c + 8 h + 2 g + i] of lane l is the columns 32 c + 8 g + 2 (l % 4) +
// {0, 1} of row 16 h + 8 i + l / 4.
__device__ __forceinline__ void read_fragments(uint32_t taddr, uint64_t (&v)[32]) {
  asm volatile(
      "{\n\t.reg .b32 r<64>;\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {r0, r1, r2, r3, r4, r5, r6, r7, "
      "r8, r9, r10, r11, r12, r13, r14, r15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {r16, r17, r18, r19, r20, r21, r22, r23, "
      "r24, r25, r26, r27, r28, r29, r30, r31}, [%33];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {r32, r33, r34, r35, r36, r37, r38, r39, "
      "r40, r41, r42, r43, r44, r45, r46, r47}, [%34];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {r48, r49, r50, r51, r52, r53, r54, r55, "
      "r56, r57, r58, r59, r60, r61, r62, r63}, [%35];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "mov.b64 %0, {r0, r1};\n\tmov.b64 %1, {r2, r3};\n\tmov.b64 %2, {r4, r5};\n\t"
      "mov.b64 %3, {r6, r7};\n\tmov.b64 %4, {r8, r9};\n\tmov.b64 %5, {r10, r11};\n\t"
      "mov.b64 %6, {r12, r13};\n\tmov.b64 %7, {r14, r15};\n\tmov.b64 %8, {r16, r17};\n\t"
      "mov.b64 %9, {r18, r19};\n\tmov.b64 %10, {r20, r21};\n\tmov.b64 %11, {r22, r23};\n\t"
      "mov.b64 %12, {r24, r25};\n\tmov.b64 %13, {r26, r27};\n\tmov.b64 %14, {r28, r29};\n\t"
      "mov.b64 %15, {r30, r31};\n\tmov.b64 %16, {r32, r33};\n\tmov.b64 %17, {r34, r35};\n\t"
      "mov.b64 %18, {r36, r37};\n\tmov.b64 %19, {r38, r39};\n\tmov.b64 %20, {r40, r41};\n\t"
      "mov.b64 %21, {r42, r43};\n\tmov.b64 %22, {r44, r45};\n\tmov.b64 %23, {r46, r47};\n\t"
      "mov.b64 %24, {r48, r49};\n\tmov.b64 %25, {r50, r51};\n\tmov.b64 %26, {r52, r53};\n\t"
      "mov.b64 %27, {r54, r55};\n\tmov.b64 %28, {r56, r57};\n\tmov.b64 %29, {r58, r59};\n\t"
      "mov.b64 %30, {r60, r61};\n\tmov.b64 %31, {r62, r63};\n\t"
      "}"
      : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]),
        "=l"(v[6]), "=l"(v[7]), "=l"(v[8]), "=l"(v[9]), "=l"(v[10]), "=l"(v[11]),
        "=l"(v[12]), "=l"(v[13]), "=l"(v[14]), "=l"(v[15]), "=l"(v[16]), "=l"(v[17]),
        "=l"(v[18]), "=l"(v[19]), "=l"(v[20]), "=l"(v[21]), "=l"(v[22]), "=l"(v[23]),
        "=l"(v[24]), "=l"(v[25]), "=l"(v[26]), "=l"(v[27]), "=l"(v[28]), "=l"(v[29]),
        "=l"(v[30]), "=l"(v[31])
      : "r"(taddr), "r"(taddr + (16u << 16)), "r"(taddr + 32), "r"(taddr + 32 + (16u << 16))
      : "memory");
}

// Pairs of fp32 in one 64-bit register: one instruction for two (the same rate per value, half the
// instructions).
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ uint64_t both(float x) {
  return pair(__float_as_uint(x), __float_as_uint(x));
}
__device__ __forceinline__ float first(uint64_t p) { return __uint_as_float((uint32_t)p); }
__device__ __forceinline__ float second(uint64_t p) { return __uint_as_float((uint32_t)(p >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}
// One arrival of a converged warp.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// The same at a barrier of the cluster. The default order of one CTA is enough: what it orders are
// reads of tensor memory, complete before it (release at cluster scope waited over 1000 cycles).
__device__ __forceinline__ void warp_arrive_cluster(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// Whether the phase is complete. try_wait lets the hardware suspend the thread meanwhile, for longer
// than most waits last; a call with a limit below that (the give-up self-test) asks without.
__device__ __forceinline__ bool phase_done_now(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred P;\n\tmbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity, const KernelArgs& a) {
  return a.wait_limit_ns >= 1000000ull ? mbar_try_wait(bar, parity) : phase_done_now(bar, parity);
}

// A value that is the same in all lanes, as the hardware's reduction gives it: in a uniform register.
__device__ __forceinline__ int uniform(int x) {
  return (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)x);
}

// A wait of the whole warp: one vote when the phase is complete; given up after the call's limit
// (then at once, and the device error word says so).
__device__ __forceinline__ void warp_wait(uint32_t bar, uint32_t parity, bool* failed,
                                          const KernelArgs& a) {
  if (*failed || __all_sync(0xFFFFFFFFu, phase_done(bar, parity, a))) return;
  const unsigned long long t0 = global_ns();
  while (!__all_sync(0xFFFFFFFFu, phase_done(bar, parity, a))) {
    // the timer ticks every 32 ns at best; a begun tick counts
    if (__any_sync(0xFFFFFFFFu, global_ns() - t0 + 32 > a.wait_limit_ns)) {
      *failed = true;
      if ((threadIdx.x & 31) == 0) atomicOr(a.err, 1u);
      return;
    }
  }
}

// ------------------------------------------------------------------------------------------
// tiles
// ------------------------------------------------------------------------------------------

// n / d and the remainder for 0 <= n < 2^31, d given with floor(2^32 / d) + 1: the estimate is right or
// one too large. (Several roles find their tile at every tile's end; the compiler's divisions there
// took half a microsecond.)
__device__ __forceinline__ int divide(int n, Divisor d, int* rest) {
  int q = d.d == 1 ? n : (int)__umulhi((uint32_t)n, d.magic), r = n - q * d.d;
  if (r < 0) {
    --q;
    r += d.d;
  }
  *rest = r;
  return q;
}
// The same for a divisor not known before: in fp32, exact to one below 2^23.
__device__ __forceinline__ int divide(int n, int d, int* rest) {
  int q = n < (1 << 23) ? (int)(__int2float_rn(n) * __frcp_rn(__int2float_rn(d))) : n / d;
  int r = n - q * d;
  if (r < 0) {
    --q;
    r += d;
  } else if (r >= d) {
    ++q;
    r -= d;
  }
  *rest = r;
  return q;
}

// p tile and q tile of tile t of a p_tiles x q_tiles grid: runs of eight p tiles cross all q
// tiles, so that the CTAs working at one time share operands in L2
__device__ __forceinline__ void raster(int t, const KernelArgs& a, int* p, int* q) {
  int in;
  const int first = divide(t, a.run, &in) * 8;
  const int height = min(8, a.p_tiles - first);
  if (height == 8) {
    *p = first + (in & 7);
    *q = in >> 3;
  } else {
    *q = divide(in, height, p);
    *p += first;
  }
}

template <typename C>
__device__ __forceinline__ int tile_count(const KernelArgs& a, const int* prefix) {
  if (C::MODE == kB128Dense) return a.p_tiles * a.q_tiles;
  if (C::MODE == kB128Wgrad) return a.p_tiles * a.q_tiles * a.E;
  return prefix[a.E] * a.q_tiles;
}

template <typename C>
__device__ __forceinline__ Tile get_tile(const KernelArgs& a, int t, const int* prefix,
                                         const int* start) {
  Tile r;
  int p, q, kb0 = 0;
  r.e = 0;
  r.nk = a.nk;
  int64_t p_first;  // first row of the P tile in its matrix
  if (C::MODE == kB128Grouped) {  // P: tokens, Q: weights
    // the last expert with prefix * q_tiles <= t: in two rounds, 32 at a time
    const int lane = threadIdx.x & 31, width = (a.E + 31) >> 5;
    const int run = __popc(__ballot_sync(
        0xFFFFFFFFu, (int64_t)prefix[min((lane + 1) * width, a.E)] * a.q_tiles <= t));
    const int at = run * width + 1 + lane;
    const int lo = run * width +
                   __popc(__ballot_sync(0xFFFFFFFFu, lane < width && at < a.E &&
                                                         (int64_t)prefix[at] * a.q_tiles <= t));
    const int local = t - prefix[lo] * a.q_tiles, row_tiles = prefix[lo + 1] - prefix[lo];
    q = local;
    p = 0;
    if (row_tiles > 1) q = divide(local, row_tiles, &p);  // one weight tile's token tiles together
    r.e = lo;
    r.n = C::kTileCols;
    r.c_col = q * C::kTileCols;
    r.q_row = (int)(lo * a.q_rows) + r.c_col;
    r.q_valid = (int)min((int64_t)C::kTileCols, a.q_rows - r.c_col);
    p_first = start[lo] + p * C::kPTile;
    r.p_row = (int)p_first;
    r.p_valid = min(C::kPTile, start[lo + 1] - r.p_row);
  } else {
    if (C::MODE == kB128Wgrad) {
      r.e = divide(t, a.per, &t);
      kb0 = prefix[r.e];
      r.nk = prefix[r.e + 1] - kb0;
    }
    raster(t, a, &p, &q);
    r.n = C::kSwap ? a.q_even : C::kTileCols;
    r.q_row = q * r.n;
    r.q_valid = (int)min((int64_t)r.n, a.q_rows - r.q_row);
    p_first = (int64_t)p * C::kPTile;
    r.p_row = (int)p_first;
    r.p_valid = (int)min((int64_t)C::kPTile, a.p_rows - p_first);
    r.c_col = r.q_row;
  }
  r.k0 = kb0 * kStepBytes;
  r.p_scale = C::kPRows ? kb0 * a.p_pitch + r.p_row
                        : (int64_t)p * C::CTAS * a.p_pitch + kb0;
  r.q_scale = C::kQRows ? kb0 * a.q_pitch + r.q_row
                        : r.e * a.b_estride + (int64_t)q * (C::kTileCols / kB128) * a.q_pitch + kb0;
  r.c = (int64_t)r.q_row * a.ldc + p_first;
  r.c_row = (int)p_first;
  if constexpr (C::CTAS == 2) {  // this CTA's own 128 rows of P
    const int rank = (int)cluster_rank(), skip = rank * kLanes;
    r.p_row += skip;
    r.p_valid = min(kLanes, r.p_valid - skip);
    r.p_scale += C::kPRows ? skip : rank * a.p_pitch;
    r.c += skip;
    r.c_row += skip;
  }
  if (C::kSwap && C::MODE == kB128Dense && a.split > 1) {  // this CTA's share of the contraction
    const int per = (r.nk + a.split - 1) / a.split, first = (int)cluster_rank() * per;
    r.k0 += first * kStepBytes;
    r.p_scale += C::kPRows ? first * a.p_pitch : first;
    r.q_scale += C::kQRows ? first * a.q_pitch : first;
    r.nk = max(0, min(per, r.nk - first));
  }
  return r;
}

// Table of the calls by expert: prefix sums of ceil(n_e / unit), and first rows. Offsets that break
// their contract are clamped and made non-decreasing, so that every later access stays inside the
// operands. All threads read the offsets (one trip to memory), one warp scans them.
template <typename C>
__device__ __forceinline__ void build_table(const KernelArgs& a, int unit, int limit, int* prefix,
                                            int* start) {
  for (int e = threadIdx.x; e <= a.E; e += kThreads) {
    start[e] = (int)min(max(load_s64(a.offsets + e), (int64_t)0), a.rows_total);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int before = 0, reach = start[0];
    if (lane == 0) prefix[0] = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      int end = e < a.E ? max(start[e + 1], reach) : reach;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {  // running maximum: non-decreasing ends
        const int up = __shfl_up_sync(0xFFFFFFFFu, end, d);
        if (lane >= d) end = max(end, up);
      }
      int first = __shfl_up_sync(0xFFFFFFFFu, end, 1);
      if (lane == 0) first = reach;
      reach = __shfl_sync(0xFFFFFFFFu, end, 31);
      int rows = e < a.E ? end - first : 0;
      if (C::MODE == kB128Grouped && (rows < a.row_min || rows > a.row_max)) rows = 0;
      int sum = (rows + unit - 1) / unit;
      if (e < a.E) start[e + 1] = end;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += up;
      }
      if (e < a.E) prefix[e + 1] = min(before + sum, limit);
      before += __shfl_sync(0xFFFFFFFFu, sum, 31);
      __syncwarp();
    }
  }
}

struct Smem {
  uint8_t* ring;
  uint8_t* staging;       // [kPromoWarps][kStagingBytes]
  float* scales;          // [kScaleSlots][kSlotFloats]
  uint64_t* full;         // [stages]: operands landed and (not swapped) accumulator read
  uint64_t* empty;        // [stages]: operands read
  uint64_t* acc_full;     // [accumulators or batches, at most 4]
  uint64_t* acc_empty;    // [2] (swapped)
  uint64_t* scale_full;   // [kScaleGroups]
  uint64_t* scale_empty;  // [kScaleGroups]
  uint64_t* done;
  uint32_t* tmem_slot;
  int* prefix;
  int* start;
};

template <typename C>
__device__ __forceinline__ int stage_count(const KernelArgs& a) {
  return C::kSwap ? a.stages : C::kStages;
}
template <typename C>
__device__ __forceinline__ int stage_bytes(const KernelArgs& a) {
  return C::kSwap ? a.stage_bytes : C::kFixedStageBytes;
}

// tiles of this CTA (or pair): t0, t0 + step, ...
template <typename C>
__device__ __forceinline__ void tile_range(const KernelArgs& a, int* t0, int* step) {
  const int group = C::kSwap && C::MODE == kB128Dense ? a.split : C::CTAS;
  *t0 = blockIdx.x / group;
  *step = gridDim.x / group;
}

// ------------------------------------------------------------------------------------------
// roles. The loading and the multiplying warp run converged and issue from one elected lane, so that
// addresses and descriptors stay in uniform registers.
// ------------------------------------------------------------------------------------------
template <typename C>
__device__ __forceinline__ void produce(const CUtensorMap& pmap, const CUtensorMap& qmap,
                                        const CUtensorMap& map16, const KernelArgs& a,
                                        const Smem& s, int tiles) {
  const int stages = stage_count<C>(a);
  bool failed = false;
  int issued = 0, st = 0, t0, step;
  uint32_t parity = 1;  // a fresh barrier's preceding phase counts as complete
  tile_range<C>(a, &t0, &step);
  for (int t = t0; t < tiles && !failed; t += step) {
    const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
    // rows this CTA loads: of Q all of the tile's columns, or its half of them; of P 128, or (narrow) the
    // sixteens that hold rows of the expert (what is left in the others reaches lanes that are not
    // written)
    const int q_rows = tile.n / C::CTAS;
    const int q_row = tile.q_row + (C::CTAS == 2 ? (int)cluster_rank() * q_rows : 0);
    const int p_rows = C::kNarrow ? min(kLanes, (tile.p_valid + 15) & ~15) : kLanes;
    const uint32_t bytes = (uint32_t)(p_rows + q_rows) * kStepBytes;
    for (int kb = 0; kb < tile.nk; ++kb) {
      warp_wait(smem_u32(s.empty + st), parity, &failed, a);
      if (failed) break;
      const uint32_t bar = smem_u32(s.full + st);
      const uint32_t dst = smem_u32(s.ring + st * stage_bytes<C>(a)), q_dst = dst + kLanes * kStepBytes;
      const int x = tile.k0 + kb * kStepBytes;
      if constexpr (C::CTAS == 2) {
        const uint32_t first = in_cta(bar, 0);
        if (elect_one()) {
          if (cluster_rank() == 0) mbar_arrive_expect_tx(bar, 2 * bytes);
          tma_load_box_pair(dst, &pmap, x, tile.p_row, first);
          tma_load_box_pair(q_dst, &qmap, x, q_row, first);
        }
      } else if (elect_one()) {
        mbar_arrive_expect_tx(bar, bytes);
        if (p_rows == kLanes) {
          tma_load_box(dst, &pmap, x, tile.p_row, bar);
        } else {
          for (int r = 0; r < p_rows; r += 16) {
            tma_load_box(dst + r * kStepBytes, &map16, x, tile.p_row + r, bar);
          }
        }
        if (!C::kSwap || q_rows == 128) {
          tma_load_box(q_dst, &qmap, x, q_row, bar);
        } else {
          for (int r = 0; r < q_rows; r += 16) {
            tma_load_box(q_dst + r * kStepBytes, &map16, x, q_row + r, bar);
          }
        }
      }
      __syncwarp();
      ++issued;
      if (++st == stages) {
        st = 0;
        parity ^= 1;
      }
    }
  }
  // A CTA that has seen every stage released has nothing more to come: its loads have landed, and the
  // commits' arrivals at its stages' barriers, which nothing else waits for (in a pair they come from the
  // other CTA), are in. After a give-up the loads are waited for by their own barriers; a
  // pair's are counted on its first CTA's, and as the two may then not have issued the same steps, each
  // also lets a millisecond pass, a thousand times what a load or an arrival takes.
  for (int i = 0; i < stages && !failed; ++i) {
    warp_wait(smem_u32(s.empty + st), parity, &failed, a);
    if (++st == stages) {
      st = 0;
      parity ^= 1;
    }
  }
  if (!failed) return;
  if constexpr (C::CTAS == 2) {
    const unsigned long long begin = global_ns();
    while (global_ns() - begin < 1000000ull) {
    }
    if (cluster_rank() != 0) return;
  }
  bool drain_failed = false;
  for (int i = issued > stages ? issued - stages : 0; i < issued; ++i) {
    mbar_wait(smem_u32(s.full + i % stages), (i / stages) & 1, &drain_failed, kWaitNs, a.err);
  }
}

template <typename C>
__device__ __forceinline__ void multiply(const KernelArgs& a, const Smem& s, int tiles,
                                         uint32_t tmem) {
  static_assert(kStepBytes == 128, "issue_step");
  const int stages = stage_count<C>(a);
  bool failed = false;
  int st = 0, t0, step;
  uint32_t full_parity = 0;
  tile_range<C>(a, &t0, &step);
  if constexpr (!C::kSwap) {
    int buf = 0;
    for (int t = t0; t < tiles && !failed; t += step) {
      const int nk = uniform(get_tile<C>(a, t, s.prefix, s.start).nk);
      for (int kb = 0; kb < nk; ++kb) {
        warp_wait(smem_u32(s.full + st), full_parity, &failed, a);
        if (failed) break;
        tc_fence_after();
        const uint64_t p = desc_sw128(smem_u32(s.ring + st * C::kFixedStageBytes));
        issue_step<C::CTAS>(tmem + buf * C::kTileCols, p, p + (kLanes * kStepBytes >> 4),
                            idesc_e4m3_f32(C::kPTile, C::kTileCols), smem_u32(s.empty + st),
                            smem_u32(s.acc_full + buf), true);
        if (++st == stages) {
          st = 0;
          full_parity ^= 1;
        }
        buf = (buf + 1) & (C::kBufs - 1);
      }
    }
  } else {
    uint32_t batch = 0;
    for (int t = t0; t < tiles && !failed; t += step) {
      const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
      const int nk = uniform(tile.nk);
      const uint32_t idesc = idesc_e4m3_f32(C::kPTile, uniform(tile.n));
      for (int kb = 0; kb < nk; ++batch) {
        const uint32_t half = batch & 1;
        warp_wait(smem_u32(s.acc_empty + half), ((batch >> 1) & 1) ^ 1, &failed, a);
        uint32_t column = tmem + half * kColumns;
        for (int left = min(a.batch, nk - kb); left > 0; --left, ++kb) {
          warp_wait(smem_u32(s.full + st), full_parity, &failed, a);
          if (failed) break;
          tc_fence_after();
          const uint64_t p = desc_sw128(smem_u32(s.ring + st * stage_bytes<C>(a)));
          issue_step<C::CTAS>(column, p, p + (kLanes * kStepBytes >> 4), idesc,
                              smem_u32(s.empty + st), smem_u32(s.acc_full + half), left == 1);
          column += a.stride;
          if (++st == stages) {
            st = 0;
            full_parity ^= 1;
          }
        }
        if (failed) break;
      }
    }
  }
  if (elect_one()) {
    if constexpr (C::CTAS == 2) {
      commit_pair(smem_u32(s.done));
    } else {
      mma_commit(smem_u32(s.done));
    }
  }
  __syncwarp();
  // every MMA issued completes before the tensor memory is freed
  bool drain_failed = false;
  mbar_wait(smem_u32(s.done), 0, &drain_failed, kWaitNs, a.err);
}

// 4-byte asynchronous copy to shared memory, `at` floats on from dst and src; zero where !ok (nothing is
// read then).
template <int AT>
__device__ __forceinline__ void copy_scale(uint32_t dst, const float* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0 + %3], [%1 + %3], 4, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 4 : 0), "n"(AT * 4)
               : "memory");
}

// One warp copies the scales into a ring, a group of steps at a time and a group ahead: the promoting
// warps then never wait for a scale's trip from L2, which is longer than a step, and meet a barrier
// for scales once in kScaleGroup steps.
template <typename C>
__device__ __forceinline__ void fetch_scales(const KernelArgs& a, const Smem& s, int tiles) {
  const int lane = threadIdx.x & 31;
  bool failed = false;
  int group = 0, t0, step;
  tile_range<C>(a, &t0, &step);
  for (int t = t0; t < tiles && !failed; t += step) {
    const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
    const int nk = tile.nk, p_valid = tile.p_valid, q_valid = tile.q_valid;
    // this lane's scales of the current step: its rows of P (or P's block), its columns (or blocks) of Q
    const float* p = a.p_scales + tile.p_scale + (C::kPRows ? lane : 0);
    const float* q = a.q_scales + tile.q_scale + (C::kQRows ? (int64_t)lane : lane * a.q_pitch);
    for (int kb0 = 0; kb0 < nk; kb0 += kScaleGroup, ++group) {
      const int g = group % kScaleGroups;
      warp_wait(smem_u32(s.scale_empty + g), ((group / kScaleGroups) & 1) ^ 1, &failed, a);
      if (failed) break;
      uint32_t dst = smem_u32(s.scales + g * kScaleGroup * C::kSlotFloats + lane);
      for (int left = min(kScaleGroup, nk - kb0); left > 0; --left) {
        if constexpr (C::kPRows) {
          copy_scale<0>(dst, p, lane < p_valid);
          copy_scale<32>(dst, p, 32 + lane < p_valid);
          copy_scale<64>(dst, p, 64 + lane < p_valid);
          copy_scale<96>(dst, p, 96 + lane < p_valid);
          p += a.p_pitch;
        } else {
          if (lane == 0) copy_scale<0>(dst, p, p_valid > 0);
          ++p;
        }
        if constexpr (C::kQRows) {
#define MXQ_COLUMNS(at) \
  if (!C::kSwap || (at) < tile.n) copy_scale<at>(dst + C::kPScales * 4, q, (at) + lane < q_valid)
          MXQ_COLUMNS(0);
          MXQ_COLUMNS(32);
          MXQ_COLUMNS(64);
          MXQ_COLUMNS(96);
          if constexpr (!C::kSwap) MXQ_COLUMNS(128);
          if constexpr (!C::kSwap) MXQ_COLUMNS(160);
          if constexpr (!C::kSwap) MXQ_COLUMNS(192);
          if constexpr (!C::kSwap) MXQ_COLUMNS(224);
#undef MXQ_COLUMNS
          q += a.q_pitch;
        } else {
          if (lane < C::kTileCols / kB128) {
            copy_scale<0>(dst + C::kPScales * 4, q, lane * kB128 < q_valid);
          }
          ++q;
        }
        dst += C::kSlotFloats * 4;
      }
      __syncwarp();
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                       smem_u32(s.scale_full + g))
                   : "memory");
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // none lands after the CTA's shared memory goes
}

// A promoting warp's way through the steps (not swapped): the barriers of one step around its reads.
// (Asking the next step's barrier before this step's sums, to have only the answer left, measured
// slower: 436 against 360 us at 8192^3; so did fetching its scales there, 392 against 340.)
template <typename C>
struct Steps {
  const KernelArgs& a;
  const Smem& s;
  uint32_t full0;        // the barriers on which read accumulators are reported
  int it = 0, st2 = C::kBufs % C::kStages;  // step, stage of the step that gets its accumulator next
  uint32_t group = 0;
  bool failed = false;

  __device__ __forceinline__ Steps(const KernelArgs& a_, const Smem& s_) : a(a_), s(s_) {
    static_assert(C::kBufs <= C::kStages, "a stage has one accumulator's arrivals under way");
    full0 = C::CTAS == 2 ? in_cta(smem_u32(s.full), 0) : smem_u32(s.full);
    for (int i = 0; i < C::kBufs; ++i) hand_back(i);  // the first steps find theirs free
  }
  __device__ __forceinline__ void hand_back(int st) {
    if constexpr (C::CTAS == 2) {
      warp_arrive_cluster(full0 + 8 * st);
    } else {
      warp_arrive(full0 + 8 * st);
    }
  }
  // scales of step kb of the tile
  __device__ __forceinline__ const float* scales(int kb) {
    const int g = group % kScaleGroups, in = kb % kScaleGroup;
    if (in == 0) {
      warp_wait(smem_u32(s.scale_full + g), (group / kScaleGroups) & 1, &failed, a);
    }
    return s.scales + (g * kScaleGroup + in) * C::kSlotFloats;
  }
  __device__ __forceinline__ bool accumulator() {
    warp_wait(smem_u32(s.acc_full + it % C::kBufs), (it / C::kBufs) & 1, &failed, a);
    if (failed) return false;
    tc_fence_after();
    return true;
  }
  __device__ __forceinline__ uint32_t column() const { return it % C::kBufs * C::kTileCols; }
  __device__ __forceinline__ void accumulator_read() {
    tc_fence_before();
    hand_back(st2);
    if (++st2 == C::kStages) st2 = 0;
  }
  __device__ __forceinline__ void end(int kb, int nk) {
    if (kb % kScaleGroup == kScaleGroup - 1 || kb == nk - 1) {
      warp_arrive(smem_u32(s.scale_empty + group % kScaleGroups));
      ++group;
    }
    ++it;
  }
  // The steps that may have been loaded are handed back unread, so that the loading warp sees its
  // copies land. Steps it .. it + kBufs - 1 have their arrivals already and their stages may still be
  // in that phase, so the steps that follow on those stages are left out: a second arrival there would
  // complete a phase before its copies do. Where the other warps went on and such steps were loaded all
  // the same, nothing completes their phases, and the loading warp's drain ends by its limit, long after
  // the copies have landed.
  __device__ __forceinline__ void give_up() {
    for (int i = 0; i < C::kStages - C::kBufs; ++i) hand_back((st2 + i) % C::kStages);
  }
};

// The same of the swapped shape, whose steps are short beside the way of their signals (about 650 cycles
// of barriers and reads a step, whatever its columns): tensor memory holds two batches of up to four
// accumulators, and a batch is handed over, read and handed back as one.
template <typename C>
struct Batches {
  const KernelArgs& a;
  const Smem& s;
  uint32_t batch = 0, group = 0;
  bool failed = false;

  __device__ __forceinline__ Batches(const KernelArgs& a_, const Smem& s_) : a(a_), s(s_) {
    static_assert(C::CTAS == 1, "the swapped shape runs on single CTAs");
  }
  // scales of the batch that begins with step kb of the tile (a batch lies in one group)
  __device__ __forceinline__ const float* scales(int kb) {
    const int g = group % kScaleGroups, in = kb % kScaleGroup;
    if (in == 0) {
      warp_wait(smem_u32(s.scale_full + g), (group / kScaleGroups) & 1, &failed, a);
    }
    return s.scales + (g * kScaleGroup + in) * C::kSlotFloats;
  }
  __device__ __forceinline__ bool accumulators() {
    warp_wait(smem_u32(s.acc_full + (batch & 1)), (batch >> 1) & 1, &failed, a);
    if (failed) return false;
    tc_fence_after();
    return true;
  }
  __device__ __forceinline__ uint32_t column(int in) const {
    return (batch & 1) * kColumns + in * a.stride;
  }
  __device__ __forceinline__ void accumulators_read() {
    tc_fence_before();
    warp_arrive(smem_u32(s.acc_empty + (batch & 1)));
  }
  __device__ __forceinline__ void end(int kb, int nk) {  // kb: the step after the batch
    if (kb % kScaleGroup == 0 || kb == nk) {
      warp_arrive(smem_u32(s.scale_empty + group % kScaleGroups));
      ++group;
    }
    ++batch;
  }
};

// Staging of a promoting warp's output: one or two boxes of 32 rows x 128 bytes, 16-byte chunk q of row
// r at q ^ (r % 8), written with tensor-map stores.
template <typename C>
struct Boxes {
  static constexpr int kCols = C::kF32 ? 32 : 64;  // columns of a box
  uint8_t* base;
  __device__ __forceinline__ void wait() {  // all are read
    if ((threadIdx.x & 31) == 0) bulk_wait_read_all();
    __syncwarp();
  }
  // the boxes, side by side; the second only where it has columns
  __device__ __forceinline__ void store(const CUtensorMap& cmap, int x, int y, int z, int cols) {
    fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      tma_store_box_3d(&cmap, x, y, z, smem_u32(base));
      if (C::kBoxes > 1 && cols > kCols) {
        tma_store_box_3d(&cmap, x + kCols, y, z, smem_u32(base + 4096));
      }
      bulk_commit_group();
    }
  }
  // The first `rows` rows and `cols` columns of box u only, by ordinary stores (the box's other rows
  // are another expert's).
  __device__ __forceinline__ void store_part(const KernelArgs& a, int u, int64_t at, int rows,
                                             int cols) {
    const int lane = threadIdx.x & 31, chunk = lane & 7, per = C::kF32 ? 4 : 8;
    __syncwarp();
    for (int r = lane >> 3; r < rows; r += 4) {
      if (chunk * per >= cols) break;
      const uint4 v =
          *reinterpret_cast<const uint4*>(base + u * 4096 + r * 128 + ((chunk ^ (r & 7)) << 4));
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.c) +
                                (at + r * a.ldc + chunk * per) * (C::kF32 ? 4 : 2)) = v;
    }
    __syncwarp();
  }
  __device__ __forceinline__ void drain() {  // read before the CTA's shared memory goes away
    if ((threadIdx.x & 31) == 0) bulk_wait_read_all();
  }
};

// Swapped shape: the groups of eight columns (tokens) first, first + every, .. of a warp's fragments to
// C [token][lane]. bf16 goes through shared memory, transposed on the way (8 tokens x 32 lanes = 64
// bytes each), so that a lane stores 16 bytes of one token.
template <typename C>
__device__ __forceinline__ void store_swapped(const KernelArgs& a, const Smem& s, const Tile& tile,
                                              int pw, const uint64_t (&sums)[C::kWarpCols / 2],
                                              int first_group, int every) {
  const int lane = threadIdx.x & 31, row0 = (pw & 3) * 32, lr = lane >> 2, lc = (lane & 3) * 2;
  const int cols = tile.n / 2, col0 = (pw >> 2) * cols;
  uint8_t* staging = s.staging + pw * C::kStagingBytes;
  // what a lane stores of a group: token lane / 4, 8 lanes' worth from 8 (lane % 4) on
  const int part = (lane & 3) * 8;
  // Slots are taken in turn by the groups that this warp stores (by the number of the group, every fourth
  // one would find the same): between two uses of one lie the barriers of three others, which order the
  // reads of the first before the writes of the second.
  int stored = 0;
#pragma unroll
  for (int gi = 0; gi < C::kWarpCols / 8; ++gi) {
    if (gi * 8 >= cols || gi % every != first_group) continue;
    if constexpr (C::kF32) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = row0 + 8 * r + lr, col = col0 + gi * 8 + lc;
        float* o = static_cast<float*>(a.c) + tile.c + col * a.ldc + row;
        if (row < tile.p_valid && col < tile.q_valid) o[0] = first(sums[gi * 4 + r]);
        if (row < tile.p_valid && col + 1 < tile.q_valid) o[a.ldc] = second(sums[gi * 4 + r]);
      }
    } else {
      uint32_t h[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) h[r] = bf16_pair(first(sums[gi * 4 + r]), second(sums[gi * 4 + r]));
      uint8_t* slot = staging + (stored++ & 3) * 8 * 80;
      asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                       smem_u32(slot + (lane & 7) * 80 + (lane >> 3) * 16)),
                   "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                   : "memory");
      __syncwarp();
      const uint4 v = *reinterpret_cast<const uint4*>(slot + lr * 80 + part * 2);
      const int col = col0 + gi * 8 + lr;
      if (col < tile.q_valid && row0 + part < tile.p_valid) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.c) + tile.c + col * a.ldc + row0 + part) = v;
      }
    }
  }
  __syncwarp();  // the staging is free again
}

// The promoting warps of the rows and narrow shapes: warp w holds lanes 32 (w % 4) .. and half w / 4 of
// the tile's columns, a row per thread.
template <typename C>
__device__ __forceinline__ void promote_rows(const CUtensorMap& cmap, const KernelArgs& a,
                                             const Smem& s, int tiles, uint32_t tmem, int pw) {
  const int lane = threadIdx.x & 31, row0 = (pw & 3) * 32, row = row0 + lane, half = pw >> 2;
  const uint32_t tbase = tmem + ((uint32_t)row0 << 16) + half * C::kWarpCols;
  Steps<C> steps(a, s);
  Boxes<C> boxes{s.staging + pw * C::kStagingBytes};
  int t0, step;
  tile_range<C>(a, &t0, &step);
  for (int t = t0; t < tiles; t += step) {
    int nk;
    bool live;  // narrow: some of the warp's rows exist, of an expert's few
    {
      const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
      nk = tile.nk;
      live = !C::kNarrow || tile.p_valid > row0;
    }
    uint64_t sums[C::kWarpCols / 2];
#pragma unroll
    for (int i = 0; i < C::kWarpCols / 2; ++i) sums[i] = 0u;
    for (int kb = 0; kb < nk; ++kb) {
      const float* sc = steps.scales(kb);
      const uint64_t m = both(sc[row] * sc[C::kPScales + half * C::kWarpCols / kB128]);
      if (!steps.accumulator()) break;
      // The accumulator goes back as soon as it is in registers; 64 columns of it fit beside the sums.
      uint64_t v[32];
      auto add = [&](int h) {
#pragma unroll
        for (int i = 0; i < 32; ++i) sums[h * 32 + i] = fma2(v[i], m, sums[h * 32 + i]);
      };
      const uint32_t src = tbase + steps.column();
      if (live) {
        read_row(src, v);
        if constexpr (C::kWarpCols == 128) {
          add(0);
          read_row(src + 64, v);
        }
      }
      steps.accumulator_read();
      if (live) add(C::kWarpCols / 64 - 1);
      steps.end(kb, nk);
    }
    if (steps.failed) {
      steps.give_up();
      break;
    }
    // found again: kept through the steps, its fields would take the sums' registers
    const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
    if (tile.p_valid <= row0) continue;  // none of the warp's rows exists
    // all boxes of the staging at a time: one fence and one wait
#pragma unroll
    for (int b = 0; b < C::kWarpCols / Boxes<C>::kCols; b += C::kBoxes) {
      const int col = half * C::kWarpCols + b * Boxes<C>::kCols;
      if (col >= tile.q_valid) break;
      boxes.wait();
#pragma unroll
      for (int u = 0; u < C::kBoxes; ++u) {
        uint8_t* line = boxes.base + u * 4096 + lane * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q) {  // 16 bytes: four fp32 or eight bf16
          const uint64_t* d = sums + ((b + u) * Boxes<C>::kCols + q * (Boxes<C>::kCols / 8)) / 2;
          uint4 o;
          if constexpr (C::kF32) {
            o = make_uint4((uint32_t)d[0], (uint32_t)(d[0] >> 32), (uint32_t)d[1],
                           (uint32_t)(d[1] >> 32));
          } else {
            o = make_uint4(bf16_pair(first(d[0]), second(d[0])), bf16_pair(first(d[1]), second(d[1])),
                           bf16_pair(first(d[2]), second(d[2])), bf16_pair(first(d[3]), second(d[3])));
          }
          *reinterpret_cast<uint4*>(line + ((q ^ (lane & 7)) << 4)) = o;
        }
      }
      if (C::MODE == kB128Grouped && tile.p_valid < row0 + 32) {
        const int64_t at = (int64_t)(tile.c_row + row0) * a.ldc + tile.c_col + col;
#pragma unroll
        for (int u = 0; u < C::kBoxes; ++u) {
          boxes.store_part(a, u, at + u * Boxes<C>::kCols, tile.p_valid - row0,
                           tile.q_valid - col - u * Boxes<C>::kCols);
        }
      } else {
        boxes.store(cmap, tile.c_col + col, tile.c_row + row0, C::MODE == kB128Wgrad ? tile.e : 0,
                    tile.q_valid - col);
      }
    }
  }
  boxes.drain();
}

// The promoting warps of the columns and swapped shapes read the accumulator in fragments: warp w holds
// lanes 32 (w % 4) .. and half w / 4 of the tile's columns, and sums[(ch * 4 + g) * 4 + r] of lane l are
// the columns 32 ch + 8 g + 2 (l % 4) + {0, 1} of row 8 r + l / 4.
// Fragments reads one accumulator and adds it, `chunks` chunks of 32 columns, two at a time in registers:
// read(): the reads, with the first two chunks' sums between them; rest(): the sums that are left.
template <typename C>
struct Fragments {
  uint64_t (&sums)[C::kWarpCols / 2];
  uint64_t m[4], q[4];  // row scales; column scales of the chunk that is added next
  uint64_t v[32];
  const float* qs;

  __device__ __forceinline__ void column_scales(int ch) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      q[g] = *reinterpret_cast<const uint64_t*>(qs + ch * 32 + g * 8);
      if (!C::kPRows) q[g] = mul2(q[g], m[0]);
    }
  }
  // ps: scales of P's rows (at this warp's first and lane / 4) or of its block; qs_: of the columns
  __device__ __forceinline__ void scales(const float* ps, const float* qs_) {
    qs = qs_;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (C::kPRows || r == 0) m[r] = both(ps[C::kPRows ? 8 * r : 0]);
    }
    column_scales(0);
  }
  // ch is known at compile time wherever this is called; w: the chunk's sixteen pairs
  __device__ __forceinline__ void add(int ch, const uint64_t* w) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint64_t& d = sums[(ch * 4 + g) * 4 + r];
        d = fma2(w[8 * (r >> 1) + 2 * g + (r & 1)], C::kPRows ? mul2(q[g], m[r]) : q[g], d);
      }
    }
  }
  __device__ __forceinline__ void add_two(int ch, bool second) {
    add(ch, v);
    if (second) {
      column_scales(ch + 1);
      add(ch + 1, v + 16);
    }
  }
  __device__ __forceinline__ void read(uint32_t src, int chunks) {  // chunks <= kWarpCols / 32
    if constexpr (C::kWarpCols > 64) {  // all four chunks
      read_fragments(src, v);
      add_two(0, true);
      column_scales(2);
      read_fragments(src + 64, v);
    } else if (chunks > 1) {
      read_fragments(src, v);
    } else {
      read_fragments(src, *reinterpret_cast<uint64_t(*)[16]>(v));
    }
  }
  __device__ __forceinline__ void rest(int chunks) {
    add_two(C::kWarpCols > 64 ? 2 : 0, chunks > 1);
  }
};

// The columns shape.
template <typename C>
__device__ __forceinline__ void promote_columns(const CUtensorMap& cmap, const KernelArgs& a,
                                                const Smem& s, int tiles, uint32_t tmem, int pw) {
  constexpr int kChunks = C::kWarpCols / 32;
  const int lane = threadIdx.x & 31, row0 = (pw & 3) * 32, lr = lane >> 2, lc = (lane & 3) * 2;
  const int col0 = (pw >> 2) * C::kWarpCols;
  const uint32_t tbase = tmem + ((uint32_t)row0 << 16) + col0;
  Steps<C> steps(a, s);
  Boxes<C> boxes{s.staging + pw * C::kStagingBytes};
  int t0, step;
  tile_range<C>(a, &t0, &step);
  for (int t = t0; t < tiles; t += step) {
    const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
    uint64_t sums[C::kWarpCols / 2];
#pragma unroll
    for (int i = 0; i < C::kWarpCols / 2; ++i) sums[i] = 0u;
    Fragments<C> f{sums};
    for (int kb = 0; kb < tile.nk; ++kb) {
      const float* sc = steps.scales(kb);
      f.scales(sc + row0 + lr, sc + C::kPScales + col0 + lc);
      if (!steps.accumulator()) break;
      f.read(tbase + steps.column(), kChunks);
      steps.accumulator_read();
      f.rest(kChunks);
      steps.end(kb, tile.nk);
    }
    if (steps.failed) {
      steps.give_up();
      break;
    }
    if (tile.p_valid <= row0) continue;
    constexpr int kBoxCols = Boxes<C>::kCols;
#pragma unroll
    for (int b = 0; b < C::kWarpCols / kBoxCols; b += 2) {
      const int col = col0 + b * kBoxCols;
      if (col >= tile.q_valid) break;
      boxes.wait();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int g = 0; g < kBoxCols / 8; ++g) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint64_t d = sums[((b + u) * (kBoxCols / 8) + g) * 4 + r];
            uint8_t* line = boxes.base + u * 4096 + (8 * r + lr) * 128;
            if constexpr (C::kF32) {
              const int byte = (g * 8 + lc) * 4;
              *reinterpret_cast<uint64_t*>(line + (((byte >> 4) ^ lr) << 4) + (byte & 15)) = d;
            } else {
              const int byte = (g * 8 + lc) * 2;
              *reinterpret_cast<uint32_t*>(line + (((byte >> 4) ^ lr) << 4) + (byte & 15)) =
                  bf16_pair(first(d), second(d));
            }
          }
        }
      }
      boxes.store(cmap, tile.c_col + col, tile.c_row + row0, C::MODE == kB128Wgrad ? tile.e : 0,
                  tile.q_valid - col);
    }
  }
  boxes.drain();
}

// The swapped shape. A call that splits the contraction has one tile, whose sums are left for add_parts.
template <typename C>
__device__ __forceinline__ void promote_swapped(const KernelArgs& a, const Smem& s, int tiles,
                                                uint32_t tmem, int pw,
                                                uint64_t (&sums)[C::kWarpCols / 2]) {
  const int lane = threadIdx.x & 31, row0 = (pw & 3) * 32, lr = lane >> 2, lc = (lane & 3) * 2;
  Batches<C> batches(a, s);
  int t0, step;
  tile_range<C>(a, &t0, &step);
  for (int t = t0; t < tiles; t += step) {
    const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
    const int cols = tile.n / 2, col0 = (pw >> 2) * cols;  // this warp's columns
    const int chunks = (cols + 31) / 32;
    const uint32_t tbase = tmem + ((uint32_t)row0 << 16) + col0;
#pragma unroll
    for (int i = 0; i < C::kWarpCols / 2; ++i) sums[i] = 0u;
    Fragments<C> f{sums};
    for (int kb = 0; kb < tile.nk; kb += a.batch) {
      const int n = min(a.batch, tile.nk - kb);
      const float* sc = batches.scales(kb);
      if (!batches.accumulators()) break;
      for (int in = 0; in < n; ++in, sc += C::kSlotFloats) {
        f.scales(sc + (C::kPRows ? row0 + lr : 0), sc + C::kPScales + col0 + lc);
        f.read(tbase + batches.column(in), chunks);
        if (in == n - 1) batches.accumulators_read();
        f.rest(chunks);
      }
      batches.end(kb + n, tile.nk);
    }
    if (batches.failed) break;
    if (C::MODE == kB128Dense && a.split > 1) break;
    store_swapped<C>(a, s, tile, pw, sums, 0, 1);
  }
}

// Adds the parts of a tile whose contraction the CTAs of a cluster shared: every CTA leaves its sums in
// its own (now idle) ring, then each takes its share of the groups of columns, adds the parts in
// rank order and writes them.
template <typename C>
__device__ __forceinline__ void add_parts(const KernelArgs& a, const Smem& s, const Tile& tile, int pw,
                                          uint64_t (&sums)[C::kWarpCols / 2]) {
  const int tid = threadIdx.x - 128, rank = (int)cluster_rank();
  const int groups = tile.n / 2 / 8;  // of eight columns, per warp
  uint64_t* mine = reinterpret_cast<uint64_t*>(s.ring) + tid;
#pragma unroll
  for (int i = 0; i < C::kWarpCols / 2; ++i) {
    if (i / 4 < groups) mine[i * (kPromoWarps * 32)] = sums[i];
  }
  cluster_sync();
  uint32_t from[kMaxSplit];
#pragma unroll
  for (int r = 0; r < kMaxSplit; ++r) from[r] = in_cta(smem_u32(mine), r < a.split ? r : 0);
#pragma unroll
  for (int gi = 0; gi < C::kWarpCols / 8; ++gi) {
    if (gi >= groups || gi % a.split != rank) continue;
    uint64_t v[kMaxSplit][4];  // all on their way before the first is added
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (r < a.split) {
          asm volatile("ld.shared::cluster.b64 %0, [%1];"
                       : "=l"(v[r][i])
                       : "r"(from[r] + (gi * 4 + i) * (kPromoWarps * 32 * 8)));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint64_t sum = v[0][i];
#pragma unroll
      for (int r = 1; r < kMaxSplit; ++r) {
        if (r < a.split) sum = add2(sum, v[r][i]);
      }
      sums[gi * 4 + i] = sum;
    }
  }
  store_swapped<C>(a, s, tile, pw, sums, rank, a.split);
  cluster_sync();  // the parts are read before their CTAs leave
}

template <typename C>
__global__ void __launch_bounds__(kThreads, 1)
    b128_gemm_kernel(const __grid_constant__ CUtensorMap pmap,
                     const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap map16,
                     const __grid_constant__ CUtensorMap cmap, KernelArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Smem s;
  s.ring = smem;
  s.staging = smem + C::kRingBytes;
  s.scales = reinterpret_cast<float*>(s.staging + kPromoWarps * C::kStagingBytes);
  s.full = reinterpret_cast<uint64_t*>(s.scales + kScaleSlots * C::kSlotFloats);
  s.empty = s.full + kMaxStages;
  s.acc_full = s.empty + kMaxStages;
  s.acc_empty = s.acc_full + 4;
  s.scale_full = s.acc_empty + 2;
  s.scale_empty = s.scale_full + kScaleGroups;
  s.done = s.scale_empty + kScaleGroups;
  s.tmem_slot = reinterpret_cast<uint32_t*>(s.done + 1);
  s.prefix = reinterpret_cast<int*>(s.tmem_slot + 2);
  s.start = s.prefix + kMaxExperts + 1;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);  // uniform
  const bool parts = C::kSwap && C::MODE == kB128Dense && a.split > 1;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < stage_count<C>(a); ++i) {
      mbar_init(smem_u32(s.full + i), C::kSwap ? 1 : 1 + C::CTAS * kPromoWarps);
      mbar_init(smem_u32(s.empty + i), 1);
    }
    for (int i = 0; i < C::kBufs; ++i) mbar_init(smem_u32(s.acc_full + i), 1);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(s.acc_empty + i), kPromoWarps);
    for (int i = 0; i < kScaleGroups; ++i) {
      mbar_init(smem_u32(s.scale_full + i), 32);
      mbar_init(smem_u32(s.scale_empty + i), kPromoWarps);
    }
    mbar_init(smem_u32(s.done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  if (warp == 1) {
    if constexpr (C::CTAS == 2) {
      tmem_alloc_pair(smem_u32(s.tmem_slot), kTmemCols);
    } else {
      tmem_alloc(smem_u32(s.tmem_slot), kTmemCols);
      tmem_relinquish();
    }
  }
  if (C::MODE == kB128Grouped) build_table<C>(a, C::kPTile, INT32_MAX, s.prefix, s.start);
  if (C::MODE == kB128Wgrad) build_table<C>(a, kB128, (int)a.blocks_total, s.prefix, s.start);
  tc_fence_before();
  __syncthreads();
  if constexpr (C::CTAS == 2) cluster_sync();  // the other CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = *s.tmem_slot;
  const int tiles = tile_count<C>(a, s.prefix);
  // The promoting warps hold their sums and two or three chunks in registers: the others give theirs
  // up.
  if (C::MODE == kB128Grouped && tiles == 0) {
    // none of this launch's experts has rows (3.2 us a launch in all, 2.6 so)
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (warp == 0) produce<C>(pmap, qmap, map16, a, s, tiles);
    if (warp == 1 && (C::CTAS == 1 || cluster_rank() == 0)) multiply<C>(a, s, tiles, tmem);
    if (warp == 2) fetch_scales<C>(a, s, tiles);
    __syncwarp();
    if (parts) {  // add_parts' two
      cluster_sync();
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kPromoRegs));
    if constexpr (C::kSwap) {
      uint64_t sums[C::kWarpCols / 2];
      promote_swapped<C>(a, s, tiles, tmem, warp - 4, sums);
      if constexpr (C::MODE == kB128Dense) {
        if (parts) {
          const Tile tile = get_tile<C>(a, blockIdx.x / a.split, s.prefix, s.start);
          add_parts<C>(a, s, tile, warp - 4, sums);
        }
      }
    } else if constexpr (C::kQRows) {
      promote_columns<C>(cmap, a, s, tiles, tmem, warp - 4);
    } else {
      promote_rows<C>(cmap, a, s, tiles, tmem, warp - 4);
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (C::CTAS == 2) cluster_sync();  // nothing of either CTA is still used by the other
  tc_fence_after();
  if (warp == 1) {
    if constexpr (C::CTAS == 2) {
      tmem_dealloc_pair(tmem, kTmemCols);
    } else {
      tmem_dealloc(tmem, kTmemCols);
    }
  }
}

// ------------------------------------------------------------------------------------------
// host
// ------------------------------------------------------------------------------------------
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// launch_pdl with clusters of `ctas` CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), unsigned grid, int threads, size_t smem,
                            int ctas, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  if (err != cudaSuccess) (void)cudaGetLastError();  // reported here, not to a later caller
  return err;
}

template <typename C>
int slot_count() {
  return resident_ctas(reinterpret_cast<const void*>(&b128_gemm_kernel<C>), kThreads,
                       smem_bytes<C>(), 1);
}

// q_even, split (swapped): columns of a tile and CTAs along the contraction; row_min, row_max (by
// expert): the experts of this launch
template <typename C>
cudaError_t launch_config(const B128GemmArgs& g, cudaStream_t stream, int q_even = 0, int split = 1,
                          int row_min = 0, int row_max = INT32_MAX) {
  const int slots = slot_count<C>();
  if (slots <= 0) return cudaErrorInvalidConfiguration;
  KernelArgs a{};
  const int64_t kblocks = ceil_div(g.K, kB128), nblocks = ceil_div(g.N, kB128);
  const bool grouped = C::MODE == kB128Grouped;
  const int64_t bmap = grouped ? g.N * g.E : g.N;  // rows of B's tensor map
  const int64_t apitch = g.M, bpitch = g.b_rows ? g.N : kblocks;
  a.p_scales = C::kSwap ? g.b_scales : g.a_scales;
  a.q_scales = C::kSwap ? g.a_scales : g.b_scales;
  a.p_rows = C::kSwap ? g.N : g.M;
  a.q_rows = C::kSwap ? g.M : g.N;
  a.p_pitch = C::kSwap ? bpitch : apitch;
  a.q_pitch = C::kSwap ? apitch : bpitch;
  a.b_estride = grouped ? nblocks * kblocks : 0;
  a.c = g.c;
  a.offsets = g.offsets;
  a.err = g.err;
  a.wait_limit_ns = g.wait_limit_ns;
  a.ldc = g.N;
  a.rows_total = C::MODE == kB128Wgrad ? g.rows_total : g.M;
  a.blocks_total = kblocks;
  a.E = g.E;
  a.nk = (int)kblocks;
  a.p_tiles = (int)ceil_div(a.p_rows, C::kPTile);
  a.q_tiles = (int)ceil_div(a.q_rows, C::kSwap ? q_even : C::kTileCols);
  auto divisor = [](int64_t d) {
    return Divisor{(int)d, (uint32_t)((uint64_t(1) << 32) / (uint64_t)d + 1)};
  };
  if ((int64_t)a.p_tiles * a.q_tiles > INT32_MAX / 8) return cudaErrorInvalidValue;
  a.run = divisor(8 * (int64_t)a.q_tiles);
  a.per = divisor((int64_t)a.p_tiles * a.q_tiles);
  a.q_even = q_even;
  a.split = split;
  a.row_min = row_min;
  a.row_max = row_max;
  if (C::kSwap) {
    a.stage_bytes = (kLanes + q_even) * kStepBytes;
    a.stages = C::kRingBytes / a.stage_bytes;
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    a.batch = q_even <= 64 ? 4 : 2;  // two batches fill tensor memory
    a.stride = kColumns / a.batch;
  }
  const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const void *pcodes = C::kSwap ? g.b_codes : g.a_codes, *qcodes = C::kSwap ? g.a_codes : g.b_codes;
  const int64_t prows = C::kSwap ? bmap : g.M, qrows = C::kSwap ? g.M : bmap;
  CUtensorMap pmap, qmap, map16, cmap;  // map16: boxes of 16 rows of the tokens
  cudaError_t err = make_tensor_map_2d(&pmap, pcodes, prows, g.K, u8, 1, kStepBytes, kLanes, swz);
  if (err == cudaSuccess) {
    err = make_tensor_map_2d(&qmap, qcodes, qrows, g.K, u8, 1, kStepBytes, 128, swz);
  }
  map16 = pmap;  // where it is not used
  if (err == cudaSuccess && (C::kSwap || C::kNarrow)) {
    err = make_tensor_map_2d(&map16, g.a_codes, g.M, g.K, u8, 1, kStepBytes, 16, swz);
  }
  if (err == cudaSuccess) {
    if (C::kSwap) {
      cmap = pmap;  // not used
    } else {
      err = make_tensor_map_3d(&cmap, g.c, C::MODE == kB128Wgrad ? g.E : 1, g.M, g.N,
                               C::kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                               C::kF32 ? 4 : 2, C::kF32 ? 32 : 64, 32, swz);
    }
  }
  if (err != cudaSuccess) return err;
  int64_t tiles = (int64_t)a.p_tiles * a.q_tiles;  // at most, by expert
  if (C::MODE == kB128Wgrad) tiles *= g.E;
  if (grouped) tiles = (g.M / C::kPTile + (g.M < g.E ? g.M : g.E)) * a.q_tiles;
  if (tiles > INT32_MAX / kMaxSplit) return cudaErrorInvalidValue;
  const int cluster = C::kSwap && C::MODE == kB128Dense ? split : C::CTAS;
  const int64_t groups = split > 1 ? tiles : slots / cluster;
  return launch_clusters(&b128_gemm_kernel<C>, (unsigned)((tiles < groups ? tiles : groups) * cluster),
                         kThreads, smem_bytes<C>(), cluster, stream, pmap, qmap, map16, cmap, a);
}

// CTAs of the swapped shape that run at once in clusters of 1, 2, 4 or 8: the parts of the chip that a
// cluster cannot cross leave SMs over. Asked once per device.
template <typename C>
int cluster_slots(int ctas) {
  constexpr int kDevices = 16;
  static std::atomic<int> cache[kDevices][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::atomic<int>& kept = cache[dev % kDevices][ctas == 8 ? 3 : ctas / 2];
  int known = dev < kDevices ? kept.load(std::memory_order_relaxed) : 0;
  if (known == 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<C>();
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, &b128_gemm_kernel<C>, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      return 0;
    }
    known = clusters * ctas;
    if (dev < kDevices) kept.store(known, std::memory_order_relaxed);
  }
  return known;
}

// Dense calls: 256 x 256 tiles on pairs, or the swapped shape, whose 128-row weight tiles, times up to
// eight CTAs along the contraction as long as all run at once, spread few tokens over the SMs. The rule
// compares what each costs by its waves, from measured steps (us): 0.32 (8192^3: 0.34) and 2.3 a tile of the pairs,
// whatever the rows; 0.25 to 0.29 up to 64 columns, 0.44 beyond (batches of two), and 4 for joining
// the parts. 8192 x 8192, swapped / pairs: 1 token 14 / 34, 128 21 / 26, 192 31 / 26, 512 59 / 27.
template <bool B_ROWS, bool F32>
cudaError_t launch_dense(const B128GemmArgs& g, cudaStream_t stream) {
  using Large = Config<2, kB128Dense, false, true, B_ROWS, F32>;
  using Small = Config<1, kB128Dense, true, B_ROWS, true, F32>;
  const int slots = slot_count<Small>();
  if (slots <= 1) return cudaErrorInvalidConfiguration;
  const int64_t nk = ceil_div(g.K, kB128);
  const int64_t q_tiles = ceil_div(g.M, Small::kTileCols);
  const int q_even = (int)ceil_div(ceil_div(g.M, q_tiles), 16) * 16;
  const int64_t tiles = ceil_div(g.M, q_even) * ceil_div(g.N, kLanes);
  int split = 1;
  while (split < kMaxSplit && nk >= 4 * split && tiles * split * 2 <= slots &&
         tiles * split * 2 <= cluster_slots<Small>(split * 2)) {
    split *= 2;
  }
  const double step = q_even <= 64 ? 0.25 + 0.0007 * q_even : 0.44;
  const double few = (double)ceil_div(tiles * split, slots) * ((double)ceil_div(nk, split) * step + 1.2) +
                     (split > 1 ? 5.8 : 2.0);
  const double many =
      (double)ceil_div(ceil_div(g.M, 256) * ceil_div(g.N, 256), slots / 2) * ((double)nk * 0.32 + 2.3) +
      2.9;
  return many <= few ? launch_config<Large>(g, stream)
                     : launch_config<Small>(g, stream, q_even, split);
}

// Calls by expert: experts of more than kFewRows rows in 256 x 256 tiles on pairs, the others in tiles of
// 128 x 128: two launches, each of which takes its experts from the offsets. A call of few rows has
// no large expert. Weights of 1024 x 2048, us: 76 experts of 128 rows 39 narrow, of 130 rows 44 and of
// 256 rows 47 in pairs; 128 experts that share 16384 rows unevenly 76, of which the narrow shape was
// taken in place of the swapped one for 86 (128 choices among them: 34.5 for 39).
constexpr int kFewRows = 128;
template <bool F32>
cudaError_t launch_grouped(const B128GemmArgs& g, cudaStream_t stream) {
  if (g.M > kFewRows) {
    const cudaError_t err = launch_config<Config<2, kB128Grouped, false, true, false, F32>>(
        g, stream, 0, 1, kFewRows + 1, INT32_MAX);
    if (err != cudaSuccess) return err;
  }
  return launch_config<Config<1, kB128Grouped, false, true, false, F32>>(g, stream, 0, 1, 0, kFewRows);
}

}  // namespace

cudaError_t launch_b128_gemm(int mode, const B128GemmArgs& g, cudaStream_t stream) {
  if (mode == kB128Wgrad) {
    return g.out_f32
               ? launch_config<Config<2, kB128Wgrad, false, true, true, true>>(g, stream)
               : launch_config<Config<2, kB128Wgrad, false, true, true, false>>(g, stream);
  }
  if (mode == kB128Grouped) {
    return g.out_f32 ? launch_grouped<true>(g, stream) : launch_grouped<false>(g, stream);
  }
  if (g.b_rows) {
    return g.out_f32 ? launch_dense<true, true>(g, stream) : launch_dense<true, false>(g, stream);
  }
  return g.out_f32 ? launch_dense<false, true>(g, stream) : launch_dense<false, false>(g, stream);
}

}  // namespace mxq
