// mx_b128_gemm.cu -- products of E4M3 operands with one fp32 scale per block of 128 along the
// contraction, on the 5th-generation tensor cores:
//   C[i][j] = sum_kb sa[kb, i] sb[kb, j] sum_{k in block kb} a[i][k] b[j][k],
// dense, by expert (rows of A by offsets, one B per expert), and by expert for weight gradients
// (the contraction runs over each expert's own rows).
#include "mx_device.cuh"
#include "mx_expert.h"
#include "mx_launch.h"
#include "mx_tcgen05.cuh"

namespace mxq {

namespace {

using namespace tc;

constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s: drains, whatever the limit

// Operand P supplies the 128 tensor-memory lanes, operand Q the BN accumulator columns.
constexpr int kLanes = 128;
constexpr int kStepBytes = 128;  // one scale block of the contraction per step

// CTAS = 2: a pair of SMs shares one 256 x BN tile (cta_group::2). Each CTA loads 128 rows of P and
// half of Q's rows, holds its 128 lanes of the accumulator and promotes them; the first CTA issues
// the MMAs for both. Per step an SM then receives 32 KB instead of 48 and reads as much: one CTA
// alone with 128 x 256 tiles was bound by shared memory (48 KB in, 48 KB read, about 750 of the
// MMAs' 512 cycles).
template <int BN, int CTAS>
struct Shape {
  static constexpr int kPromoWarps = BN >= 256 ? 8 : 4;
  static constexpr int kThreads = 128 + kPromoWarps * 32;
  static constexpr int kCols = BN / (kPromoWarps / 4);  // accumulator columns of a promoting warp
  static constexpr int kChunk = kCols < 32 ? kCols : 32;
  static constexpr int kQRowsLoaded = BN / CTAS;
  static constexpr int kStageBytes = (kLanes + kQRowsLoaded) * kStepBytes;
  static constexpr int kStages = BN >= 128 ? 6 : 8;
  static constexpr uint32_t kTmemCols = 2 * BN;  // two accumulators: 32 .. 512 columns
  static_assert(kStages % 2 == 0, "a stage always meets the same accumulator");
};
// scales travel and are released by groups of steps
constexpr int kScaleGroup = 4, kScaleGroups = 2, kScaleSlots = kScaleGroup * kScaleGroups;

// tile table of the calls by expert: prefix[E + 1] (tiles or blocks before each expert), then
// start[E + 1] (its first row) -- both int32, E <= 1024
constexpr int kMaxExperts = 1024;

struct KernelArgs {
  const float* p_scales;
  const float* q_scales;
  void* c;
  const int64_t* offsets;
  unsigned int* err;
  unsigned long long wait_limit_ns;
  int64_t p_rows, q_rows;      // rows of P and Q: of one expert's matrix, or of the whole of A
  int64_t p_pitch, q_pitch;    // rows form: floats per scale row; blocks form: floats per block row
  int64_t p_estride, q_estride;  // blocks form: floats of one expert
  int64_t ldc;                 // floats / elements per row of C
  int64_t c_estride;           // elements of one expert's C (wgrad)
  int64_t rows_total;          // rows the offsets may name
  int64_t blocks_total;        // wgrad: 128-row blocks of the padded operands
  int E;
  int nk;                      // steps of the contraction (dense, grouped)
  int p_tiles, q_tiles;        // tiles of the fixed operands (grouped: of the weights only)
  int tok_tile;                // grouped: rows of one tile of tokens
};

struct Tile {
  int p_row, q_row;        // first rows in the tensor maps
  int p_valid, q_valid;    // rows of the tile that exist
  int k0;                  // first byte along the contraction
  int kb0, nk;             // first scale block, steps
  int64_t p_scale, q_scale;  // first scale: rows form [kb0][row], blocks form [row / 128][kb0]
  int64_t c;               // element of C at (lane 0, column 0)
};

// The MMAs of one step (K = 128 in four of 32, the first overwriting the accumulator) and the
// commits that free the operands' stage and hand the accumulator over, issued by one elected lane of
// a converged warp. One statement with every operand computed outside: in a branch of the elected
// lane the descriptors went through vector registers and a step took 400 cycles to issue.
template <int CTAS>
__device__ __forceinline__ void issue_step(uint32_t d, uint64_t p, uint64_t q, uint32_t idesc,
                                           uint32_t empty, uint32_t acc_full) {
  if constexpr (CTAS == 1) {
    asm volatile(
        "{\n\t.reg .pred e, on, off;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\tsetp.ne.b32 off, 0, 0;\n\tsetp.eq.b32 on, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %5, %9, off;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %2, %6, %9, on;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %3, %7, %9, on;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %4, %8, %9, on;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%10];\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%11];\n\t"
        "}" ::"r"(d),
        "l"(p), "l"(p + 2), "l"(p + 4), "l"(p + 6), "l"(q), "l"(q + 2), "l"(q + 4), "l"(q + 6),
        "r"(idesc), "r"(empty), "r"(acc_full)
        : "memory");
  } else {  // the commits arrive at the same barriers of both CTAs
    asm volatile(
        "{\n\t.reg .pred e, on, off;\n\t.reg .b16 both;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\tsetp.ne.b32 off, 0, 0;\n\tsetp.eq.b32 on, 0, 0;\n\t"
        "mov.b16 both, 3;\n\t"
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

// The pair's rank, barrier and addresses.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t in_first_cta(uint32_t addr) {  // the same address of CTA 0
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
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

// Instruction descriptor, kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), A and B E4M3 (bits 7-9
// and 10-12 = 0), both K-major, N >> 3 at bits 17-22, M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// N consecutive 32-bit columns of this thread's tensor-memory lane: the load is only issued; the
// values are there after wait_columns, which names them so that no use moves before it.
__device__ __forceinline__ void issue_columns(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void issue_columns(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void wait_columns(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void wait_columns(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// Pairs of fp32 in one 64-bit register: one instruction for two (the same rate per value, half the
// instructions, which the warp that issues the MMAs competes with for fetch and issue).
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  return ((uint64_t)hi << 32) | lo;
}
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

// Scale forms of an operand and orientation of the output.
template <int BN_, int CTAS_, int MODE_, bool SWAP_, bool P_ROWS_, bool Q_ROWS_, bool F32_>
struct Config {
  static constexpr int BN = BN_, CTAS = CTAS_, MODE = MODE_;
  using S = Shape<BN_, CTAS_>;
  static constexpr int kPRowsTile = kLanes * CTAS_;  // rows of P in a tile
  static constexpr bool kSwap = SWAP_;    // P is B (weights), C written [column][lane]
  static constexpr bool kPRows = P_ROWS_, kQRows = Q_ROWS_;
  static constexpr bool kF32 = F32_;
  // floats of a scale slot: one per lane / column (rows form) or one per block of 128
  static constexpr int kPScales = P_ROWS_ ? kLanes : 4, kQScales = Q_ROWS_ ? BN_ : 4;
  static constexpr int kSlotFloats = kPScales + kQScales;
};

template <typename C>
constexpr int smem_bytes() {
  using S = typename C::S;
  return 1024 + S::kStages * S::kStageBytes + kScaleSlots * C::kSlotFloats * 4 +
         (2 * S::kStages + 2 * kScaleGroups + 3) * 8 + 16 +
         (C::MODE != kB128Dense ? 2 * (kMaxExperts + 1) * 4 : 0);
}

// tiles in all; grouped and wgrad calls read the table
template <typename C>
__device__ __forceinline__ int tile_count(const KernelArgs& a, const int* prefix) {
  if (C::MODE == kB128Dense) return a.p_tiles * a.q_tiles;
  if (C::MODE == kB128Wgrad) return a.p_tiles * a.q_tiles * a.E;
  return prefix[a.E] * (C::kSwap ? a.p_tiles : a.q_tiles);
}

// p tile and q tile of tile t of a p_tiles x q_tiles grid: runs of eight p tiles cross all q
// tiles, so that the CTAs working at one time share operands in L2
__device__ __forceinline__ void raster(int t, int p_tiles, int q_tiles, int* p, int* q) {
  const int run = 8 * q_tiles, first = t / run * 8;
  const int height = min(8, p_tiles - first);
  const int in = t % run;
  *p = first + in % height;
  *q = in / height;
}

// The tile as this CTA of a pair sees it: its own 128 rows of P.
template <typename C>
__device__ __forceinline__ Tile own_half(const KernelArgs& a, Tile r) {
  if constexpr (C::CTAS == 2) {
    const int rank = (int)cluster_rank(), skip = rank * kLanes;
    r.p_row += skip;
    r.p_valid = min(kLanes, r.p_valid - skip);  // <= 0: nothing of it exists
    r.p_scale += C::kPRows ? skip : rank * a.p_pitch;
    r.c += C::kSwap ? (int64_t)skip : skip * a.ldc;
  }
  return r;
}

template <typename C>
__device__ __forceinline__ Tile get_tile(const KernelArgs& a, int t, const int* prefix,
                                         const int* start) {
  Tile r;
  int e = 0, p, q;
  if (C::MODE == kB128Grouped) {
    const int fixed = C::kSwap ? a.p_tiles : a.q_tiles;
    int lo = 0, hi = a.E;  // largest e with prefix[e] * fixed <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)prefix[mid] * fixed <= t) {
        lo = mid;
      } else {
        hi = mid;
      }
    }
    e = lo;
    const int local = t - prefix[e] * fixed, n = prefix[e + 1] - prefix[e];
    const int tok = local % n, w = local / n;  // token tiles of one weight tile run together
    const int row = start[e] + tok * a.tok_tile;
    const int left = start[e + 1] - row;
    if (C::kSwap) {
      p = w;
      r.p_row = (int)(e * a.p_rows) + p * C::kPRowsTile;
      r.p_valid = (int)min((int64_t)C::kPRowsTile, a.p_rows - (int64_t)p * C::kPRowsTile);
      r.q_row = row;
      r.q_valid = min(C::BN, left);
      r.p_scale = e * a.p_estride + (int64_t)p * C::CTAS * a.p_pitch;
      r.q_scale = row;
      r.c = (int64_t)row * a.ldc + p * C::kPRowsTile;
    } else {
      q = w;
      r.p_row = row;
      r.p_valid = min(C::kPRowsTile, left);
      r.q_row = (int)(e * a.q_rows) + q * C::BN;
      r.q_valid = (int)min((int64_t)C::BN, a.q_rows - (int64_t)q * C::BN);
      r.p_scale = row;
      r.q_scale = e * a.q_estride + (int64_t)q * (C::BN / kB128) * a.q_pitch;
      r.c = (int64_t)row * a.ldc + (int64_t)q * C::BN;
    }
    r.k0 = r.kb0 = 0;
    r.nk = a.nk;
    return own_half<C>(a, r);
  }
  r.kb0 = 0;
  r.nk = a.nk;
  if (C::MODE == kB128Wgrad) {
    const int per = a.p_tiles * a.q_tiles;
    e = t / per;
    t -= e * per;
    r.kb0 = prefix[e];
    r.nk = prefix[e + 1] - prefix[e];
  }
  raster(t, a.p_tiles, a.q_tiles, &p, &q);
  r.k0 = r.kb0 * kStepBytes;
  r.p_row = p * C::kPRowsTile;
  r.q_row = q * C::BN;
  r.p_valid = (int)min((int64_t)C::kPRowsTile, a.p_rows - r.p_row);
  r.q_valid = (int)min((int64_t)C::BN, a.q_rows - r.q_row);
  r.p_scale = C::kPRows ? r.kb0 * a.p_pitch + r.p_row : (int64_t)p * C::CTAS * a.p_pitch + r.kb0;
  r.q_scale = C::kQRows ? r.kb0 * a.q_pitch + r.q_row
                        : (int64_t)q * (C::BN / kB128) * a.q_pitch + r.kb0;
  r.c = e * a.c_estride + (C::kSwap ? (int64_t)r.q_row * a.ldc + r.p_row
                                    : (int64_t)r.p_row * a.ldc + r.q_row);
  return own_half<C>(a, r);
}

// Table of the calls by expert: prefix sums of ceil(n_e / unit). Offsets that break their contract
// are clamped, so that every later access stays inside the operands.
__device__ __forceinline__ void build_table(const KernelArgs& a, int unit, int limit, int* prefix,
                                            int* start) {
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  int before = 0;
  if (lane == 0) prefix[0] = 0;
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    const int e = e0 + lane;
    int64_t lo = 0, hi = 0;
    if (e < a.E) {
      lo = min(max(load_s64(a.offsets + e), (int64_t)0), a.rows_total);
      hi = min(max(load_s64(a.offsets + e + 1), lo), a.rows_total);
      start[e] = (int)lo;
      if (e == a.E - 1) start[a.E] = (int)hi;
    }
    int sum = (int)((hi - lo + unit - 1) / unit);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += up;
    }
    if (e < a.E) prefix[e + 1] = min(before + sum, limit);
    before += __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
}

struct Smem {
  uint8_t* ring;
  float* scales;        // [kScaleSlots][kSlotFloats]
  uint64_t* full;
  uint64_t* empty;
  uint64_t* acc_full;   // [2]
  uint64_t* scale_full;   // [kScaleGroups]
  uint64_t* scale_empty;  // [kScaleGroups]
  uint64_t* done;
  uint32_t* tmem_slot;
  int* prefix;
  int* start;
};

// One lane of a warp that runs converged.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Whether the phase is complete. try_wait lets the hardware suspend the thread meanwhile, for longer
// than most waits last; a call with a limit below that (the give-up self-test) asks without.
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity, const KernelArgs& a) {
  if (a.wait_limit_ns >= 1000000ull) return mbar_try_wait(bar, parity);
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred P;\n\tmbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
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

// The loading and the multiplying warp run converged and issue from one elected lane: addresses
// and descriptors then stay in uniform registers. Issued from a lone lane's own branch instead,
// the four MMAs and two commits of a step took over 600 cycles, more than the MMAs themselves.
template <typename C>
__device__ __forceinline__ void produce(const CUtensorMap& pmap, const CUtensorMap& qmap,
                                        const KernelArgs& a, const Smem& s, int tiles) {
  using S = typename C::S;
  bool failed = false;
  int issued = 0, st = 0;
  uint32_t parity = 1;  // a fresh barrier's preceding phase counts as complete
  for (int t = blockIdx.x / C::CTAS; t < tiles && !failed; t += gridDim.x / C::CTAS) {
    const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
    for (int kb = 0; kb < tile.nk; ++kb) {
      warp_wait(smem_u32(s.empty + st), parity, &failed, a);
      if (failed) break;
      const uint32_t bar = smem_u32(s.full + st), dst = smem_u32(s.ring + st * S::kStageBytes);
      const int x = tile.k0 + kb * kStepBytes;
      if constexpr (C::CTAS == 2) {
        const uint32_t first = in_first_cta(bar);
        const int q_row = tile.q_row + (int)cluster_rank() * S::kQRowsLoaded;
        if (elect_one()) {
          if (cluster_rank() == 0) mbar_arrive_expect_tx(bar, 2 * S::kStageBytes);
          tma_load_box_pair(dst, &pmap, x, tile.p_row, first);
          tma_load_box_pair(dst + kLanes * kStepBytes, &qmap, x, q_row, first);
        }
      } else if (elect_one()) {
        mbar_arrive_expect_tx(bar, S::kStageBytes);
        tma_load_box(dst, &pmap, x, tile.p_row, bar);
        tma_load_box(dst + kLanes * kStepBytes, &qmap, x, tile.q_row, bar);
      }
      ++issued;
      if (++st == S::kStages) {
        st = 0;
        parity ^= 1;
      }
    }
  }
  // Loads in flight land before the CTA's shared memory goes away. The first CTA of a pair sees both
  // CTAs' on its barriers, and both leave together; after a give-up, in which the two may not have
  // issued the same steps, each also lets a millisecond pass, a thousand times what a load takes.
  if (C::CTAS == 2 && failed) {
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < 1000000ull) {
    }
  }
  if (C::CTAS == 2 && cluster_rank() != 0) return;
  bool drain_failed = false;
  for (int i = issued > S::kStages ? issued - S::kStages : 0; i < issued; ++i) {
    mbar_wait(smem_u32(s.full + i % S::kStages), (i / S::kStages) & 1, &drain_failed, kWaitNs, a.err);
  }
}

template <typename C>
__device__ __forceinline__ void multiply(const KernelArgs& a, const Smem& s, int tiles,
                                         uint32_t tmem) {
  using S = typename C::S;
  constexpr uint32_t idesc = idesc_e4m3_f32(C::kPRowsTile, C::BN);
  static_assert(kStepBytes == 128, "issue_step");
  bool failed = false;
  int st = 0, buf = 0;
  uint32_t full_parity = 0;
  for (int t = blockIdx.x / C::CTAS; t < tiles && !failed; t += gridDim.x / C::CTAS) {
    const int nk = get_tile<C>(a, t, s.prefix, s.start).nk;
    for (int kb = 0; kb < nk; ++kb) {
      warp_wait(smem_u32(s.full + st), full_parity, &failed, a);
      if (failed) break;
      tc_fence_after();
      const uint64_t p = desc_sw128(smem_u32(s.ring + st * S::kStageBytes));
      issue_step<C::CTAS>(tmem + buf * C::BN, p, p + (kLanes * kStepBytes >> 4), idesc, smem_u32(s.empty + st),
                 smem_u32(s.acc_full + buf));
      if (++st == S::kStages) {
        st = 0;
        full_parity ^= 1;
      }
      buf ^= 1;
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

// 4-byte asynchronous copy to shared memory; zero where !ok (nothing is read then).
__device__ __forceinline__ void copy_scale(float* dst, const float* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(ok ? 4 : 0)
               : "memory");
}

// One warp copies the scales into a ring, a group of steps at a time and a group ahead: the promoting
// warps then never wait for a scale's trip from L2, which is longer than a step, and meet a barrier
// for scales once in kScaleGroup steps.
template <typename C>
__device__ __forceinline__ void fetch_scales(const KernelArgs& a, const Smem& s, int tiles) {
  const int lane = threadIdx.x & 31;
  bool failed = false;
  int group = 0;
  for (int t = blockIdx.x / C::CTAS; t < tiles && !failed; t += gridDim.x / C::CTAS) {
    const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
    for (int kb0 = 0; kb0 < tile.nk; kb0 += kScaleGroup, ++group) {
      const int g = group % kScaleGroups;
      warp_wait(smem_u32(s.scale_empty + g), ((group / kScaleGroups) & 1) ^ 1, &failed, a);
      if (failed) break;
      for (int kb = kb0; kb < min(kb0 + kScaleGroup, tile.nk); ++kb) {
        float* dst = s.scales + (g * kScaleGroup + kb - kb0) * C::kSlotFloats;
        if (C::kPRows) {
          const float* src = a.p_scales + tile.p_scale + kb * a.p_pitch;
#pragma unroll
          for (int i = 0; i < kLanes / 32; ++i) {
            const int r = 32 * i + lane;
            const bool ok = r < tile.p_valid;
            copy_scale(dst + r, ok ? src + r : a.p_scales, ok);
          }
        } else if (lane == 0) {
          const bool ok = tile.p_valid > 0;
          copy_scale(dst, ok ? a.p_scales + tile.p_scale + kb : a.p_scales, ok);
        }
        dst += C::kPScales;
        if (C::kQRows) {
          const float* src = a.q_scales + tile.q_scale + kb * a.q_pitch;
#pragma unroll
          for (int i = 0; i < (C::BN + 31) / 32; ++i) {
            const int c = 32 * i + lane;
            const bool ok = c < tile.q_valid;
            if (c < C::BN) copy_scale(dst + c, ok ? src + c : a.q_scales, ok);
          }
        } else if (lane < C::BN / kB128) {
          const bool ok = lane * kB128 < tile.q_valid;
          copy_scale(dst + lane,
                     ok ? a.q_scales + tile.q_scale + lane * a.q_pitch + kb : a.q_scales, ok);
        }
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                       smem_u32(s.scale_full + g))
                   : "memory");
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // none lands after the CTA's shared memory goes
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

// The promoting warps: warp w holds lanes 32 (w % 4) .. and columns kCols (w / 4) .. of the tile in
// registers, adds each step's accumulator times the step's scales, and writes the tile.
template <typename C>
__device__ __forceinline__ void promote(const KernelArgs& a, const Smem& s, int tiles,
                                        uint32_t tmem, int pw) {
  using S = typename C::S;
  constexpr int kCols = S::kCols, kChunk = S::kChunk;
  const int lane = threadIdx.x & 31;
  const int row = (pw & 3) * 32 + lane, col0 = (pw >> 2) * kCols;
  const uint32_t tbase = tmem + ((uint32_t)((pw & 3) * 32) << 16) + col0;
  bool failed = false;
  int it = 0;
  // A step's stage is full once its operands have landed and its accumulator has been read: both
  // arrive on one barrier, so the multiplying warp waits once per step. The first two steps find
  // their accumulators free.
  const uint32_t full0 = C::CTAS == 2 ? in_first_cta(smem_u32(s.full)) : smem_u32(s.full);
  auto hand_back = [&](int st) {
    if constexpr (C::CTAS == 2) {
      warp_arrive_cluster(full0 + 8 * st);
    } else {
      warp_arrive(full0 + 8 * st);
    }
  };
  hand_back(0);
  hand_back(1);
  int st2 = 2;  // stage of the step after next
  uint32_t group = 0;
  for (int t = blockIdx.x / C::CTAS; t < tiles; t += gridDim.x / C::CTAS) {
    const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
    const bool live = row < tile.p_valid;
    uint64_t sums[kCols / 2];  // fp32 pairs
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) sums[i] = 0u;
    for (int kb = 0; kb < tile.nk; ++kb, ++it) {
      const int buf = it & 1, g = group % kScaleGroups, in = kb % kScaleGroup;
      const float* ps = s.scales + (g * kScaleGroup + in) * C::kSlotFloats;
      const float* cs = ps + C::kPScales + (C::kQRows ? col0 : col0 / kB128);
      if (in == 0) {
        warp_wait(smem_u32(s.scale_full + g), (group / kScaleGroups) & 1, &failed, a);
      }
      const float m = ps[C::kPRows ? row : 0] * (C::kQRows ? 1.0f : cs[0]);
      const uint64_t m2 = pair(__float_as_uint(m), __float_as_uint(m));
      warp_wait(smem_u32(s.acc_full + buf), (it >> 1) & 1, &failed, a);
      if (failed) break;
      tc_fence_after();
      // The accumulator goes back to the MMAs as soon as it is in registers: with two of them, a
      // step cannot be shorter than half of (MMA + signal + read + signal), so the reads come first
      // and the sums after. Three of four chunks fit beside the sums; the fourth follows the first's.
      // With a scale per column two chunks at a time: the scales' own reads from shared memory need
      // registers to run ahead, else each of them is waited for (1300 cycles a step).
      constexpr int kChunks = kCols / kChunk;
      constexpr int kFirst = kChunks > 3 ? (C::kQRows ? 2 : 3) : kChunks;
      uint32_t v[kFirst][kChunk];
      auto add = [&](int ch, const uint32_t (&w)[kChunk]) {
#pragma unroll
        for (int i = 0; i < kChunk; i += 4) {
          uint64_t* d = sums + (ch * kChunk + i) / 2;
          uint64_t m01 = m2, m23 = m2;
          if (C::kQRows) {
            const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(cs + ch * kChunk + i);
            m01 = mul2(m2, q.x);
            m23 = mul2(m2, q.y);
          }
          d[0] = fma2(pair(w[i], w[i + 1]), m01, d[0]);
          d[1] = fma2(pair(w[i + 2], w[i + 3]), m23, d[1]);
        }
      };
      const uint32_t src = tbase + buf * C::BN;
#pragma unroll
      for (int ch = 0; ch < kFirst; ++ch) issue_columns(src + ch * kChunk, v[ch]);
#pragma unroll
      for (int ch = 0; ch < kFirst; ++ch) wait_columns(v[ch]);
#pragma unroll
      for (int ch = kFirst; ch < kChunks; ++ch) {
        add(ch - kFirst, v[ch - kFirst]);
        issue_columns(src + ch * kChunk, v[ch - kFirst]);
      }
#pragma unroll
      for (int ch = kFirst; ch < kChunks; ++ch) wait_columns(v[ch - kFirst]);
      tc_fence_before();
      hand_back(st2);
      if (++st2 == S::kStages) st2 = 0;
#pragma unroll
      for (int ch = kChunks - kFirst; ch < kChunks; ++ch) add(ch, v[ch % kFirst]);
      if (in == kScaleGroup - 1 || kb == tile.nk - 1) {
        warp_arrive(smem_u32(s.scale_empty + g));
        ++group;
      }
    }
    if (failed) {
      // The steps that may have been loaded are handed back unread, so that the loading warp sees
      // its copies land. Steps it and it + 1 have their arrivals already and their stages may still
      // be in that phase, so the steps that follow on those two stages are left out: a second
      // arrival there would complete a phase before its copies do.
      for (int i = 0; i < S::kStages - 2; ++i) hand_back((st2 + i) % S::kStages);
      return;
    }
    if (!live) continue;
    float acc[kCols];
#pragma unroll
    for (int i = 0; i < kCols; i += 2) {
      acc[i] = __uint_as_float((uint32_t)sums[i / 2]);
      acc[i + 1] = __uint_as_float((uint32_t)(sums[i / 2] >> 32));
    }
    if (C::kSwap) {  // lane = column of C, a warp writes 32 neighbours of each row
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        if (col0 + i >= tile.q_valid) break;
        const int64_t at = tile.c + (int64_t)(col0 + i) * a.ldc + row;
        if (C::kF32) {
          static_cast<float*>(a.c)[at] = acc[i];
        } else {
          uint16_t h;
          asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(acc[i]));
          static_cast<uint16_t*>(a.c)[at] = h;
        }
      }
    } else {  // lane = row of C, 16-byte pieces (columns in eights: N % 8 == 0)
      const int64_t at = tile.c + (int64_t)row * a.ldc + col0;
#pragma unroll
      for (int i = 0; i < kCols; i += 8) {
        if (col0 + i >= tile.q_valid) break;
        if (C::kF32) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.c) + at + i);
          o[0] = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
          o[1] = make_float4(acc[i + 4], acc[i + 5], acc[i + 6], acc[i + 7]);
        } else {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            asm("cvt.rn.bf16x2.f32 %0, %2, %1;"
                : "=r"(o[j])
                : "f"(acc[i + 2 * j]), "f"(acc[i + 2 * j + 1]));
          }
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.c) + at + i) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }
}

template <typename C>
__global__ void __launch_bounds__(C::S::kThreads, 1)
    b128_gemm_kernel(const __grid_constant__ CUtensorMap pmap,
                     const __grid_constant__ CUtensorMap qmap, KernelArgs a) {
  using S = typename C::S;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Smem s;
  s.ring = smem;
  s.scales = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes);
  s.full = reinterpret_cast<uint64_t*>(s.scales + kScaleSlots * C::kSlotFloats);
  s.empty = s.full + S::kStages;
  s.acc_full = s.empty + S::kStages;
  s.scale_full = s.acc_full + 2;
  s.scale_empty = s.scale_full + kScaleGroups;
  s.done = s.scale_empty + kScaleGroups;
  s.tmem_slot = reinterpret_cast<uint32_t*>(s.done + 1);
  s.prefix = reinterpret_cast<int*>(s.tmem_slot + 2);
  s.start = s.prefix + kMaxExperts + 1;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);  // uniform

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(smem_u32(s.full + i), 1 + C::CTAS * S::kPromoWarps);
      mbar_init(smem_u32(s.empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(s.acc_full + i), 1);
    for (int i = 0; i < kScaleGroups; ++i) {
      mbar_init(smem_u32(s.scale_full + i), 32);
      mbar_init(smem_u32(s.scale_empty + i), S::kPromoWarps);
    }
    mbar_init(smem_u32(s.done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  if (warp == 1) {
    if constexpr (C::CTAS == 2) {
      tmem_alloc_pair(smem_u32(s.tmem_slot), S::kTmemCols);
    } else {
      tmem_alloc(smem_u32(s.tmem_slot), S::kTmemCols);
      tmem_relinquish();
    }
  }
  if (C::MODE == kB128Grouped) build_table(a, a.tok_tile, INT32_MAX, s.prefix, s.start);
  if (C::MODE == kB128Wgrad) build_table(a, kB128, (int)a.blocks_total, s.prefix, s.start);
  tc_fence_before();
  __syncthreads();
  if constexpr (C::CTAS == 2) cluster_sync();  // the other CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = *s.tmem_slot;
  const int tiles = tile_count<C>(a, s.prefix);
  // The promoting warps hold kCols sums and two chunks in registers: of a launch with eight of them
  // the others give theirs up (40 x 128 + 232 x 256 = 168 x 384, the launch's total).
  if (warp < 4) {
    if (S::kPromoWarps == 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) produce<C>(pmap, qmap, a, s, tiles);
    if (warp == 1 && (C::CTAS == 1 || cluster_rank() == 0)) multiply<C>(a, s, tiles, tmem);
    if (warp == 2) fetch_scales<C>(a, s, tiles);
  } else {
    if (S::kPromoWarps == 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    promote<C>(a, s, tiles, tmem, warp - 4);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (C::CTAS == 2) cluster_sync();  // nothing of either CTA is still used by the other
  tc_fence_after();
  if (warp == 1) {
    if constexpr (C::CTAS == 2) {
      tmem_dealloc_pair(tmem, S::kTmemCols);
    } else {
      tmem_dealloc(tmem, S::kTmemCols);
    }
  }
}

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
cudaError_t launch_config(const B128GemmArgs& g, cudaStream_t stream) {
  using S = typename C::S;
  auto* kernel = &b128_gemm_kernel<C>;
  constexpr int smem = smem_bytes<C>();
  const int slots = resident_ctas(reinterpret_cast<const void*>(kernel), S::kThreads, smem, 1);
  if (slots <= 0) return cudaErrorInvalidConfiguration;
  KernelArgs a{};
  const int64_t kblocks = ceil_div(g.K, kB128), nblocks = ceil_div(g.N, kB128);
  const bool grouped = C::MODE == kB128Grouped;
  // rows of one matrix of each operand, and of all of its tensor map
  const int64_t arows = g.M, brows = g.N, bmap = grouped ? g.N * g.E : g.N;
  const int64_t apitch = g.M;
  const int64_t bpitch = g.b_rows ? g.N : kblocks;
  const int64_t bestride = g.b_rows ? 0 : nblocks * kblocks;
  a.p_scales = C::kSwap ? g.b_scales : g.a_scales;
  a.q_scales = C::kSwap ? g.a_scales : g.b_scales;
  a.p_rows = C::kSwap ? brows : arows;
  a.q_rows = C::kSwap ? arows : brows;
  a.p_pitch = C::kSwap ? bpitch : apitch;
  a.q_pitch = C::kSwap ? apitch : bpitch;
  a.p_estride = C::kSwap ? bestride : 0;
  a.q_estride = C::kSwap ? 0 : bestride;
  a.c = g.c;
  a.offsets = g.offsets;
  a.err = g.err;
  a.wait_limit_ns = g.wait_limit_ns;
  a.ldc = g.N;
  a.c_estride = g.M * g.N;
  a.rows_total = C::MODE == kB128Wgrad ? g.rows_total : g.M;
  a.blocks_total = kblocks;
  a.E = g.E;
  a.nk = (int)kblocks;
  a.p_tiles = (int)ceil_div(a.p_rows, C::kPRowsTile);
  a.q_tiles = (int)ceil_div(a.q_rows, C::BN);
  a.tok_tile = C::kSwap ? C::BN : C::kPRowsTile;
  CUtensorMap pmap, qmap;
  const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
  cudaError_t err = make_tensor_map_2d(&pmap, C::kSwap ? g.b_codes : g.a_codes,
                                       C::kSwap ? bmap : arows, g.K, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1,
                                       kStepBytes, kLanes, swz);
  if (err != cudaSuccess) return err;
  err = make_tensor_map_2d(&qmap, C::kSwap ? g.a_codes : g.b_codes, C::kSwap ? arows : bmap, g.K,
                           CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kStepBytes, S::kQRowsLoaded, swz);
  if (err != cudaSuccess) return err;
  int64_t tiles = (int64_t)a.p_tiles * a.q_tiles;  // at most, by expert
  if (C::MODE == kB128Wgrad) tiles *= g.E;
  if (grouped) {
    tiles = (g.M / a.tok_tile + (g.M < g.E ? g.M : g.E)) * (C::kSwap ? a.p_tiles : a.q_tiles);
  }
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  const int64_t groups = slots / C::CTAS;
  return launch_clusters(kernel, (unsigned)((tiles < groups ? tiles : groups) * C::CTAS), S::kThreads,
                         smem, C::CTAS, stream, pmap, qmap, a);
}

}  // namespace

cudaError_t launch_b128_gemm(int mode, const B128GemmArgs& g, cudaStream_t stream) {
  if (mode == kB128Wgrad) {
    return g.out_f32 ? launch_config<Config<256, 2, kB128Wgrad, false, true, true, true>>(g, stream)
                     : launch_config<Config<256, 2, kB128Wgrad, false, true, true, false>>(g, stream);
  }
  if (mode == kB128Grouped) {
    return g.out_f32 ? launch_config<Config<256, 2, kB128Grouped, false, true, false, true>>(g, stream)
                     : launch_config<Config<256, 2, kB128Grouped, false, true, false, false>>(g, stream);
  }
  if (g.b_rows) {
    return g.out_f32 ? launch_config<Config<256, 2, kB128Dense, false, true, true, true>>(g, stream)
                     : launch_config<Config<256, 2, kB128Dense, false, true, true, false>>(g, stream);
  }
  return g.out_f32 ? launch_config<Config<256, 2, kB128Dense, false, true, false, true>>(g, stream)
                   : launch_config<Config<256, 2, kB128Dense, false, true, false, false>>(g, stream);
}

}  // namespace mxq
