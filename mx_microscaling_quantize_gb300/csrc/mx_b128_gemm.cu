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

template <int BN>
struct Shape {
  static constexpr int kPromoWarps = BN >= 256 ? 8 : 4;
  static constexpr int kThreads = 128 + kPromoWarps * 32;
  static constexpr int kCols = BN / (kPromoWarps / 4);  // accumulator columns of a promoting warp
  static constexpr int kChunk = kCols < 32 ? kCols : 32;
  static constexpr int kStageBytes = (kLanes + BN) * kStepBytes;
  static constexpr int kStages = BN >= 256 ? 4 : (BN >= 128 ? 6 : 8);
  static constexpr uint32_t kTmemCols = 2 * BN;  // two accumulators: 32 .. 512 columns
};

// tile table of the calls by expert: prefix[E + 1] (tiles or blocks before each expert), then
// start[E + 1] (its first row) -- both int32, E <= 1024
constexpr int kMaxExperts = 1024;

template <int BN>
constexpr int smem_bytes(bool by_expert) {
  using S = Shape<BN>;
  return 1024 + S::kStages * S::kStageBytes + S::kPromoWarps * 2 * S::kCols * 4 +
         (2 * S::kStages + 5) * 8 + 16 + (by_expert ? 2 * (kMaxExperts + 1) * 4 : 0);
}

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

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
// Instruction descriptor, kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), A and B E4M3 (bits 7-9
// and 10-12 = 0), both K-major, N >> 3 at bits 17-22, M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// N consecutive fp32 columns of this thread's tensor-memory lane (issue and wait in one statement,
// so that no use of the values moves in between)
__device__ __forceinline__ void load_columns(uint32_t taddr, float (&y)[32]) { tmem_ld32(taddr, y); }
__device__ __forceinline__ void load_columns(uint32_t taddr, float (&y)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(r[i]);
}

// (a0, a1) += (v0, v1) * (m0, m1), one packed fp32 FMA
__device__ __forceinline__ void fma2(float& a0, float& a1, float v0, float v1, float m0, float m1) {
  asm("{\n\t.reg .b64 a, v, m;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "mov.b64 m, {%4, %5};\n\tfma.rn.f32x2 a, v, m, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(v0), "f"(v1), "f"(m0), "f"(m1));
}
__device__ __forceinline__ void mul2v(float& v0, float& v1, float m0, float m1) {
  asm("{\n\t.reg .b64 v, m;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 m, {%2, %3};\n\t"
      "mul.rn.f32x2 v, v, m;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(v0), "+f"(v1)
      : "f"(m0), "f"(m1));
}

// Scale forms of an operand and orientation of the output.
template <int BN_, int MODE_, bool SWAP_, bool P_ROWS_, bool Q_ROWS_, bool F32_>
struct Config {
  static constexpr int BN = BN_, MODE = MODE_;
  static constexpr bool kSwap = SWAP_;    // P is B (weights), C written [column][lane]
  static constexpr bool kPRows = P_ROWS_, kQRows = Q_ROWS_;
  static constexpr bool kF32 = F32_;
};

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
      r.p_row = (int)(e * a.p_rows) + p * kLanes;
      r.p_valid = (int)min((int64_t)kLanes, a.p_rows - (int64_t)p * kLanes);
      r.q_row = row;
      r.q_valid = min(C::BN, left);
      r.p_scale = e * a.p_estride + (int64_t)p * a.p_pitch;
      r.q_scale = row;
      r.c = (int64_t)row * a.ldc + p * kLanes;
    } else {
      q = w;
      r.p_row = row;
      r.p_valid = min(kLanes, left);
      r.q_row = (int)(e * a.q_rows) + q * C::BN;
      r.q_valid = (int)min((int64_t)C::BN, a.q_rows - (int64_t)q * C::BN);
      r.p_scale = row;
      r.q_scale = e * a.q_estride + (int64_t)q * (C::BN / kB128) * a.q_pitch;
      r.c = (int64_t)row * a.ldc + (int64_t)q * C::BN;
    }
    r.k0 = r.kb0 = 0;
    r.nk = a.nk;
    return r;
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
  r.p_row = p * kLanes;
  r.q_row = q * C::BN;
  r.p_valid = (int)min((int64_t)kLanes, a.p_rows - r.p_row);
  r.q_valid = (int)min((int64_t)C::BN, a.q_rows - r.q_row);
  r.p_scale = C::kPRows ? r.kb0 * a.p_pitch + r.p_row : (int64_t)p * a.p_pitch + r.kb0;
  r.q_scale = C::kQRows ? r.kb0 * a.q_pitch + r.q_row
                        : (int64_t)q * (C::BN / kB128) * a.q_pitch + r.kb0;
  r.c = e * a.c_estride + (C::kSwap ? (int64_t)r.q_row * a.ldc + r.p_row
                                    : (int64_t)r.p_row * a.ldc + r.q_row);
  return r;
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
  float* cols;      // promoting warps: two buffers of kCols column scales each
  uint64_t* full;
  uint64_t* empty;
  uint64_t* acc_full;   // [2]
  uint64_t* acc_empty;  // [2]
  uint64_t* done;
  uint32_t* tmem_slot;
  int* prefix;
  int* start;
};

template <typename C>
__device__ __forceinline__ void produce(const CUtensorMap& pmap, const CUtensorMap& qmap,
                                        const KernelArgs& a, const Smem& s, int tiles) {
  using S = Shape<C::BN>;
  bool failed = false;
  int it = 0;
  for (int t = blockIdx.x; t < tiles && !failed; t += gridDim.x) {
    const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
    for (int kb = 0; kb < tile.nk; ++kb, ++it) {
      const int st = it % S::kStages;
      if (it >= S::kStages) {
        mbar_wait(smem_u32(s.empty + st), ((it / S::kStages) & 1) ^ 1, &failed, a.wait_limit_ns,
                  a.err);
        if (failed) break;
      }
      const uint32_t bar = smem_u32(s.full + st), dst = smem_u32(s.ring + st * S::kStageBytes);
      mbar_arrive_expect_tx(bar, S::kStageBytes);
      tma_load_box(dst, &pmap, tile.k0 + kb * kStepBytes, tile.p_row, bar);
      tma_load_box(dst + kLanes * kStepBytes, &qmap, tile.k0 + kb * kStepBytes, tile.q_row, bar);
    }
  }
  // loads in flight land before the CTA's shared memory goes away
  bool drain_failed = false;
  for (int i = it > S::kStages ? it - S::kStages : 0; i < it; ++i) {
    mbar_wait(smem_u32(s.full + i % S::kStages), (i / S::kStages) & 1, &drain_failed, kWaitNs, a.err);
  }
}

template <typename C>
__device__ __forceinline__ void multiply(const KernelArgs& a, const Smem& s, int tiles,
                                         uint32_t tmem) {
  using S = Shape<C::BN>;
  constexpr uint32_t idesc = idesc_e4m3_f32(kLanes, C::BN);
  bool failed = false;
  int it = 0;
  for (int t = blockIdx.x; t < tiles && !failed; t += gridDim.x) {
    const int nk = get_tile<C>(a, t, s.prefix, s.start).nk;
    for (int kb = 0; kb < nk; ++kb, ++it) {
      const int st = it % S::kStages, buf = it & 1;
      if (it >= 2) {
        mbar_wait(smem_u32(s.acc_empty + buf), ((it >> 1) & 1) ^ 1, &failed, a.wait_limit_ns, a.err);
      }
      mbar_wait(smem_u32(s.full + st), (it / S::kStages) & 1, &failed, a.wait_limit_ns, a.err);
      if (failed) break;
      tc_fence_after();
      const uint32_t p0 = smem_u32(s.ring + st * S::kStageBytes), q0 = p0 + kLanes * kStepBytes;
#pragma unroll
      for (int k = 0; k < kStepBytes / 32; ++k) {
        mma_e4m3(tmem + buf * C::BN, desc_sw128(p0 + 32 * k), desc_sw128(q0 + 32 * k), idesc,
                 k > 0 ? 1u : 0u);
      }
      mma_commit(smem_u32(s.empty + st));
      mma_commit(smem_u32(s.acc_full + buf));
    }
  }
  mma_commit(smem_u32(s.done));  // every MMA issued completes before the tensor memory is freed
  bool drain_failed = false;
  mbar_wait(smem_u32(s.done), 0, &drain_failed, kWaitNs, a.err);
}

// The promoting warps: warp w holds lanes 32 (w % 4) .. and columns kCols (w / 4) .. of the tile in
// registers, adds each step's accumulator times the step's scales, and writes the tile.
template <typename C>
__device__ __forceinline__ void promote(const KernelArgs& a, const Smem& s, int tiles,
                                        uint32_t tmem, int pw) {
  using S = Shape<C::BN>;
  constexpr int kCols = S::kCols, kChunk = S::kChunk;
  const int lane = threadIdx.x & 31;
  const int row = (pw & 3) * 32 + lane, col0 = (pw >> 2) * kCols;
  float* mine = s.cols + pw * 2 * kCols;
  const uint32_t tbase = tmem + ((uint32_t)((pw & 3) * 32) << 16) + col0;
  bool failed = false;
  int it = 0;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const Tile tile = get_tile<C>(a, t, s.prefix, s.start);
    const bool live = row < tile.p_valid;
    float acc[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
    // scales of step kb: the lane's (or its block's) and, rows form, the columns'
    const float* ps = a.p_scales + tile.p_scale + (C::kPRows ? row : 0);
    const int qblock = col0 / kB128;
    const bool qlive = qblock * kB128 < tile.q_valid;
    const float* qs = a.q_scales + tile.q_scale + (C::kQRows ? col0 : qblock * a.q_pitch);
    auto lane_scale = [&](int kb) -> float {
      if (kb >= tile.nk) return 0.0f;
      float v = live ? load_f32(ps + (C::kPRows ? kb * a.p_pitch : (int64_t)kb)) : 0.0f;
      if (!C::kQRows) v *= qlive ? load_f32(qs + kb) : 0.0f;
      return v;
    };
    constexpr int kPer = (kCols + 31) / 32;
    float next_cols[kPer];
    auto col_scales = [&](int kb) {
      if constexpr (C::kQRows) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int c = i * 32 + lane;
          next_cols[i] = kb < tile.nk && c < kCols && col0 + c < tile.q_valid
                             ? load_f32(qs + kb * a.q_pitch + c)
                             : 0.0f;
        }
      }
    };
    float next_lane = lane_scale(0);
    col_scales(0);
    for (int kb = 0; kb < tile.nk; ++kb, ++it) {
      const int buf = it & 1;
      const float m = next_lane;
      float* cs = mine + buf * kCols;
      if (C::kQRows) {
        __syncwarp();  // the buffer's readers of two steps ago are done
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (i * 32 + lane < kCols) cs[i * 32 + lane] = next_cols[i];
        }
        __syncwarp();
      }
      next_lane = lane_scale(kb + 1);
      col_scales(kb + 1);
      mbar_wait(smem_u32(s.acc_full + buf), (it >> 1) & 1, &failed, a.wait_limit_ns, a.err);
      failed = __any_sync(0xFFFFFFFFu, failed);
      if (failed) break;
      tc_fence_after();
#pragma unroll
      for (int ch = 0; ch < kCols / kChunk; ++ch) {
        float v[kChunk];
        load_columns(tbase + buf * C::BN + ch * kChunk, v);
        if (ch == kCols / kChunk - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(s.acc_empty + buf));
        }
#pragma unroll
        for (int i = 0; i < kChunk; i += 4) {
          if (C::kQRows) {
            const float4 q = *reinterpret_cast<const float4*>(cs + ch * kChunk + i);
            mul2v(v[i], v[i + 1], q.x, q.y);
            mul2v(v[i + 2], v[i + 3], q.z, q.w);
          }
          float* d = acc + ch * kChunk + i;
          fma2(d[0], d[1], v[i], v[i + 1], m, m);
          fma2(d[2], d[3], v[i + 2], v[i + 3], m, m);
        }
      }
    }
    if (failed) return;
    if (!live) continue;
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
__global__ void __launch_bounds__(Shape<C::BN>::kThreads, 1)
    b128_gemm_kernel(const __grid_constant__ CUtensorMap pmap,
                     const __grid_constant__ CUtensorMap qmap, KernelArgs a) {
  using S = Shape<C::BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Smem s;
  s.ring = smem;
  s.cols = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes);
  s.full = reinterpret_cast<uint64_t*>(s.cols + S::kPromoWarps * 2 * S::kCols);
  s.empty = s.full + S::kStages;
  s.acc_full = s.empty + S::kStages;
  s.acc_empty = s.acc_full + 2;
  s.done = s.acc_empty + 2;
  s.tmem_slot = reinterpret_cast<uint32_t*>(s.done + 1);
  s.prefix = reinterpret_cast<int*>(s.tmem_slot + 2);
  s.start = s.prefix + kMaxExperts + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(smem_u32(s.full + i), 1);
      mbar_init(smem_u32(s.empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(s.acc_full + i), 1);
      mbar_init(smem_u32(s.acc_empty + i), S::kPromoWarps);
    }
    mbar_init(smem_u32(s.done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  if (warp == 1) {
    tmem_alloc(smem_u32(s.tmem_slot), S::kTmemCols);
    tmem_relinquish();
  }
  if (C::MODE == kB128Grouped) build_table(a, a.tok_tile, INT32_MAX, s.prefix, s.start);
  if (C::MODE == kB128Wgrad) build_table(a, kB128, (int)a.blocks_total, s.prefix, s.start);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s.tmem_slot;
  const int tiles = tile_count<C>(a, s.prefix);
  if (warp == 0) {
    if (lane == 0) produce<C>(pmap, qmap, a, s, tiles);
  } else if (warp == 1) {
    if (lane == 0) multiply<C>(a, s, tiles, tmem);
  } else if (warp >= 4) {
    promote<C>(a, s, tiles, tmem, warp - 4);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, S::kTmemCols);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename C>
cudaError_t launch_config(const B128GemmArgs& g, cudaStream_t stream) {
  using S = Shape<C::BN>;
  auto* kernel = &b128_gemm_kernel<C>;
  constexpr int smem = smem_bytes<C::BN>(C::MODE != kB128Dense);
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
  a.p_tiles = (int)ceil_div(a.p_rows, kLanes);
  a.q_tiles = (int)ceil_div(a.q_rows, C::BN);
  a.tok_tile = C::kSwap ? C::BN : kLanes;
  CUtensorMap pmap, qmap;
  const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
  cudaError_t err = make_tensor_map_2d(&pmap, C::kSwap ? g.b_codes : g.a_codes,
                                       C::kSwap ? bmap : arows, g.K, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1,
                                       kStepBytes, kLanes, swz);
  if (err != cudaSuccess) return err;
  err = make_tensor_map_2d(&qmap, C::kSwap ? g.a_codes : g.b_codes, C::kSwap ? arows : bmap, g.K,
                           CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kStepBytes, C::BN, swz);
  if (err != cudaSuccess) return err;
  int64_t tiles = (int64_t)a.p_tiles * a.q_tiles;  // at most, by expert
  if (C::MODE == kB128Wgrad) tiles *= g.E;
  if (grouped) {
    tiles = (g.M / a.tok_tile + (g.M < g.E ? g.M : g.E)) * (C::kSwap ? a.p_tiles : a.q_tiles);
  }
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(kernel, dim3((unsigned)(tiles < slots ? tiles : slots)), dim3(S::kThreads), smem,
                    stream, pmap, qmap, a);
}

}  // namespace

cudaError_t launch_b128_gemm(int mode, const B128GemmArgs& g, cudaStream_t stream) {
  if (mode == kB128Wgrad) {
    return g.out_f32 ? launch_config<Config<256, kB128Wgrad, false, true, true, true>>(g, stream)
                     : launch_config<Config<256, kB128Wgrad, false, true, true, false>>(g, stream);
  }
  if (mode == kB128Grouped) {
    return g.out_f32 ? launch_config<Config<256, kB128Grouped, false, true, false, true>>(g, stream)
                     : launch_config<Config<256, kB128Grouped, false, true, false, false>>(g, stream);
  }
  if (g.b_rows) {
    return g.out_f32 ? launch_config<Config<256, kB128Dense, false, true, true, true>>(g, stream)
                     : launch_config<Config<256, kB128Dense, false, true, true, false>>(g, stream);
  }
  return g.out_f32 ? launch_config<Config<256, kB128Dense, false, true, false, true>>(g, stream)
                   : launch_config<Config<256, kB128Dense, false, true, false, false>>(g, stream);
}

}  // namespace mxq
