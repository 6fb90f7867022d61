// mx_b128_quant.cu -- E4M3 operands with one fp32 scale per block of 128 along the contraction.
//
// For a block with abs-max A (1 x 128 of a row, 128 x 1 of a column, or a 128 x 128 square):
//   a = max(A, 2^-100);  r = 448 / a;  scale = a / 448;  code_i = E4M3(x_i * r),
// every step one fp32 operation rounded to nearest even, the code saturating at 448 and keeping
// the sign of zero. A block holding a NaN or an infinity gets scale NaN and codes 0x7F.
// The floor 2^-100 keeps r finite for zero and tiny blocks. x * r (one fp32 rounding before the
// rounding to E4M3) is the definition, not x / scale: the division would cost ten times the
// multiplication and differ only next to a rounding midpoint.
//
// All three kernels are bound by memory: 2 bytes read and 1 written per element (2 written when
// the square kernel writes both orders), scales 1/32 of a byte. x[8192, 8192], where a plain copy of
// as many bytes takes 30 us: rows 30 us (6.7 TB/s), columns 32 (6.3), squares 30 (6.7), squares in both
// orders 42 (6.4). The transposed squares of a matrix whose rows are no multiple of 16 leave byte by byte:
// 8200 rows 210 us.
#include "mx_device.cuh"
#include "mx_expert.h"
#include "mx_launch.h"

namespace mxq {

namespace {

struct Factors {
  float r, scale;
};

__device__ __forceinline__ Factors block_factors_b128(uint32_t amax_bits) {
  Factors f;
  const float a = fmaxf(__uint_as_float(amax_bits), kB128AmaxFloor);
  f.r = __fdiv_rn(448.0f, a);
  f.scale = __fdiv_rn(a, 448.0f);
  if (amax_bits >= 0x7F800000u) f.r = f.scale = __uint_as_float(0x7FC00000u);
  return f;
}

// Sign-free bf16x2 abs-max accumulation; the two halves are joined by amax_bits. NaN propagates:
// the patterns are compared as integers, and those of NaN lie above that of infinity.
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t amax_join(uint32_t m) {  // -> fp32 bits
  return max(m & 0xFFFFu, m >> 16) << 16;
}

// four values (bf16x2 words w0, w1: lower index in the low half) times r -> four code bytes
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float r) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(d)
      : "f"(__fmul_rn(bf16_lo(w0), r)), "f"(__fmul_rn(bf16_hi(w0), r)),
        "f"(__fmul_rn(bf16_lo(w1), r)), "f"(__fmul_rn(bf16_hi(w1), r)));
  return d;
}

// two values (separate fp32) -> two code bytes
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(d) : "f"(lo), "f"(hi));
  return d;
}

// Codes are written once and not read again here: evict-first.
__device__ __forceinline__ void store16B(void* p, const uint32_t* r) {
  asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

constexpr int kRowsCols = 512;  // columns of a warp's tile: 4 blocks of 128, 8 lanes each

// 1 x 128 blocks. A warp takes RW rows of 512 columns: lane l holds 16 elements (32 bytes) of
// block l / 8 of every row, so the RW loads of a thread are in flight together, eight lanes
// reduce a block's abs-max in three shuffles, and the RW scales of a block, which are adjacent in
// the [K / 128, R] layout, leave as one segment.
template <int RW, bool GATHER>
__global__ void __launch_bounds__(256) b128_rows_kernel(B128QuantArgs a, int64_t col_tiles,
                                                        int64_t tiles) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, sub = lane & 7, blk = lane >> 3;
  const int64_t tile = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (tile >= tiles) return;
  const int64_t r0 = tile / col_tiles * RW;
  const int64_t col = tile % col_tiles * kRowsCols + blk * kB128 + sub * 16;
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  int32_t src[RW];  // gathered rows' sources (-1: zeros), asked for together
  if constexpr (GATHER) {
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      src[i] = r0 + i < a.R && col < a.K ? load_s32(a.index + r0 + i) : -1;
    }
  }
  uint32_t w[RW][8];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int64_t row = GATHER ? src[i] : r0 + i;
    if (GATHER ? row >= 0 && row < a.M : row < a.R && col < a.K) {
      load32B(x + row * a.K + col, w[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = 0u;
    }
  }
  float mine = 0.0f;  // lane sub keeps the scale of row sub
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = amax2(m, w[i][j]);
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
    const Factors f = block_factors_b128(amax_join(m));
    if (sub == i) mine = f.scale;
    if (r0 + i < a.R && col < a.K) {
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = codes4(w[i][2 * j], w[i][2 * j + 1], f.r);
      store16B(a.codes + (r0 + i) * a.K + col, c);
    }
  }
  const int64_t kb = tile % col_tiles * (kRowsCols / kB128) + blk;
  if (sub < RW && r0 + sub < a.R && kb * kB128 < a.K) a.scales[kb * a.R + r0 + sub] = mine;
}

// 128 x 128 tiles, 256 threads: thread (rg, cg) holds rows 8 rg .. and columns 8 cg .. (16-byte
// loads, 16 lanes per row). The transposed codes (eight rows of one column are eight bytes of a
// thread) pass through shared memory, 8-byte chunk rg of column c at chunk rg ^ (c / 8) so that
// neither side meets a bank twice, and leave as full 128-byte lines.
constexpr int kTileThreads = 256;

__device__ __forceinline__ void load_tile(const uint16_t* x, int64_t K, int64_t row0, int64_t row_end,
                                          int64_t col, uint32_t (&w)[8][4]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (row0 + i < row_end && col < K) {
      load16B(x + (row0 + i) * K + col, w[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i][j] = 0u;
    }
  }
}

__device__ __forceinline__ void copy16B_async(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(to)),
               "l"(from)
               : "memory");
}

__device__ __forceinline__ void stage_transposed(uint8_t* sm, int rg, int cg, int j,
                                                 const uint32_t (&v)[2]) {
  *reinterpret_cast<uint2*>(sm + (cg * 8 + j) * 128 + ((rg ^ cg) << 3)) = make_uint2(v[0], v[1]);
}

// Writes the staged tile: column c of the tile to dst + c * pitch, `valid` bytes of each.
__device__ __forceinline__ void store_transposed(const uint8_t* sm, uint8_t* dst, int64_t pitch,
                                                 int valid, int cols) {
  const int q = threadIdx.x & 7;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int c = p * 32 + (threadIdx.x >> 3);
    const int s = c >> 3;
    uint4 v = *reinterpret_cast<const uint4*>(sm + c * 128 + ((q ^ (s >> 1)) << 4));
    if (s & 1) v = make_uint4(v.z, v.w, v.x, v.y);
    if (c >= cols) continue;
    uint8_t* o = dst + c * pitch + q * 16;
    if ((pitch & 15) == 0) {
      if (q * 16 < valid) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        store16B(o, u);
      }
    } else {  // rows that are not whole 16-byte pieces: byte by byte
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      for (int b = 0; b < 16 && q * 16 + b < valid; ++b) o[b] = (uint8_t)(u[b >> 2] >> (8 * (b & 3)));
    }
  }
}

// Expert owning 128-row block b of a buffer in which every expert's rows start a new block, from the
// (clamped) offsets in shared memory: source rows [*row0, *row_end) of the block, false when b lies
// past the last expert. One warp.
__device__ __forceinline__ bool find_block(const int* offsets, int E, int64_t b, int* row0,
                                           int* row_end) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const int lo = e < E ? offsets[e] : 0, hi = e < E ? max(offsets[e + 1], lo) : 0;
    const int n = (hi - lo + kB128 - 1) / kB128;
    int sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += up;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + sum > b);
    if (past) {
      const int who = __ffs(past) - 1;
      const int first = before + sum - n;
      *row0 = __shfl_sync(0xFFFFFFFFu, lo + ((int)b - first) * kB128, who);
      *row_end = __shfl_sync(0xFFFFFFFFu, hi, who);
      return true;
    }
    before += __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
  return false;
}

// Blocks of 128 rows of the buffer above that belong to experts. One warp.
__device__ __forceinline__ int64_t count_blocks(const int* offsets, int E) {
  int n = 0;
  for (int e = threadIdx.x & 31; e < E; e += 32) {
    n += (max(offsets[e + 1] - offsets[e], 0) + kB128 - 1) / kB128;
  }
  return (int64_t)__reduce_add_sync(0xFFFFFFFFu, (unsigned)n);
}

// 128 x 1 blocks, written transposed (codes [K, 128 * blocks], scales [blocks, K]): the operand
// of a product that contracts over the rows of x. The transposition goes through shared memory, a tile
// of 128 rows being one block. A CTA walks a run of tiles along x's rows, and while it reduces, converts
// and writes one, the next is on its way into shared memory, every thread's pieces to places of its
// own: four CTAs keep 128 KB of an SM's loads in flight (x[8192, 8192] 32 us; a tile's own loads in
// registers, nothing on its way meanwhile, 36.6).
struct ColsShared {
  uint4 next[8][kTileThreads];  // the tile on its way
  uint8_t out[128 * 128];
  uint32_t part[8][64];
  float factor[128];
  int64_t blocks;
  int offsets[1024 + 1];
};
template <bool GATHER>
__global__ void __launch_bounds__(kTileThreads, 4) b128_cols_kernel(B128QuantArgs a) {
  extern __shared__ __align__(128) uint8_t cols_shared[];
  ColsShared& s = *reinterpret_cast<ColsShared*>(cols_shared);
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4, warp = tid >> 5;
  int64_t blocks = a.blocks;
  if (a.offsets) {
    for (int e = tid; e <= a.E; e += kTileThreads) {  // one trip to memory
      s.offsets[e] = (int)min(max(load_s64(a.offsets + e), (int64_t)0), a.R);
    }
    __syncthreads();
    if (warp == 0) {
      const int64_t n = count_blocks(s.offsets, a.E);
      if (tid == 0) s.blocks = min(n, a.blocks);
    }
    __syncthreads();
    blocks = s.blocks;  // those past the last expert's are never read by the product
  }
  const int64_t cols = (a.K + kB128 - 1) / kB128, tiles = blocks * cols;
  const int64_t t0 = tiles * blockIdx.x / gridDim.x, t1 = tiles * (blockIdx.x + 1) / gridDim.x;
  if (t0 == t1) return;
  const int64_t pitch = a.blocks * kB128;
  int64_t b = t0 / cols, c = t0 - b * cols;
  int row0 = 0, row_end = 0;  // source rows of block b
  auto find = [&] {
    if (a.offsets) {
      find_block(s.offsets, a.E, b, &row0, &row_end);
    } else {
      row0 = (int)(b * kB128);
      row_end = (int)a.R;
    }
  };
  auto load = [&] {  // tile (b, c)
    const int64_t col = c * kB128 + cg * 8, first = (int64_t)row0 + rg * 8;
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
      int32_t src[4];  // gathered rows' sources (-1: zeros), asked for together
      if constexpr (GATHER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          src[i] = first + h + i < row_end && col < a.K ? load_s32(a.index + first + h + i) : -1;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = GATHER ? src[i] : first + h + i;
        if (GATHER ? row >= 0 && row < a.M : row < row_end && col < a.K) {
          copy16B_async(&s.next[h + i][tid], static_cast<const uint16_t*>(a.x) + row * a.K + col);
        } else {
          s.next[h + i][tid] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  find();
  load();
  for (int64_t t = t0; t < t1; ++t) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // a thread reads only what it copied
    uint32_t w[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 v = s.next[i][tid];
      w[i][0] = v.x;
      w[i][1] = v.y;
      w[i][2] = v.z;
      w[i][3] = v.w;
    }
    uint32_t m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) m[j] = amax2(m[j], w[i][j]);
      m[j] = __vmaxu2(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 16));
    }
    if ((tid & 16) == 0) {  // eight columns' halves, still in pairs
      *reinterpret_cast<uint4*>(&s.part[warp][cg * 4]) = make_uint4(m[0], m[1], m[2], m[3]);
    }
    __syncthreads();
    const int64_t at = b, c0 = c * kB128;
    if (t + 1 < t1) {
      if (++c == cols) {
        c = 0;
        ++b;
        find();
      }
      load();
    }
    if (tid < 128) {
      uint32_t top = s.part[0][tid >> 1];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = __vmaxu2(top, s.part[i][tid >> 1]);
      const Factors f = block_factors_b128((tid & 1) ? top & 0xFFFF0000u : top << 16);
      s.factor[tid] = f.r;
      if (c0 + tid < a.K) a.scales[at * a.K + c0 + tid] = f.scale;
    }
    __syncthreads();
    float r8[8];
    *reinterpret_cast<float4*>(r8) = *reinterpret_cast<const float4*>(s.factor + cg * 8);
    *reinterpret_cast<float4*>(r8 + 4) = *reinterpret_cast<const float4*>(s.factor + cg * 8 + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float r = r8[j];
      uint32_t v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = w[4 * h + i][j >> 1];
          f[i] = __fmul_rn((j & 1) ? bf16_hi(u) : bf16_lo(u), r);
        }
        v[h] = codes2(f[0], f[1]) | codes2(f[2], f[3]) << 16;
      }
      stage_transposed(s.out, rg, cg, j, v);
    }
    __syncthreads();
    // (the next tile's first barriers keep its codes from overtaking these reads)
    store_transposed(s.out, a.codes + c0 * pitch + at * kB128, pitch, kB128,
                     (int)min((int64_t)kB128, a.K - c0));
  }
}

// 128 x 128 squares of every matrix of a batch (blockIdx.z), in the order of x and, when codes_t
// is given, transposed as well.
__global__ void __launch_bounds__(kTileThreads) b128_blocks_kernel(B128QuantArgs a) {
  __shared__ __align__(16) uint8_t sm[128 * 128];
  __shared__ uint32_t part[8];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  const int64_t row_blocks = (a.M + kB128 - 1) / kB128, col_blocks = (a.K + kB128 - 1) / kB128;
  const int64_t cb = blockIdx.x % col_blocks, rb = blockIdx.x / col_blocks, z = blockIdx.y;
  const int64_t r0 = rb * kB128, c0 = cb * kB128;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + z * a.M * a.K;
  uint32_t w[8][4];
  load_tile(x, a.K, r0 + rg * 8, a.M, c0 + cg * 8, w);
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) m = amax2(m, w[i][j]);
  }
  m = __reduce_max_sync(0xFFFFFFFFu, amax_join(m));
  if ((tid & 31) == 0) part[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, part[i]);
  const Factors f = block_factors_b128(m);
  if (tid == 0) {
    a.scales[(z * row_blocks + rb) * col_blocks + cb] = f.scale;
    if (a.scales_t) a.scales_t[(z * col_blocks + cb) * row_blocks + rb] = f.scale;
  }
  uint32_t c[8][2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i][0] = codes4(w[i][0], w[i][1], f.r);
    c[i][1] = codes4(w[i][2], w[i][3], f.r);
    const int64_t row = r0 + rg * 8 + i, col = c0 + cg * 8;
    if (row < a.M && col < a.K) {
      *reinterpret_cast<uint2*>(a.codes + (z * a.M + row) * a.K + col) = make_uint2(c[i][0], c[i][1]);
    }
  }
  if (!a.codes_t) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {  // byte j of eight rows
    uint32_t v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo = __byte_perm(c[4 * h][j >> 2], c[4 * h + 1][j >> 2], (j & 3) | (4 + (j & 3)) << 4);
      const uint32_t hi = __byte_perm(c[4 * h + 2][j >> 2], c[4 * h + 3][j >> 2], (j & 3) | (4 + (j & 3)) << 4);
      v[h] = __byte_perm(lo, hi, 0x5410);
    }
    stage_transposed(sm, rg, cg, j, v);
  }
  __syncthreads();
  store_transposed(sm, a.codes_t + (z * a.K + c0) * a.M + r0, a.M,
                   (int)min((int64_t)kB128, a.M - r0), (int)min((int64_t)kB128, a.K - c0));
}

}  // namespace

template <bool GATHER>
static cudaError_t rows_launch(const B128QuantArgs& a, cudaStream_t stream) {
  const int64_t col_tiles = (a.K + kRowsCols - 1) / kRowsCols;
  // Four rows per warp once that leaves every SM work (x[8192, 8192]: 30.9 us; eight rows, whose 91
  // registers halve the resident warps, 36.1); one row per warp for small calls, where the latency
  // of a warp's own chain counts.
  constexpr int kRows = 4;
  if (a.R * col_tiles >= kRows * 8 * 152) {
    const int64_t tiles = (a.R + kRows - 1) / kRows * col_tiles;
    return launch_pdl(&b128_rows_kernel<kRows, GATHER>, dim3((unsigned)((tiles + 7) / 8)), dim3(256), 0,
                      stream, a, col_tiles, tiles);
  }
  const int64_t tiles = a.R * col_tiles;
  return launch_pdl(&b128_rows_kernel<1, GATHER>, dim3((unsigned)((tiles + 3) / 4)), dim3(128), 0,
                    stream, a, col_tiles, tiles);
}

cudaError_t launch_b128_rows(const B128QuantArgs& a, cudaStream_t stream) {
  return a.index ? rows_launch<true>(a, stream) : rows_launch<false>(a, stream);
}

template <bool GATHER>
static cudaError_t cols_launch(const B128QuantArgs& a, cudaStream_t stream) {
  const int64_t tiles = a.blocks * ((a.K + kB128 - 1) / kB128);  // by expert: at most
  const int64_t slots = resident_ctas(reinterpret_cast<const void*>(&b128_cols_kernel<GATHER>), kTileThreads,
                                      sizeof(ColsShared), 0);
  if (slots <= 0) return cudaErrorInvalidConfiguration;
  return launch_pdl(&b128_cols_kernel<GATHER>, dim3((unsigned)(tiles < slots ? tiles : slots)),
                    dim3(kTileThreads), sizeof(ColsShared), stream, a);
}

cudaError_t launch_b128_cols(const B128QuantArgs& a, cudaStream_t stream) {
  return a.index ? cols_launch<true>(a, stream) : cols_launch<false>(a, stream);
}

cudaError_t launch_b128_blocks(const B128QuantArgs& a, cudaStream_t stream) {
  const int64_t tiles = (a.M + kB128 - 1) / kB128 * ((a.K + kB128 - 1) / kB128);
  return launch_pdl(&b128_blocks_kernel, dim3((unsigned)tiles, (unsigned)a.batch),
                    dim3(kTileThreads), 0, stream, a);
}

}  // namespace mxq
