// dense_gemm.cu -- the dense products beside the experts on the tcgen05 tensor
// cores: moe_linear, moe_gated_linear and their gradients.
//
//   D[m, n] = sum_k A(m, k) B(n, k)      bf16 or fp16 in, fp32 sums
// with A and B each stored along k (K-major) or along their rows (M/N-major),
// so that no gradient needs a transposed copy:
//   forward   a   = x W^T      A = x [n, C],    B = W [R, C]      both K-major
//   d_x       dx  = d_a W      A = d_a [n, R],  B = W [R, C]      B N-major
//   d_w       dw  = d_a^T x    A = d_a [n, R],  B = x [n, C]      both M/N-major
// (the two gradients in one launch, which also adds up a bias's gradient)
// and an epilogue on the sums while they are in registers (dense.cuh): bias,
// activation and residual; the gated product; the gradients of either.
//
// A persistent kernel, one CTA pair (cta_group::2) per two SMs: tiles of 256
// rows (128 per CTA) x tn columns (tn / 2 of B's rows per CTA), K steps of 128
// bytes through a ring of TMA-fed stages, two accumulators of tn TMEM columns,
// so that the epilogue of one tile runs under the products of the next.
//   warp 0      TMA producer (each CTA its own halves; bytes counted on the
//               leader's barrier)
//   warp 1      TMEM allocation; the leader's issues the MMAs
//   warps 2..   epilogue, two to four per TMEM lane quarter, column chunks in turn
// MXFP8 operands (moe_linear_mx8, moe_gated_linear_mx8) take the same kernel:
// E4M3 codes with one power of two per 32 of them, which the tensor core
// applies itself (kind::mxf8f6f4, block_scale), so nothing is converted and
// the rate is twice that of bf16. A stage then holds 128 codes of each row and
// the rows' four scales, which tcgen05.cp spreads into TMEM beside the
// accumulators (224 columns each, so that both fit). The scales come row by
// row with C / 32 bytes at no alignment: a small kernel lays them out in the
// blocks that the copy wants first, x and w together.
// Where the tiles are fewer than the pairs of SMs can take, the K range is
// split: parts write fp32 sums and a second kernel adds them in order and
// applies the epilogue. No atomics: the bits depend on the inputs and sizes.
// Every mbarrier wait is bounded.
#include "dense.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kRowsCta = 128;                    // A rows of a CTA's half tile
constexpr int kStepBytes = 128;                  // K bytes of a stage
constexpr int kABytes = kRowsCta * kStepBytes;   // 16 KB
constexpr int kMaxTn = 256;
// Epilogue warps, two to four per TMEM lane quarter: with four a tile's
// epilogue has the latency of two column chunks; a group of 32 8-bit results
// takes 64 columns and twice the registers, rows off 16 bytes 128 registers
// (922 x 5281 x 280: 24.9 us with four, where they spill, 16.0 with three,
// 16.9 with two), an activation's gradient 115 (with four, 52 bytes of spills).
constexpr int epi_warps(int epi) {
  return epi == EPI_GATED_MX ? 8 : epi == EPI_COLUMNS || epi == EPI_DACT ? 12 : 16;
}
constexpr int gemm_threads(int epi) { return (2 + epi_warps(epi)) * 32; }
constexpr int kRingBytes = 220 * 1024;
constexpr int kMaxStages = 8;
constexpr int kNumBars = 2 * kMaxStages + 2 + 2 + 1;
constexpr int kGemmSmem = 1024 + kRingBytes + kNumBars * 8 + 16;
constexpr int kTmemCols = 512;
// MXFP8: stages, accumulator columns, and the scales of a stage: blocks of 512
// bytes (128 rows, 4 scales each; 4 TMEM columns), one of x and two of w.
constexpr int kMxStages = 5;
constexpr int kMxTn = 224;
constexpr int kScaleBlock = 512;
constexpr int kScaleBytes = 3 * kScaleBlock;
constexpr int kScaleCols = 12;
constexpr int kScaleOffset = kRingBytes - kMxStages * kScaleBytes;
static_assert(2 * kMxTn + kMxStages * kScaleCols <= kTmemCols, "TMEM columns");
static_assert(kMxStages * (kABytes + kMxTn / 2 * kStepBytes) <= kScaleOffset, "stages and scales");
static_assert(kScaleOffset % kScaleBlock == 0, "scale blocks");
constexpr int acc_cols(bool mx) { return mx ? kMxTn : kMaxTn; }
static_assert(kGemmSmem <= 227 * 1024, "shared memory per CTA");

// One product. Gradients come two at a time.
struct GemmProblem {
  DenseEpi e;
  int64_t part_stride;  // floats between the parts of a split sum
  int m_tiles, n_tiles, splits;
  int num_kb;           // K steps of the whole sum
  int tn, b_bytes;      // columns of a tile, B bytes per CTA and stage
  int tn_last, b_bytes_last, n_full;  // the last tile of a row of tiles, if narrower
  int a_k_major, partial;             // gradients: how A is stored; fp32 parts of a split sum
  int units;            // tiles x parts
  uint32_t idesc;
};

// Sums over the rows of part [rows, cols], for the epilogue warps to make while
// the first products run (a bias's gradient).
struct ColumnJoin {
  const float *part;
  void *out;  // null: none
  int rows, cols, half;
};

struct GemmArgs {
  GemmProblem p[2];
  ColumnJoin join;
  int stages, stage_bytes;
  int pairs;  // B rows come interleaved through a 3-D map
  uint32_t *status;
  unsigned long long timeout_ns;
};

// Tensor maps of a launch: A, B, B of narrow last tiles, scale blocks of A and
// of B; or A and B of two gradients.
enum { kMapA = 0, kMapB = 1, kMapBLast = 2, kMapSa = 3, kMapSb = 4, kMaps = 5 };
struct GemmMaps {
  CUtensorMap m[kMaps];
};

// Shared-memory descriptor of an operand stored along its rows (M/N-major),
// 128-byte swizzle: atoms of 64 rows x 8 k (a 128-byte line per k), 8-k groups
// 1024 bytes apart (SBO), atoms along the rows 8 KB apart (LBO; a stage holds
// 64 k of each).
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// 512 bytes (32 lines of 16: line l holds the scales of rows l, l + 32, l + 64
// and l + 96) to 4 TMEM columns of all lane quarters, in both CTAs of the pair
// from their own shared memory.
__device__ __forceinline__ void copy_scales_pair(uint32_t tmem, uint32_t saddr) {
  const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) |
                        ((uint64_t)1 << 46);
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
               : "memory");
}

__device__ __forceinline__ void st_shared_cluster(uint32_t cluster_addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

__device__ __forceinline__ void umma_mx8_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                              uint32_t sa, uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}

// Unit u: a tile of a product and its part of the sum. The narrow last tiles
// come behind all others, to fill what the last wave of whole tiles leaves.
struct Unit {
  int p, m, n, s, k_lo, k_hi, tn, b_bytes;
};
template <bool GRAD>
__device__ __forceinline__ Unit unit_of(int u, const GemmArgs &args) {
  Unit w;
  w.p = GRAD && u >= args.p[0].units ? 1 : 0;
  const GemmProblem &a = args.p[w.p];
  if (w.p) u -= args.p[0].units;
  const int tiles = a.m_tiles * a.n_tiles, full = a.m_tiles * a.n_full;
  w.s = u / tiles;
  const int t = u - w.s * tiles;
  if (t < full) {
    w.m = t / a.n_full;
    w.n = t - w.m * a.n_full;
    w.tn = a.tn;
    w.b_bytes = a.b_bytes;
  } else {
    w.m = t - full;
    w.n = a.n_full;
    w.tn = a.tn_last;
    w.b_bytes = a.b_bytes_last;
  }
  w.k_lo = (int)((int64_t)a.num_kb * w.s / a.splits);
  w.k_hi = (int)((int64_t)a.num_kb * (w.s + 1) / a.splits);
  return w;
}

// ---------------------------------------------- epilogue of the tile's warps --
// A warp reads 32 rows x 32 columns of sums from TMEM, a row per lane. Before
// the epilogue the four lanes of a group exchange them, so that a lane has 8
// columns of its group's 4 rows: v[8 k + i] is row 4 (lane / 4) + k, column 8
// (lane % 4) + i. Rows are then read and written 64 bytes side by side (128 of
// fp32) and not 16 per row: 4945 x 3632 x 1152 36 -> 31 us.
__device__ __forceinline__ void regroup(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 2; h > 0; h >>= 1)
#pragma unroll
    for (int p = 0; p < 4; ++p)
      if ((p & h) == 0)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float got =
              __shfl_xor_sync(0xffffffffu, lane & h ? v[8 * p + i] : v[8 * (p + h) + i], h);
          if (lane & h) v[8 * p + i] = got;
          else v[8 * (p + h) + i] = got;
        }
}

// What a lane's epilogue reads: fetched ahead, while the sums are still being
// made. The loads are volatile: plain ones were moved down to their use,
// behind the wait.
struct RowsAddend {
  uint4 q[4];  // of e.add, a row each (EPI_DGATED: 4 values, in x and y)
  uint4 bias;
};
template <int EPI>
__device__ __forceinline__ void fetch_rows(const DenseEpi &e, int64_t row0, int c, RowsAddend &a) {
  const int lane = threadIdx.x & 31, col = c + (lane & 3) * 8;
  const int64_t row = row0 + (lane >> 2) * 4;
  if (col >= e.cols) return;
  if constexpr (EPI == EPI_LINEAR || EPI == EPI_DACT) {
    if (e.bias) {
      const uint16_t *b = static_cast<const uint16_t *>(e.bias) + col;
      if (e.vec) {
        a.bias = load_now(reinterpret_cast<const uint4 *>(b));
      } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = (uint32_t)load_now(b + 2 * i) | (uint32_t)load_now(b + 2 * i + 1) << 16;
        a.bias = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (e.add) {
      const uint16_t *p = static_cast<const uint16_t *>(e.add) + row * e.cols + col;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (row + k < e.rows) a.q[k] = load_now(reinterpret_cast<const uint4 *>(p + (int64_t)k * e.cols));
    }
  } else if constexpr (EPI == EPI_DGATED) {
    const int I = e.cols / 2;
    const uint16_t *p = static_cast<const uint16_t *>(e.add) + row * I + col / 2;
#pragma unroll
    for (int k = 0; k < 4; ++k, p += I)
      if (row + k < e.rows) {
        if (e.vec) {
          const uint2 w = load_now(reinterpret_cast<const uint2 *>(p));
          a.q[k].x = w.x;
          a.q[k].y = w.y;
        } else {
          a.q[k].x = (uint32_t)load_now(p) | (uint32_t)load_now(p + 1) << 16;
          a.q[k].y = (uint32_t)load_now(p + 2) | (uint32_t)load_now(p + 3) << 16;
        }
      }
  }
}

__device__ __forceinline__ void store4(uint16_t *p, const float (&f)[4], int half) {
  const float g[8] = {f[0], f[1], f[2], f[3], 0.f, 0.f, 0.f, 0.f};
  const uint4 q = pack8(g, half);
  *reinterpret_cast<uint2 *>(p) = make_uint2(q.x, q.y);
}

// The regrouped sums of columns [c, c + 32) of rows [row0, row0 + 32), row0 <
// e.rows. Every lane of the warp comes here.
template <int EPI>
__device__ __forceinline__ void rows_epilogue(const DenseEpi &e, int64_t row0, int c,
                                              float (&v)[32], const RowsAddend &a) {
  const int lane = threadIdx.x & 31, col = c + (lane & 3) * 8;
  const int64_t row = row0 + (lane >> 2) * 4;
  const int rows = col >= e.cols ? 0 : e.rows - row >= 4 ? 4 : e.rows > row ? (int)(e.rows - row) : 0;
  const int64_t at = row * e.cols + col;
  if constexpr (EPI == EPI_LINEAR || EPI == EPI_DACT) {
    if (e.bias) {
      float b[8];
      unpack8(a.bias, e.half, b);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += b[i & 7];
    }
  }
  uint16_t *out = static_cast<uint16_t *>(e.out) + at;
  if constexpr (EPI == EPI_LINEAR) {
    if (e.act != MOE_LINEAR_NONE) by_eights(v, [&](float f) { return linear_act(f, e.act); });
  } else if constexpr (EPI == EPI_DACT) {
    by_eights(v, [&](float f) { return linear_slope(f, e.act); });
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v[8 * k + i];
    if constexpr (EPI == EPI_LINEAR || EPI == EPI_DACT) {
      if (e.add) {
        float d[8];
        unpack8(a.q[k], e.half, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = EPI == EPI_DACT ? f[i] * d[i] : f[i] + d[i];
      }
    }
    if constexpr (EPI == EPI_DGATED) {
      const int I = e.cols / 2;
      float d[8], g[4], u[4];
      unpack8(make_uint4(a.q[k].x, a.q[k].y, 0u, 0u), e.half, d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        gated_backward(f[2 * i], f[2 * i + 1], d[i], e.gate, g[i], u[i]);
      if (k < rows) {
        if (e.gate.layout == MOE_W13_PACKED) {
          uint16_t *p = static_cast<uint16_t *>(e.out) + (row + k) * e.cols + col / 2;
          store4(p, g, e.half);
          store4(p + I, u, e.half);
        } else {
          const float o[8] = {g[0], u[0], g[1], u[1], g[2], u[2], g[3], u[3]};
          *reinterpret_cast<uint4 *>(out + (int64_t)k * e.cols) = pack8(o, e.half);
        }
      }
    } else if (k < rows) {
      *reinterpret_cast<uint4 *>(out + (int64_t)k * e.cols) = pack8(f, e.half);
    }
    if constexpr (EPI == EPI_DACT) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * k + i] = k < rows ? f[i] : 0.f;
    }
  }
  if constexpr (EPI == EPI_DACT) {
    if (e.column_part) {  // over the lane's rows, then over the groups
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float f = (v[i] + v[8 + i]) + (v[16 + i] + v[24 + i]);
#pragma unroll
        for (int h = 4; h < 32; h <<= 1) f += __shfl_xor_sync(0xffffffffu, f, h);
        v[i] = f;
      }
      if (lane < 4 && col < e.cols) {
        float4 *p = reinterpret_cast<float4 *>(e.column_part + row0 / 32 * e.cols + col);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  }
}

// The same of a part of a split sum [rows, part_columns(cols)].
__device__ __forceinline__ void store_partial(float *part, int64_t rows, int cols, int64_t row0,
                                              int c, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  const int64_t row = row0 + (lane >> 2) * 4, wide = part_columns(cols);
  float *p = part + row * wide + c + (lane & 3) * 8;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (row + k < rows) {
      uint4 q[2];
      memcpy(q, v + 8 * k, 32);
      store32(p + k * wide, q[0], q[1]);
    }
}

// v[c] of lane r to v[r] of lane c.
__device__ __forceinline__ void transpose32(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 16; h > 0; h >>= 1)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if ((i & h) == 0) {
        const float got = __shfl_xor_sync(0xffffffffu, lane & h ? v[i] : v[i + h], h);
        if (lane & h) v[i] = got;
        else v[i + h] = got;
      }
}

// EPI_COLUMNS, 32 rows x 32 columns of a warp: a lane per column, so that a
// row's values are read and written side by side (922 x 5281 x 280 with bias
// and residual: 95 us with a lane per row).
struct ColumnAddend {
  uint16_t r[32];
};
__device__ __forceinline__ void fetch_columns(const DenseEpi &e, int64_t row0, int c,
                                              ColumnAddend &a) {
  const int col = c + (int)(threadIdx.x & 31);
  const uint16_t *p = static_cast<const uint16_t *>(e.add) + row0 * e.cols + col;
  if (e.add && col < e.cols) {
    const int rows = e.rows - row0 < 32 ? (int)(e.rows - row0) : 32;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      a.r[i] = 0;
      if (i < rows) a.r[i] = load_now(p + (int64_t)i * e.cols);
    }
  }
}
__device__ __forceinline__ void linear_columns(const DenseEpi &e, int64_t row0, int c,
                                               float (&v)[32], const ColumnAddend &a) {
  const int col = c + (int)(threadIdx.x & 31);
  transpose32(v);
  if (col >= e.cols) return;
  const int rows = e.rows - row0 < 32 ? (int)(e.rows - row0) : 32;
  uint16_t *out = static_cast<uint16_t *>(e.out) + row0 * e.cols + col;
  const float b = e.bias ? from16(static_cast<const uint16_t *>(e.bias)[col], e.half) : 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] += b;
  if (e.act != MOE_LINEAR_NONE) by_eights(v, [&](float f) { return linear_act(f, e.act); });
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (e.add) v[i] += from16(a.r[i], e.half);
    if (i < rows) out[(int64_t)i * e.cols] = to16(v[i], e.half);
  }
}

// The epilogue warps' share of a ColumnJoin: 32 columns per CTA at a time, one
// row per warp, then over the warps.
template <int WARPS>
__device__ __forceinline__ void join_columns(const ColumnJoin &j, int warp, int lane,
                                             float (*s_sum)[33]) {
  for (int c0 = (int)blockIdx.x * 32; c0 < j.cols; c0 += (int)gridDim.x * 32) {
    float acc = 0.f;
    if (c0 + lane < j.cols) {
#pragma unroll 8
      for (int r = warp; r < j.rows; r += WARPS)
        acc += __ldcg(j.part + (int64_t)r * j.cols + c0 + lane);
    }
    s_sum[warp][lane] = acc;
    asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
    if (warp == 0 && c0 + lane < j.cols) {
      acc = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) acc += s_sum[w][lane];
      static_cast<uint16_t *>(j.out)[c0 + lane] = to16(acc, j.half);
    }
    asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
  }
}

// GRAD: up to two gradients, B stored along its rows, A either way; else both
// operands K-major. MX: both are MXFP8.
template <bool GRAD, int EPI, bool MX>
__global__ void __launch_bounds__(gemm_threads(EPI), 1)
    dense_gemm_kernel(const __grid_constant__ GemmMaps maps,
                      const __grid_constant__ GemmArgs args) {
  static_assert(GRAD == (EPI == EPI_GRAD), "gradients have an epilogue of their own");
  constexpr int kStepK = MX ? 128 : 64;  // elements of a K step
  __shared__ float s_join[GRAD ? epi_warps(EPI) : 1][33];
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kRingBytes);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
  volatile int *s_abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const uint32_t stage0 = smem_u32(smem), full0 = smem_u32(bars);
  const int stages = args.stages, stage_bytes = args.stage_bytes;
  auto full_bar = [&](int s) { return full0 + 8u * s; };
  auto empty_bar = [&](int s) { return full0 + 8u * (kMaxStages + s); };
  auto tfull_bar = [&](int b) { return full0 + 8u * (2 * kMaxStages + b); };
  auto tempty_bar = [&](int b) { return full0 + 8u * (2 * kMaxStages + 2 + b); };
  const uint32_t drain_bar = full0 + 8u * (2 * kMaxStages + 4);
  auto a_addr = [&](int s) { return stage0 + (uint32_t)(s * stage_bytes); };
  auto b_addr = [&](int s) { return stage0 + (uint32_t)(s * stage_bytes + kABytes); };
  auto scale_addr = [&](int s) { return stage0 + (uint32_t)(kScaleOffset + s * kScaleBytes); };

  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int first = (int)(blockIdx.x >> 1), step = (int)(gridDim.x >> 1);
  const int total = args.p[0].units + (GRAD ? args.p[1].units : 0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 2 * epi_warps(EPI));  // the leader's counts both CTAs
    }
    mbar_init(drain_bar, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    prefetch_tmap(&maps.m[kMapA]);
    prefetch_tmap(&maps.m[kMapB]);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  // MXFP8: the preceding kernel lays out the scales and has itself waited for
  // all before it, so only the scales' loads wait for it
  pdl_launch_dependents();
  if constexpr (!MX) pdl_wait();
  __syncthreads();
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers and TMEM exist before any cross-CTA use
  tc_fence_after();
  const uint32_t tmem_base = (uint32_t)uniform((int)*tmem_slot);

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer --
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int u = first; ok && u < total; u += step) {
      const Unit w = unit_of<GRAD>(u, args);
      const GemmProblem &p = args.p[w.p];
      const int m0 = w.m * 2 * kRowsCta + (int)rank * kRowsCta;
      const int n0 = w.n * p.tn + (int)rank * (w.tn / 2);
      const uint32_t tx = 2u * (uint32_t)(kABytes + w.b_bytes + (MX ? kScaleBytes : 0));
      const CUtensorMap *ma = &maps.m[2 * w.p + kMapA];
      const CUtensorMap *mb = GRAD              ? &maps.m[2 * w.p + kMapB]
                              : w.n < p.n_full ? &maps.m[kMapB]
                                               : &maps.m[kMapBLast];
      auto load_operands = [&](int s, int kb) {
        const uint32_t fb = map_to_rank(full_bar(s), 0);
        if (leader) mbar_arrive_expect_tx(full_bar(s), tx);
        const int k0 = kb * kStepK;
        if (!GRAD || p.a_k_major) {
          tma_load_2d_pair(a_addr(s), ma, fb, k0, m0);
        } else {
          tma_load_2d_pair(a_addr(s), ma, fb, m0, k0);
          tma_load_2d_pair(a_addr(s) + 8192u, ma, fb, m0 + 64, k0);
        }
        if constexpr (GRAD) {
          tma_load_2d_pair(b_addr(s), mb, fb, n0, k0);
          if (w.b_bytes > 8192) tma_load_2d_pair(b_addr(s) + 8192u, mb, fb, n0 + 64, k0);
        } else if (args.pairs) {
          tma_load_3d_pair(b_addr(s), mb, fb, k0, 0, n0 / 2);
        } else {
          tma_load_2d_pair(b_addr(s), mb, fb, k0, n0);
        }
      };
      auto load_scales = [&](int s, int kb) {  // x's own rows, w's all: each CTA
        const uint32_t fb = map_to_rank(full_bar(s), 0);  // multiplies every column
        tma_load_2d_pair(scale_addr(s), &maps.m[kMapSa], fb, 0,
                         (w.m * 2 + (int)rank) * p.num_kb + kb);
        tma_load_2d_pair(scale_addr(s) + kScaleBlock, &maps.m[kMapSb], fb, 0,
                         (w.n * p.num_kb + kb) * 2);
      };
      int kb = w.k_lo;
      if constexpr (MX) {
        if (u == first) {  // the ring's first codes, ahead of the scales
          const int ahead = w.k_hi - w.k_lo < stages ? w.k_hi - w.k_lo : stages;
          for (int i = 0; i < ahead; ++i)
            if (elect_one()) load_operands(i, kb + i);
          pdl_wait();
          for (int i = 0; i < ahead; ++i)
            if (elect_one()) load_scales(i, kb + i);
          kb += ahead;
          issued = (uint32_t)ahead;
          stage = ahead == stages ? 0 : ahead;
          phase = ahead == stages ? 1u : 0u;
        }
      }
      for (; kb < w.k_hi; ++kb) {
        ok = wait_bounded(empty_bar(stage), phase ^ 1u, s_abort, args.status, args.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (elect_one()) {
          load_operands(stage, kb);
          if constexpr (MX) load_scales(stage, kb);
        }
        issued = issued < (uint32_t)stages ? issued + 1 : (uint32_t)stages;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // A pair's copies are counted on the leader's barriers. Where a wait gave up,
    // here or in the MMA warp after the last copy was issued, nobody else waits for
    // those in flight. drain_bar says that the MMA warp is done, whichever way.
    if (leader) {
      wait_drain(drain_bar, 0, (kMaxStages + 2) * args.timeout_ns);
      if (*s_abort) {
        for (uint32_t i = 0; i < issued; ++i) {
          int s = stage - 1 - (int)i;
          uint32_t ph = phase;
          if (s < 0) {
            s += stages;
            ph ^= 1u;
          }
          wait_drain(full_bar(s), ph, args.timeout_ns / 10);
        }
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------- MMA issuer (the leader) --
    if (leader) {
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = first; ok && u < total; u += step, ++local) {
        const Unit w = unit_of<GRAD>(u, args);
        const GemmProblem &p = args.p[w.p];
        const bool a_k = !GRAD || p.a_k_major;
        // descriptor steps (16-byte units) between the four MMAs of a stage
        const uint32_t a_step = a_k ? 2u : 128u;
        constexpr uint32_t b_step = GRAD ? 128u : 2u;
        const int acc = local & 1;
        ok = wait_bounded(tempty_bar(acc), ((uint32_t)(local >> 1) & 1u) ^ 1u, s_abort,
                          args.status, args.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * acc_cols(MX));
        const uint32_t idesc = p.idesc | ((uint32_t)(w.tn >> 3) << 17);
        for (int kb = w.k_lo; kb < w.k_hi; ++kb) {
          ok = wait_bounded(full_bar(stage), phase, s_abort, args.status, args.timeout_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = a_k ? sw128_desc(a_addr(stage)) : sw128_desc_mn(a_addr(stage));
          const uint64_t bd = GRAD ? sw128_desc_mn(b_addr(stage)) : sw128_desc(b_addr(stage));
          if (elect_one()) {
            if constexpr (MX) {
              // the columns belong to the stage: the MMAs that read them last
              // were complete before the stage was filled again
              const uint32_t sa = tmem_base + 2u * kMxTn + (uint32_t)(stage * kScaleCols);
              copy_scales_pair(sa, scale_addr(stage));
              copy_scales_pair(sa + 4u, scale_addr(stage) + kScaleBlock);
              if (w.tn > 128) copy_scales_pair(sa + 8u, scale_addr(stage) + 2 * kScaleBlock);
#pragma unroll
              for (uint32_t kk = 0; kk < 4; ++kk)  // the kk-th byte of each scale word
                umma_mx8_pair(d_tmem, ad + a_step * kk, bd + b_step * kk,
                              idesc | (kk << 4) | (kk << 29), sa, sa + 4u,
                              kb != w.k_lo || kk != 0);
            } else {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16_pair(d_tmem, ad + a_step * kk, bd + b_step * kk, idesc,
                               kb != w.k_lo || kk != 0);
            }
            umma_commit_pair(empty_bar(stage), 0x3);
          }
          __syncwarp();
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok && elect_one()) umma_commit_pair(tfull_bar(acc), 0x3);
        __syncwarp();
      }
      if (elect_one()) umma_commit_pair(drain_bar, 0x1);
      __syncwarp();
      wait_drain(drain_bar, 0, 100000000ull);
    }
  } else {
    // ----------------------------------------------------------- epilogue --
    constexpr int W = EPI == EPI_GATED_MX ? 64 : 32;
    const int q = warp & 3;            // TMEM lane quarter this warp may read
    const int part = (warp - 2) >> 2;  // which of the quarter's warps
    constexpr int kHop = epi_warps(EPI) / 4 * W;  // columns from one of its chunks to the next
    if constexpr (GRAD)
      if (args.join.out) join_columns<epi_warps(EPI)>(args.join, warp - 2, lane, s_join);
    int local = 0;
    for (int u = first; u < total; u += step, ++local) {
      const Unit w = unit_of<GRAD>(u, args);
      const GemmProblem &p = args.p[w.p];
      const int acc = local & 1;
      const int64_t row0 = (int64_t)w.m * 2 * kRowsCta + rank * kRowsCta + q * 32;
      const int c0 = w.n * p.tn;
      RowsAddend add;  // of the first columns, while the last products run
      ColumnAddend column_add;
      if (row0 < p.e.rows && part * W < w.tn && c0 + part * W < p.e.cols) {
        if constexpr (EPI == EPI_COLUMNS) fetch_columns(p.e, row0, c0 + part * W, column_add);
        else fetch_rows<EPI>(p.e, row0, c0 + part * W, add);
      }
      const bool ok = wait_bounded(tfull_bar(acc), (uint32_t)(local >> 1) & 1u, s_abort,
                                   args.status, args.timeout_ns);
      // all lanes or none: the loads from TMEM and the exchanges below take the whole warp
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * acc_cols(MX));
      const bool partial = EPI == EPI_PARTIAL || (GRAD && p.partial);
#pragma unroll 1
      for (int c = part * W; c < w.tn; c += kHop) {
        if (c0 + c >= p.e.cols) break;
        float v[W];
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < W; i += 32) {
          TMEM_LD32(taddr + c + i, r);
          tmem_wait_ld(r);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[i + j] = __uint_as_float(r[j]);
        }
        if (row0 >= p.e.rows) continue;
        const bool more = c + kHop < w.tn && c0 + c + kHop < p.e.cols;
        if constexpr (EPI == EPI_GATED || EPI == EPI_GATED_MX) {
          if (row0 + lane < p.e.rows) dense_epilogue<EPI, W>(p.e, row0 + lane, c0 + c, v);
        } else if constexpr (EPI == EPI_COLUMNS) {
          const ColumnAddend now = column_add;
          if (more) fetch_columns(p.e, row0, c0 + c + kHop, column_add);
          linear_columns(p.e, row0, c0 + c, v, now);
        } else {
          const RowsAddend now = add;
          if (more) fetch_rows<EPI>(p.e, row0, c0 + c + kHop, add);
          regroup(v);
          if (partial)
            store_partial(static_cast<float *>(p.e.out) + w.s * p.part_stride, p.e.rows, p.e.cols,
                          row0, c0 + c, v);
          else
            rows_epilogue<EPI>(p.e, row0, c0 + c, v, now);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(tempty_bar(acc));
        else
          mbar_arrive_cluster(map_to_rank(tempty_bar(acc), 0));
      }
    }
  }

  // a CTA that gave up tells its peer, which still has to reach the barrier
  if (lane == 0 && *s_abort)
    st_shared_cluster(map_to_rank(smem_u32((const void *)s_abort), rank ^ 1u), 1);
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // the leader's MMAs into the peer's TMEM are complete
  if (*s_abort) {
    // Nothing more is issued. Copies of the peer that the leader's barriers no
    // longer expected have a millisecond to land before either CTA leaves.
    const long long until = wait_deadline(1000000ull);
    while (clock64() < until) __nanosleep(1000);
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// The parts of a split sum [splits][rows, part_columns(cols)], added in order,
// and the epilogue. One thread per W columns; where rows do not start on 16
// bytes (EPI_LINEAR only) per column.
template <int EPI>
constexpr int join_width(bool vec) {
  return EPI == EPI_GATED_MX ? 64 : EPI == EPI_GATED || EPI == EPI_DGATED ? 16 : vec ? 8 : 1;
}
template <int EPI, bool VEC>
__global__ void __launch_bounds__(256)
dense_join_kernel(const float *part, int64_t stride, int splits, const __grid_constant__ DenseEpi e) {
  constexpr int W = join_width<EPI>(VEC);
  pdl_launch_dependents();
  pdl_wait();
  const int chunks = (e.cols + W - 1) / W;
  const int64_t total = e.rows * chunks;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / chunks;
    const int c = (int)(i - row * chunks) * W;
    const float *p = part + row * part_columns(e.cols) + c;
    if constexpr (W == 1) {
      float v = 0.f;
      for (int s = 0; s < splits; ++s, p += stride) v += __ldcg(p);
      const int64_t at = row * e.cols + c;
      if (e.bias) v += from16(static_cast<const uint16_t *>(e.bias)[c], e.half);
      if (e.act != MOE_LINEAR_NONE) v = linear_act(v, e.act);
      if (e.add) v += from16(static_cast<const uint16_t *>(e.add)[at], e.half);
      static_cast<uint16_t *>(e.out)[at] = to16(v, e.half);
    } else {
      float v[W];
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = 0.f;
      for (int s = 0; s < splits; ++s, p += stride) {
#pragma unroll
        for (int j = 0; j < W; j += 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4 *>(p + j));
          v[j] += f.x;
          v[j + 1] += f.y;
          v[j + 2] += f.z;
          v[j + 3] += f.w;
        }
      }
      dense_epilogue<EPI, W>(e, row, c, v);
    }
  }
}

// 16-bit [rows, cols] row-major in boxes of 64 columns x box_rows rows (fp16
// and bf16 are copied alike).
bool map_rows(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int box_rows) {
  return map_2d(m, base, (uint64_t)rows, (uint64_t)cols, (uint32_t)box_rows);
}

// A packed w13 [2, I, cols]: rows gate_i, up_i alternate in the box of
// 64 columns x 2 x box_pairs.
bool map_pairs(CUtensorMap *m, const void *base, int64_t I, int64_t cols, int box_pairs) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, 2, (cuuint64_t)I};
  cuuint64_t strides[2] = {(cuuint64_t)(I * cols * 2), (cuuint64_t)(cols * 2)};
  cuuint32_t box[3] = {64, 2, (cuuint32_t)box_pairs};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale bytes [rows, G] to blocks: one thread per line of a block (four rows'
// four scales), K steps fastest, so that a warp reads its rows' bytes in a
// piece. Rows and groups that do not exist get 1 (their codes are zeros).
struct ScaleLayout {
  const uint8_t *src;
  uint8_t *dst;
  int64_t rows;
  int tiles, tile_rows, blocks;  // blocks of 128 rows per tile
  int pairs;                     // tile rows 2i, 2i + 1 are rows i and i + rows / 2
};
// Bytes of the widest load that every row's scales allow (4, 2 or 1).
template <int BYTES>
__device__ __forceinline__ uint32_t scale_word(const uint8_t *p, int left) {
  uint32_t word = 0;
#pragma unroll
  for (int t = 0; t < 4; t += BYTES) {
    uint32_t part;
    if constexpr (BYTES == 4) part = left >= 4 ? __ldg(reinterpret_cast<const uint32_t *>(p)) : 0u;
    else if constexpr (BYTES == 2)
      part = t < left ? __ldg(reinterpret_cast<const uint16_t *>(p + t)) : 0x7f7fu;
    else part = t < left ? __ldg(p + t) : 0x7fu;
    word |= part << (8 * t);
  }
  return word;
}
template <int BYTES>
__global__ void __launch_bounds__(256)
mx8_layout_kernel(const ScaleLayout a, const ScaleLayout b, int G, int num_kb) {
  pdl_wait();  // first: the product that follows starts on this kernel's word
  pdl_launch_dependents();
  const int64_t na = (int64_t)a.tiles * a.blocks * num_kb * 32;
  const int64_t nb = (int64_t)b.tiles * b.blocks * num_kb * 32;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < na + nb;
       i += (int64_t)gridDim.x * blockDim.x) {
    const ScaleLayout &l = i < na ? a : b;
    const int64_t j = i < na ? i : i - na;  // [tile][block][line][kb]
    const int64_t lines = j / num_kb;
    const int kb = (int)(j - lines * num_kb), left = G - kb * 4;
    const int line = (int)(lines & 31);
    const int64_t tb = lines >> 5, tile = tb / l.blocks;
    const int block = (int)(tb - tile * l.blocks);
    uint32_t word[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = block * 128 + q * 32 + line;
      const int64_t row = tile * l.tile_rows + r;
      word[q] = 0x7f7f7f7fu;
      if (r < l.tile_rows && row < l.rows) {
        const int64_t from = l.pairs ? (row >> 1) + (row & 1) * (l.rows / 2) : row;
        word[q] = scale_word<BYTES>(l.src + from * G + kb * 4, left);
      }
    }
    reinterpret_cast<uint4 *>(l.dst)[((tile * num_kb + kb) * l.blocks + block) * 32 + line] =
        make_uint4(word[0], word[1], word[2], word[3]);
  }
}

// MXFP8 codes [rows, cols] in boxes of 128 columns; with `pairs` as map_pairs.
bool map_codes(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int box_rows,
               bool pairs) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const int64_t I = rows / 2;
  cuuint64_t dims[3] = {(cuuint64_t)cols, pairs ? 2 : (cuuint64_t)rows, (cuuint64_t)I};
  cuuint64_t strides[2] = {(cuuint64_t)(pairs ? I * cols : cols), (cuuint64_t)cols};
  cuuint32_t box[3] = {128, pairs ? 2 : (cuuint32_t)box_rows, (cuuint32_t)(box_rows / 2)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, pairs ? 3 : 2, const_cast<void *>(base), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale blocks, `box` of them at a time.
bool map_blocks(CUtensorMap *m, const void *base, int64_t blocks, int box_blocks) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {kScaleBlock / 4, (cuuint64_t)blocks};
  cuuint64_t strides[1] = {kScaleBlock};
  cuuint32_t box[2] = {kScaleBlock / 4, (cuuint32_t)box_blocks};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool GRAD, int EPI, bool MX>
cudaError_t launch_gemm(const GemmMaps &m, const GemmArgs &a, cudaStream_t s) {
  auto kern = dense_gemm_kernel<GRAD, EPI, MX>;
  static PerDeviceOnce once;
  static std::atomic<int> resident[PerDeviceOnce::kMaxDevices] = {};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(device_sm_count() & ~1);
  cfg.blockDim = dim3(gemm_threads(EPI));
  cfg.dynamicSmemBytes = kGemmSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  err = once.run([&] {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kGemmSmem);
    if (e == cudaSuccess) e = uniform_carveout(kern);
    int n = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e == cudaSuccess) resident[dev].store(n < 1 ? 1 : n, std::memory_order_relaxed);
    return e;
  });
  if (err != cudaSuccess) return err;
  const int64_t units = (int64_t)a.p[0].units + a.p[1].units;
  int64_t pairs = resident[dev].load(std::memory_order_relaxed);
  if (units < pairs) pairs = units;
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  err = cudaLaunchKernelEx(&cfg, kern, m, a);
  return err != cudaSuccess ? err : cudaGetLastError();
}

template <int EPI, bool VEC = true>
cudaError_t launch_join(const float *part, int64_t stride, int splits, const DenseEpi &e,
                        cudaStream_t s) {
  constexpr int W = join_width<EPI>(VEC);
  const int64_t threads = e.rows * ((e.cols + W - 1) / W);
  int64_t blocks = (threads + 255) / 256;
  const int64_t cap = (int64_t)device_sm_count() * 8;
  if (blocks > cap) blocks = cap;
  return launch_dependent(dense_join_kernel<EPI, VEC>, dim3((unsigned)blocks), dim3(256), 0, s, part,
                          stride, splits, e);
}

template <bool MX>
cudaError_t launch_kind(int kind, const GemmMaps &m, const GemmArgs &a, cudaStream_t s) {
  if constexpr (!MX) {
    if (kind == EPI_DACT) return launch_gemm<false, EPI_DACT, MX>(m, a, s);
    if (kind == EPI_DGATED) return launch_gemm<false, EPI_DGATED, MX>(m, a, s);
  }
  switch (kind) {
    case EPI_GATED: return launch_gemm<false, EPI_GATED, MX>(m, a, s);
    case EPI_GATED_MX: return launch_gemm<false, EPI_GATED_MX, MX>(m, a, s);
    case EPI_PARTIAL: return launch_gemm<false, EPI_PARTIAL, MX>(m, a, s);
    case EPI_COLUMNS: return launch_gemm<false, EPI_COLUMNS, MX>(m, a, s);
    default: return launch_gemm<false, EPI_LINEAR, MX>(m, a, s);
  }
}

cudaError_t join_parts(const DenseProduct &p, const DensePlan &plan, const float *partial,
                       cudaStream_t s) {
  const int64_t stride = p.M * part_columns((int)p.N);
  const int n = plan.splits;
  switch (p.kind) {
    case EPI_DACT: return launch_join<EPI_DACT>(partial, stride, n, p.epi, s);
    case EPI_GATED: return launch_join<EPI_GATED>(partial, stride, n, p.epi, s);
    case EPI_GATED_MX: return launch_join<EPI_GATED_MX>(partial, stride, n, p.epi, s);
    case EPI_DGATED: return launch_join<EPI_DGATED>(partial, stride, n, p.epi, s);
    default:
      return p.epi.vec ? launch_join<EPI_LINEAR>(partial, stride, n, p.epi, s)
                       : launch_join<EPI_LINEAR, false>(partial, stride, n, p.epi, s);
  }
}

// Estimated SM cycles of a K step of a tile of tn columns on a CTA pair: 2 per
// column (256 x tn x 64 products at 4096 per cycle and SM; MXFP8 twice the
// products at twice the rate) and no less than its operands' way into shared
// memory. The constants choose between tile widths and do not foretell times: 74
// bytes per cycle and SM rank the widths of small products as they measured (2048 x
// 2880 x 2880: 36, 26, 22 and 30 us at 64, 128, 160 and 256 columns), while large ones on
// all SMs take in 52 to 54 (567 cycles per step of 224 columns, 8192 x 2880 x 2880 in bf16;
// 620 in MXFP8, 2047 x 5760 x 2880; 582 of 192 columns, MXFP8, 8192 x 5760 x 2880).
double step_cycles(int tn, bool mx) {
  const double mma = 2.08 * tn, load = (16384.0 + (mx ? kScaleBytes : 0) + 64.0 * tn) / 74.0;
  return mma > load ? mma : load;
}
constexpr double kUnitCycles = 800.0;   // of a unit beside its steps
constexpr double kJoinCycles = 5000.0;  // of the kernel that joins the parts
constexpr int kPairs = 76;  // of the GB300's 152 SMs: a plan does not depend on the device

DensePlan plan_of(int64_t M, int64_t N, int tn, int last, int splits) {
  DensePlan p{};
  p.tn = tn;
  p.tn_last = last;
  p.m_tiles = (int)((M + 255) / 256);
  p.n_tiles = (int)((N + tn - 1) / tn);
  p.splits = splits;
  p.partial = splits > 1 ? (size_t)M * part_columns((int)N) * 4 * splits : 0;
  return p;
}

void set_problem(GemmProblem &g, const DenseProduct &p, const DensePlan &plan, bool grad, bool mx,
                 float *partial) {
  auto b_bytes = [&](int cols) {
    return grad ? (cols / 2 + 63) / 64 * 8192 : cols / 2 * kStepBytes;
  };
  g.e = p.epi;
  g.m_tiles = plan.m_tiles;
  g.n_tiles = plan.n_tiles;
  g.splits = plan.splits;
  g.num_kb = (int)((p.K + (mx ? 127 : 63)) / (mx ? 128 : 64));
  g.tn = plan.tn;
  g.b_bytes = b_bytes(plan.tn);
  g.tn_last = plan.tn_last;
  g.b_bytes_last = b_bytes(plan.tn_last);
  g.n_full = plan.tn_last == plan.tn ? plan.n_tiles : plan.n_tiles - 1;
  g.a_k_major = p.a.k_major;
  g.units = plan.m_tiles * plan.n_tiles * plan.splits;
  if (mx) {  // scale type E8M0 (bit 23); both codes E4M3
    g.idesc = (1u << 23) | ((uint32_t)(256 >> 4) << 24);
  } else {
    const uint32_t type = p.epi.half ? 0u : 1u;  // fp16 / bf16
    g.idesc = (1u << 4) | (type << 7) | (type << 10) | ((p.a.k_major ? 0u : 1u) << 15) |
              ((p.b.k_major ? 0u : 1u) << 16) | ((uint32_t)(256 >> 4) << 24);
  }
  if (plan.splits > 1) {
    g.partial = 1;
    g.e.out = partial;
    g.part_stride = p.M * part_columns((int)p.N);
  }
}

// Where calls without a status word of the caller's record a wait that gave up.
__device__ uint32_t g_wait_status;

cudaError_t wait_status_word(uint32_t **out) {
  static PerDeviceOnce once;
  static std::atomic<uint32_t *> word[PerDeviceOnce::kMaxDevices] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess)
    err = once.run([&] {
      void *p = nullptr;
      const cudaError_t e = cudaGetSymbolAddress(&p, g_wait_status);
      if (e == cudaSuccess) word[dev].store(static_cast<uint32_t *>(p), std::memory_order_relaxed);
      return e;
    });
  if (err == cudaSuccess) *out = word[dev].load(std::memory_order_relaxed);
  return err;
}

cudaError_t set_ring(GemmArgs &a, int b_bytes, bool mx, int32_t *status) {
  a.stage_bytes = kABytes + b_bytes;
  const int most = mx ? kMxStages : kMaxStages;
  a.stages = kRingBytes / a.stage_bytes < most ? kRingBytes / a.stage_bytes : most;
  a.status = reinterpret_cast<uint32_t *>(status);
  a.timeout_ns = kWaitTimeoutNs;
  return status ? cudaSuccess : wait_status_word(&a.status);
}

}  // namespace

// Tile width and number of parts of the sum: the choice with the least
// estimated time. A split costs its partial sums' way through L2 and the
// joining kernel.
DensePlan dense_plan(int64_t M, int64_t N, int64_t K, int kind, bool mx) {
  DensePlan best{};
  double best_t = 1e300;
  const int gran = kind == EPI_GATED_MX ? 64 : 32;
  const int64_t kb = mx ? (K + 127) / 128 : (K + 63) / 64, mt = (M + 255) / 256;
  for (int tn = acc_cols(mx) / gran * gran; tn >= 64; tn -= gran) {
    const int64_t nt = (N + tn - 1) / tn;
    const int last = (int)((N - (nt - 1) * tn + gran - 1) / gran * gran);
    const int64_t nf = last == tn ? nt : nt - 1;
    for (int s = 1; s <= 16; ++s) {
      if (s > 1 && (kb / s < 4 || mt * nt * s > 2 * kPairs)) break;
      const double steps = (double)((kb + s - 1) / s);
      // whole tiles in waves, the narrow ones in the room that the last leaves
      const int64_t full = mt * nf * s, waves = (full + kPairs - 1) / kPairs;
      int64_t narrow = (nt - nf) * mt * s - (waves * kPairs - full);
      if (narrow < 0) narrow = 0;
      double t = (double)waves * (steps * step_cycles(tn, mx) + kUnitCycles) +
                 (double)((narrow + kPairs - 1) / kPairs) *
                     (steps * step_cycles(last, mx) + kUnitCycles);
      if (s > 1) t += kJoinCycles + (double)M * N * 4.0 * (s + 1) / 2500.0;
      if (t < best_t) {
        best_t = t;
        best = plan_of(M, N, tn, last, s);
      }
    }
  }
  if (mx)
    best.blocks = (size_t)kb * kScaleBlock * 2 * ((size_t)best.m_tiles + (size_t)best.n_tiles);
  return best;
}

// The same for two gradients in one launch, whose units are dealt out one
// after the other to the pairs in turn (x: the one that comes first).
void dense_plan_two(int64_t M0, int64_t N0, int64_t K0, int64_t M1, int64_t N1, int64_t K1,
                    DensePlan *plan0, DensePlan *plan1) {
  struct Choice {
    int tn, last, splits;
    int64_t units;
    double time, extra;
  };
  auto choices = [](int64_t M, int64_t N, int64_t K, Choice *out) {
    int count = 0;
    const int64_t kb = (K + 63) / 64, mt = (M + 255) / 256;
    const int splits[] = {1, 2, 3, 4, 6, 8, 12};
    for (int tn = 256; tn >= 64; tn -= 64) {
      const int64_t nt = (N + tn - 1) / tn;
      if (tn > 64 && N <= tn / 2) continue;  // a narrower tile holds all columns
      const int last = (int)((N - (nt - 1) * tn + 31) / 32 * 32);
      for (int s : splits) {
        if (s > 1 && (kb / s < 4 || mt * nt * s > 2 * kPairs)) break;
        out[count++] = {tn, last, s, mt * nt * s,
                        (double)((kb + s - 1) / s) * step_cycles(tn, false) + kUnitCycles,
                        s > 1 ? kJoinCycles + (double)M * N * 4.0 * (s + 1) / 2500.0 : 0.0};
      }
    }
    return count;
  };
  Choice c0[28], c1[28];
  const int n0 = choices(M0, N0, K0, c0), n1 = choices(M1, N1, K1, c1);
  double best = 1e300;
  int b0 = 0, b1 = 0;
  for (int i = 0; i < n0; ++i)
    for (int j = 0; j < n1; ++j) {
      const Choice &x = c0[i], &y = c1[j];
      const int64_t fx = x.units / kPairs, rx = x.units % kPairs;
      const int64_t fy = y.units / kPairs, ry = y.units % kPairs;
      // pairs [0, rx) take one unit more of x, the ry pairs behind them (in a
      // ring) one more of y
      double t = (double)fx * x.time + (double)fy * y.time;
      if (rx + ry > kPairs) t += x.time + y.time;
      else if (rx > 0 && (ry == 0 || x.time >= y.time)) t += x.time;
      else if (ry > 0) t += y.time;
      t += x.extra + y.extra;
      if (t < best) {
        best = t;
        b0 = i;
        b1 = j;
      }
    }
  *plan0 = plan_of(M0, N0, c0[b0].tn, c0[b0].last, c0[b0].splits);
  *plan1 = plan_of(M1, N1, c1[b1].tn, c1[b1].last, c1[b1].splits);
}

cudaError_t launch_dense(const DenseProduct &p, const DensePlan &plan, uint8_t *blocks,
                         float *partial, int32_t *status, cudaStream_t s) {
  GemmMaps maps;
  CUtensorMap *m = maps.m;
  const bool mx = p.a.scales != nullptr;
  GemmArgs a{};
  set_problem(a.p[0], p, plan, false, mx, partial);
  cudaError_t err = set_ring(a, a.p[0].b_bytes, mx, status);
  if (err != cudaSuccess) return err;
  if (p.starve_ns) {  // each step waits for bytes that nobody sends
    a.timeout_ns = p.starve_ns;
    a.p[0].b_bytes += 16;
    a.p[0].b_bytes_last += 16;
  }
  a.pairs = p.b.pairs;
  const GemmProblem &g = a.p[0];
  auto map_b = [&](CUtensorMap *t, int cols) {
    if (mx) return map_codes(t, p.b.p, p.N, p.K, cols / 2, p.b.pairs);
    if (p.b.pairs) return map_pairs(t, p.b.p, p.N / 2, p.K, cols / 4);
    return map_rows(t, p.b.p, p.N, p.K, cols / 2);
  };
  bool ok = mx ? map_codes(&m[kMapA], p.a.p, p.M, p.K, kRowsCta, false)
               : map_rows(&m[kMapA], p.a.p, p.M, p.K, kRowsCta);
  ok = ok && map_b(&m[kMapB], plan.tn);
  m[kMapBLast] = m[kMapB];
  if (plan.tn_last != plan.tn) ok = ok && map_b(&m[kMapBLast], plan.tn_last);
  m[kMapSa] = m[kMapSb] = m[kMapA];
  if (mx) {
    const int64_t a_blocks = (int64_t)2 * plan.m_tiles * g.num_kb;
    const int64_t b_blocks = (int64_t)2 * plan.n_tiles * g.num_kb;
    uint8_t *sb = blocks + a_blocks * kScaleBlock;
    ok = ok && map_blocks(&m[kMapSa], blocks, a_blocks, 1) &&
         map_blocks(&m[kMapSb], sb, b_blocks, 2);
    if (!ok) return cudaErrorInvalidValue;
    const ScaleLayout la{p.a.scales, blocks, p.M, 2 * plan.m_tiles, kRowsCta, 1, 0};
    const ScaleLayout lb{p.b.scales, sb, p.N, plan.n_tiles, plan.tn, 2, p.b.pairs};
    int64_t grid = ((a_blocks + b_blocks) * 32 + 255) / 256;
    const int64_t cap = (int64_t)device_sm_count() * 4;  // room for the product's CTAs
    if (grid > cap) grid = cap;
    const int G = (int)(p.K / 32);
    const uintptr_t bits = (uintptr_t)p.a.scales | (uintptr_t)p.b.scales | (uintptr_t)G;
    err = launch_dependent(bits % 4 == 0   ? mx8_layout_kernel<4>
                           : bits % 2 == 0 ? mx8_layout_kernel<2>
                                           : mx8_layout_kernel<1>,
                           dim3((unsigned)grid), dim3(256), 0, s, la, lb, G, g.num_kb);
    if (err != cudaSuccess) return err;
  }
  if (!ok) return cudaErrorInvalidValue;
  const int kind = plan.splits > 1                         ? (int)EPI_PARTIAL
                   : p.kind == EPI_LINEAR && !p.epi.vec ? (int)EPI_COLUMNS
                                                        : p.kind;
  err = mx ? launch_kind<true>(kind, maps, a, s) : launch_kind<false>(kind, maps, a, s);
  return err != cudaSuccess || plan.splits == 1 ? err : join_parts(p, plan, partial, s);
}

cudaError_t read_wait_status(int32_t *out, bool reset, cudaStream_t s) {
  uint32_t *word = nullptr;
  cudaError_t err = wait_status_word(&word);
  if (err == cudaSuccess) err = cudaMemcpyAsync(out, word, 4, cudaMemcpyDeviceToHost, s);
  if (err == cudaSuccess && reset) err = cudaMemsetAsync(word, 0, 4, s);
  return err != cudaSuccess ? err : cudaStreamSynchronize(s);
}

cudaError_t launch_dense_gradients(const DenseProduct *const *p, const DensePlan *const *plan,
                                   float *const *partial, int count, const float *column_part,
                                   int column_rows, int columns, int half, void *column_out,
                                   int32_t *status, cudaStream_t s) {
  GemmMaps maps{};
  GemmArgs a{};
  int most = 0;
  for (int i = 0; i < count; ++i) {
    const DenseProduct &d = *p[i];
    set_problem(a.p[i], d, *plan[i], true, false, partial[i]);
    most = a.p[i].b_bytes > most ? a.p[i].b_bytes : most;
    CUtensorMap *m = maps.m + 2 * i;
    if (!(d.a.k_major ? map_rows(&m[kMapA], d.a.p, d.M, d.K, kRowsCta)
                      : map_rows(&m[kMapA], d.a.p, d.K, d.M, 64)) ||
        !map_rows(&m[kMapB], d.b.p, d.K, d.N, 64))
      return cudaErrorInvalidValue;
  }
  for (int i = 2 * count; i < kMaps; ++i) maps.m[i] = maps.m[0];
  cudaError_t err = set_ring(a, most, false, status);
  if (err != cudaSuccess) return err;
  a.join = {column_part, column_out, column_rows, columns, half};
  err = launch_gemm<true, EPI_GRAD, false>(maps, a, s);
  for (int i = 0; i < count && err == cudaSuccess; ++i)
    if (plan[i]->splits > 1) err = join_parts(*p[i], *plan[i], partial[i], s);
  return err;
}

}  // namespace moe
