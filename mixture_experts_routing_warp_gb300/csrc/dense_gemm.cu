// dense_gemm.cu -- the dense products beside the experts on the tcgen05 tensor
// cores: moe_linear, moe_gated_linear and their gradients.
//
//   D[m, n] = sum_k A(m, k) B(n, k)      bf16 or fp16 in, fp32 sums
// with A and B each stored along k (K-major) or along their rows (M/N-major),
// so that no gradient needs a transposed copy:
//   forward   a   = x W^T      A = x [n, C],    B = W [R, C]      both K-major
//   d_x       dx  = d_a W      A = d_a [n, R],  B = W [R, C]      B N-major
//   d_w       dw  = d_a^T x    A = d_a [n, R],  B = x [n, C]      both M/N-major
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
//   warps 2..   epilogue, two or four per TMEM lane quarter, column chunks in turn
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
#ifdef DENSE_TUNE
#include <stdio.h>
#include <stdlib.h>
#endif

namespace moe {
namespace {

using namespace tc;

constexpr int kRowsCta = 128;                    // A rows of a CTA's half tile
constexpr int kStepBytes = 128;                  // K bytes of a stage
constexpr int kABytes = kRowsCta * kStepBytes;   // 16 KB
constexpr int kMaxTn = 256;
// Epilogue warps, two or four per TMEM lane quarter: with four a tile's
// epilogue has the latency of two column chunks; a group of 32 8-bit results
// takes 64 columns and twice the registers.
#ifndef EPI_WARPS
#define EPI_WARPS 16
#endif
constexpr int epi_warps(int epi) { return epi == EPI_GATED_MX ? 8 : EPI_WARPS; }
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

struct GemmArgs {
  DenseEpi e;
  int64_t part_stride;  // floats between the parts of a split sum
  int m_tiles, n_tiles, splits;
  int num_kb;           // K steps of the whole sum
  int tn, stages, b_bytes;
  int tn_last, b_bytes_last, n_full;  // the last tile of a row of tiles, if narrower
  int pairs;            // B rows come interleaved through a 3-D map
  uint32_t idesc;
  uint32_t *status;
  unsigned long long timeout_ns;
};

// Shared-memory descriptor of an operand stored along its rows (M/N-major),
// 128-byte swizzle: atoms of 64 rows x 8 k (a 128-byte line per k), 8-k groups
// 1024 bytes apart (SBO), atoms along the rows 8 KB apart (LBO; a stage holds
// 64 k of each).
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Unit u: a tile and its part of the sum. The narrow last tiles come behind
// all others, to fill what the last wave of whole tiles leaves idle.
// 512 bytes (32 lines of 16: line l holds the scales of rows l, l + 32, l + 64
// and l + 96) to 4 TMEM columns of all lane quarters, in both CTAs of the pair
// from their own shared memory.
__device__ __forceinline__ void copy_scales_pair(uint32_t tmem, uint32_t saddr) {
  const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) |
                        ((uint64_t)1 << 46);
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
               : "memory");
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

struct Unit {
  int m, n, s, k_lo, k_hi, tn, b_bytes;
};
__device__ __forceinline__ Unit unit_of(int u, const GemmArgs &a) {
  Unit w;
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

// AK / BK: the operand is K-major. MX: both are MXFP8.
template <bool AK, bool BK, int EPI, bool MX>
__global__ void __launch_bounds__(gemm_threads(EPI), 1)
    dense_gemm_kernel(const __grid_constant__ CUtensorMap map_a,
                      const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ CUtensorMap map_b_last,
                      const __grid_constant__ CUtensorMap map_sa,
                      const __grid_constant__ CUtensorMap map_sb,
                      const __grid_constant__ GemmArgs args) {
  constexpr int kStepK = MX ? 128 : 64;  // elements of a K step
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kRingBytes);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
  volatile int *s_abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const uint32_t stage0 = smem_u32(smem), full0 = smem_u32(bars);
  const int stages = args.stages, stage_bytes = kABytes + args.b_bytes;
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
  const int total = args.m_tiles * args.n_tiles * args.splits;
  const int tn = args.tn;

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
    prefetch_tmap(&map_a);
    prefetch_tmap(&map_b);
    prefetch_tmap(&map_b_last);
    if constexpr (MX) {
      prefetch_tmap(&map_sa);
      prefetch_tmap(&map_sb);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  pdl_launch_dependents();
  pdl_wait();
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
      const Unit w = unit_of(u, args);
      const int m0 = w.m * 2 * kRowsCta + (int)rank * kRowsCta;
      const int n0 = w.n * tn + (int)rank * (w.tn / 2);
      const uint32_t tx = 2u * (uint32_t)(kABytes + w.b_bytes + (MX ? kScaleBytes : 0));
      const CUtensorMap *mb = w.n < args.n_full ? &map_b : &map_b_last;
      for (int kb = w.k_lo; kb < w.k_hi; ++kb) {
        ok = wait_bounded(empty_bar(stage), phase ^ 1u, s_abort, args.status, args.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t fb = map_to_rank(full_bar(stage), 0);
          if (leader) mbar_arrive_expect_tx(full_bar(stage), tx);
          const int k0 = kb * kStepK;
          if constexpr (AK) {
            tma_load_2d_pair(a_addr(stage), &map_a, fb, k0, m0);
          } else {
            tma_load_2d_pair(a_addr(stage), &map_a, fb, m0, k0);
            tma_load_2d_pair(a_addr(stage) + 8192u, &map_a, fb, m0 + 64, k0);
          }
          if constexpr (BK) {
            if (args.pairs)
              tma_load_3d_pair(b_addr(stage), mb, fb, k0, 0, n0 / 2);
            else
              tma_load_2d_pair(b_addr(stage), mb, fb, k0, n0);
          } else {
            tma_load_2d_pair(b_addr(stage), &map_b, fb, n0, k0);
            if (w.b_bytes > 8192)
              tma_load_2d_pair(b_addr(stage) + 8192u, &map_b, fb, n0 + 64, k0);
          }
          if constexpr (MX) {  // x's own rows, w's all: each CTA multiplies every column
            tma_load_2d_pair(scale_addr(stage), &map_sa, fb, 0,
                             (w.m * 2 + (int)rank) * args.num_kb + kb);
            tma_load_2d_pair(scale_addr(stage) + kScaleBlock, &map_sb, fb, 0,
                             (w.n * args.num_kb + kb) * 2);
          }
        }
        issued = issued < (uint32_t)stages ? issued + 1 : (uint32_t)stages;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // a pair's copies complete on the leader's barriers: the leader drains
    // (the peer stays resident until the final cluster barrier)
    if (!ok && leader) {
      for (uint32_t i = 0; i < issued; ++i) {
        int s = stage - 1 - (int)i;
        uint32_t ph = phase;
        if (s < 0) {
          s += stages;
          ph ^= 1u;
        }
        wait_drain(full_bar(s), ph, 100000000ull);
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------- MMA issuer (the leader) --
    if (leader) {
      // descriptor steps (16-byte units) between the four MMAs of a stage
      constexpr uint32_t a_step = AK ? 2u : 128u, b_step = BK ? 2u : 128u;
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = first; ok && u < total; u += step, ++local) {
        const Unit w = unit_of(u, args);
        const int acc = local & 1;
        ok = wait_bounded(tempty_bar(acc), ((uint32_t)(local >> 1) & 1u) ^ 1u, s_abort,
                          args.status, args.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * acc_cols(MX));
        const uint32_t idesc = args.idesc | ((uint32_t)(w.tn >> 3) << 17);
        for (int kb = w.k_lo; kb < w.k_hi; ++kb) {
          ok = wait_bounded(full_bar(stage), phase, s_abort, args.status, args.timeout_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = AK ? sw128_desc(a_addr(stage)) : sw128_desc_mn(a_addr(stage));
          const uint64_t bd = BK ? sw128_desc(b_addr(stage)) : sw128_desc_mn(b_addr(stage));
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
    int local = 0;
    for (int u = first; u < total; u += step, ++local) {
      const Unit w = unit_of(u, args);
      const int acc = local & 1;
      const int64_t row = (int64_t)w.m * 2 * kRowsCta + rank * kRowsCta + q * 32 + lane;
      const int c0 = w.n * tn;
      const bool live = row < args.e.rows;
      Addend<EPI, W> add;  // of the first columns, while the last products run
      if (live && part * W < w.tn && c0 + part * W < args.e.cols)
        fetch_addend<EPI, W>(args.e, row, c0 + part * W, add);
      if (!wait_bounded(tfull_bar(acc), (uint32_t)(local >> 1) & 1u, s_abort, args.status,
                        args.timeout_ns))
        break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * acc_cols(MX));
      DenseEpi e = args.e;
      if constexpr (EPI == EPI_PARTIAL) e.out = static_cast<float *>(e.out) + w.s * args.part_stride;
#pragma unroll 1
      for (int c = part * W; c < w.tn; c += kHop) {
        if (c0 + c >= args.e.cols) break;
        float v[W];
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < W; i += 32) {
          TMEM_LD32(taddr + c + i, r);
          tmem_wait_ld(r);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[i + j] = __uint_as_float(r[j]);
        }
        if (live) {
          const Addend<EPI, W> now = add;
          if (c + kHop < w.tn && c0 + c + kHop < args.e.cols)
            fetch_addend<EPI, W>(e, row, c0 + c + kHop, add);
          dense_epilogue<EPI, W>(e, row, c0 + c, v, now);
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

  tc_fence_before();
  cluster_sync();  // the leader's MMAs into the peer's TMEM are complete
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// The parts of a split sum, added in order, and the epilogue. One thread per
// W columns.
template <int EPI>
__global__ void __launch_bounds__(256)
dense_join_kernel(const float *part, int64_t stride, int splits, const __grid_constant__ DenseEpi e) {
  constexpr int W = EPI == EPI_GATED_MX ? 64 : EPI == EPI_GATED || EPI == EPI_DGATED ? 16 : 8;
  pdl_launch_dependents();
  pdl_wait();
  const int chunks = (e.cols + W - 1) / W;
  const int64_t total = e.rows * chunks;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / chunks;
    const int c = (int)(i - row * chunks) * W;
    float v[W];
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = 0.f;
    const float *p = part + row * e.cols + c;
    Addend<EPI, W> add;
    fetch_addend<EPI, W>(e, row, c, add);
    const bool full = c + W <= e.cols && e.cols % 4 == 0;
    for (int s = 0; s < splits; ++s, p += stride) {
      if (full) {
#pragma unroll
        for (int j = 0; j < W; j += 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4 *>(p + j));
          v[j] += f.x;
          v[j + 1] += f.y;
          v[j + 2] += f.z;
          v[j + 3] += f.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (c + j < e.cols) v[j] += __ldcg(p + j);
      }
    }
    dense_epilogue<EPI, W>(e, row, c, v, add);
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
  pdl_launch_dependents();
  pdl_wait();
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

struct GemmMaps {
  CUtensorMap a, b, b_last, sa, sb;
};

template <bool AK, bool BK, int EPI, bool MX = false>
cudaError_t launch_gemm(const GemmMaps &m, const GemmArgs &a, cudaStream_t s) {
  auto kern = dense_gemm_kernel<AK, BK, EPI, MX>;
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
  const int64_t units = (int64_t)a.m_tiles * a.n_tiles * a.splits;
  int64_t pairs = resident[dev].load(std::memory_order_relaxed);
  if (units < pairs) pairs = units;
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  err = cudaLaunchKernelEx(&cfg, kern, m.a, m.b, m.b_last, m.sa, m.sb, a);
  return err != cudaSuccess ? err : cudaGetLastError();
}

template <int EPI>
cudaError_t launch_join(const float *part, int64_t stride, int splits, const DenseEpi &e,
                        cudaStream_t s) {
  constexpr int W = EPI == EPI_GATED_MX ? 64 : EPI == EPI_GATED || EPI == EPI_DGATED ? 16 : 8;
  const int64_t threads = e.rows * ((e.cols + W - 1) / W);
  int64_t blocks = (threads + 255) / 256;
  const int64_t cap = (int64_t)device_sm_count() * 8;
  if (blocks > cap) blocks = cap;
  return launch_dependent(dense_join_kernel<EPI>, dim3((unsigned)blocks), dim3(256), 0, s, part,
                          stride, splits, e);
}

template <bool AK, bool BK>
cudaError_t launch_kind(int kind, const GemmMaps &m, const GemmArgs &a, cudaStream_t s) {
  if constexpr (AK && BK) {
    switch (kind) {
      case EPI_DACT: return launch_gemm<AK, BK, EPI_DACT>(m, a, s);
      case EPI_GATED: return launch_gemm<AK, BK, EPI_GATED>(m, a, s);
      case EPI_GATED_MX: return launch_gemm<AK, BK, EPI_GATED_MX>(m, a, s);
      case EPI_DGATED: return launch_gemm<AK, BK, EPI_DGATED>(m, a, s);
    }
  }
  if (kind == EPI_PARTIAL) return launch_gemm<AK, BK, EPI_PARTIAL>(m, a, s);
  return launch_gemm<AK, BK, EPI_LINEAR>(m, a, s);
}

cudaError_t launch_mx(int kind, const GemmMaps &m, const GemmArgs &a, cudaStream_t s) {
  switch (kind) {
    case EPI_GATED: return launch_gemm<true, true, EPI_GATED, true>(m, a, s);
    case EPI_GATED_MX: return launch_gemm<true, true, EPI_GATED_MX, true>(m, a, s);
    case EPI_PARTIAL: return launch_gemm<true, true, EPI_PARTIAL, true>(m, a, s);
    default: return launch_gemm<true, true, EPI_LINEAR, true>(m, a, s);
  }
}

}  // namespace

// Tile width and number of parts of the sum: the choice with the least
// estimated time, in SM cycles. A K step of a pair takes 2 cycles per column
// (256 x tn x 64 products at 8192 per cycle and SM; MXFP8 twice the products at
// twice the rate) and no less than its operands' way into shared memory
// (kIngress bytes per cycle and SM) nor than its issue; a unit costs about
// kUnit cycles beside its steps; a split costs its partial sums' way through
// L2 and the joining kernel.
DensePlan dense_plan(int64_t M, int64_t N, int64_t K, int kind, bool mx) {
  constexpr int kPairs = 76;  // of the GB300's 152 SMs: a plan does not depend on the device
  constexpr double kIngress = 60.0, kIssue = 200.0, kUnit = 800.0;
  DensePlan best{};
  double best_t = 1e300;
  const int gran = kind == EPI_GATED_MX ? 64 : 32;
  const int64_t kb = mx ? (K + 127) / 128 : (K + 63) / 64, mt = (M + 255) / 256;
  auto step = [&](int tn) {
    const double mma = 2.0 * tn, load = (16384.0 + (mx ? kScaleBytes : 0) + 64.0 * tn) / kIngress;
    const double t = mma > load ? mma : load;
    return t > kIssue ? t : kIssue;
  };
#ifdef DENSE_TUNE
  const char *env_tn = getenv("DENSE_TN"), *env_s = getenv("DENSE_SPLIT");
#endif
  for (int tn = acc_cols(mx) / gran * gran; tn >= 64; tn -= gran) {
#ifdef DENSE_TUNE
    if (env_tn && atoi(env_tn) != tn) continue;
#endif
    const int64_t nt = (N + tn - 1) / tn;
    const int last = (int)((N - (nt - 1) * tn + gran - 1) / gran * gran);
    const int64_t nf = last == tn ? nt : nt - 1;
    for (int s = 1; s <= 16; ++s) {
#ifdef DENSE_TUNE
      if (env_s && atoi(env_s) != s) continue;
#endif
      if (s > 1 && (kb / s < 4 || mt * nt * s > 2 * kPairs)) break;
      const double steps = (double)((kb + s - 1) / s);
      // whole tiles in waves, the narrow ones in the room that the last leaves
      const int64_t full = mt * nf * s, waves = (full + kPairs - 1) / kPairs;
      int64_t narrow = (nt - nf) * mt * s - (waves * kPairs - full);
      if (narrow < 0) narrow = 0;
      double t = (double)waves * (steps * step(tn) + kUnit) +
                 (double)((narrow + kPairs - 1) / kPairs) * (steps * step(last) + kUnit);
      if (s > 1) t += 5000.0 + (double)M * N * 4.0 * (s + 1) / 2500.0;
      if (t < best_t) {
        best_t = t;
        best.tn = tn;
        best.tn_last = last;
        best.m_tiles = (int)mt;
        best.n_tiles = (int)nt;
        best.splits = s;
      }
    }
  }
  best.partial = best.splits > 1 ? (size_t)M * N * 4 * best.splits : 0;
  best.blocks = mx ? (size_t)kb * kScaleBlock * 2 * ((size_t)best.m_tiles + (size_t)best.n_tiles) : 0;
#ifdef DENSE_TUNE
  if (getenv("DENSE_SHOW")) fprintf(stderr, "plan M %ld N %ld K %ld: tn %d last %d splits %d tiles %dx%d est %.0f\n", (long)M, (long)N, (long)K, best.tn, best.tn_last, best.splits, best.m_tiles, best.n_tiles, best_t);
#endif
  return best;
}

cudaError_t launch_dense(const DenseProduct &p, const DensePlan &plan, uint8_t *blocks,
                         float *partial, int32_t *status, cudaStream_t s) {
  GemmMaps m;
  const int tn = plan.tn;
  const bool ak = p.a.k_major, bk = p.b.k_major, mx = p.a.scales != nullptr;
  GemmArgs a{};
  a.e = p.epi;
  a.m_tiles = plan.m_tiles;
  a.n_tiles = plan.n_tiles;
  a.splits = plan.splits;
  a.num_kb = (int)((p.K + (mx ? 127 : 63)) / (mx ? 128 : 64));
  a.tn = tn;
  auto b_bytes = [&](int cols) { return bk ? cols / 2 * kStepBytes : (cols / 2 + 63) / 64 * 8192; };
  a.b_bytes = b_bytes(tn);
  a.tn_last = plan.tn_last;
  a.b_bytes_last = b_bytes(plan.tn_last);
  a.n_full = plan.tn_last == tn ? plan.n_tiles : plan.n_tiles - 1;
  a.stages = kRingBytes / (kABytes + a.b_bytes);
  const int most = mx ? kMxStages : kMaxStages;
  if (a.stages > most) a.stages = most;
  a.pairs = p.b.pairs;
  a.status = reinterpret_cast<uint32_t *>(status);
  a.timeout_ns = kWaitTimeoutNs;

  auto map_b = [&](CUtensorMap *t, int cols) {
    if (mx) return map_codes(t, p.b.p, p.N, p.K, cols / 2, p.b.pairs);
    if (p.b.pairs) return map_pairs(t, p.b.p, p.N / 2, p.K, cols / 4);
    return bk ? map_rows(t, p.b.p, p.N, p.K, cols / 2) : map_rows(t, p.b.p, p.K, p.N, 64);
  };
  bool ok = mx   ? map_codes(&m.a, p.a.p, p.M, p.K, kRowsCta, false)
            : ak ? map_rows(&m.a, p.a.p, p.M, p.K, kRowsCta)
                 : map_rows(&m.a, p.a.p, p.K, p.M, 64);
  ok = ok && map_b(&m.b, tn);
  m.b_last = m.b;
  if (plan.tn_last != tn) ok = ok && map_b(&m.b_last, plan.tn_last);
  m.sa = m.sb = m.a;
  if (mx) {
    // scale type E8M0 (bit 23); both codes E4M3
    a.idesc = (1u << 23) | ((uint32_t)(256 >> 4) << 24);
    const int64_t a_blocks = (int64_t)2 * plan.m_tiles * a.num_kb;
    const int64_t b_blocks = (int64_t)2 * plan.n_tiles * a.num_kb;
    uint8_t *sb = blocks + a_blocks * kScaleBlock;
    ok = ok && map_blocks(&m.sa, blocks, a_blocks, 1) && map_blocks(&m.sb, sb, b_blocks, 2);
    if (!ok) return cudaErrorInvalidValue;
    const ScaleLayout la{p.a.scales, blocks, p.M, 2 * plan.m_tiles, kRowsCta, 1, 0};
    const ScaleLayout lb{p.b.scales, sb, p.N, plan.n_tiles, tn, 2, p.b.pairs};
    int64_t grid = ((a_blocks + b_blocks) * 32 + 255) / 256;
    const int64_t cap = (int64_t)device_sm_count() * 8;
    if (grid > cap) grid = cap;
    const int G = (int)(p.K / 32);
    const uintptr_t bits = (uintptr_t)p.a.scales | (uintptr_t)p.b.scales | (uintptr_t)G;
    const cudaError_t err =
        launch_dependent(bits % 4 == 0   ? mx8_layout_kernel<4>
                         : bits % 2 == 0 ? mx8_layout_kernel<2>
                                         : mx8_layout_kernel<1>,
                         dim3((unsigned)grid), dim3(256), 0, s, la, lb, G, a.num_kb);
    if (err != cudaSuccess) return err;
  } else {
    const uint32_t type = p.epi.half ? 0u : 1u;  // fp16 / bf16
    a.idesc = (1u << 4) | (type << 7) | (type << 10) | ((ak ? 0u : 1u) << 15) |
              ((bk ? 0u : 1u) << 16) | ((uint32_t)(256 >> 4) << 24);
  }
  if (!ok) return cudaErrorInvalidValue;
  int kind = p.kind;
  if (plan.splits > 1) {
    kind = EPI_PARTIAL;
    a.e.out = partial;
    a.part_stride = p.M * p.N;
  }
  const cudaError_t err = mx         ? launch_mx(kind, m, a, s)
                          : ak && bk ? launch_kind<true, true>(kind, m, a, s)
                          : ak       ? launch_kind<true, false>(kind, m, a, s)
                                     : launch_kind<false, false>(kind, m, a, s);
  return err != cudaSuccess || plan.splits == 1 ? err : launch_dense_join(p, plan, partial, s);
}

cudaError_t launch_dense_join(const DenseProduct &p, const DensePlan &plan, const float *partial,
                              cudaStream_t s) {
  switch (p.kind) {
    case EPI_DACT: return launch_join<EPI_DACT>(partial, p.M * p.N, plan.splits, p.epi, s);
    case EPI_GATED: return launch_join<EPI_GATED>(partial, p.M * p.N, plan.splits, p.epi, s);
    case EPI_GATED_MX: return launch_join<EPI_GATED_MX>(partial, p.M * p.N, plan.splits, p.epi, s);
    case EPI_DGATED: return launch_join<EPI_DGATED>(partial, p.M * p.N, plan.splits, p.epi, s);
    default: return launch_join<EPI_LINEAR>(partial, p.M * p.N, plan.splits, p.epi, s);
  }
}

}  // namespace moe
