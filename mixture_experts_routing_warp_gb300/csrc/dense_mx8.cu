// dense_mx8.cu -- products of MXFP8 rows and weights on the tcgen05 tensor
// cores (moe_linear_mx8, moe_gated_linear_mx8):
//   a[m, n] = sum_k x[m, k] 2^(sx[m, k/32]) w[n, k] 2^(sw[n, k/32])
// E4M3 codes, one power of two per 32 of them, applied by the tensor core
// itself (kind::mxf8f6f4, block_scale, one scale per row and 32 k): the codes
// go through it at twice the bf16 rate and nothing is converted.
//
// A persistent kernel, one CTA per SM: tiles of 128 rows x tn <= 192 columns,
// K steps of 128. Per step a stage holds 128 x 128 codes of x, tn x 128 of w
// (TMA, 128-byte swizzle) and their scales, which tcgen05.cp spreads into
// TMEM: a block of 128 rows and 4 scales is 32 lines of 16 bytes, line l
// holding rows l, l + 32, l + 64, l + 96, and takes 4 columns. Two
// accumulators of tn columns and the scales of every stage share the 512
// columns: with 256-column tiles they would not fit.
//   warp 0      TMA producer        warp 1  scale copies and MMAs
//   warps 2-9   epilogue, two per TMEM lane quarter (dense.cuh)
// The scales come row by row with C / 32 bytes each, at no alignment: a small
// kernel lays them out in those blocks first (x and w together, 1/32 of their
// bytes).
#include "dense.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kRows = 128, kStep = 128;
constexpr int kABytes = kRows * kStep;
constexpr int kMaxTn = 192;
constexpr int kStages = 5;
constexpr int kStageBytes = kABytes + kMaxTn * kStep;  // 40 KB
constexpr int kScaleA = 512, kScaleB = 1024;           // bytes of a stage's scales
constexpr int kScaleBytes = kScaleA + kScaleB;
constexpr int kScaleCols = 12;                         // TMEM columns of a stage's scales
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kNumBars = 2 * kStages + 5;
constexpr int kSmem = 1024 + kStages * (kStageBytes + kScaleBytes) + kNumBars * 8 + 16;
constexpr int kTmemCols = 512;
static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
static_assert(2 * kMaxTn + kStages * kScaleCols <= kTmemCols, "TMEM columns");

struct Mx8Args {
  DenseEpi e;
  int64_t part_stride;
  const uint8_t *sa, *sb;  // scale blocks: [m_tiles][num_kb][512], [n_tiles][num_kb][1024]
  int m_tiles, n_tiles, splits, num_kb, tn, pairs;
  uint32_t idesc;
  uint32_t *status;
  unsigned long long timeout_ns;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"((uint64_t)src), "r"(bytes), "r"(bar)
      : "memory");
}

// 512 bytes (32 lines of 16) to 4 TMEM columns of all four lane quarters: rows
// unswizzled, groups of 8 lines 128 bytes apart.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t saddr) {
  const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) |
                        ((uint64_t)1 << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
               : "memory");
}

__device__ __forceinline__ void umma_mx8(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                         uint32_t sa, uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}

struct Unit {
  int m, n, s, k_lo, k_hi;
};
__device__ __forceinline__ Unit unit_of(int u, const Mx8Args &a) {
  Unit w;
  const int tiles = a.m_tiles * a.n_tiles;
  w.s = u / tiles;
  const int t = u - w.s * tiles;
  w.m = t / a.n_tiles;
  w.n = t - w.m * a.n_tiles;
  w.k_lo = (int)((int64_t)a.num_kb * w.s / a.splits);
  w.k_hi = (int)((int64_t)a.num_kb * (w.s + 1) / a.splits);
  return w;
}

template <int EPI>
__global__ void __launch_bounds__(kThreads, 1)
    dense_mx8_kernel(const __grid_constant__ CUtensorMap map_a,
                     const __grid_constant__ CUtensorMap map_b,
                     const __grid_constant__ Mx8Args args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kStages * (kStageBytes + kScaleBytes));
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
  volatile int *s_abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const uint32_t stage0 = smem_u32(smem), full0 = smem_u32(bars);
  const uint32_t scale0 = stage0 + kStages * kStageBytes;
  auto full_bar = [&](int s) { return full0 + 8u * s; };
  auto empty_bar = [&](int s) { return full0 + 8u * (kStages + s); };
  auto tfull_bar = [&](int b) { return full0 + 8u * (2 * kStages + b); };
  auto tempty_bar = [&](int b) { return full0 + 8u * (2 * kStages + 2 + b); };
  const uint32_t drain_bar = full0 + 8u * (2 * kStages + 4);
  auto a_addr = [&](int s) { return stage0 + (uint32_t)(s * kStageBytes); };
  auto b_addr = [&](int s) { return stage0 + (uint32_t)(s * kStageBytes + kABytes); };
  auto scale_addr = [&](int s) { return scale0 + (uint32_t)(s * kScaleBytes); };

  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int total = args.m_tiles * args.n_tiles * args.splits;
  const int tn = args.tn;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    prefetch_tmap(&map_a);
    prefetch_tmap(&map_b);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_launch_dependents();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = (uint32_t)uniform((int)*tmem_slot);

  if (warp == 0) {
    const uint32_t sb_bytes = tn > 128 ? 1024u : 512u;
    const uint32_t tx = (uint32_t)(kABytes + tn * kStep + kScaleA) + sb_bytes;
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
      const Unit w = unit_of(u, args);
      for (int kb = w.k_lo; kb < w.k_hi; ++kb) {
        ok = wait_bounded(empty_bar(stage), phase ^ 1u, s_abort, args.status, args.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t fb = full_bar(stage);
          mbar_arrive_expect_tx(fb, tx);
          tma_load_2d(a_addr(stage), &map_a, fb, kb * kStep, w.m * kRows);
          if (args.pairs)
            tma_load_3d(b_addr(stage), &map_b, fb, kb * kStep, 0, w.n * tn / 2);
          else
            tma_load_2d(b_addr(stage), &map_b, fb, kb * kStep, w.n * tn);
          bulk_load(scale_addr(stage), args.sa + ((int64_t)w.m * args.num_kb + kb) * kScaleA,
                    kScaleA, fb);
          bulk_load(scale_addr(stage) + kScaleA,
                    args.sb + ((int64_t)w.n * args.num_kb + kb) * kScaleB, sb_bytes, fb);
        }
        issued = issued < (uint32_t)kStages ? issued + 1 : (uint32_t)kStages;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      for (uint32_t i = 0; i < issued; ++i) {
        int s = stage - 1 - (int)i;
        uint32_t ph = phase;
        if (s < 0) {
          s += kStages;
          ph ^= 1u;
        }
        wait_drain(full_bar(s), ph, 100000000ull);
      }
    }
  } else if (warp == 1) {
    int stage = 0, local = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < total; u += gridDim.x, ++local) {
      const Unit w = unit_of(u, args);
      const int acc = local & 1;
      ok = wait_bounded(tempty_bar(acc), ((uint32_t)(local >> 1) & 1u) ^ 1u, s_abort, args.status,
                        args.timeout_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kMaxTn);
      for (int kb = w.k_lo; kb < w.k_hi; ++kb) {
        ok = wait_bounded(full_bar(stage), phase, s_abort, args.status, args.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // the scales' columns belong to the stage: the MMAs that read them
        // last were complete before the stage was filled again
        const uint32_t sfa = tmem_base + 2u * kMaxTn + (uint32_t)(stage * kScaleCols);
        const uint32_t sfb = sfa + 4u;
        const uint64_t ad = sw128_desc(a_addr(stage)), bd = sw128_desc(b_addr(stage));
        if (elect_one()) {
          copy_scales(sfa, scale_addr(stage));
          copy_scales(sfb, scale_addr(stage) + kScaleA);
          if (tn > 128) copy_scales(sfb + 4u, scale_addr(stage) + kScaleA + 512u);
#pragma unroll
          for (uint32_t kk = 0; kk < 4; ++kk)  // the kk-th byte of each scale word
            umma_mx8(d_tmem, ad + 2u * kk, bd + 2u * kk, args.idesc | (kk << 4) | (kk << 29), sfa,
                     sfb, kb != w.k_lo || kk != 0);
          umma_commit(empty_bar(stage));
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok && elect_one()) umma_commit(tfull_bar(acc));
      __syncwarp();
    }
    if (elect_one()) umma_commit(drain_bar);
    __syncwarp();
    wait_drain(drain_bar, 0, 100000000ull);
  } else {
    constexpr int W = EPI == EPI_GATED_MX ? 64 : 32;
    const int q = warp & 3, part = (warp - 2) >> 2;
    int local = 0;
    for (int u = blockIdx.x; u < total; u += gridDim.x, ++local) {
      const Unit w = unit_of(u, args);
      const int acc = local & 1;
      const int64_t row = (int64_t)w.m * kRows + q * 32 + lane;
      const int c0 = w.n * tn;
      const bool live = row < args.e.rows;
      Addend<EPI, W> add;  // of the first columns, while the last products run
      if (live && c0 + part * W < args.e.cols) fetch_addend<EPI, W>(args.e, row, c0 + part * W, add);
      if (!wait_bounded(tfull_bar(acc), (uint32_t)(local >> 1) & 1u, s_abort, args.status,
                        args.timeout_ns))
        break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kMaxTn);
      DenseEpi e = args.e;
      if constexpr (EPI == EPI_PARTIAL) e.out = static_cast<float *>(e.out) + w.s * args.part_stride;
#pragma unroll 1
      for (int c = part * W; c < tn; c += 2 * W) {
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
          if (c + 2 * W < tn && c0 + c + 2 * W < args.e.cols)
            fetch_addend<EPI, W>(e, row, c0 + c + 2 * W, add);
          dense_epilogue<EPI, W>(e, row, c0 + c, v, now);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(acc));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// Scale bytes [rows, G] to the blocks of the tiles: one thread per row of a
// tile and K step, four bytes each. Rows and groups that do not exist get 1
// (their codes are zeros).
struct Layout {
  const uint8_t *src;
  uint8_t *dst;
  int64_t rows;
  int tiles, tile_rows, block;  // rows of a tile, bytes of its block
  int pairs;                    // tile rows 2i, 2i + 1 are rows i and i + rows / 2
};
__global__ void __launch_bounds__(256)
mx8_layout_kernel(const Layout a, const Layout b, int G, int num_kb) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t na = (int64_t)a.tiles * a.tile_rows * num_kb;
  const int64_t nb = (int64_t)b.tiles * b.tile_rows * num_kb;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < na + nb;
       i += (int64_t)gridDim.x * blockDim.x) {
    const Layout &l = i < na ? a : b;
    const int64_t j = i < na ? i : i - na;
    const int64_t row = j / num_kb;
    const int kb = (int)(j - row * num_kb);
    const int64_t tile = row / l.tile_rows;
    const int r = (int)(row - tile * l.tile_rows);
    uint32_t word = 0x7f7f7f7fu;
    if (row < l.rows) {
      const int64_t from = l.pairs ? (row >> 1) + (row & 1) * (l.rows / 2) : row;
      const uint8_t *p = l.src + from * G + kb * 4;
      const int left = G - kb * 4;
      word = 0;
#pragma unroll
      for (int t = 0; t < 4; ++t) word |= (uint32_t)(t < left ? p[t] : 0x7f) << (8 * t);
    }
    *reinterpret_cast<uint32_t *>(l.dst + (tile * num_kb + kb) * l.block + (r >> 7) * 512 +
                                  (r & 31) * 16 + ((r >> 5) & 3) * 4) = word;
  }
}

bool map_codes(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)cols};
  cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_code_pairs(CUtensorMap *m, const void *base, int64_t I, int64_t cols, int box_pairs) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, 2, (cuuint64_t)I};
  cuuint64_t strides[2] = {(cuuint64_t)(I * cols), (cuuint64_t)cols};
  cuuint32_t box[3] = {128, 2, (cuuint32_t)box_pairs};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int EPI>
cudaError_t launch_mx8(const CUtensorMap &ma, const CUtensorMap &mb, const Mx8Args &a,
                       cudaStream_t s) {
  auto kern = dense_mx8_kernel<EPI>;
  static PerDeviceOnce once;
  const cudaError_t err = once.run([&] {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    return e != cudaSuccess ? e : uniform_carveout(kern);
  });
  if (err != cudaSuccess) return err;
  const int64_t units = (int64_t)a.m_tiles * a.n_tiles * a.splits;
  const int64_t sms = device_sm_count();
  return launch_dependent(kern, dim3((unsigned)(units < sms ? units : sms)), dim3(kThreads), kSmem,
                          s, ma, mb, a);
}

}  // namespace

size_t mx8_scale_blocks(const DensePlan &plan, int64_t K) {
  const int64_t num_kb = (K + kStep - 1) / kStep;
  return (size_t)num_kb * ((size_t)plan.m_tiles * kScaleA + (size_t)plan.n_tiles * kScaleB);
}

cudaError_t launch_dense_mx8(const DenseProduct &p, const DensePlan &plan, uint8_t *blocks,
                             float *partial, int32_t *status, cudaStream_t s) {
  CUtensorMap ma, mb;
  const int tn = plan.tn;
  if (!map_codes(&ma, p.a.p, p.M, p.K, kRows) ||
      !(p.b.pairs ? map_code_pairs(&mb, p.b.p, p.N / 2, p.K, tn / 2)
                  : map_codes(&mb, p.b.p, p.N, p.K, tn)))
    return cudaErrorInvalidValue;
  Mx8Args a{};
  a.e = p.epi;
  a.m_tiles = plan.m_tiles;
  a.n_tiles = plan.n_tiles;
  a.splits = plan.splits;
  a.num_kb = (int)((p.K + kStep - 1) / kStep);
  a.tn = tn;
  a.pairs = p.b.pairs;
  a.idesc = ((uint32_t)(tn >> 3) << 17) | (1u << 23) | ((uint32_t)(kRows >> 4) << 24);
  a.status = reinterpret_cast<uint32_t *>(status);
  a.timeout_ns = kWaitTimeoutNs;
  uint8_t *sb = blocks + (size_t)plan.m_tiles * a.num_kb * kScaleA;
  a.sa = blocks;
  a.sb = sb;
  const Layout la{p.a.scales, blocks, p.M, plan.m_tiles, kRows, kScaleA, 0};
  const Layout lb{p.b.scales, sb, p.N, plan.n_tiles, tn, kScaleB, p.b.pairs};
  const int64_t threads = ((int64_t)plan.m_tiles * kRows + (int64_t)plan.n_tiles * tn) * a.num_kb;
  int64_t grid = (threads + 255) / 256;
  const int64_t cap = (int64_t)device_sm_count() * 8;
  if (grid > cap) grid = cap;
  cudaError_t err = launch_dependent(mx8_layout_kernel, dim3((unsigned)grid), dim3(256), 0, s, la,
                                     lb, (int)(p.K / 32), a.num_kb);
  if (err != cudaSuccess) return err;
  if (plan.splits > 1) {
    a.e.out = partial;
    a.part_stride = p.M * p.N;
    err = launch_mx8<EPI_PARTIAL>(ma, mb, a, s);
    return err != cudaSuccess ? err : launch_dense_join(p, plan, partial, s);
  }
  switch (p.kind) {
    case EPI_GATED: return launch_mx8<EPI_GATED>(ma, mb, a, s);
    case EPI_GATED_MX: return launch_mx8<EPI_GATED_MX>(ma, mb, a, s);
    default: return launch_mx8<EPI_LINEAR>(ma, mb, a, s);
  }
}

}  // namespace moe
