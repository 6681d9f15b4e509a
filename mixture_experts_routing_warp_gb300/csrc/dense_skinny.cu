// dense_skinny.cu -- moe_linear and moe_gated_linear, and the sums that their
// gradients compute again, for a handful of rows (decode): y[t, r] = sum_k
// x[t, k] w[r, k] with every weight read once.
//
// Bound by HBM for the weights, and at a few MB by latency: one launch, no
// partial sums through memory. A CTA takes 16 rows of w (gated: 8 gate and
// their 8 up rows; 8-bit results: four times that, a group of 32) over the
// whole of K, its warps a slice of K each, and adds the warps' sums in shared
// memory in a fixed order. Weights go from global memory straight into the
// fragments of mma.sync m16n8k16: a lane loads 16 bytes of rows g and g + 8, 8
// consecutive k, which serve as the k slots of two MMAs; x's fragment takes
// the same 8 k of its token, so the products pair up although the slots are
// not in order. tcgen05 has no use here: its tiles would wait for the same
// bytes, and need their sums split over K to reach all SMs, with a second
// launch (2880 x 2880, one row: 11.2 us that way, 4.2 here). From HBM, over inputs that
// together exceed twice the L2, one row takes 5.5 us and 2880 x 5760 gated 7.3 (their bytes alone
// 2.5 and 4.9); the other figures here are of weights in L2.
//
// MXFP8: a lane loads the 8 codes of its k's in a group of 32, as fp16 (exact);
// the two MMAs of a group start from zero, and their sums enter the total
// times both scales, which the CTA has laid out as floats in shared memory (with
// the bytes fetched and converted group by group 155 instructions for 84, and
// 2880 x 2880 8.7 us for 6.0).
//
// Before the wait for the preceding kernel the CTA asks L2 for its weights:
// they come from HBM while that kernel ends, and L2 is coherent with whatever
// it still writes.
#include <type_traits>

#include "dense.cuh"

namespace moe {
namespace {

enum { IN_BF16 = 0, IN_FP16 = 1, IN_MX8 = 2 };

constexpr int kRows = 16;    // of w per m tile
constexpr int kMaxGroups = 256;  // MXFP8: rows of up to 8192 values
constexpr int kAhead = 64;   // lines of each weight row that are asked for ahead

// m tiles of a CTA and the K slices of each: a warp per tile and slice.
constexpr int m_tiles(int epi) { return epi == EPI_GATED_MX ? 4 : 1; }
constexpr int k_slices(int epi) { return epi == EPI_GATED_MX ? 4 : 8; }
constexpr int skinny_threads(int epi) { return m_tiles(epi) * k_slices(epi) * 32; }

__device__ __forceinline__ uint4 load_weights(const uint16_t *p, bool live) {
  uint4 q = make_uint4(0u, 0u, 0u, 0u);
  if (live)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                 : "l"(p));
  return q;
}
__device__ __forceinline__ uint2 load_codes(const uint8_t *p, bool live) {
  uint2 q = make_uint2(0u, 0u);
  if (live)
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "l"(p));
  return q;
}

// Four E4M3 codes as two pairs of fp16.
__device__ __forceinline__ void codes_to_half(uint32_t q, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(q));
}

// 2^(b - 127); 255 is NaN
__device__ __forceinline__ float scale_of(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7fc00000u : b << 23);
}

// The smaller and the larger of two scales, NaN where either is.
__device__ __forceinline__ float lesser(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float greater(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// part s t + acc for a group's sum, 0 or 2^-18 to 2^22.6, and two scales, powers of two from
// 2^-127 to 2^127. s t first is right wherever it is in fp32's range, as it is for bytes from
// kNearLo to kNearHi: then nothing is rounded before acc is added. Else (WIDE) the lesser
// scale goes first: that is exact (part is a multiple of 2^-18, and 2^-145 is in fp32),
// and too large only where the result is. Four instructions more per group and
// token pair: 16 rows, 2880 x 2880 9.2 us for 8.7.
constexpr uint32_t kNearLo = 53, kNearHi = 190;  // 2^-74 and 2^63: products from 2^-148 to 2^126
template <bool WIDE>
__device__ __forceinline__ float scaled(float part, float s, float t, float acc) {
  if constexpr (WIDE) return fmaf(part * lesser(s, t), greater(s, t), acc);
  else return fmaf(part, s * t, acc);
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1, bool half) {
  if (half)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct SkinnyArgs {
  const void *x, *w;
  const uint8_t *x_scales, *w_scales;
  int n, rows, K;  // rows of w; gated: of h (pairs)
  int packed;
  DenseEpi e;
};

// The CTA's weight row j of m tile mt: gated, gates first, then their ups.
template <int EPI>
__device__ __forceinline__ int64_t weight_row(const SkinnyArgs &a, int mt, int j, bool &live) {
  const int64_t tile = (int64_t)blockIdx.x * m_tiles(EPI) + mt;
  if constexpr (EPI == EPI_LINEAR || EPI == EPI_DACT) {
    const int64_t r = tile * kRows + j;
    live = r < a.rows;
    return r;
  }
  const int64_t i = tile * (kRows / 2) + (j & 7);
  live = i < a.rows;
  return a.packed ? i + (j >> 3) * (int64_t)a.rows : 2 * i + (j >> 3);
}

// The warp's sums over its slice of K, 16-bit operands.
template <int EPI, bool HALF, int NB>
__device__ __forceinline__ void sum16(const SkinnyArgs &a, int mt, int slice, int lane,
                                      float (&acc)[NB][4]) {
  constexpr int U = NB == 4 ? 2 : 4;  // blocks of 32 k in flight
  const int g = lane >> 2, t = lane & 3;
  const uint16_t *x = static_cast<const uint16_t *>(a.x), *w = static_cast<const uint16_t *>(a.w);
  bool live0, live1;
  const uint16_t *w0 = w + weight_row<EPI>(a, mt, g, live0) * a.K;
  const uint16_t *w1 = w + weight_row<EPI>(a, mt, g + 8, live1) * a.K;
  const int blocks = (a.K + 31) / 32;
  const int b_lo = blocks * slice / k_slices(EPI), b_hi = blocks * (slice + 1) / k_slices(EPI);
  for (int b = b_lo; b < b_hi; b += U) {
    uint4 q0[U], q1[U], xq[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (b + u) * 32 + t * 8;
      const bool in = b + u < b_hi && k < a.K;
      q0[u] = load_weights(w0 + k, in && live0);
      q1[u] = load_weights(w1 + k, in && live1);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int tok = nb * 8 + g;
        xq[u][nb] = make_uint4(0u, 0u, 0u, 0u);
        if (in && tok < a.n)
          xq[u][nb] = __ldg(reinterpret_cast<const uint4 *>(x + (int64_t)tok * a.K + k));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        mma_16x8x16(acc[nb], q0[u].x, q1[u].x, q0[u].y, q1[u].y, xq[u][nb].x, xq[u][nb].y, HALF);
        mma_16x8x16(acc[nb], q0[u].z, q1[u].z, q0[u].w, q1[u].w, xq[u][nb].z, xq[u][nb].w, HALF);
      }
  }
}

// The same of MXFP8 operands. s_w, s_x: the scales of the CTA's weight rows and
// of the tokens, a row of `wide` each; far: this thread saw one outside [kNearLo,
// kNearHi]. A weight row that does not exist is read as row 0, a token as the last one;
// their sums go nowhere. U groups of 32 k in flight: four, and two of 9 to 16 rows at four CTAs per
// SM, whose registers hold no more (8192 x 2880, 9 rows: 10.1 us for 12.3 with spills).
template <int EPI, int NB, int U>
__device__ __forceinline__ void sum8(const SkinnyArgs &a, int mt, int slice, int lane,
                                     const float *s_w, const float *s_x, int wide, bool far,
                                     float (&acc)[NB][4]) {
  const int g = lane >> 2, t = lane & 3, G = a.K / 32;
  bool live;
  int64_t r0 = weight_row<EPI>(a, mt, g, live);
  if (!live) r0 = 0;
  int64_t r1 = weight_row<EPI>(a, mt, g + 8, live);
  if (!live) r1 = 0;
  const int lo = G * slice / k_slices(EPI), hi = G * (slice + 1) / k_slices(EPI);
  const uint8_t *w0 = static_cast<const uint8_t *>(a.w) + r0 * a.K + lo * 32 + t * 8;
  const uint8_t *w1 = static_cast<const uint8_t *>(a.w) + r1 * a.K + lo * 32 + t * 8;
  const uint8_t *x[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int tok = nb * 8 + g < a.n ? nb * 8 + g : a.n - 1;
    x[nb] = static_cast<const uint8_t *>(a.x) + (int64_t)tok * a.K + lo * 32 + t * 8;
  }
  const float *sw0 = s_w + (mt * kRows + g) * wide + lo, *sw1 = sw0 + 8 * wide;
  const float *sx = s_x + 2 * t * wide + lo;
  const int count = hi - lo;
  uint2 q0[U], q1[U], xq[U][NB];
  auto fetch = [&](int b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = b + u < count;
      q0[u] = load_codes(w0 + (b + u) * 32, in);
      q1[u] = load_codes(w1 + (b + u) * 32, in);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        xq[u][nb] = make_uint2(0u, 0u);
        if (in) xq[u][nb] = __ldg(reinterpret_cast<const uint2 *>(x[nb] + (b + u) * 32));
      }
    }
  };
  auto sum = [&](auto is_far) {
    for (int b = 0; b < count; b += U) {
      if (b > 0) fetch(b);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (b + u >= count) break;
        uint32_t a0[4], a1[4];
        codes_to_half(q0[u].x, a0[0], a0[1]);
        codes_to_half(q0[u].y, a0[2], a0[3]);
        codes_to_half(q1[u].x, a1[0], a1[1]);
        codes_to_half(q1[u].y, a1[2], a1[3]);
        const float s0 = sw0[b + u], s1 = sw1[b + u];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          uint32_t x0, x1, x2, x3;
          codes_to_half(xq[u][nb].x, x0, x1);
          codes_to_half(xq[u][nb].y, x2, x3);
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          mma_16x8x16(part, a0[0], a1[0], a0[1], a1[1], x0, x1, true);
          mma_16x8x16(part, a0[2], a1[2], a0[3], a1[3], x2, x3, true);
          const float t0 = sx[nb * 8 * wide + b + u], t1 = sx[(nb * 8 + 1) * wide + b + u];
          acc[nb][0] = scaled<decltype(is_far)::value>(part[0], s0, t0, acc[nb][0]);
          acc[nb][1] = scaled<decltype(is_far)::value>(part[1], s0, t1, acc[nb][1]);
          acc[nb][2] = scaled<decltype(is_far)::value>(part[2], s1, t0, acc[nb][2]);
          acc[nb][3] = scaled<decltype(is_far)::value>(part[3], s1, t1, acc[nb][3]);
        }
      }
    }
  };
  fetch(0);
  // the CTA's scales, with the first codes on their way
  if (__syncthreads_or(far)) sum(std::true_type{});
  else sum(std::false_type{});
}

// NB blocks of 8 tokens; CTAS per SM that registers are left for.
template <int EPI, int IN, int NB, int CTAS>
__global__ void __launch_bounds__(skinny_threads(EPI), CTAS)
    dense_skinny_kernel(const __grid_constant__ SkinnyArgs a) {
  constexpr bool PAIRS = EPI != EPI_LINEAR && EPI != EPI_DACT;
  constexpr int MT = m_tiles(EPI), KS = k_slices(EPI), kThreads = skinny_threads(EPI);
  __shared__ float s_sum[MT * KS][NB][4][32];
  __shared__ float s_d[EPI == EPI_DACT ? NB * 8 : 1][kRows + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  {
    const int64_t bytes = (int64_t)a.K * (IN == IN_MX8 ? 1 : 2);
    const int lines = (int)((bytes + 127) / 128), most = lines < kAhead ? lines : kAhead;
    for (int i = threadIdx.x; i < MT * kRows * most; i += kThreads) {
      bool live;
      const int j = i / most;
      const int64_t r = weight_row<EPI>(a, j / kRows, j % kRows, live);
      const char *p = static_cast<const char *>(a.w) + r * bytes + (i % most) * 128;
      if (live) asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
    }
  }
  pdl_launch_dependents();
  pdl_wait();

  float acc[NB][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;
  if constexpr (IN == IN_MX8) {
    extern __shared__ float s_scale[];  // [rows of the CTA and tokens][G | 1]
    const int G = a.K / 32, wide = G | 1;
    bool far = false;
    for (int r = warp; r < MT * kRows + NB * 8; r += MT * KS) {
      const int tok = r - MT * kRows;
      bool live;
      const int64_t row = weight_row<EPI>(a, r / kRows, r % kRows, live);
      const uint8_t *src = tok < 0 ? a.w_scales + row * G : a.x_scales + (int64_t)tok * G;
      if (tok >= 0) live = tok < a.n;
      for (int i = lane; i < G; i += 32) {
        const uint32_t byte = live ? __ldg(src + i) : kNearLo;
        far |= byte < kNearLo || byte > kNearHi;
        s_scale[r * wide + i] = live ? scale_of(byte) : 0.f;
      }
    }
    sum8<EPI, NB, NB == 2 && CTAS == 4 ? 2 : 4>(a, warp / KS, warp % KS, lane, s_scale, s_scale + MT * kRows * wide, wide, far,
                  acc);
  } else sum16<EPI, IN == IN_FP16, NB>(a, warp / KS, warp % KS, lane, acc);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_sum[warp][nb][i][lane] = acc[nb][i];
  __syncthreads();

  // the sum of row j of m tile mt and token tok over the warps: register
  // (tok & 1) + 2 (j >= 8) of lane (j & 7) * 4 + (tok & 7) / 2
  auto total = [&](int mt, int j, int tok) {
    float f = 0.f;
#pragma unroll
    for (int w = 0; w < KS; ++w)
      f += s_sum[mt * KS + w][tok >> 3][(tok & 1) + 2 * (j >> 3)][(j & 7) * 4 + ((tok & 7) >> 1)];
    return f;
  };
  const DenseEpi &e = a.e;
  const int half = IN == IN_MX8 ? e.half : IN == IN_FP16;
  if constexpr (EPI == EPI_GATED_MX) {
    // a warp per token, a lane per value of its group of 32
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    for (int tok = warp; tok < a.n; tok += MT * KS) {
      const int mt = lane >> 3, j = lane & 7;
      const float h = gated(total(mt, j, tok), total(mt, j + 8, tok), e.gate);
      const uint32_t b = mx8_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu));
      const int64_t at = (int64_t)tok * a.rows + c;
      e.codes[at] = (uint8_t)__nv_cvt_float_to_fp8(h * mx8_inverse(b), __NV_SATFINITE, __NV_E4M3);
      if (lane == 0) e.scales[at / 32] = (uint8_t)b;
    }
    return;
  }
  constexpr int kOut = PAIRS ? kRows / 2 : kRows;  // results per token
  for (int i = threadIdx.x; i < kOut * NB * 8; i += kThreads) {
    const int j = i % kOut, tok = i / kOut;
    const int64_t c = (int64_t)blockIdx.x * kOut + j;
    const bool live = tok < a.n && c < a.rows;
    const int64_t at = (int64_t)tok * a.rows + c;
    uint16_t *out = static_cast<uint16_t *>(e.out) + at;
    auto add = [&] { return from16(static_cast<const uint16_t *>(e.add)[at], half); };
    if constexpr (PAIRS) {
      if (!live) continue;
      const float g = total(0, j, tok), u = total(0, j + 8, tok);
      if constexpr (EPI == EPI_GATED) {
        *out = to16(gated(g, u, e.gate), half);
      } else {  // in w13's row order
        float d_g, d_u;
        gated_backward(g, u, add(), e.gate, d_g, d_u);
        uint16_t *d = static_cast<uint16_t *>(e.out) + (int64_t)tok * 2 * a.rows +
                      (a.packed ? c : 2 * c);
        d[0] = to16(d_g, half);
        d[a.packed ? a.rows : 1] = to16(d_u, half);
      }
    } else {
      float v = 0.f;
      if (live) {
        v = total(0, j, tok);
        if (e.bias) v += from16(static_cast<const uint16_t *>(e.bias)[c], half);
        if constexpr (EPI == EPI_DACT) {
          v = add() * linear_slope(v, e.act);
        } else {
          if (e.act != MOE_LINEAR_NONE) v = linear_act(v, e.act);
          if (e.add) v += add();
        }
        *out = to16(v, half);
      }
      if constexpr (EPI == EPI_DACT) s_d[tok][j] = v;
    }
  }
  if constexpr (EPI == EPI_DACT) {
    if (!e.column_part) return;
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * kRows + threadIdx.x;
    if (threadIdx.x < kRows && c < a.rows) {
      float f = 0.f;
      for (int tok = 0; tok < a.n; ++tok) f += s_d[tok][threadIdx.x];
      e.column_part[c] = f;
    }
  }
}

// More registers, and with them more loads in flight per warp, as long as the
// SMs hold all CTAs at once; else one CTA more per SM. One row, in a graph:
// 2880 x 5760 gated (360 CTAs) 5.1 us at three CTAs per SM and 6.4 at four,
// 8192 x 8192 (512) 26.8 and 20.9; 32 rows: 2880 x 2880 (180) 7.9 us at two
// and 9.5 at three, 2880 x 5760 gated 13.6 and 10.3.
template <int EPI, int IN, int NB, int CTAS>
cudaError_t launch_ctas(const SkinnyArgs &a, int ctas, cudaStream_t s) {
  auto kern = dense_skinny_kernel<EPI, IN, NB, CTAS>;
  size_t smem = 0;
  if constexpr (IN == IN_MX8) {
    constexpr int kScaleRows = m_tiles(EPI) * kRows + NB * 8;
    static PerDeviceOnce once;
    const cudaError_t err = once.run([&] {
      return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  kScaleRows * (kMaxGroups | 1) * 4);
    });
    if (err != cudaSuccess) return err;
    smem = (size_t)kScaleRows * (a.K / 32 | 1) * 4;
  }
  return launch_dependent(kern, dim3((unsigned)ctas), dim3(skinny_threads(EPI)), smem, s, a);
}
template <int EPI, int IN, int NB>
cudaError_t launch_nb(const SkinnyArgs &a, cudaStream_t s) {
  const int per = (EPI == EPI_LINEAR || EPI == EPI_DACT ? kRows : kRows / 2) * m_tiles(EPI);
  const int ctas = (a.rows + per - 1) / per;
  if constexpr (EPI == EPI_GATED_MX) {
    return launch_ctas<EPI, IN, NB, 1>(a, ctas, s);
  } else {
    constexpr int kFew = NB == 4 ? 2 : 3;
    return ctas <= kFew * device_sm_count() ? launch_ctas<EPI, IN, NB, kFew>(a, ctas, s)
                                            : launch_ctas<EPI, IN, NB, kFew + 1>(a, ctas, s);
  }
}

template <int EPI, int IN>
cudaError_t launch_n(const SkinnyArgs &a, cudaStream_t s) {
  if (a.n <= 8) return launch_nb<EPI, IN, 1>(a, s);
  if constexpr (IN != IN_MX8 && EPI != EPI_GATED_MX)
    if (a.n > 16) return launch_nb<EPI, IN, 4>(a, s);
  return launch_nb<EPI, IN, 2>(a, s);
}

template <int EPI>
cudaError_t launch_in(const SkinnyArgs &a, cudaStream_t s) {
  if constexpr (EPI != EPI_DACT && EPI != EPI_DGATED)
    if (a.x_scales) return launch_n<EPI, IN_MX8>(a, s);
  return a.e.half ? launch_n<EPI, IN_FP16>(a, s) : launch_n<EPI, IN_BF16>(a, s);
}

}  // namespace

// Up to 16 rows, 16-bit ones with 16-bit results up to 32 where the weights are
// few: a CTA reads all of x for its 16 weight rows, and at 32 rows that is
// twice the weights' bytes (from L2). 2880 x 2880: 32 rows 7.9 us for 10.1 on the
// tensor tiles, 2880 x 5760 gated 10.3 for 11.6; 8192 x 8192: 16 rows 26.5 for
// 28.1, 32 rows 47 for 29. MXFP8 is bound by issue (84 instructions for 512
// codes): 2880 x 2880: 1 / 8 / 16 rows 6.0 / 6.5 / 8.7 us for 14 / 12.7 / 13 on the
// tensor tiles; 8192 x 8192: 20.8 / 23.9 / 32.3 for 28.9 / 24.6 / 22.6.
bool dense_skinny(int64_t n, int64_t out, int64_t in, int kind, bool mx) {
  if (mx) return in <= 32 * kMaxGroups && (n <= 8 || (n <= 16 && out * in <= (1 << 25)));
  if (kind == EPI_GATED_MX) return n <= 16;
  return n <= 16 || (n <= 32 && out * in <= (1 << 24));
}

cudaError_t launch_dense_skinny(const DenseProduct &p, cudaStream_t s) {
  const bool pairs = p.kind != EPI_LINEAR && p.kind != EPI_DACT;
  const SkinnyArgs a{p.a.p, p.b.p, p.a.scales, p.b.scales, (int)p.M,
                     (int)(pairs ? p.N / 2 : p.N), (int)p.K, p.b.pairs, p.epi};
  switch (p.kind) {
    case EPI_GATED: return launch_in<EPI_GATED>(a, s);
    case EPI_GATED_MX: return launch_in<EPI_GATED_MX>(a, s);
    case EPI_DGATED: return launch_in<EPI_DGATED>(a, s);
    case EPI_DACT: return launch_in<EPI_DACT>(a, s);
    default: return launch_in<EPI_LINEAR>(a, s);
  }
}

}  // namespace moe
