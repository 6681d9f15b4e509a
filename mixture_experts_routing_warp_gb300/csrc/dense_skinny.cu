// dense_skinny.cu -- moe_linear and moe_gated_linear, and the sums that their
// gradients compute again, for a handful of rows (decode): y[t, r] = sum_k
// x[t, k] w[r, k] with every weight read once.
//
// Bound by HBM for the weights, and at a few MB by latency: one launch, no
// partial sums through memory. A CTA takes 16 rows of w (gated: 8 gate and
// their 8 up rows) over the whole of K, its warps a slice of K each, and adds
// the warps' sums in shared memory in a fixed order. Weights go from global
// memory straight into the fragments of mma.sync m16n8k16: a lane loads 16
// bytes of rows g and g + 8, 8 consecutive k, which serve as the k slots of
// two MMAs; x's fragment takes the same 8 k of its token, so the products pair
// up although the slots are not in order. tcgen05 has no use here: its tiles
// would wait for the same bytes, and need their sums split over K to reach all
// SMs, with a second launch (2880 x 2880, one row: 11.2 us that way, 4.2 here).
// Before the wait for the preceding kernel the CTA asks L2 for its weights:
// they come from HBM while that kernel ends, and L2 is coherent with whatever
// it still writes.
#include "dense.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;  // of w per CTA
constexpr int kAhead = 64;  // lines of each weight row that are asked for ahead

__device__ __forceinline__ uint4 load_weights(const uint16_t *p, bool live) {
  uint4 q = make_uint4(0u, 0u, 0u, 0u);
  if (live)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                 : "l"(p));
  return q;
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
  const uint16_t *x, *w;
  int n, rows, K;  // rows of w; gated: of h (pairs)
  int packed;
  DenseEpi e;
};

// The CTA's weight row j of 16: gated, gates first, then their ups.
template <bool PAIRS>
__device__ __forceinline__ int64_t weight_row(const SkinnyArgs &a, int j, bool &live) {
  if constexpr (!PAIRS) {
    const int64_t r = (int64_t)blockIdx.x * kRows + j;
    live = r < a.rows;
    return r;
  }
  const int64_t i = (int64_t)blockIdx.x * (kRows / 2) + (j & 7);
  live = i < a.rows;
  return a.packed ? i + (j >> 3) * (int64_t)a.rows : 2 * i + (j >> 3);
}

// NB blocks of 8 tokens; CTAS per SM that registers are left for.
template <int EPI, bool HALF, int NB, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS)
    dense_skinny_kernel(const __grid_constant__ SkinnyArgs a) {
  constexpr bool PAIRS = EPI == EPI_GATED || EPI == EPI_DGATED;
  __shared__ float s_d[EPI == EPI_DACT ? NB * 8 : 1][kRows + 1];
  constexpr int U = NB == 4 ? 2 : 4;  // blocks of 32 k in flight per warp
  __shared__ float s_sum[kWarps][NB][4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  {
    const int lines = (a.K * 2 + 127) / 128;
    const int most = lines < kAhead ? lines : kAhead;
    for (int i = threadIdx.x; i < kRows * most; i += kThreads) {
      bool live;
      const int64_t r = weight_row<PAIRS>(a, i / most, live);
      const char *p = reinterpret_cast<const char *>(a.w + r * a.K) + (i % most) * 128;
      if (live) asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
    }
  }
  pdl_launch_dependents();
  pdl_wait();

  bool live0, live1;
  const uint16_t *w0 = a.w + weight_row<PAIRS>(a, g, live0) * a.K;
  const uint16_t *w1 = a.w + weight_row<PAIRS>(a, g + 8, live1) * a.K;
  const int blocks = (a.K + 31) / 32;
  const int b_lo = blocks * warp / kWarps, b_hi = blocks * (warp + 1) / kWarps;
  float acc[NB][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;
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
          xq[u][nb] = __ldg(reinterpret_cast<const uint4 *>(a.x + (int64_t)tok * a.K + k));
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
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_sum[warp][nb][i][lane] = acc[nb][i];
  __syncthreads();

  // the sum of CTA row j and token tok over the warps: register (tok & 1) + 2
  // (j >= 8) of lane (j & 7) * 4 + (tok & 7) / 2
  auto total = [&](int j, int tok) {
    float f = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      f += s_sum[w][tok >> 3][(tok & 1) + 2 * (j >> 3)][(j & 7) * 4 + ((tok & 7) >> 1)];
    return f;
  };
  const DenseEpi &e = a.e;
  constexpr int kOut = PAIRS ? kRows / 2 : kRows;  // results per token
  for (int i = threadIdx.x; i < kOut * NB * 8; i += kThreads) {
    const int j = i % kOut, tok = i / kOut;
    const int64_t c = (int64_t)blockIdx.x * kOut + j;
    const bool live = tok < a.n && c < a.rows;
    const int64_t at = (int64_t)tok * a.rows + c;
    uint16_t *out = static_cast<uint16_t *>(e.out) + at;
    auto add = [&] { return from16(static_cast<const uint16_t *>(e.add)[at], HALF); };
    if constexpr (PAIRS) {
      if (!live) continue;
      const float g = total(j, tok), u = total(j + 8, tok);
      if constexpr (EPI == EPI_GATED) {
        *out = to16(gated(g, u, e.gate), HALF);
      } else {  // in w13's row order
        float d_g, d_u;
        gated_backward(g, u, add(), e.gate, d_g, d_u);
        uint16_t *d = static_cast<uint16_t *>(e.out) + (int64_t)tok * 2 * a.rows +
                      (a.packed ? c : 2 * c);
        d[0] = to16(d_g, HALF);
        d[a.packed ? a.rows : 1] = to16(d_u, HALF);
      }
    } else {
      float v = 0.f;
      if (live) {
        v = total(j, tok);
        if (e.bias) v += from16(static_cast<const uint16_t *>(e.bias)[c], HALF);
        if constexpr (EPI == EPI_DACT) {
          v = add() * linear_slope(v, e.act);
        } else {
          if (e.act != MOE_LINEAR_NONE) v = linear_act(v, e.act);
          if (e.add) v += add();
        }
        *out = to16(v, HALF);
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
template <int EPI, bool HALF, int NB>
cudaError_t launch_nb(const SkinnyArgs &a, cudaStream_t s) {
  constexpr bool PAIRS = EPI == EPI_GATED || EPI == EPI_DGATED;
  constexpr int kFew = NB == 4 ? 2 : 3, per = PAIRS ? kRows / 2 : kRows;
  const int ctas = (a.rows + per - 1) / per;
  return launch_dependent(ctas <= kFew * device_sm_count()
                              ? dense_skinny_kernel<EPI, HALF, NB, kFew>
                              : dense_skinny_kernel<EPI, HALF, NB, kFew + 1>,
                          dim3((unsigned)ctas), dim3(kThreads), 0, s, a);
}

template <int EPI, bool HALF>
cudaError_t launch_n(const SkinnyArgs &a, cudaStream_t s) {
  if (a.n <= 8) return launch_nb<EPI, HALF, 1>(a, s);
  return a.n <= 16 ? launch_nb<EPI, HALF, 2>(a, s) : launch_nb<EPI, HALF, 4>(a, s);
}

template <int EPI>
cudaError_t launch_epi(const SkinnyArgs &a, cudaStream_t s) {
  return a.e.half ? launch_n<EPI, true>(a, s) : launch_n<EPI, false>(a, s);
}

}  // namespace

// Up to 16 rows always, up to 32 where the weights are few: a CTA reads all of
// x for its 16 weight rows, and at 32 rows that is twice the weights' bytes
// (from L2). 2880 x 2880: 32 rows 7.9 us for 10.1 on the tensor tiles, 2880 x
// 5760 gated 10.3 for 11.6; 8192 x 8192: 16 rows 26.5 for 28.1, 32 rows 47 for 29.
bool dense_skinny(int64_t n, int64_t out, int64_t in) {
  return n <= 16 || (n <= 32 && out * in <= (1 << 24));
}

cudaError_t launch_dense_skinny(const DenseProduct &p, cudaStream_t s) {
  const bool pairs = p.kind == EPI_GATED || p.kind == EPI_DGATED;
  const SkinnyArgs a{static_cast<const uint16_t *>(p.a.p), static_cast<const uint16_t *>(p.b.p),
                     (int)p.M, (int)(pairs ? p.N / 2 : p.N), (int)p.K, p.b.pairs, p.epi};
  switch (p.kind) {
    case EPI_GATED: return launch_epi<EPI_GATED>(a, s);
    case EPI_DGATED: return launch_epi<EPI_DGATED>(a, s);
    case EPI_DACT: return launch_epi<EPI_DACT>(a, s);
    default: return launch_epi<EPI_LINEAR>(a, s);
  }
}

}  // namespace moe
