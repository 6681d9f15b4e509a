// permute.cu -- token rows to expert-sorted order and back, with the gate
// weights applied, and the gradients (moe_dispatch, moe_combine_weighted and
// their backward passes), plus the gradient of the gate weights to the logits
// (moe_route_backward).
//
// With p(t,j) = row_sorted[t*k + j] (-1: the slot is dropped):
//   dispatch           x_sorted[p(t,j)] = x[t]
//   dispatch backward  dx[t]            = sum_j d_sorted[p(t,j)]
//   combine            out[t]           = sum_j w[t,j] * y_sorted[p(t,j)]
//   combine backward   d_sorted[p(t,j)] = w[t,j] * d_out[t]
//                      dw[t,j]          = <d_out[t], y_sorted[p(t,j)]>
// All of them move rows and compute next to nothing: bound by HBM. The work
// is token-major, so that the token-side row crosses HBM once whatever k is,
// and every sum runs in slot order in fp32: no atomics, so the bits of a
// result depend on its inputs only.
#include "moe_internal.cuh"

#include <cuda_fp16.h>

#include <type_traits>

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxThreads = 256;
constexpr int kMaxRowThreads = 512;

template <int B>
struct Vec;
template <>
struct Vec<16> { using type = uint4; };
template <>
struct Vec<4> { using type = uint32_t; };
template <>
struct Vec<2> { using type = uint16_t; };

template <int B>
__device__ __forceinline__ typename Vec<B>::type vec_zero() {
  typename Vec<B>::type z;
  memset(&z, 0, sizeof z);
  return z;
}

// The B / sizeof(T) elements of a vector as floats, and back (rounded once,
// to nearest even); 16-bit types by pairs, one conversion instruction each.
template <typename T, int B>
__device__ __forceinline__ void unpack(typename Vec<B>::type v, float *f) {
  if constexpr (sizeof(T) == 4) {
    memcpy(f, &v, B);
  } else if constexpr (B == 2) {
    T e;
    memcpy(&e, &v, 2);
    f[0] = (float)e;
  } else {
    uint32_t w[B / 4];
    memcpy(w, &v, B);
#pragma unroll
    for (int i = 0; i < B / 4; ++i) {
      if constexpr (std::is_same_v<T, __half>) {
        __half2 h;
        memcpy(&h, &w[i], 4);
        const float2 d = __half22float2(h);
        f[2 * i] = d.x;
        f[2 * i + 1] = d.y;
      } else {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
}

template <typename T, int B>
__device__ __forceinline__ typename Vec<B>::type pack(const float *f) {
  typename Vec<B>::type v;
  if constexpr (sizeof(T) == 4) {
    memcpy(&v, f, B);
  } else if constexpr (B == 2) {
    const T e = (T)f[0];
    memcpy(&v, &e, 2);
  } else {
    uint32_t w[B / 4];
#pragma unroll
    for (int i = 0; i < B / 4; ++i) {
      if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        memcpy(&w[i], &h, 4);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        memcpy(&w[i], &h, 4);
      }
    }
    memcpy(&v, w, B);
  }
  return v;
}

// Positions (-1: dropped) and weights (1 where w is null) of the slots f ..
// f + 3 as far as `left` of them exist: all loads before their first use, so
// that the rows' loads wait for one latency and not for four.
__device__ __forceinline__ void load_slots(const int32_t *row_sorted, const void *w, int w_dtype,
                                           int64_t f, int left, int64_t N, int64_t *p, float *wj) {
  int32_t at[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) at[j] = j < left ? __ldg(row_sorted + f + j) : -1;
  if (!w) {
#pragma unroll
    for (int j = 0; j < 4; ++j) wj[j] = 1.f;
  } else if (w_dtype == MOE_FP32) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      wj[j] = j < left ? __ldg(static_cast<const float *>(w) + f + j) : 0.f;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      wj[j] = j < left ? bf16_bits_to_float(__ldg(static_cast<const uint16_t *>(w) + f + j)) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = at[j] >= 0 && at[j] < N ? at[j] : -1;
}

// How a kernel's CTA covers rows: `lanes` threads (a power of two) per token's
// row, U vectors each at a time. The whole row is in flight at once where
// 3 * 256 vectors hold it: one row's bytes, contiguous in HBM, are then read
// and written together (the dispatch of 8192 tokens, H 2880, k 4: 41.8 us with
// rows in pieces of 64 vectors by different CTAs, 37.0 us so).
struct RowMap {
  int lanes, per_cta, vpr;  // threads per row, rows per CTA, vectors per row
};

// Zeros for the rows of no kept slot, [*n_kept, N), dealt out like tokens.
template <int B>
__device__ __forceinline__ void zero_tail(void *dst, const int32_t *n_kept, int64_t N,
                                          const RowMap &m, int64_t first, int lane) {
  if (!n_kept) return;
  using V = typename Vec<B>::type;
  const int64_t kept = max(__ldg(n_kept), 0);
  for (int64_t r = kept + first; r < N; r += (int64_t)gridDim.x * m.per_cta)
    for (int c = lane; c < m.vpr; c += m.lanes) static_cast<V *>(dst)[r * m.vpr + c] = vec_zero<B>();
}

template <int B, int U>
__global__ void __launch_bounds__(kMaxThreads)
dispatch_kernel(const void *x, const int32_t *row_sorted, const int32_t *n_kept, int64_t n, int k,
                RowMap m, void *x_sorted) {
  using V = typename Vec<B>::type;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & (m.lanes - 1);
  const int64_t N = n * k, t = (int64_t)blockIdx.x * m.per_cta + threadIdx.x / m.lanes;
  if (t < n)
    for (int c0 = lane; c0 < m.vpr; c0 += U * m.lanes) {
      V v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * m.lanes < m.vpr) v[u] = static_cast<const V *>(x)[t * m.vpr + c0 + u * m.lanes];
      for (int j0 = 0; j0 < k; j0 += 4) {
        int64_t p[4];
        float one[4];
        load_slots(row_sorted, nullptr, MOE_FP32, t * k + j0, k - j0, N, p, one);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (p[j] >= 0 && c0 + u * m.lanes < m.vpr)
              static_cast<V *>(x_sorted)[p[j] * m.vpr + c0 + u * m.lanes] = v[u];
      }
    }
  zero_tail<B>(x_sorted, n_kept, N, m, t, lane);
}

// One vector per thread and row, four rows in flight; blockDim.x threads along
// the row, blockDim.y tokens. `w` null: all weights 1 (the dispatch's backward
// pass). One vector a thread keeps the kernel at 40 registers and the SM full:
// three vectors a thread measured 98 us where this takes 70 (16384 tokens,
// H 2880, k 4). The sums leave by streaming stores (74 us without).
template <typename T, int B>
__global__ void __launch_bounds__(kMaxRowThreads, 3)
combine_weighted_kernel(const void *y_sorted, const int32_t *row_sorted, const void *w,
                        int w_dtype, int64_t n, int k, int vpr, void *out) {
  using V = typename Vec<B>::type;
  constexpr int EPV = B / sizeof(T);
  pdl_wait();
  pdl_launch_dependents();
  const int64_t N = n * k, t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= n) return;
  for (int c = threadIdx.x; c < vpr; c += blockDim.x) {
    float acc[EPV] = {};
    for (int j0 = 0; j0 < k; j0 += 4) {
      V v[4];
      int64_t p[4];
      float wj[4];
      load_slots(row_sorted, w, w_dtype, t * k + j0, k - j0, N, p, wj);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = p[j] >= 0 ? __ldcs(static_cast<const V *>(y_sorted) + p[j] * vpr + c)
                         : vec_zero<B>();
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (p[j] >= 0) {
          float f[EPV];
          unpack<T, B>(v[j], f);
#pragma unroll
          for (int i = 0; i < EPV; ++i) acc[i] = fmaf(wj[j], f[i], acc[i]);
        }
    }
    __stcs(static_cast<V *>(out) + t * vpr + c, pack<T, B>(acc));
  }
}

// A row's threads read their share of d_out[t] once, write the k scaled
// copies and add up the k dot products with the sorted rows; those are joined
// over lanes, then over the row's warps. K: 4, or 8 where k > 4. The register
// limits keep five CTAs of 128 threads on an SM (K = 4, U = 3: 67.5 us for
// 8192 tokens, H 2880; 72.8 with the compiler's own 127 registers).
template <typename T, int B, int U, int K>
__global__ void __maxnreg__(K == 4 ? (U == 3 ? 96 : 80) : (U == 3 ? 128 : 104))
combine_backward_kernel(const void *d_out, const void *y_sorted, const int32_t *row_sorted,
                        const void *w, int w_dtype, const int32_t *n_kept, int64_t n, int k,
                        RowMap m, void *d_sorted, float *d_weights) {
  using V = typename Vec<B>::type;
  constexpr int EPV = B / sizeof(T);
  __shared__ float s_dot[kMaxThreads / 32][K];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & (m.lanes - 1), wid = threadIdx.x >> 5;
  const int64_t N = n * k, t = (int64_t)blockIdx.x * m.per_cta + threadIdx.x / m.lanes;
  float dot[K] = {};
  if (t < n) {
#pragma unroll 1
    for (int c0 = lane; c0 < m.vpr; c0 += U * m.lanes) {
      V g[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        g[u] = c0 + u * m.lanes < m.vpr
                   ? __ldcs(static_cast<const V *>(d_out) + t * m.vpr + c0 + u * m.lanes)
                   : vec_zero<B>();
#pragma unroll
      for (int j0 = 0; j0 < K; j0 += 4) {
        if (j0 >= k) break;
        V v[4][U];
        int64_t p[4];
        float wj[4];
        load_slots(row_sorted, w, w_dtype, t * k + j0, k - j0, N, p, wj);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int u = 0; u < U; ++u)
            v[j][u] = p[j] >= 0 && c0 + u * m.lanes < m.vpr
                          ? __ldcs(static_cast<const V *>(y_sorted) + p[j] * m.vpr + c0 +
                                   u * m.lanes)
                          : vec_zero<B>();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (p[j] >= 0)
#pragma unroll
            for (int u = 0; u < U; ++u) {
              if (c0 + u * m.lanes >= m.vpr) continue;
              float d[EPV], f[EPV], o[EPV];
              unpack<T, B>(g[u], d);
              unpack<T, B>(v[j][u], f);
#pragma unroll
              for (int i = 0; i < EPV; ++i) {
                dot[j0 + j] = fmaf(d[i], f[i], dot[j0 + j]);
                o[i] = wj[j] * d[i];
              }
              static_cast<V *>(d_sorted)[p[j] * m.vpr + c0 + u * m.lanes] = pack<T, B>(o);
            }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < K; ++j)
    if (j < k) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if ((threadIdx.x & 31) == 0) s_dot[wid][j] = dot[j];
    }
  __syncthreads();
  if (t < n && lane < k) {
    float sum = 0.f;
    for (int q = 0; q < m.lanes / 32; ++q) sum += s_dot[wid + q][lane];
    d_weights[t * k + lane] = sum;
  }
  zero_tail<B>(d_sorted, n_kept, N, m, t, lane);
}

// dz = p * (up - <p, up>) over the softmax's support (the k selected experts
// or all E), up = d_vals at the selected experts and 0 elsewhere. G lanes hold
// one token's E logits, V of them per load, NQ loads per lane; every lane
// looks through the k selected ids for its own experts, so that no load waits
// for another, and the two sums of the softmax are joined over the lanes
// together. One group per token: a chain of one load, some 100 instructions
// and two joins, so tokens are best all in flight at once. K: 4, or 8 where k > 4.
template <int V, int NQ, int K>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(const float *logits, const int32_t *topk_indx, const float *d_vals,
                      int64_t n, int E, int k, int gating, int G, float *d_logits) {
  pdl_wait();
  pdl_launch_dependents();
  const int g = threadIdx.x & (G - 1);
  const bool all = gating == MOE_GATING_SOFTMAX_ALL;
  const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / G;
  const bool on = t < n;
  float z[NQ][V], up[NQ][V];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int e = (q * G + g) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      z[q][i] = -INFINITY;
      up[q][i] = 0.f;
    }
    if (on && e < E) {
      if constexpr (V == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(logits + t * E + e);
        z[q][0] = v.x, z[q][1] = v.y, z[q][2] = v.z, z[q][3] = v.w;
      } else {
        z[q][0] = logits[t * E + e];
      }
    }
  }
  int idx[K];
  float d[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    idx[j] = on && j < k ? __ldg(topk_indx + t * k + j) : -1;
    d[j] = on && j < k ? __ldg(d_vals + t * k + j) : 0.f;
  }
  float top = -INFINITY;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = (q * G + g) * V + i;
      bool chosen = false;
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (j < k && idx[j] == e) {
          up[q][i] = d[j];
          chosen = true;
        }
      if (!all && !chosen) z[q][i] = -INFINITY;
      top = fmaxf(top, z[q][i]);
    }
  for (int o = G >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float den = 0.f, dot = 0.f;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      z[q][i] = z[q][i] == -INFINITY ? 0.f : expf(z[q][i] - top);
      den += z[q][i];
      dot = fmaf(z[q][i], up[q][i], dot);
    }
  for (int o = G >> 1; o > 0; o >>= 1) {
    den += __shfl_xor_sync(0xffffffffu, den, o);
    dot += __shfl_xor_sync(0xffffffffu, dot, o);
  }
  const float scale = den > 0.f ? 1.f / den : 0.f, mean = dot * scale;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int e = (q * G + g) * V;
    if (!on || e >= E) continue;
    float o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = z[q][i] * scale * (up[q][i] - mean);
    if constexpr (V == 4)
      *reinterpret_cast<float4 *>(d_logits + t * E + e) = make_float4(o[0], o[1], o[2], o[3]);
    else
      d_logits[t * E + e] = o[0];
  }
}

inline int elem_bytes(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }

// The widest vector (16, 4 or 2 bytes) that divides a row's bytes and both
// row arrays' base addresses: every row then starts on it.
inline int vec_bytes(size_t row_bytes, const void *a, const void *b) {
  const uintptr_t bits = (uintptr_t)row_bytes | (uintptr_t)a | (uintptr_t)b;
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
}

// The fewest threads per row (32, 64, 128 or 256) with at most 3 vectors each;
// rows beyond 768 vectors go round.
inline RowMap row_map(int vpr) {
  int lanes = 32;
  while (lanes < kMaxThreads && vpr > 3 * lanes) lanes *= 2;
  const int cta = lanes < kThreads ? kThreads : lanes;
  return {lanes, cta / lanes, vpr};
}

// These kernels keep the default split of L1 and shared memory: with the
// library's usual one (all shared) L1 is too small for the rows in flight, and
// the combine above takes 96 us in place of 70.
template <auto Kern, typename... Args>
cudaError_t go(dim3 grid, dim3 block, cudaStream_t s, Args... args) {
  const cudaError_t err = launch_dependent(Kern, grid, block, 0, s, args...);
  return err == cudaSuccess ? cudaGetLastError() : err;
}

// One CTA per per_cta tokens; F<U>::kern is the kernel for U vectors a thread.
template <template <int> class F, typename... Args>
cudaError_t go_rows(int64_t n, const RowMap &m, cudaStream_t s, Args... args) {
  const dim3 grid((unsigned)((n + m.per_cta - 1) / m.per_cta));
  const dim3 threads(m.lanes * m.per_cta);
  if (m.vpr <= m.lanes) return go<F<1>::kern>(grid, threads, s, args...);
  if (m.vpr <= 2 * m.lanes) return go<F<2>::kern>(grid, threads, s, args...);
  return go<F<3>::kern>(grid, threads, s, args...);
}
template <int B>
struct Dispatch {
  template <int U>
  struct F {
    static constexpr auto kern = dispatch_kernel<B, U>;
  };
};
template <typename T, int B, int K>
struct Backward {
  template <int U>
  struct F {
    static constexpr auto kern = combine_backward_kernel<T, B, U, K>;
  };
};

}  // namespace

cudaError_t launch_dispatch(const void *x, const int32_t *row_sorted, const int32_t *n_kept,
                            int64_t n, int k, int H, int dtype, void *x_sorted, cudaStream_t s) {
  const size_t rb = (size_t)H * elem_bytes(dtype);
  const int vb = vec_bytes(rb, x, x_sorted);
  const RowMap m = row_map((int)(rb / vb));
  if (vb == 16)
    return go_rows<Dispatch<16>::F>(n, m, s, x, row_sorted, n_kept, n, k, m, x_sorted);
  if (vb == 4) return go_rows<Dispatch<4>::F>(n, m, s, x, row_sorted, n_kept, n, k, m, x_sorted);
  return go_rows<Dispatch<2>::F>(n, m, s, x, row_sorted, n_kept, n, k, m, x_sorted);
}

template <typename T>
static cudaError_t combine_typed(const void *y, const int32_t *row_sorted, const void *w, int wd,
                                 int64_t n, int k, int H, void *out, cudaStream_t s) {
  const size_t rb = (size_t)H * sizeof(T);
  const int vb = vec_bytes(rb, y, out), vpr = (int)(rb / vb);
  // a thread per vector of the row, rows of up to 128 vectors several to a CTA
  int lanes = (vpr + 31) / 32 * 32;
  if (lanes > kMaxRowThreads) lanes = kMaxRowThreads;
  const int per_cta = lanes < 256 ? 256 / lanes : 1;
  const dim3 grid((unsigned)((n + per_cta - 1) / per_cta)), block(lanes, per_cta);
  if (vb == 16)
    return go<combine_weighted_kernel<T, 16>>(grid, block, s, y, row_sorted, w, wd, n, k, vpr, out);
  if (vb == 4)
    return go<combine_weighted_kernel<T, 4>>(grid, block, s, y, row_sorted, w, wd, n, k, vpr, out);
  if constexpr (sizeof(T) == 2)
    return go<combine_weighted_kernel<T, 2>>(grid, block, s, y, row_sorted, w, wd, n, k, vpr, out);
  return cudaErrorInvalidValue;
}

cudaError_t launch_combine_weighted(const void *y_sorted, const int32_t *row_sorted,
                                    const void *weights, int w_dtype, int64_t n, int k, int H,
                                    int dtype, void *out, cudaStream_t s) {
  if (dtype == MOE_FP32)
    return combine_typed<float>(y_sorted, row_sorted, weights, w_dtype, n, k, H, out, s);
  if (dtype == MOE_FP16)
    return combine_typed<__half>(y_sorted, row_sorted, weights, w_dtype, n, k, H, out, s);
  return combine_typed<__nv_bfloat16>(y_sorted, row_sorted, weights, w_dtype, n, k, H, out, s);
}

template <typename T>
static cudaError_t backward_typed(const void *d_out, const void *y, const int32_t *row_sorted,
                                  const void *w, int wd, const int32_t *n_kept, int64_t n, int k,
                                  int H, void *d_sorted, float *dw, cudaStream_t s) {
  const size_t rb = (size_t)H * sizeof(T);
  const int va = vec_bytes(rb, d_out, y), vd = vec_bytes(rb, d_sorted, d_sorted);
  const int vb = va < vd ? va : vd;
  const RowMap m = row_map((int)(rb / vb));
#define MOE_BACKWARD(B_)                                                                       \
  return k <= 4 ? go_rows<Backward<T, B_, 4>::template F>(n, m, s, d_out, y, row_sorted, w, wd, \
                                                          n_kept, n, k, m, d_sorted, dw)       \
                : go_rows<Backward<T, B_, 8>::template F>(n, m, s, d_out, y, row_sorted, w, wd, \
                                                          n_kept, n, k, m, d_sorted, dw)
  if (vb == 16) MOE_BACKWARD(16);
  if (vb == 4) MOE_BACKWARD(4);
  if constexpr (sizeof(T) == 2) MOE_BACKWARD(2);
  return cudaErrorInvalidValue;
#undef MOE_BACKWARD
}

cudaError_t launch_combine_backward(const void *d_out, const void *y_sorted,
                                    const int32_t *row_sorted, const void *weights, int w_dtype,
                                    const int32_t *n_kept, int64_t n, int k, int H, int dtype,
                                    void *d_sorted, float *d_weights, cudaStream_t s) {
  if (dtype == MOE_FP32)
    return backward_typed<float>(d_out, y_sorted, row_sorted, weights, w_dtype, n_kept, n, k, H,
                                 d_sorted, d_weights, s);
  if (dtype == MOE_FP16)
    return backward_typed<__half>(d_out, y_sorted, row_sorted, weights, w_dtype, n_kept, n, k, H,
                                  d_sorted, d_weights, s);
  return backward_typed<__nv_bfloat16>(d_out, y_sorted, row_sorted, weights, w_dtype, n_kept, n,
                                       k, H, d_sorted, d_weights, s);
}

cudaError_t launch_route_backward(const float *logits, const int32_t *topk_indx,
                                  const float *d_vals, int64_t n, int E, int k, int gating,
                                  float *d_logits, cudaStream_t s) {
  const bool vec = E % 4 == 0 && ((uintptr_t)logits | (uintptr_t)d_logits) % 16 == 0;
  const int per = vec ? E / 4 : E;
  int G = 1;
  while (G < 32 && G < per) G *= 2;
  const int nq = (per + G - 1) / G;
  const dim3 grid((unsigned)((n * G + kThreads - 1) / kThreads));
#define MOE_ROUTE_BACKWARD(V_, NQ_)                                                          \
  return k <= 4 ? go<route_backward_kernel<V_, NQ_, 4>>(grid, dim3(kThreads), s, logits,     \
                                                        topk_indx, d_vals, n, E, k, gating, \
                                                        G, d_logits)                         \
                : go<route_backward_kernel<V_, NQ_, 8>>(grid, dim3(kThreads), s, logits,     \
                                                        topk_indx, d_vals, n, E, k, gating, \
                                                        G, d_logits)
  if (vec) {
    if (nq == 1) MOE_ROUTE_BACKWARD(4, 1);
    MOE_ROUTE_BACKWARD(4, 2);
  }
  if (nq == 1) MOE_ROUTE_BACKWARD(1, 1);
  if (nq == 2) MOE_ROUTE_BACKWARD(1, 2);
  if (nq <= 4) MOE_ROUTE_BACKWARD(1, 4);
  MOE_ROUTE_BACKWARD(1, 8);
#undef MOE_ROUTE_BACKWARD
}

}  // namespace moe
