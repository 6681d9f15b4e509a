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

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

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
// to nearest even).
template <typename T, int B>
__device__ __forceinline__ void unpack(typename Vec<B>::type v, float *f) {
  T e[B / sizeof(T)];
  memcpy(e, &v, B);
#pragma unroll
  for (int i = 0; i < (int)(B / sizeof(T)); ++i) f[i] = (float)e[i];
}

template <typename T, int B>
__device__ __forceinline__ typename Vec<B>::type pack(const float *f) {
  T e[B / sizeof(T)];
#pragma unroll
  for (int i = 0; i < (int)(B / sizeof(T)); ++i) e[i] = (T)f[i];
  typename Vec<B>::type v;
  memcpy(&v, e, B);
  return v;
}

__device__ __forceinline__ float load_weight(const void *w, int w_dtype, int64_t f) {
  return w_dtype == MOE_FP32 ? __ldg(static_cast<const float *>(w) + f)
                             : bf16_bits_to_float(__ldg(static_cast<const uint16_t *>(w) + f));
}

// Zeros for the rows of no kept slot, [*n_kept, N): warp `warp` of `warps`
// takes every warps-th row, `vecs` vectors from `c0`, 32 lanes apart.
template <int B>
__device__ __forceinline__ void zero_tail(void *dst, const int32_t *n_kept, int64_t N, int vpr,
                                          int c0, int c1, int64_t warp, int64_t warps) {
  if (!n_kept) return;
  using V = typename Vec<B>::type;
  const int64_t kept = max(__ldg(n_kept), 0);
  for (int64_t r = kept + warp; r < N; r += warps)
    for (int c = c0; c < c1; c += 32) static_cast<V *>(dst)[r * vpr + c] = vec_zero<B>();
}

// A warp copies 32 * CPL vectors (column block blockIdx.y) of one token's
// row to the token's k sorted rows.
template <int B, int CPL>
__global__ void __launch_bounds__(kThreads)
dispatch_kernel(const void *x, const int32_t *row_sorted, const int32_t *n_kept, int64_t n, int k,
                int vpr, void *x_sorted) {
  using V = typename Vec<B>::type;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t warps = (int64_t)gridDim.x * kWarps, N = n * k;
  const int64_t warp = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int c0 = blockIdx.y * 32 * CPL + (threadIdx.x & 31);
  for (int64_t t = warp; t < n; t += warps) {
    V v[CPL];
#pragma unroll
    for (int q = 0; q < CPL; ++q)
      if (c0 + 32 * q < vpr) v[q] = static_cast<const V *>(x)[t * vpr + c0 + 32 * q];
    for (int j = 0; j < k; ++j) {
      const int64_t p = __ldg(row_sorted + t * k + j);
      if (p < 0 || p >= N) continue;
#pragma unroll
      for (int q = 0; q < CPL; ++q)
        if (c0 + 32 * q < vpr) static_cast<V *>(x_sorted)[p * vpr + c0 + 32 * q] = v[q];
    }
  }
  zero_tail<B>(x_sorted, n_kept, N, vpr, c0, min(vpr, (int)(blockIdx.y + 1) * 32 * CPL), warp,
               warps);
}

// A warp sums 32 * CPL vectors of one token's k sorted rows. Four rows are in
// flight at a time; `w` null: all weights 1 (the dispatch's backward pass).
template <typename T, int B, int CPL>
__global__ void __launch_bounds__(kThreads)
combine_weighted_kernel(const void *y_sorted, const int32_t *row_sorted, const void *w,
                        int w_dtype, int64_t n, int k, int vpr, void *out) {
  using V = typename Vec<B>::type;
  constexpr int EPV = B / sizeof(T);
  pdl_wait();
  pdl_launch_dependents();
  const int64_t warps = (int64_t)gridDim.x * kWarps, N = n * k;
  const int64_t warp = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int c0 = blockIdx.y * 32 * CPL + (threadIdx.x & 31);
  for (int64_t t = warp; t < n; t += warps) {
    float acc[CPL][EPV] = {};
    for (int j0 = 0; j0 < k; j0 += 4) {
      V v[4][CPL];
      float wj[4];
      bool live[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t f = t * k + j0 + j;
        const int64_t p = j0 + j < k ? __ldg(row_sorted + f) : -1;
        live[j] = p >= 0 && p < N;
        wj[j] = live[j] && w ? load_weight(w, w_dtype, f) : 1.f;
#pragma unroll
        for (int q = 0; q < CPL; ++q)
          v[j][q] = live[j] && c0 + 32 * q < vpr
                        ? __ldcs(static_cast<const V *>(y_sorted) + p * vpr + c0 + 32 * q)
                        : vec_zero<B>();
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (live[j])
#pragma unroll
          for (int q = 0; q < CPL; ++q) {
            float f[EPV];
            unpack<T, B>(v[j][q], f);
#pragma unroll
            for (int i = 0; i < EPV; ++i) acc[q][i] = fmaf(wj[j], f[i], acc[q][i]);
          }
    }
#pragma unroll
    for (int q = 0; q < CPL; ++q)
      if (c0 + 32 * q < vpr)
        static_cast<V *>(out)[t * vpr + c0 + 32 * q] = pack<T, B>(acc[q]);
  }
}

// WPT warps hold one token: each reads its share of d_out[t] once, writes the
// k scaled copies and adds up the k dot products with the sorted rows; the
// dot products are joined over lanes, then over the WPT warps.
template <typename T, int B, int WPT>
__global__ void __launch_bounds__(kThreads)
combine_backward_kernel(const void *d_out, const void *y_sorted, const int32_t *row_sorted,
                        const void *w, int w_dtype, const int32_t *n_kept, int64_t n, int k,
                        int vpr, void *d_sorted, float *d_weights) {
  using V = typename Vec<B>::type;
  constexpr int EPV = B / sizeof(T), TPB = kWarps / WPT;
  __shared__ float s_dot[TPB][WPT][kMaxTopk];
  pdl_wait();
  pdl_launch_dependents();
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = wid / WPT, part = wid % WPT;
  const int64_t N = n * k;
  // every warp of a block makes the same number of rounds (__syncthreads)
  for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < n; t0 += (int64_t)gridDim.x * TPB) {
    const int64_t t = t0 + slot;
    float dot[kMaxTopk] = {};
    if (t < n) {
      int64_t p[kMaxTopk];
      float wj[kMaxTopk];
#pragma unroll
      for (int j = 0; j < kMaxTopk; ++j) {
        p[j] = j < k ? __ldg(row_sorted + t * k + j) : -1;
        if (p[j] >= N) p[j] = -1;
        wj[j] = p[j] >= 0 ? load_weight(w, w_dtype, t * k + j) : 0.f;
      }
      for (int c = part * 32 + lane; c < vpr; c += WPT * 32) {
        float d[EPV];
        unpack<T, B>(static_cast<const V *>(d_out)[t * vpr + c], d);
#pragma unroll
        for (int j0 = 0; j0 < kMaxTopk; j0 += 4) {
          if (j0 >= k) break;
          V v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[j] = p[j0 + j] >= 0
                       ? __ldcs(static_cast<const V *>(y_sorted) + p[j0 + j] * vpr + c)
                       : vec_zero<B>();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (p[j0 + j] >= 0) {
              float f[EPV], g[EPV];
              unpack<T, B>(v[j], f);
#pragma unroll
              for (int i = 0; i < EPV; ++i) {
                dot[j0 + j] = fmaf(d[i], f[i], dot[j0 + j]);
                g[i] = wj[j0 + j] * d[i];
              }
              static_cast<V *>(d_sorted)[p[j0 + j] * vpr + c] = pack<T, B>(g);
            }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kMaxTopk; ++j)
      if (j < k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
    if (WPT == 1) {
#pragma unroll
      for (int j = 0; j < kMaxTopk; ++j)
        if (t < n && j < k && lane == j) d_weights[t * k + j] = dot[j];
    } else {
#pragma unroll
      for (int j = 0; j < kMaxTopk; ++j)
        if (lane == 0 && j < k) s_dot[slot][part][j] = dot[j];
      __syncthreads();
      if (part == 0 && lane < k && t < n) {
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < WPT; ++q) sum += s_dot[slot][q][lane];
        d_weights[t * k + lane] = sum;
      }
      __syncthreads();
    }
  }
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  zero_tail<B>(d_sorted, n_kept, N, vpr, lane, vpr, (int64_t)blockIdx.x * kWarps + wid, warps);
}

// dz = p * (up - <p, up>) over the softmax's support (the k selected experts
// or all E), up = d_vals at the selected experts and 0 elsewhere. G lanes
// hold one token's E logits, V of them per load, NQ loads per lane.
template <int V, int NQ>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(const float *logits, const int32_t *topk_indx, const float *d_vals,
                      int64_t n, int E, int k, int gating, int G, float *d_logits) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane & (G - 1);
  const int64_t groups = (int64_t)gridDim.x * (kThreads / G);
  const bool all = gating == MOE_GATING_SOFTMAX_ALL;
  // every lane of a warp makes the same number of rounds (full-warp shuffles)
  for (int64_t t0 = ((int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31)) / G; t0 < n;
       t0 += groups) {
    const int64_t t = t0 + lane / G;
    const bool on = t < n;
    float z[NQ][V];
    float top = -INFINITY;
    if (all) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int e = (q * G + g) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) z[q][i] = -INFINITY;
        if (on && e < E) {
          if (V == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(logits + t * E + e);
            z[q][0] = v.x, z[q][V > 1 ? 1 : 0] = v.y, z[q][V > 2 ? 2 : 0] = v.z;
            z[q][V > 3 ? 3 : 0] = v.w;
          } else {
            z[q][0] = logits[t * E + e];
          }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, z[q][i]);
      }
    }
    // the k selected: every lane of the group holds all of them
    int idx[kMaxTopk];
    float up[kMaxTopk], zs[kMaxTopk];
#pragma unroll
    for (int j = 0; j < kMaxTopk; ++j) {
      idx[j] = on && j < k ? __ldg(topk_indx + t * k + j) : -1;
      if (idx[j] >= E) idx[j] = -1;
      up[j] = idx[j] >= 0 ? __ldg(d_vals + t * k + j) : 0.f;
      zs[j] = idx[j] >= 0 ? __ldg(logits + t * E + idx[j]) : -INFINITY;
      top = fmaxf(top, zs[j]);
    }
    if (all)
      for (int o = G >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float den = 0.f, mean = 0.f, p[kMaxTopk];
    if (all) {
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          z[q][i] = z[q][i] == -INFINITY ? 0.f : expf(z[q][i] - top);
          den += z[q][i];
        }
      for (int o = G >> 1; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    }
#pragma unroll
    for (int j = 0; j < kMaxTopk; ++j) {
      p[j] = idx[j] >= 0 ? expf(zs[j] - top) : 0.f;
      if (!all) den += p[j];
    }
#pragma unroll
    for (int j = 0; j < kMaxTopk; ++j)
      if (idx[j] >= 0) {
        p[j] /= den;
        mean = fmaf(p[j], up[j], mean);
      }
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int e = (q * G + g) * V;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        o[i] = all ? -(z[q][i] / den) * mean : 0.f;
#pragma unroll
        for (int j = 0; j < kMaxTopk; ++j)
          if (idx[j] == e + i) o[i] = p[j] * (up[j] - mean);
      }
      if (on && e < E) {
        if (V == 4)
          *reinterpret_cast<float4 *>(d_logits + t * E + e) =
              make_float4(o[0], o[V > 1 ? 1 : 0], o[V > 2 ? 2 : 0], o[V > 3 ? 3 : 0]);
        else
          d_logits[t * E + e] = o[0];
      }
    }
  }
}

inline int elem_bytes(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }

// The widest vector (16, 4 or 2 bytes) that divides a row's bytes and both
// row arrays' base addresses: every row then starts on it.
inline int vec_bytes(size_t row_bytes, const void *a, const void *b) {
  const uintptr_t bits = (uintptr_t)row_bytes | (uintptr_t)a | (uintptr_t)b;
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
}

// Column blocks of 32 * cpl vectors on y, enough CTAs on x for one warp per
// token, at most 16 per SM in all.
inline dim3 row_grid(int64_t n, int vpr, int cpl) {
  const int64_t gy = (vpr + 32 * cpl - 1) / (32 * cpl);
  int64_t gx = (n + kWarps - 1) / kWarps;
  const int64_t cap = ((int64_t)device_sm_count() * 16 + gy - 1) / gy;
  if (gx > cap) gx = cap;
  return dim3((unsigned)gx, (unsigned)gy);
}

template <auto Kern, typename... Args>
cudaError_t go(dim3 grid, cudaStream_t s, Args... args) {
  static PerDeviceOnce configured;
  cudaError_t err = configured.run([] { return uniform_carveout(Kern); });
  if (err != cudaSuccess) return err;
  err = launch_dependent(Kern, grid, dim3(kThreads), 0, s, args...);
  return err == cudaSuccess ? cudaGetLastError() : err;
}

}  // namespace

cudaError_t launch_dispatch(const void *x, const int32_t *row_sorted, const int32_t *n_kept,
                            int64_t n, int k, int H, int dtype, void *x_sorted, cudaStream_t s) {
  const size_t rb = (size_t)H * elem_bytes(dtype);
  const int vb = vec_bytes(rb, x, x_sorted), vpr = (int)(rb / vb);
  if (vb == 16)
    return go<dispatch_kernel<16, 2>>(row_grid(n, vpr, 2), s, x, row_sorted, n_kept, n, k, vpr,
              x_sorted);
  if (vb == 4)
    return go<dispatch_kernel<4, 4>>(row_grid(n, vpr, 4), s, x, row_sorted, n_kept, n, k, vpr,
              x_sorted);
  return go<dispatch_kernel<2, 4>>(row_grid(n, vpr, 4), s, x, row_sorted, n_kept, n, k, vpr,
            x_sorted);
}

template <typename T>
static cudaError_t combine_typed(const void *y, const int32_t *row_sorted, const void *w, int wd,
                                 int64_t n, int k, int H, void *out, cudaStream_t s) {
  const size_t rb = (size_t)H * sizeof(T);
  const int vb = vec_bytes(rb, y, out), vpr = (int)(rb / vb);
  if (vb == 16)
    return go<combine_weighted_kernel<T, 16, 2>>(row_grid(n, vpr, 2), s, y, row_sorted, w, wd, n,
              k, vpr, out);
  if (vb == 4)
    return go<combine_weighted_kernel<T, 4, 4>>(row_grid(n, vpr, 4), s, y, row_sorted, w, wd, n,
              k, vpr, out);
  if constexpr (sizeof(T) == 2)
    return go<combine_weighted_kernel<T, 2, 4>>(row_grid(n, vpr, 4), s, y, row_sorted, w, wd, n,
              k, vpr, out);
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

template <typename T, int B>
static cudaError_t backward_vec(const void *d_out, const void *y, const int32_t *row_sorted,
                                const void *w, int wd, const int32_t *n_kept, int64_t n, int k,
                                int vpr, void *d_sorted, float *dw, cudaStream_t s) {
  // Rows beyond a couple of vectors per lane are shared by the block's four warps.
  const bool wide = vpr > 64;
  int64_t blocks = wide ? n : (n + kWarps - 1) / kWarps;
  const int64_t cap = (int64_t)device_sm_count() * 16;
  if (blocks > cap) blocks = cap;
  const dim3 grid((unsigned)blocks);
  if (wide)
    return go<combine_backward_kernel<T, B, kWarps>>(grid, s, d_out, y, row_sorted, w, wd, n_kept,
              n, k, vpr, d_sorted, dw);
  return go<combine_backward_kernel<T, B, 1>>(grid, s, d_out, y, row_sorted, w, wd, n_kept, n, k,
            vpr, d_sorted, dw);
}

template <typename T>
static cudaError_t backward_typed(const void *d_out, const void *y, const int32_t *row_sorted,
                                  const void *w, int wd, const int32_t *n_kept, int64_t n, int k,
                                  int H, void *d_sorted, float *dw, cudaStream_t s) {
  const size_t rb = (size_t)H * sizeof(T);
  int vb = vec_bytes(rb, d_out, y);
  if (vec_bytes(rb, d_sorted, d_sorted) < vb) vb = vec_bytes(rb, d_sorted, d_sorted);
  const int vpr = (int)(rb / vb);
  if (vb == 16)
    return backward_vec<T, 16>(d_out, y, row_sorted, w, wd, n_kept, n, k, vpr, d_sorted, dw, s);
  if (vb == 4)
    return backward_vec<T, 4>(d_out, y, row_sorted, w, wd, n_kept, n, k, vpr, d_sorted, dw, s);
  if constexpr (sizeof(T) == 2)
    return backward_vec<T, 2>(d_out, y, row_sorted, w, wd, n_kept, n, k, vpr, d_sorted, dw, s);
  return cudaErrorInvalidValue;
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
  int64_t blocks = (n * G + kThreads - 1) / kThreads;
  const int64_t cap = (int64_t)device_sm_count() * 16;
  if (blocks > cap) blocks = cap;
  const dim3 grid((unsigned)blocks);
#define MOE_ROUTE_BACKWARD(V_, NQ_)                                                            \
  return go<route_backward_kernel<V_, NQ_>>(grid, s, logits, topk_indx, d_vals, n, E, k, gating, \
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
