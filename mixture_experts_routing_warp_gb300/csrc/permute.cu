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
#include "operators.cuh"

#include <cuda_fp16.h>

#include <type_traits>

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxThreads = 256;
constexpr int kMaxRowThreads = 512;
constexpr int kShiftThreads = 128;

// The elements of 16 bytes as floats, and back (rounded once, to nearest
// even); 16-bit types by pairs, one conversion instruction each.
template <typename T>
__device__ __forceinline__ void unpack(const uint4 &v, float *f) {
  if constexpr (sizeof(T) == 4) {
    memcpy(f, &v, 16);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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

template <typename T>
__device__ __forceinline__ uint4 pack(const float *f) {
  uint4 v;
  if constexpr (sizeof(T) == 4) {
    memcpy(&v, f, 16);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        memcpy(&w[i], &h, 4);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        memcpy(&w[i], &h, 4);
      }
    }
    memcpy(&v, w, 16);
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
__device__ __forceinline__ void zero_tail(void *dst, const int32_t *n_kept, int64_t N,
                                          const RowMap &m, int64_t first, int lane) {
  if (!n_kept) return;
  const int64_t kept = max(__ldg(n_kept), 0);
  for (int64_t r = kept + first; r < N; r += (int64_t)gridDim.x * m.per_cta)
    for (int c = lane; c < m.vpr; c += m.lanes)
      static_cast<uint4 *>(dst)[r * m.vpr + c] = make_uint4(0u, 0u, 0u, 0u);
}

template <int U>
__global__ void __launch_bounds__(kMaxThreads)
dispatch_kernel(const void *x, const int32_t *row_sorted, const int32_t *n_kept, int64_t n, int k,
                RowMap m, void *x_sorted) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & (m.lanes - 1);
  const int64_t N = n * k, t = (int64_t)blockIdx.x * m.per_cta + threadIdx.x / m.lanes;
  if (t < n)
    for (int c0 = lane; c0 < m.vpr; c0 += U * m.lanes) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * m.lanes < m.vpr) v[u] = static_cast<const uint4 *>(x)[t * m.vpr + c0 + u * m.lanes];
      for (int j0 = 0; j0 < k; j0 += 4) {
        int64_t p[4];
        float one[4];
        load_slots(row_sorted, nullptr, MOE_FP32, t * k + j0, k - j0, N, p, one);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (p[j] >= 0 && c0 + u * m.lanes < m.vpr)
              static_cast<uint4 *>(x_sorted)[p[j] * m.vpr + c0 + u * m.lanes] = v[u];
      }
    }
  zero_tail(x_sorted, n_kept, N, m, t, lane);
}

// One vector per thread and row, four rows in flight; blockDim.x threads along
// the row, blockDim.y tokens. `w` null: all weights 1 (the dispatch's backward
// pass). One vector a thread keeps the kernel at 40 registers (16-bit rows: at
// the price of 24 bytes of spills) and the SM full: three vectors a thread
// measured 98 us where this takes 76 (16384 tokens, H 2880, k 4). The sums leave
// by streaming stores (81 us without). TOK: tokens per thread, 1, or for
// k = 4 / TOK so many that four rows are in flight.
template <typename T, int TOK>
__global__ void __launch_bounds__(kMaxRowThreads, TOK == 1 ? 3 : 2)
combine_weighted_kernel(const void *y_sorted, const int32_t *row_sorted, const void *w,
                        int w_dtype, int64_t n, int k, int vpr, void *out) {
  constexpr int EPV = 16 / sizeof(T);
  pdl_wait();
  pdl_launch_dependents();
  const int64_t N = n * k, t = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * TOK;
  if (t >= n) return;
  for (int c = threadIdx.x; c < vpr; c += blockDim.x) {
    float acc[TOK][EPV] = {};
    for (int j0 = 0; j0 < (TOK > 1 ? 1 : k); j0 += 4) {
      uint4 v[4];
      int64_t p[4];
      float wj[4];
      const int64_t left = TOK > 1 ? N - t * k : k - j0;
      load_slots(row_sorted, w, w_dtype, t * k + j0, (int)min(left, (int64_t)4), N, p, wj);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = p[j] >= 0 ? __ldcs(static_cast<const uint4 *>(y_sorted) + p[j] * vpr + c)
                         : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (p[j] >= 0) {
          float f[EPV];
          unpack<T>(v[j], f);
          float *sum = acc[j * TOK / 4];
#pragma unroll
          for (int i = 0; i < EPV; ++i) sum[i] = fmaf(wj[j], f[i], sum[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < TOK; ++i)
      if (TOK == 1 || t + i < n)
        __stcs(static_cast<uint4 *>(out) + (t + i) * vpr + c, pack<T>(acc[i]));
  }
}

// A row's threads read their share of d_out[t] once, write the k scaled
// copies and add up the k dot products with the sorted rows; those are joined
// over lanes, then over the row's warps. K: 1, 2, 4 or 8, the least that holds
// k. The register limits keep five CTAs of 128 threads on an SM (K = 4, U = 3:
// 67.5 us for 8192 tokens, H 2880; 72.8 with the compiler's own 127 registers),
// seven with K = 2 and nine with K = 1 (16384 tokens, H 1440, k 1: 32.5 us with
// K = 4's kernel, 22.0 so; 8192, k 2: 22.0 and 17.9).
template <typename T, int U, int K>
__global__ void __maxnreg__(K == 1 ? 56 : K == 2 ? 72 : K == 4 ? (U == 3 ? 96 : 80) : (U == 3 ? 128 : 104))
combine_backward_kernel(const void *d_out, const void *y_sorted, const int32_t *row_sorted,
                        const void *w, int w_dtype, const int32_t *n_kept, int64_t n, int k,
                        RowMap m, void *d_sorted, float *d_weights) {
  constexpr int EPV = 16 / sizeof(T), J = K < 4 ? K : 4;
  __shared__ float s_dot[kMaxThreads / 32][K];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & (m.lanes - 1), wid = threadIdx.x >> 5;
  const int64_t N = n * k, t = (int64_t)blockIdx.x * m.per_cta + threadIdx.x / m.lanes;
  float dot[K] = {};
  if (t < n) {
#pragma unroll 1
    for (int c0 = lane; c0 < m.vpr; c0 += U * m.lanes) {
      uint4 g[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        g[u] = c0 + u * m.lanes < m.vpr
                   ? __ldcs(static_cast<const uint4 *>(d_out) + t * m.vpr + c0 + u * m.lanes)
                   : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int j0 = 0; j0 < K; j0 += J) {
        if (j0 >= k) break;
        uint4 v[J][U];
        int64_t p[4];
        float wj[4];
        load_slots(row_sorted, w, w_dtype, t * k + j0, min(J, k - j0), N, p, wj);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int u = 0; u < U; ++u)
            v[j][u] = p[j] >= 0 && c0 + u * m.lanes < m.vpr
                          ? __ldcs(static_cast<const uint4 *>(y_sorted) + p[j] * m.vpr + c0 +
                                   u * m.lanes)
                          : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (p[j] >= 0)
#pragma unroll
            for (int u = 0; u < U; ++u) {
              if (c0 + u * m.lanes >= m.vpr) continue;
              float d[EPV], f[EPV], o[EPV];
              unpack<T>(g[u], d);
              unpack<T>(v[j][u], f);
#pragma unroll
              for (int i = 0; i < EPV; ++i) {
                dot[j0 + j] = fmaf(d[i], f[i], dot[j0 + j]);
                o[i] = wj[j] * d[i];
              }
              static_cast<uint4 *>(d_sorted)[p[j] * m.vpr + c0 + u * m.lanes] = pack<T>(o);
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
  zero_tail(d_sorted, n_kept, N, m, t, lane);
}

// ---- Rows that do not all start on 16 bytes (their length or an array's
// address is no multiple). The vectors are cut where the written row has its
// 16-byte words, so that stores stay whole; what a vector needs of another row
// starts at any element and is joined from the two aligned words around it.
// The second word is the next thread's first: HBM sees every byte once. In
// place of vectors of 2 (4) bytes, bf16, 8192 tokens, k 4, H 2879 (2878):
// combine 135 (79) -> 47 us, dispatch 71 (46) -> 43, the combine's gradients
// 169 (109) -> 99. Bound by instructions and the latency of few threads: each
// join is 19 instructions, so what belongs to the row (slots, places, whether
// it lies away from the array's ends) is worked out once and not per vector,
// and the register limits below trade rows in flight per thread for threads:
// dispatch two and 10 CTAs of 128 (four and 8: 46.5 us), combine four and 7
// (four and 6: 50; two and 9: 50), gradients four and 5 (two and 7: 103). They
// cost spills: 40 bytes in the combine of 16-bit rows (92 with k > 4), 36 to 88
// in the gradients of k > 4.
struct Window {
  uint4 a, b;
};

// Whether the two aligned words from the one that holds byte q of an array of
// `size` bytes on lie in the array, wherever it starts. They do for every
// vector of a row that has `margin` rows before and after it.
__device__ __forceinline__ bool words_inside(int64_t q, int64_t size) {
  return q >= 15 && q + 32 <= size;
}
inline int row_margin(int rb) { return 30 / rb + 1; }

// The two words `c` bytes (a multiple of 16) on from the one that holds s.
__device__ __forceinline__ Window load_window(uintptr_t s, int c) {
  const uint4 *w = reinterpret_cast<const uint4 *>((s & ~(uintptr_t)15) + c);
  return {w[0], w[1]};
}

// The 16 bytes that start s & 15 bytes into the window.
__device__ __forceinline__ uint4 join_window(const Window &r, uintptr_t s) {
  uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = s & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = s & 4 ? w[i + 1] : w[i];
  const uint32_t bits = (uint32_t)(s & 2) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// Bytes [at, at + 16) of a row of rb bytes as far as it has them: for the
// array's first and last words, and for the ends of a written row.
__device__ __forceinline__ uint4 load_part(uintptr_t row, int at, int rb) {
  uint32_t w[4] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (at + 2 * i >= 0 && at + 2 * i < rb)
      w[i >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t *>(row + at + 2 * i)
                   << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_part(uintptr_t row, int at, int rb, const uint4 &v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (at + 2 * i >= 0 && at + 2 * i < rb)
      *reinterpret_cast<uint16_t *>(row + at + 2 * i) = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}
__device__ __forceinline__ bool whole(int at, int rb) { return at >= 0 && at + 16 <= rb; }

// Zeros for the bytes of the rows [*n_kept, N).
__device__ __forceinline__ void zero_tail_bytes(uintptr_t dst, const int32_t *n_kept, int64_t N,
                                                int rb) {
  if (!n_kept) return;
  const int64_t kept = min((int64_t)max(__ldg(n_kept), 0), N);
  const uintptr_t lo = dst + kept * rb, hi = dst + N * rb;
  const int64_t threads = blockDim.x * blockDim.y, all = 16 * threads * gridDim.x;
  for (uintptr_t w = (lo & ~(uintptr_t)15) +
                     16 * (blockIdx.x * threads + threadIdx.y * blockDim.x + threadIdx.x);
       w < hi; w += all) {
    if (w >= lo && w + 16 <= hi) {
      *reinterpret_cast<uint4 *>(w) = make_uint4(0u, 0u, 0u, 0u);
    } else {
      for (uintptr_t e = w > lo ? w : lo; e < w + 16 && e < hi; e += 2)
        *reinterpret_cast<uint16_t *>(e) = 0;
    }
  }
}

// FEW: k <= 4, a token's slots and places are worked out once for its row.
template <bool FEW>
__global__ void __launch_bounds__(kShiftThreads, 10)
dispatch_shift_kernel(const void *x, const int32_t *row_sorted, const int32_t *n_kept, int64_t n,
                      int k, int rb, int margin, void *x_sorted) {
  pdl_wait();
  pdl_launch_dependents();
  const uintptr_t x0 = (uintptr_t)x, d0 = (uintptr_t)x_sorted;
  const int64_t N = n * k, t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t < n) {
    const uintptr_t row = x0 + t * rb;
    const bool inner = t >= margin && t < n - margin;
    uintptr_t to[4];  // the written row's first word
    int h[4];         // the row starts so many bytes into it; a dropped slot's never does
    auto place = [&](int j0) {
      int64_t p[4];
      float one[4];
      load_slots(row_sorted, nullptr, MOE_FP32, t * k + j0, k - j0, N, p, one);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        to[j] = d0 + p[j] * rb;
        h[j] = p[j] >= 0 ? (int)(to[j] & 15) : -rb;
        to[j] &= ~(uintptr_t)15;
      }
    };
    if (FEW) place(0);
    for (int c = 16 * threadIdx.x; c < rb + 15; c += 16 * blockDim.x)
      for (int j0 = 0; j0 < (FEW ? 1 : k); j0 += 4) {
        if (!FEW) place(j0);
        // vectors start c - 15 to c bytes into the row
        const bool inside = inner || words_inside(t * rb + c - 15, n * rb - 15);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          Window v[2];
#pragma unroll
          for (int j = i; j < i + 2; ++j)
            if (c < rb + h[j] && inside) v[j - i] = load_window(row - h[j], c);
#pragma unroll
          for (int j = i; j < i + 2; ++j)
            if (c < rb + h[j]) {
              const uint4 o =
                  inside ? join_window(v[j - i], row - h[j]) : load_part(row, c - h[j], rb);
              if (whole(c - h[j], rb))
                *reinterpret_cast<uint4 *>(to[j] + c) = o;
              else
                store_part(to[j] + h[j], c - h[j], rb, o);
            }
        }
      }
  }
  zero_tail_bytes(d0, n_kept, N, rb);
}

template <typename T, bool FEW>
__global__ void __launch_bounds__(kShiftThreads, 7)
combine_shift_kernel(const void *y_sorted, const int32_t *row_sorted, const void *w, int w_dtype,
                     int64_t n, int k, int rb, int margin, void *out) {
  constexpr int EPV = 16 / sizeof(T);
  pdl_wait();
  pdl_launch_dependents();
  const int64_t N = n * k, t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= n) return;
  const uintptr_t y0 = (uintptr_t)y_sorted;
  const int h = (int)(((uintptr_t)out + t * rb) & 15);
  const uintptr_t to = (uintptr_t)out + t * rb - h;  // the written row's first word
  uintptr_t from[4];  // the same place of the rows that are read; 0: dropped
  float wj[4];
  bool inner = true;
  auto place = [&](int j0) {
    int64_t p[4];
    load_slots(row_sorted, w, w_dtype, t * k + j0, k - j0, N, p, wj);
    inner = true;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      from[j] = p[j] >= 0 ? y0 + p[j] * rb - h : 0;
      inner &= p[j] < 0 || (p[j] >= margin && p[j] < N - margin);
    }
  };
  if (FEW) place(0);
  for (int c = 16 * threadIdx.x; c < rb + h; c += 16 * blockDim.x) {
    float acc[EPV] = {};
    for (int j0 = 0; j0 < (FEW ? 1 : k); j0 += 4) {
      if (!FEW) place(j0);
      bool inside = true;
      if (!inner) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          inside &= !from[j] || words_inside((int64_t)(from[j] - y0) + c, N * rb);
      }
      if (inside) {
        Window v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (from[j]) v[j] = load_window(from[j], c);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (from[j]) {
            float f[EPV];
            unpack<T>(join_window(v[j], from[j]), f);
#pragma unroll
            for (int i = 0; i < EPV; ++i) acc[i] = fmaf(wj[j], f[i], acc[i]);
          }
      } else {  // the array's first or last words: one slot at a time
#pragma unroll 1
        for (int j = j0; j < min(j0 + 4, k); ++j) {
          int64_t p[4];
          float w1[4];
          load_slots(row_sorted, w, w_dtype, t * k + j, 1, N, p, w1);
          if (p[0] < 0) continue;
          float f[EPV];
          unpack<T>(load_part(y0 + p[0] * rb, c - h, rb), f);
#pragma unroll
          for (int i = 0; i < EPV; ++i) acc[i] = fmaf(w1[0], f[i], acc[i]);
        }
      }
    }
    if (whole(c - h, rb))
      __stcs(reinterpret_cast<uint4 *>(to + c), pack<T>(acc));
    else
      store_part(to + h, c - h, rb, pack<T>(acc));
  }
}

// One slot's share of the vector `at` bytes into its rows: the scaled copy,
// and the sum `dot` over the elements that the row has.
template <typename T>
__device__ __forceinline__ float backward_vector(const uint4 &gv, const uint4 &yv, float wj,
                                                 uintptr_t to, int at, int rb, float dot) {
  constexpr int EPV = 16 / sizeof(T);
  float d[EPV], f[EPV], o[EPV];
  unpack<T>(gv, d);
  unpack<T>(yv, f);
  const bool all = whole(at, rb);
#pragma unroll
  for (int i = 0; i < EPV; ++i) {
    const int b = at + i * (int)sizeof(T);
    if (all || (b >= 0 && b < rb)) dot = fmaf(d[i], f[i], dot);
    o[i] = wj * d[i];
  }
  if (all)
    *reinterpret_cast<uint4 *>(to + at) = pack<T>(o);
  else
    store_part(to, at, rb, pack<T>(o));
  return dot;
}

// SAME: y_sorted and d_sorted have the same address modulo 16, so that the
// vectors of their rows are words of both.
template <typename T, int K, bool SAME>
__global__ void __launch_bounds__(kShiftThreads, (SAME ? 5 : 4) + (K == 1 ? 4 : K == 2 ? 2 : 0))
combine_backward_shift_kernel(const void *d_out, const void *y_sorted, const int32_t *row_sorted,
                              const void *w, int w_dtype, const int32_t *n_kept, int64_t n, int k,
                              int rb, int margin, void *d_sorted, float *d_weights) {
  constexpr bool FEW = K <= 4;
  constexpr int J = K < 4 ? K : 4;
  __shared__ float s_dot[kShiftThreads / 32][K];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t N = n * k, t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const uintptr_t y0 = (uintptr_t)y_sorted, d0 = (uintptr_t)d_sorted, yd = y0 - d0,
                  g_row = (uintptr_t)d_out + t * rb;
  float dot[K] = {};
  if (t < n) {
    uintptr_t to[J];  // the written row's first word; yd on from it, the read one's
    int h[J];         // the rows start so many bytes on; a dropped slot's never do
    float wj[4];
    bool inner = true;
    auto place = [&](int j0) {
      int64_t p[4];
      load_slots(row_sorted, w, w_dtype, t * k + j0, min(J, k - j0), N, p, wj);
      inner = t >= margin && t < n - margin;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        to[j] = d0 + p[j] * rb;
        h[j] = p[j] >= 0 ? (int)(to[j] & 15) : -rb;
        to[j] &= ~(uintptr_t)15;
        inner &= p[j] < 0 || (p[j] >= margin && p[j] < N - margin);
      }
    };
    if (FEW) place(0);
#pragma unroll 1
    for (int c = 16 * threadIdx.x; c < rb + 15; c += 16 * blockDim.x) {
#pragma unroll
      for (int j0 = 0; j0 < K; j0 += J) {
        if (j0 >= k) break;
        if (!FEW) place(j0);
        bool inside = true;
        if (!inner) {  // vectors start c - 15 to c bytes into the row
          inside = words_inside(t * rb + c - 15, n * rb - 15);
#pragma unroll
          for (int j = 0; j < J; ++j)
            inside &= c >= rb + h[j] || words_inside((int64_t)(to[j] - d0) + c, N * rb);
        }
        if (inside) {
          Window g[J], v[J];
#pragma unroll
          for (int j = 0; j < J; ++j)
            if (c < rb + h[j]) {
              if (SAME)
                v[j].a = __ldcs(reinterpret_cast<const uint4 *>(to[j] + yd + c));
              else
                v[j] = load_window(to[j] + yd, c);
              g[j] = load_window(g_row - h[j], c);
            }
#pragma unroll
          for (int j = 0; j < J; ++j)
            if (c < rb + h[j])
              dot[j0 + j] = backward_vector<T>(
                  join_window(g[j], g_row - h[j]),
                  SAME ? v[j].a : join_window(v[j], to[j] + yd), wj[j], to[j] + h[j], c - h[j],
                  rb, dot[j0 + j]);
        } else {  // an array's first or last words: one slot at a time
#pragma unroll 1
          for (int j = 0; j < min(J, k - j0); ++j) {
            int64_t p[4];
            float w1[4];
            load_slots(row_sorted, w, w_dtype, t * k + j0 + j, 1, N, p, w1);
            if (p[0] < 0) continue;
            const uintptr_t row = d0 + p[0] * rb;
            const int at = c - (int)(row & 15);
            if (at >= rb) continue;
            const float add = backward_vector<T>(load_part(g_row, at, rb),
                                                 load_part(row + yd, at, rb), w1[0], row, at, rb,
                                                 0.f);
#pragma unroll
            for (int i = 0; i < J; ++i)
              if (i == j) dot[j0 + i] += add;
          }
        }
      }
    }
  }
  const int warps = blockDim.x / 32, first = threadIdx.y * warps;  // of the token
#pragma unroll
  for (int j = 0; j < K; ++j)
    if (j < k) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if ((threadIdx.x & 31) == 0) s_dot[first + threadIdx.x / 32][j] = dot[j];
    }
  __syncthreads();
  if (t < n && threadIdx.x < k) {
    float sum = 0.f;
    for (int q = 0; q < warps; ++q) sum += s_dot[first + q][threadIdx.x];
    d_weights[t * k + threadIdx.x] = sum;
  }
  zero_tail_bytes(d0, n_kept, N, rb);
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
  // den is NaN beside a NaN or +inf logit and 0 where every one is -inf: NaN for
  // the softmax's support, like the gate weights themselves
  const float scale = 1.f / den, mean = dot * scale;
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
  // Experts outside the support stay 0 beside such a logit or gradient too: the
  // rare token looks its experts up once more (a mask kept for every token took
  // 7.3 us for 6.5 at 16384 tokens and 128 experts).
  if (on && !all && !(fabsf(mean) < INFINITY)) {
#pragma unroll 1
    for (int q = 0; q < NQ * V; ++q) {
      const int e = (q / V * G + g) * V + q % V;
      bool chosen = e >= E;
      for (int j = 0; j < k; ++j) chosen |= __ldg(topk_indx + t * k + j) == e;
      if (!chosen) d_logits[t * E + e] = 0.f;
    }
  }
}

inline int elem_bytes(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }

// Whether every row of both arrays starts on 16 bytes.
inline bool rows_aligned(size_t row_bytes, const void *a, const void *b) {
  return ((uintptr_t)row_bytes | (uintptr_t)a | (uintptr_t)b) % 16 == 0;
}

// Threads along a row of so many vectors, at most `most`: the fewest rounds,
// and the fewest warps for that many; short rows share a CTA.
struct RowBlock {
  dim3 grid, block;
  RowBlock(int64_t n, int vectors, int most) {
    const int rounds = (vectors + most - 1) / most;
    const int lanes = ((vectors + rounds - 1) / rounds + 31) / 32 * 32;
    const int cta = most < 256 ? most : 256, per_cta = lanes < cta ? cta / lanes : 1;
    grid = dim3((unsigned)((n + per_cta - 1) / per_cta));
    block = dim3(lanes, per_cta);
  }
};
// Vectors that rows of rb bytes need wherever they start.
inline int shifted_vectors(size_t rb) { return (int)((rb + 29) / 16); }

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
// the combine above takes 99 us in place of 76, its gradients (8192 tokens) 81
// in place of 69.
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
template <int U>
struct Dispatch {
  static constexpr auto kern = dispatch_kernel<U>;
};
template <typename T, int K>
struct Backward {
  template <int U>
  struct F {
    static constexpr auto kern = combine_backward_kernel<T, U, K>;
  };
};

}  // namespace

cudaError_t launch_dispatch(const void *x, const int32_t *row_sorted, const int32_t *n_kept,
                            int64_t n, int k, int H, int dtype, void *x_sorted, cudaStream_t s) {
  const size_t rb = (size_t)H * elem_bytes(dtype);
  if (!rows_aligned(rb, x, x_sorted)) {
    const RowBlock b(n, shifted_vectors(rb), kShiftThreads);
    const int margin = row_margin((int)rb);
    if (k <= 4)
      return go<dispatch_shift_kernel<true>>(b.grid, b.block, s, x, row_sorted, n_kept, n, k,
                                             (int)rb, margin, x_sorted);
    return go<dispatch_shift_kernel<false>>(b.grid, b.block, s, x, row_sorted, n_kept, n, k,
                                            (int)rb, margin, x_sorted);
  }
  const RowMap m = row_map((int)(rb / 16));
  return go_rows<Dispatch>(n, m, s, x, row_sorted, n_kept, n, k, m, x_sorted);
}

template <typename T>
static cudaError_t combine_typed(const void *y, const int32_t *row_sorted, const void *w, int wd,
                                 int64_t n, int k, int H, void *out, cudaStream_t s) {
  const size_t rb = (size_t)H * sizeof(T);
  if (!rows_aligned(rb, y, out)) {
    const RowBlock b(n, shifted_vectors(rb), kShiftThreads);
    const int margin = row_margin((int)rb);
    if (k <= 4)
      return go<combine_shift_kernel<T, true>>(b.grid, b.block, s, y, row_sorted, w, wd, n, k,
                                               (int)rb, margin, out);
    return go<combine_shift_kernel<T, false>>(b.grid, b.block, s, y, row_sorted, w, wd, n, k,
                                              (int)rb, margin, out);
  }
  const int vpr = (int)(rb / 16);
  // bf16, k 1, one and four tokens a thread: H 1440, 512 tokens 2.2 and 2.0 us,
  // 1024 3.2 and 2.4, 16384 24.6 and 13.7; H 512, 512 tokens 1.6 and 2.0, 1024
  // 1.8 and 2.0, 2048 3.1 and 2.3 (few are better spread over the SMs)
  const int tok = n >= 1024 && k <= 2 ? 4 / k : 1;
  const RowBlock b((n + tok - 1) / tok, vpr, kMaxRowThreads);
#define MOE_COMBINE(TOK_) \
  return go<combine_weighted_kernel<T, TOK_>>(b.grid, b.block, s, y, row_sorted, w, wd, n, k, vpr, out)
  if (tok == 4) MOE_COMBINE(4);
  if (tok == 2) MOE_COMBINE(2);
  MOE_COMBINE(1);
#undef MOE_COMBINE
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
  if (!rows_aligned(rb, d_out, y) || (uintptr_t)d_sorted % 16) {
    const RowBlock b(n, shifted_vectors(rb), kShiftThreads);
    const bool same = ((uintptr_t)y ^ (uintptr_t)d_sorted) % 16 == 0;
#define MOE_BACKWARD(K_, SAME_)                                                              \
  return go<combine_backward_shift_kernel<T, K_, SAME_>>(b.grid, b.block, s, d_out, y,       \
                                                         row_sorted, w, wd, n_kept, n, k,    \
                                                         (int)rb, row_margin((int)rb),       \
                                                         d_sorted, dw)
    if (k == 1 && same) MOE_BACKWARD(1, true);
    if (k == 1) MOE_BACKWARD(1, false);
    if (k == 2 && same) MOE_BACKWARD(2, true);
    if (k == 2) MOE_BACKWARD(2, false);
    if (k <= 4 && same) MOE_BACKWARD(4, true);
    if (k <= 4) MOE_BACKWARD(4, false);
    if (same) MOE_BACKWARD(8, true);
    MOE_BACKWARD(8, false);
#undef MOE_BACKWARD
  }
  const RowMap m = row_map((int)(rb / 16));
  if (k == 1)
    return go_rows<Backward<T, 1>::template F>(n, m, s, d_out, y, row_sorted, w, wd, n_kept, n, k,
                                               m, d_sorted, dw);
  if (k == 2)
    return go_rows<Backward<T, 2>::template F>(n, m, s, d_out, y, row_sorted, w, wd, n_kept, n, k,
                                               m, d_sorted, dw);
  if (k <= 4)
    return go_rows<Backward<T, 4>::template F>(n, m, s, d_out, y, row_sorted, w, wd, n_kept, n, k,
                                               m, d_sorted, dw);
  return go_rows<Backward<T, 8>::template F>(n, m, s, d_out, y, row_sorted, w, wd, n_kept, n, k, m,
                                             d_sorted, dw);
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
