// norm_backward.cu -- the gradients of the root-mean-square norm (formulas and
// the shape of a row's threads: norm.cu), and the column sums that they and a
// bias's gradient need.
//
// A block's groups keep their rows' share of d_w in registers, add it up in
// shared memory at the end and write a row of partial sums; a second kernel
// adds those rows in order. Two vectors per thread and two blocks of 384 per
// SM: 8192 x 2880 with d_sum 41 us (the HBM copy rate: 28), V = 1 53, V = 3 44; rows fetched
// one ahead 57 - 68 us (the registers cost more warps than the wait).
// Neither limit is reached, 60 % of the issue slots and 56 % of HBM: a block's loads wait until
// its previous rows are done, at 5.9 warps per scheduler. Spills: 16 bytes at V = 2 (40 with fp32
// weights, 64 - 72 where rows are shifted), 128 - 168 at V = 4 (16-bit rows of 12289 elements and more).
#include "norm.cuh"

namespace moe {
namespace {

using namespace norm;

struct NormGradArgs {
  const void *d_y, *x, *weight, *d_sum;
  void *d_x;
  float *part;   // [blocks, H] sums of d v over a block's rows, or null
  float *rstd;   // [n], rows read twice only
  int64_t n;
  int H, G;
  float eps, inv_h;
};

// Threads of a block at V vectors per thread, two blocks per SM up to V = 2.
constexpr int grad_threads(int V) { return V == 2 ? 384 : kNormThreads; }

template <typename T, typename WT, bool SHIFT, int V>
__global__ void __launch_bounds__(grad_threads(V), V <= 2 ? 2 : 1)
rms_norm_backward_kernel(const NormGradArgs a) {
  constexpr int VEC = 16 / sizeof(T);
  __shared__ float scratch[2][kNormThreads / 32][2];
  extern __shared__ float s_acc[];  // [groups, H]: the groups' d_w, where there are several
  pdl_launch_dependents();
  pdl_wait();
  const int G = a.G, group = threadIdx.x / G, t = threadIdx.x % G;
  const int per_block = (int)blockDim.x / G;
  float acc[V][VEC];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[v][i] = 0.f;
  // a group's rows are a multiple of VEC apart, so they all start alike and a
  // thread's columns stay its own
  const int64_t first = (int64_t)blockIdx.x * per_block + group;
  const int shift = row_shift<SHIFT, VEC>(first, a.H);
  auto column = [&](int v) { return (t + v * G) * VEC - shift; };
  // the weights of this thread's columns: kept for all rows where they are of
  // the rows' type and a thread has one vector, else loaded again (from L1)
  constexpr bool kKeep = std::is_same_v<T, WT> && V == 1;
  Raw<T, VEC> kept[kKeep ? V : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float w[VEC];
      load_weight<WT, VEC, SHIFT>(column(v) < a.H ? a.weight : nullptr, column(v), w, a.H);
      kept[v].set(w);
    }
  }
  auto weights = [&](int v, float (&w)[VEC]) {
    if constexpr (kKeep) kept[v].get(w);
    else load_weight<WT, VEC, SHIFT>(column(v) < a.H ? a.weight : nullptr, column(v), w, a.H);
  };
  int slot = 0;
  for (int64_t row = first; row < a.n; row += (int64_t)gridDim.x * per_block, slot ^= 1) {
    const int64_t at = row * a.H;
    Raw<T, VEC> s[V], d[V], e[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      load_span<SHIFT>(static_cast<const T *>(a.x) + at, column(v), a.H, s[v]);
      load_span<SHIFT>(static_cast<const T *>(a.d_y) + at, column(v), a.H, d[v]);
      e[v].zero();
      if (a.d_sum) load_span<SHIFT>(static_cast<const T *>(a.d_sum) + at, column(v), a.H, e[v]);
    }
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[VEC], g[VEC], w[VEC];
      s[v].get(f);
      d[v].get(g);
      weights(v, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        q[0] += f[i] * f[i];
        q[1] += f[i] * (g[i] * w[i]);
      }
    }
    group_sum<2>(q, G, group, slot, scratch);
    const float r = inverse_rms(q[0], a.inv_h, a.eps);
    const float m = -(r * r) * (r * q[1] * a.inv_h);  // d_x = r d w + m x
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[VEC], g[VEC], w[VEC], o[VEC];
      s[v].get(f);
      d[v].get(g);
      e[v].get(o);
      weights(v, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float p = g[i] * r;
        o[i] = fmaf(m, f[i], fmaf(p, w[i], o[i]));
        acc[v][i] = fmaf(p, f[i], acc[v][i]);
      }
      Raw<T, VEC> out;
      out.set(o);
      store_span<SHIFT>(static_cast<T *>(a.d_x) + at, column(v), a.H, out);
    }
  }
  if (!a.part) return;
  float *dst = a.part + (int64_t)blockIdx.x * a.H;
  if (per_block > 1) dst = s_acc + group * a.H;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = column(v) + i;
      if ((!SHIFT || c >= 0) && c < a.H) dst[c] = acc[v][i];
    }
  if (per_block > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
      float f = 0.f;
      for (int g = 0; g < per_block; ++g) f += s_acc[g * a.H + c];
      a.part[(int64_t)blockIdx.x * a.H + c] = f;
    }
  }
}

template <typename T, typename WT>
__global__ void __launch_bounds__(kNormThreads)
rms_norm_backward_long_kernel(const NormGradArgs a) {
  __shared__ float scratch[2][kNormThreads / 32][2];
  pdl_launch_dependents();
  pdl_wait();
  int slot = 0;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, slot ^= 1) {
    const T *x = static_cast<const T *>(a.x) + row * a.H;
    const T *dy = static_cast<const T *>(a.d_y) + row * a.H;
    float q[2] = {0.f, 0.f}, w[1];
    for (int c = threadIdx.x; c < a.H; c += kNormThreads) {
      load_weight<WT, 1>(a.weight, c, w);
      const float s = to_float(x[c]);
      q[0] += s * s;
      q[1] += s * (to_float(dy[c]) * w[0]);
    }
    group_sum<2>(q, kNormThreads, 0, slot, scratch);
    const float r = inverse_rms(q[0], a.inv_h, a.eps);
    const float m = r * r * (q[1] * a.inv_h);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
    for (int c = threadIdx.x; c < a.H; c += kNormThreads) {
      load_weight<WT, 1>(a.weight, c, w);
      float o = r * (to_float(dy[c]) * w[0] - to_float(x[c]) * m);
      if (a.d_sum) o += to_float(static_cast<const T *>(a.d_sum)[row * a.H + c]);
      static_cast<T *>(a.d_x)[row * a.H + c] = from_float<T>(o);
    }
  }
}

// Partial column sums of d [n, cols] (times x r with x given): one block per
// 32 vectors of columns and slice of rows; part [gridDim.y, cols].
constexpr int kColThreads = 256;
template <typename T, int VEC>
__global__ void __launch_bounds__(kColThreads)
column_sum_kernel(const void *d, const void *x, const float *rstd, int64_t n, int cols,
                  float *part) {
  __shared__ float s_sum[kColThreads / 32][32 * VEC];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = ((int)blockIdx.x * 32 + lane) * VEC;
  const int64_t lo = n * blockIdx.y / gridDim.y, hi = n * (blockIdx.y + 1) / gridDim.y;
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int64_t row = lo + warp; row < hi; row += kColThreads / 32) {
      float f[VEC];
      load_pack<T, VEC>(static_cast<const T *>(d) + row * cols + c, f);
      if (x) {
        float g[VEC];
        load_pack<T, VEC>(static_cast<const T *>(x) + row * cols + c, g);
        const float r = rstd[row];
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] *= g[i] * r;
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += f[i];
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) s_sum[warp][lane * VEC + i] = acc[i];
  __syncthreads();
  for (int j = threadIdx.x; j < 32 * VEC; j += kColThreads) {
    float f = 0.f;
#pragma unroll
    for (int w = 0; w < kColThreads / 32; ++w) f += s_sum[w][j];
    const int cc = (int)blockIdx.x * 32 * VEC + j;
    if (cc < cols) part[(int64_t)blockIdx.y * cols + cc] = f;
  }
}

// out[c] = sum over the P rows of part [P, cols]: 32 columns per block, one row
// per warp at a time (all of a warp's loads in flight), then over the warps.
constexpr int kJoinThreads = 1024;
__global__ void __launch_bounds__(kJoinThreads)
column_join_kernel(const float *part, int P, int cols, int dtype, void *out) {
  __shared__ float s_sum[kJoinThreads / 32][33];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (int)blockIdx.x * 32 + lane;
  float acc = 0.f;
  if (c < cols) {
#pragma unroll 10
    for (int p = warp; p < P; p += kJoinThreads / 32) acc += __ldcg(part + (int64_t)p * cols + c);
  }
  s_sum[warp][lane] = acc;
  __syncthreads();
  float f = s_sum[lane][warp];  // column `warp` of the block, one row's sum per lane
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) f += __shfl_xor_sync(0xffffffffu, f, off);
  const int mine = (int)blockIdx.x * 32 + warp;
  if (lane == 0 && mine < cols) {
    if (dtype == MOE_FP32) static_cast<float *>(out)[mine] = f;
    else static_cast<uint16_t *>(out)[mine] = to16(f, dtype == MOE_FP16);
  }
}

template <typename T, typename WT, bool SHIFT, int V>
cudaError_t norm_grad_k(const NormGradArgs &a, dim3 grid, size_t smem, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  auto kern = rms_norm_backward_kernel<T, WT, SHIFT, V>;
  static PerDeviceOnce once;  // 512 threads x V vectors of fp32 sums: up to 64 KB
  const cudaError_t err = once.run([&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kNormThreads * V * VEC * 4);
  });
  if (err != cudaSuccess) return err;
  return launch_dependent(kern, grid, dim3((unsigned)(grad_threads(V) / a.G * a.G)), smem, s, a);
}

template <typename T, typename WT, bool SHIFT>
cudaError_t norm_grad_v(const NormGradArgs &a, int V, dim3 grid, size_t smem, cudaStream_t s) {
  switch (V) {
    case 1: return norm_grad_k<T, WT, SHIFT, 1>(a, grid, smem, s);
    case 2: return norm_grad_k<T, WT, SHIFT, 2>(a, grid, smem, s);
    case 3: return norm_grad_k<T, WT, SHIFT, 3>(a, grid, smem, s);
    default: return norm_grad_k<T, WT, SHIFT, 4>(a, grid, smem, s);
  }
}

// Blocks of the backward pass, and rows of their sums: a multiple of 8, so that a
// group's rows start alike (rms_norm_backward_kernel).
constexpr int kPartRows = 2 * 152;
static_assert(kPartRows % 8 == 0, "rows of a group");

template <typename T, typename WT>
cudaError_t norm_grad_t(NormGradArgs a, int w_dtype, void *d_weight, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  const bool based = on16(a.x) && on16(a.d_y) && on16(a.weight) && on16(a.d_sum) && on16(a.d_x);
  const bool shift = a.H % VEC != 0;
  const RowShape r = row_shape(a.n, (a.H + VEC - 1) / VEC + shift, 2, 4, grad_threads(2));
  int P;
  cudaError_t err;
  if (!based || r.V == 0) {
    const int64_t cap = (int64_t)device_sm_count() * 4;
    if (d_weight) a.rstd = a.part + (int64_t)kPartRows * a.H;
    err = launch_dependent(rms_norm_backward_long_kernel<T, WT>,
                           dim3((unsigned)(a.n < cap ? a.n : cap)), dim3(kNormThreads), 0, s, a);
    if (err != cudaSuccess || !d_weight) return err;
    P = (int)(a.n < 64 ? a.n : 64);
    err = launch_dependent(column_sum_kernel<T, 1>, dim3((unsigned)((a.H + 31) / 32), (unsigned)P),
                           dim3(kColThreads), 0, s, a.d_y, a.x, (const float *)a.rstd, a.n, a.H,
                           a.part);
  } else {
    a.G = r.G;
    if (!d_weight) a.part = nullptr;
    const int per_block = grad_threads(r.V) / r.G;
    int64_t blocks = (a.n + per_block - 1) / per_block;
    P = (int)(blocks < kPartRows ? blocks : kPartRows);
    const size_t smem = d_weight && per_block > 1 ? (size_t)per_block * a.H * 4 : 0;
    err = shift ? norm_grad_v<T, WT, true>(a, r.V, dim3((unsigned)P), smem, s)
                : norm_grad_v<T, WT, false>(a, r.V, dim3((unsigned)P), smem, s);
  }
  if (err != cudaSuccess || !d_weight) return err;
  return launch_column_join(a.part, P, a.H, w_dtype, d_weight, s);
}

}  // namespace

// Floats: the blocks' sums, and 1 / rms of each row where rows are read twice.
size_t rms_norm_backward_scratch(int64_t n, int H) {
  return ((size_t)kPartRows * H + (size_t)n) * 4;
}

cudaError_t launch_rms_norm_backward(const void *d_y, const void *x, const void *weight,
                                     int w_dtype, const void *d_sum, int64_t n, int H, int dtype,
                                     float eps, void *d_x, void *d_weight, float *scratch,
                                     cudaStream_t s) {
  const NormGradArgs a{d_y, x, weight, d_sum, d_x, scratch, nullptr, n, H, 0, eps, 1.0f / (float)H};
  const bool w32 = weight && w_dtype == MOE_FP32;
  switch (dtype) {
    case MOE_BF16:
      return w32 ? norm_grad_t<__nv_bfloat16, float>(a, w_dtype, d_weight, s)
                 : norm_grad_t<__nv_bfloat16, __nv_bfloat16>(a, w_dtype, d_weight, s);
    case MOE_FP16:
      return w32 ? norm_grad_t<__half, float>(a, w_dtype, d_weight, s)
                 : norm_grad_t<__half, __half>(a, w_dtype, d_weight, s);
    default: return norm_grad_t<float, float>(a, w_dtype, d_weight, s);
  }
}

cudaError_t launch_column_join(const float *part, int rows, int cols, int dtype, void *out,
                               cudaStream_t s) {
  return launch_dependent(column_join_kernel, dim3((unsigned)((cols + 31) / 32)),
                          dim3(kJoinThreads), 0, s, part, rows, cols, dtype, out);
}

size_t column_sum_scratch(int cols) { return (size_t)64 * cols * 4; }

cudaError_t launch_column_sum(const void *d, int64_t n, int cols, int dtype, void *out,
                              float *scratch, cudaStream_t s) {
  const bool wide = cols % 8 == 0 && on16(d);
  const int per = 32 * (wide ? 8 : 1);
  const int bx = (cols + per - 1) / per;
  int64_t P = (n + 63) / 64;  // at least 64 rows per slice, about four blocks per SM
  const int64_t most = (4 * 152 + bx - 1) / bx;
  if (P > most) P = most;
  if (P > 64) P = 64;
  if (P < 1) P = 1;
  const dim3 grid((unsigned)bx, (unsigned)P);
  cudaError_t err;
  if (dtype == MOE_FP16)
    err = wide ? launch_dependent(column_sum_kernel<__half, 8>, grid, dim3(kColThreads), 0, s, d,
                                  (const void *)nullptr, (const float *)nullptr, n, cols, scratch)
               : launch_dependent(column_sum_kernel<__half, 1>, grid, dim3(kColThreads), 0, s, d,
                                  (const void *)nullptr, (const float *)nullptr, n, cols, scratch);
  else
    err = wide ? launch_dependent(column_sum_kernel<__nv_bfloat16, 8>, grid, dim3(kColThreads), 0,
                                  s, d, (const void *)nullptr, (const float *)nullptr, n, cols,
                                  scratch)
               : launch_dependent(column_sum_kernel<__nv_bfloat16, 1>, grid, dim3(kColThreads), 0,
                                  s, d, (const void *)nullptr, (const float *)nullptr, n, cols,
                                  scratch);
  if (err != cudaSuccess) return err;
  return launch_column_join(scratch, (int)P, cols, dtype, out, s);
}

}  // namespace moe
