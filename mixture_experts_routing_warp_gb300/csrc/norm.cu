// norm.cu -- the root-mean-square norm in front of a layer, with the
// residual's addition and an 8-bit output, its gradients, and the column sums
// that a bias's gradient is.
//
//   s = x + residual (rounded to the rows' type: what the residual stream
//       keeps, and what the backward pass sees again)
//   r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//   backward, v = s r:  d_s = r (d w - v mean(d w v)) + d_sum,  d_w = sum d v
// Each row crosses HBM once: it stays in registers between its sum of squares
// and its result. A row belongs to a group of G threads (a warp up to the
// whole block of 512) with V vectors of 16 bytes each; a block's groups take
// rows independently and meet at barriers of their own. Rows that do not start
// on 16 bytes go element by element, rows too long for the registers by a
// kernel that reads them twice. All sums are fp32; d_w and the column sums
// run over a block's rows in registers, then over the blocks in a fixed order
// (no atomics: the bits depend on inputs and sizes alone).
#include "dense.cuh"

#include <type_traits>

namespace moe {
namespace {

constexpr int kNormThreads = 512;

template <typename T>
__device__ __forceinline__ float to_float(T v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else if constexpr (std::is_same_v<T, __half>) return __half2float(v);
  else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_float(float f) {
  if constexpr (std::is_same_v<T, float>) return f;
  else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(f);
  else return __float2bfloat16_rn(f);
}

// VEC elements of T as one load: 16 bytes, or one element.
template <typename T, int VEC>
struct Pack {
  T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ void load_pack(const T *p, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = to_float(*p);
  } else {
    static_assert(VEC * sizeof(T) == 16, "a 16-byte vector");
    const uint4 q = *reinterpret_cast<const uint4 *>(p);
    if constexpr (sizeof(T) == 4) memcpy(f, &q, 16);
    else unpack8(q, std::is_same_v<T, __half>, f);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T *p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    *p = from_float<T>(f[0]);
  } else {
    uint4 q;
    if constexpr (sizeof(T) == 4) memcpy(&q, f, 16);
    else q = pack8(f, std::is_same_v<T, __half>);
    *reinterpret_cast<uint4 *>(p) = q;
  }
}
// VEC weights of T or, with w32, of fp32.
template <typename T, int VEC>
__device__ __forceinline__ void load_weight(const void *w, bool w32, int c, float (&f)[VEC]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = 1.f;
  } else if (w32 && !std::is_same_v<T, float>) {
    const float *p = static_cast<const float *>(w) + c;
    if constexpr (VEC == 1) {
      f[0] = __ldg(p);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const float4 q = __ldg(reinterpret_cast<const float4 *>(p + i));
        f[i] = q.x;
        f[i + 1] = q.y;
        f[i + 2] = q.z;
        f[i + 3] = q.w;
      }
    }
  } else {
    load_pack<T, VEC>(static_cast<const T *>(w) + c, f);
  }
}

// Sums of up to two values over the group of G threads (a power of two, 32 or
// more); `slot` alternates between the two halves of the scratch, so that one
// barrier per call is enough.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int G, int group, int slot,
                                          float (*scratch)[kNormThreads / 32][N]) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
  if (G == 32) return;
  const int warp = threadIdx.x >> 5, warps = G >> 5, w0 = group * warps;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) scratch[slot][warp][i] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(G) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += scratch[slot][w0 + w][i];
}

struct NormArgs {
  const void *x, *residual, *weight;
  void *y, *sum;
  uint8_t *codes, *scales;
  int64_t n;
  int H, G, w32;
  float eps;
};

// VEC values of a row to 8-bit codes; the 32 / VEC lanes of a group of 32
// values share its largest. Every lane of the warp comes here.
template <int VEC>
__device__ __forceinline__ void store_mx8(const NormArgs &a, int64_t row, int c, bool live,
                                          const float (&f)[VEC]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < VEC; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
#pragma unroll
  for (int off = 16 / VEC; off > 0; off >>= 1)
    top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (!live) return;
  const uint32_t b = mx8_scale(top);
  const float inv = mx8_inverse(b);
  const int64_t at = row * a.H + c;
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint2 *>(a.codes + at) = make_uint2(mx8_codes4(f, inv), mx8_codes4(f + 4, inv));
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<uint32_t *>(a.codes + at) = mx8_codes4(f, inv);
  } else {
    a.codes[at] = (uint8_t)__nv_cvt_float_to_fp8(f[0] * inv, __NV_SATFINITE, __NV_E4M3);
  }
  if (c % 32 == 0) a.scales[at / 32] = (uint8_t)b;
}

template <typename T, int VEC, int V, bool MX>
__global__ void __launch_bounds__(kNormThreads)
rms_norm_kernel(const NormArgs a) {
  __shared__ float scratch[2][kNormThreads / 32][1];
  pdl_launch_dependents();
  pdl_wait();
  const int G = a.G, group = threadIdx.x / G, t = threadIdx.x % G;
  const int per_block = (int)blockDim.x / G;
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * per_block + group; row < a.n;
       row += (int64_t)gridDim.x * per_block, slot ^= 1) {
    const T *x = static_cast<const T *>(a.x) + row * a.H;
    float s[V][VEC];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (t + v * G) * VEC;
      if (c < a.H) {
        load_pack<T, VEC>(x + c, s[v]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[v][i] = 0.f;
      }
    }
    if (a.residual) {
      const T *res = static_cast<const T *>(a.residual) + row * a.H;
      float d[V][VEC];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (t + v * G) * VEC;
        if (c < a.H) load_pack<T, VEC>(res + c, d[v]);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (t + v * G) * VEC;
        if (c < a.H) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) s[v][i] = to_float(from_float<T>(s[v][i] + d[v][i]));
          if (a.sum) store_pack<T, VEC>(static_cast<T *>(a.sum) + row * a.H + c, s[v]);
        }
      }
    }
    float q[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < VEC; ++i) q[0] += s[v][i] * s[v][i];
    group_sum<1>(q, G, group, slot, scratch);
    const float r = 1.0f / sqrtf(q[0] / (float)a.H + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (t + v * G) * VEC;
      const bool live = c < a.H;
      float w[VEC];
      if (live) load_weight<T, VEC>(a.weight, a.w32, c, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[v][i] = live ? s[v][i] * r * w[i] : 0.f;
      if constexpr (MX)
        store_mx8<VEC>(a, row, c, live, s[v]);
      else if (live)
        store_pack<T, VEC>(static_cast<T *>(a.y) + row * a.H + c, s[v]);
    }
  }
}

// Rows that the registers do not hold: read twice, element by element.
template <typename T, bool MX>
__global__ void __launch_bounds__(kNormThreads)
rms_norm_long_kernel(const NormArgs a) {
  __shared__ float scratch[2][kNormThreads / 32][1];
  pdl_launch_dependents();
  pdl_wait();
  int slot = 0;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, slot ^= 1) {
    const T *x = static_cast<const T *>(a.x) + row * a.H;
    const T *res = a.residual ? static_cast<const T *>(a.residual) + row * a.H : nullptr;
    auto value = [&](int c) {
      const float f = to_float(x[c]);
      return res ? to_float(from_float<T>(f + to_float(res[c]))) : f;
    };
    float q[1] = {0.f};
    for (int c = threadIdx.x; c < a.H; c += kNormThreads) {
      const float s = value(c);
      q[0] += s * s;
    }
    group_sum<1>(q, kNormThreads, 0, slot, scratch);
    const float r = 1.0f / sqrtf(q[0] / (float)a.H + a.eps);
    for (int c0 = 0; c0 < a.H; c0 += kNormThreads) {
      const int c = c0 + (int)threadIdx.x;
      const bool live = c < a.H;
      float s = 0.f, w[1] = {0.f};
      if (live) {
        s = value(c);
        if (res && a.sum) static_cast<T *>(a.sum)[row * a.H + c] = from_float<T>(s);
        load_weight<T, 1>(a.weight, a.w32, c, w);
      }
      float f[1] = {live ? s * r * w[0] : 0.f};
      if constexpr (MX)
        store_mx8<1>(a, row, c, live, f);
      else if (live)
        static_cast<T *>(a.y)[row * a.H + c] = from_float<T>(f[0]);
    }
  }
}

struct NormGradArgs {
  const void *d_y, *x, *weight, *d_sum;
  void *d_x;
  float *part;   // [blocks, H] sums of d v over a block's rows, or null
  float *rstd;   // [n], rows read twice only
  int64_t n;
  int H, G, w32;
  float eps;
};

template <typename T, int VEC, int V>
__global__ void __launch_bounds__(kNormThreads)
rms_norm_backward_kernel(const NormGradArgs a) {
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
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * per_block + group; row < a.n;
       row += (int64_t)gridDim.x * per_block, slot ^= 1) {
    const T *x = static_cast<const T *>(a.x) + row * a.H;
    const T *dy = static_cast<const T *>(a.d_y) + row * a.H;
    float s[V][VEC], d[V][VEC];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (t + v * G) * VEC;
      if (c < a.H) {
        load_pack<T, VEC>(x + c, s[v]);
        load_pack<T, VEC>(dy + c, d[v]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[v][i] = d[v][i] = 0.f;
      }
    }
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (t + v * G) * VEC;
      float w[VEC];
      if (c < a.H) {
        load_weight<T, VEC>(a.weight, a.w32, c, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          q[0] += s[v][i] * s[v][i];
          q[1] += s[v][i] * (d[v][i] * w[i]);
        }
      }
    }
    group_sum<2>(q, G, group, slot, scratch);
    const float r = 1.0f / sqrtf(q[0] / (float)a.H + a.eps);
    const float m = r * r * (q[1] / (float)a.H);  // mean(d w v) r, to be times s
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (t + v * G) * VEC;
      if (c < a.H) {
        float w[VEC], o[VEC];
        load_weight<T, VEC>(a.weight, a.w32, c, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          o[i] = r * (d[v][i] * w[i] - s[v][i] * m);
          acc[v][i] += d[v][i] * (s[v][i] * r);
        }
        if (a.d_sum) {
          float e[VEC];
          load_pack<T, VEC>(static_cast<const T *>(a.d_sum) + row * a.H + c, e);
#pragma unroll
          for (int i = 0; i < VEC; ++i) o[i] += e[i];
        }
        store_pack<T, VEC>(static_cast<T *>(a.d_x) + row * a.H + c, o);
      }
    }
  }
  if (!a.part) return;
  float *dst = a.part + (int64_t)blockIdx.x * a.H;
  if (per_block > 1) dst = s_acc + group * a.H;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (t + v * G) * VEC;
    if (c < a.H)
#pragma unroll
      for (int i = 0; i < VEC; ++i) dst[c + i] = acc[v][i];
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

template <typename T>
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
      load_weight<T, 1>(a.weight, a.w32, c, w);
      const float s = to_float(x[c]);
      q[0] += s * s;
      q[1] += s * (to_float(dy[c]) * w[0]);
    }
    group_sum<2>(q, kNormThreads, 0, slot, scratch);
    const float r = 1.0f / sqrtf(q[0] / (float)a.H + a.eps);
    const float m = r * r * (q[1] / (float)a.H);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
    for (int c = threadIdx.x; c < a.H; c += kNormThreads) {
      load_weight<T, 1>(a.weight, a.w32, c, w);
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

// out[c] = sum over the P rows of part [P, cols]: 32 columns per block, eight
// rows at a time, then over the eight.
__global__ void __launch_bounds__(256)
column_join_kernel(const float *part, int P, int cols, int dtype, void *out) {
  __shared__ float s_sum[8][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (int)blockIdx.x * 32 + lane;
  float acc = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int p = warp; p < P; p += 8) acc += __ldcg(part + (int64_t)p * cols + c);
  }
  s_sum[warp][lane] = acc;
  __syncthreads();
  if (warp == 0 && c < cols) {
    float f = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) f += s_sum[w][lane];
    if (dtype == MOE_FP32) static_cast<float *>(out)[c] = f;
    else static_cast<uint16_t *>(out)[c] = to16(f, dtype == MOE_FP16);
  }
}

// ------------------------------------------------------------------- host --
// Threads per row (a power of two from 32 to 512) and vectors per thread.
struct RowShape {
  int G, V;
};
// Few rows: as many threads per row as have a vector, for latency; many:
// about three vectors per thread.
RowShape row_shape(int64_t n, int64_t vectors, int most) {
  const int target = n <= 2 * 152 ? 1 : 3;
  RowShape s{32, 1};
  while (s.G < kNormThreads && (int64_t)s.G * target < vectors) s.G *= 2;
  s.V = (int)((vectors + s.G - 1) / s.G);
  if (s.V > most) s.V = 0;  // not in registers
  return s;
}

template <typename T, int VEC, bool MX>
cudaError_t norm_v(const NormArgs &a, int V, dim3 grid, cudaStream_t s) {
  const dim3 block(kNormThreads);
  switch (V) {
    case 1: return launch_dependent(rms_norm_kernel<T, VEC, 1, MX>, grid, block, 0, s, a);
    case 2: return launch_dependent(rms_norm_kernel<T, VEC, 2, MX>, grid, block, 0, s, a);
    case 3: return launch_dependent(rms_norm_kernel<T, VEC, 3, MX>, grid, block, 0, s, a);
    case 4: return launch_dependent(rms_norm_kernel<T, VEC, 4, MX>, grid, block, 0, s, a);
    default: return launch_dependent(rms_norm_kernel<T, VEC, 8, MX>, grid, block, 0, s, a);
  }
}

inline bool on16(const void *p) { return ((uintptr_t)p & 15) == 0; }

template <typename T, bool MX>
cudaError_t norm_t(NormArgs a, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  const bool wide = a.H % VEC == 0 && on16(a.x) && on16(a.residual) && on16(a.weight) &&
                    on16(a.y) && on16(a.sum);
  const RowShape r = row_shape(a.n, wide ? a.H / VEC : a.H, 8);
  const int64_t cap = (int64_t)device_sm_count() * 4 * 16;
  if (r.V == 0) {
    const dim3 grid((unsigned)(a.n < cap ? a.n : cap));
    return launch_dependent(rms_norm_long_kernel<T, MX>, grid, dim3(kNormThreads), 0, s, a);
  }
  a.G = r.G;
  int64_t blocks = (a.n * r.G + kNormThreads - 1) / kNormThreads;
  if (blocks > cap) blocks = cap;
  return wide ? norm_v<T, VEC, MX>(a, r.V, dim3((unsigned)blocks), s)
              : norm_v<T, 1, MX>(a, r.V, dim3((unsigned)blocks), s);
}

template <typename T, int VEC, int V>
cudaError_t norm_grad_k(const NormGradArgs &a, dim3 grid, size_t smem, cudaStream_t s) {
  auto kern = rms_norm_backward_kernel<T, VEC, V>;
  static PerDeviceOnce once;  // 512 threads x V vectors of fp32 sums: up to 64 KB
  const cudaError_t err = once.run([&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kNormThreads * V * VEC * 4);
  });
  if (err != cudaSuccess) return err;
  return launch_dependent(kern, grid, dim3(kNormThreads), smem, s, a);
}

template <typename T, int VEC>
cudaError_t norm_grad_v(const NormGradArgs &a, int V, dim3 grid, size_t smem, cudaStream_t s) {
  switch (V) {
    case 1: return norm_grad_k<T, VEC, 1>(a, grid, smem, s);
    case 2: return norm_grad_k<T, VEC, 2>(a, grid, smem, s);
    case 3: return norm_grad_k<T, VEC, 3>(a, grid, smem, s);
    default: return norm_grad_k<T, VEC, 4>(a, grid, smem, s);
  }
}

constexpr int kPartRows = 2 * 152;  // blocks of the backward pass, and rows of their sums

template <typename T>
cudaError_t norm_grad_t(NormGradArgs a, int w_dtype, void *d_weight, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  const bool wide = a.H % VEC == 0 && on16(a.x) && on16(a.d_y) && on16(a.weight) &&
                    on16(a.d_sum) && on16(a.d_x);
  const RowShape r = row_shape(a.n, wide ? a.H / VEC : a.H, 4);
  int P;
  cudaError_t err;
  if (r.V == 0) {
    const int64_t cap = (int64_t)device_sm_count() * 4;
    if (d_weight) a.rstd = a.part + (int64_t)kPartRows * a.H;
    err = launch_dependent(rms_norm_backward_long_kernel<T>,
                           dim3((unsigned)(a.n < cap ? a.n : cap)), dim3(kNormThreads), 0, s, a);
    if (err != cudaSuccess || !d_weight) return err;
    P = (int)(a.n < 64 ? a.n : 64);
    err = launch_dependent(column_sum_kernel<T, 1>, dim3((unsigned)((a.H + 31) / 32), (unsigned)P),
                           dim3(kColThreads), 0, s, a.d_y, a.x, (const float *)a.rstd, a.n, a.H,
                           a.part);
  } else {
    a.G = r.G;
    if (!d_weight) a.part = nullptr;
    const int per_block = kNormThreads / r.G;
    int64_t blocks = (a.n + per_block - 1) / per_block;
    P = (int)(blocks < kPartRows ? blocks : kPartRows);
    const size_t smem = d_weight && per_block > 1 ? (size_t)per_block * a.H * 4 : 0;
    err = wide ? norm_grad_v<T, VEC>(a, r.V, dim3((unsigned)P), smem, s)
               : norm_grad_v<T, 1>(a, r.V, dim3((unsigned)P), smem, s);
  }
  if (err != cudaSuccess || !d_weight) return err;
  return launch_dependent(column_join_kernel, dim3((unsigned)((a.H + 31) / 32)), dim3(256), 0, s,
                          (const float *)a.part, P, a.H, w_dtype, d_weight);
}

}  // namespace

cudaError_t launch_rms_norm(const void *x, const void *residual, const void *weight, int w_dtype,
                            int64_t n, int H, int dtype, float eps, void *y, void *sum,
                            uint8_t *codes, uint8_t *scales, cudaStream_t s) {
  NormArgs a{x, residual, weight, y, sum, codes, scales, n, H, 0, w_dtype == MOE_FP32, eps};
  switch (dtype) {
    case MOE_BF16: return codes ? norm_t<__nv_bfloat16, true>(a, s) : norm_t<__nv_bfloat16, false>(a, s);
    case MOE_FP16: return codes ? norm_t<__half, true>(a, s) : norm_t<__half, false>(a, s);
    default: return codes ? norm_t<float, true>(a, s) : norm_t<float, false>(a, s);
  }
}

// Floats: the blocks' sums, and 1 / rms of each row where rows are read twice.
size_t rms_norm_backward_scratch(int64_t n, int H) {
  return ((size_t)kPartRows * H + (size_t)n) * 4;
}

cudaError_t launch_rms_norm_backward(const void *d_y, const void *x, const void *weight,
                                     int w_dtype, const void *d_sum, int64_t n, int H, int dtype,
                                     float eps, void *d_x, void *d_weight, float *scratch,
                                     cudaStream_t s) {
  NormGradArgs a{d_y, x, weight, d_sum, d_x, scratch, nullptr, n, H, 0, w_dtype == MOE_FP32, eps};
  switch (dtype) {
    case MOE_BF16: return norm_grad_t<__nv_bfloat16>(a, w_dtype, d_weight, s);
    case MOE_FP16: return norm_grad_t<__half>(a, w_dtype, d_weight, s);
    default: return norm_grad_t<float>(a, w_dtype, d_weight, s);
  }
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
  return launch_dependent(column_join_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, s,
                          (const float *)scratch, (int)P, cols, dtype, out);
}

}  // namespace moe
