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

// VEC elements of T, 16 bytes or one element, as they lie in memory: rows wait
// in registers in this form (half the registers of floats for 16-bit types).
template <typename T, int VEC>
struct Raw {
  static_assert(VEC * sizeof(T) == 16, "a 16-byte vector");
  uint4 q;
  __device__ __forceinline__ void load(const T *p) { q = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = q; }
  __device__ __forceinline__ void zero() { q = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
    if constexpr (sizeof(T) == 4) memcpy(f, &q, 16);
    else unpack8(q, std::is_same_v<T, __half>, f);
  }
  __device__ __forceinline__ void set(const float (&f)[VEC]) {
    if constexpr (sizeof(T) == 4) memcpy(&q, f, 16);
    else q = pack8(f, std::is_same_v<T, __half>);
  }
};
template <typename T>
struct Raw<T, 1> {
  T q;
  __device__ __forceinline__ void load(const T *p) { q = *p; }
  __device__ __forceinline__ void store(T *p) const { *p = q; }
  __device__ __forceinline__ void zero() { q = from_float<T>(0.f); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_float(q); }
  __device__ __forceinline__ void set(const float (&f)[1]) { q = from_float<T>(f[0]); }
};
template <typename T, int VEC>
__device__ __forceinline__ void load_pack(const T *p, float (&f)[VEC]) {
  Raw<T, VEC> r;
  r.load(p);
  r.get(f);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T *p, const float (&f)[VEC]) {
  Raw<T, VEC> r;
  r.set(f);
  r.store(p);
}
// VEC weights of WT (the rows' type or fp32); ones where there are none.
template <typename WT, int VEC>
__device__ __forceinline__ void load_weight(const void *w, int c, float (&f)[VEC]) {
  const WT *p = static_cast<const WT *>(w) + c;
  if (!w) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = 1.f;
  } else if constexpr (VEC * sizeof(WT) <= 16) {
    load_pack<WT, VEC>(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(p + i);
      memcpy(f + i, &q, 16);
    }
  }
}

// 1 / rms: rsqrt.approx, good to 2^-22
__device__ __forceinline__ float inverse_rms(float squares, float inv_h, float eps) {
  return rsqrtf(fmaf(squares, inv_h, eps));
}

// Sums of up to two values over the group of G threads (whole warps, 32 or
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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = G >> 5;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) scratch[slot][warp][i] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(G) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < warps ? scratch[slot][group * warps + lane][i] : 0.f;
#pragma unroll
  for (int off = kNormThreads / 64; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
}

struct NormArgs {
  const void *x, *residual, *weight;
  void *y, *sum;
  uint8_t *codes, *scales;
  int64_t n;
  int H, G;
  float eps, inv_h;
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

// Blocks per SM that a kernel with V vectors per thread leaves registers for.
constexpr int norm_blocks(int V) { return V == 1 ? 3 : V <= 4 ? 2 : 1; }

template <typename T, typename WT, int VEC, int V, bool MX>
__global__ void __launch_bounds__(kNormThreads, norm_blocks(V))
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
    Raw<T, VEC> s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (t + v * G) * VEC;
      if (c < a.H) s[v].load(x + c);
      else s[v].zero();
    }
    if (a.residual) {
      const T *res = static_cast<const T *>(a.residual) + row * a.H;
      Raw<T, VEC> d[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (t + v * G) * VEC;
        if (c < a.H) d[v].load(res + c);
        else d[v].zero();
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (t + v * G) * VEC;
        float f[VEC], g[VEC];
        s[v].get(f);
        d[v].get(g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] += g[i];
        s[v].set(f);
        if (a.sum && c < a.H) s[v].store(static_cast<T *>(a.sum) + row * a.H + c);
      }
    }
    float q[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[VEC];
      s[v].get(f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) q[0] += f[i] * f[i];
    }
    group_sum<1>(q, G, group, slot, scratch);
    const float r = inverse_rms(q[0], a.inv_h, a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (t + v * G) * VEC;
      const bool live = c < a.H;
      float f[VEC], w[VEC];
      s[v].get(f);
      if (live) load_weight<WT, VEC>(a.weight, c, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = live ? f[i] * r * w[i] : 0.f;
      if constexpr (MX)
        store_mx8<VEC>(a, row, c, live, f);
      else if (live)
        store_pack<T, VEC>(static_cast<T *>(a.y) + row * a.H + c, f);
    }
  }
}

// Rows that the registers do not hold: read twice, element by element.
template <typename T, typename WT, bool MX>
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
    const float r = inverse_rms(q[0], a.inv_h, a.eps);
    for (int c0 = 0; c0 < a.H; c0 += kNormThreads) {
      const int c = c0 + (int)threadIdx.x;
      const bool live = c < a.H;
      float s = 0.f, w[1] = {0.f};
      if (live) {
        s = value(c);
        if (res && a.sum) static_cast<T *>(a.sum)[row * a.H + c] = from_float<T>(s);
        load_weight<WT, 1>(a.weight, c, w);
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
  int H, G;
  float eps, inv_h;
};

#ifndef GRAD_THREADS2
#define GRAD_THREADS2 384
#endif
#ifndef GRAD_KEEP
#define GRAD_KEEP 1
#endif
// Threads of a block at V vectors per thread, two blocks per SM up to V = 2.
constexpr int grad_threads(int V) { return V == 2 ? GRAD_THREADS2 : kNormThreads; }

template <typename T, typename WT, int VEC, int V>
__global__ void __launch_bounds__(grad_threads(V), V <= 2 ? 2 : 1)
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
  // the weights of this thread's columns: kept for all rows where they are of
  // the rows' type, else loaded again (from L1)
  constexpr bool kKeep = std::is_same_v<T, WT> && V <= GRAD_KEEP;
  Raw<T, VEC> kept[kKeep ? V : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (t + v * G) * VEC;
      float one[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) one[i] = 1.f;
      kept[v].set(one);
      if (a.weight && c < a.H) kept[v].load(static_cast<const T *>(a.weight) + c);
    }
  }
  auto weights = [&](int v, float (&w)[VEC]) {
    if constexpr (kKeep) kept[v].get(w);
    else load_weight<WT, VEC>((t + v * G) * VEC < a.H ? a.weight : nullptr, (t + v * G) * VEC, w);
  };
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * per_block + group; row < a.n;
       row += (int64_t)gridDim.x * per_block, slot ^= 1) {
    const int64_t at = row * a.H;
    Raw<T, VEC> s[V], d[V], e[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (t + v * G) * VEC;
      e[v].zero();
      if (c < a.H) {
        s[v].load(static_cast<const T *>(a.x) + at + c);
        d[v].load(static_cast<const T *>(a.d_y) + at + c);
        if (a.d_sum) e[v].load(static_cast<const T *>(a.d_sum) + at + c);
      } else {
        s[v].zero();
        d[v].zero();
      }
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
      const int c = (t + v * G) * VEC;
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
      if (c < a.H) store_pack<T, VEC>(static_cast<T *>(a.d_x) + at + c, o);
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

// ------------------------------------------------------------------- host --
// Threads per row (whole warps, at most 512) and vectors per thread, at most
// `most`; V = 0: the row does not stay in registers. Few rows take one vector
// per thread, for latency.
#ifndef NORM_TARGET
#define NORM_TARGET 3
#endif
#ifndef NORM_GRAD_TARGET
#define NORM_GRAD_TARGET 2
#endif
struct RowShape {
  int G, V;
};
RowShape row_shape(int64_t n, int64_t vectors, int target, int most, int two = kNormThreads) {
  if (n <= 2 * 152) target = 1;
  const int64_t fit = (vectors + kNormThreads - 1) / kNormThreads;
  int V = (int)(fit > target ? fit : target);
  if (V == 2 && vectors > 2 * two) V = 3;
  if (fit > most) return {kNormThreads, 0};
  if (vectors < 32 * V) V = (int)((vectors + 31) / 32);
  const int64_t per = (vectors + V - 1) / V;
  return {(int)((per + 31) / 32 * 32), V};
}

template <typename T, typename WT, int VEC, bool MX>
cudaError_t norm_v(const NormArgs &a, int V, dim3 grid, cudaStream_t s) {
  const dim3 block((unsigned)(kNormThreads / a.G * a.G));  // whole groups
  switch (V) {
    case 1: return launch_dependent(rms_norm_kernel<T, WT, VEC, 1, MX>, grid, block, 0, s, a);
    case 2: return launch_dependent(rms_norm_kernel<T, WT, VEC, 2, MX>, grid, block, 0, s, a);
    case 3: return launch_dependent(rms_norm_kernel<T, WT, VEC, 3, MX>, grid, block, 0, s, a);
    case 4: return launch_dependent(rms_norm_kernel<T, WT, VEC, 4, MX>, grid, block, 0, s, a);
    case 5:
    case 6: return launch_dependent(rms_norm_kernel<T, WT, VEC, 6, MX>, grid, block, 0, s, a);
    case 7:
    case 8: return launch_dependent(rms_norm_kernel<T, WT, VEC, 8, MX>, grid, block, 0, s, a);
    default: return launch_dependent(rms_norm_kernel<T, WT, VEC, 12, MX>, grid, block, 0, s, a);
  }
}

inline bool on16(const void *p) { return ((uintptr_t)p & 15) == 0; }

template <typename T, typename WT, bool MX>
cudaError_t norm_t(NormArgs a, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  const bool wide = a.H % VEC == 0 && on16(a.x) && on16(a.residual) && on16(a.weight) &&
                    on16(a.y) && on16(a.sum);
  const RowShape r = row_shape(a.n, wide ? a.H / VEC : a.H, NORM_TARGET, 12);
  const int64_t cap = (int64_t)device_sm_count() * 4 * 16;
  if (r.V == 0) {
    const dim3 grid((unsigned)(a.n < cap ? a.n : cap));
    return launch_dependent(rms_norm_long_kernel<T, WT, MX>, grid, dim3(kNormThreads), 0, s, a);
  }
  a.G = r.G;
  const int per_block = kNormThreads / r.G;
  int64_t blocks = (a.n + per_block - 1) / per_block;
  if (blocks > cap) blocks = cap;
  return wide ? norm_v<T, WT, VEC, MX>(a, r.V, dim3((unsigned)blocks), s)
              : norm_v<T, WT, 1, MX>(a, r.V, dim3((unsigned)blocks), s);
}

template <typename T, typename WT>
cudaError_t norm_w(const NormArgs &a, cudaStream_t s) {
  return a.codes ? norm_t<T, WT, true>(a, s) : norm_t<T, WT, false>(a, s);
}

template <typename T, typename WT, int VEC, int V>
cudaError_t norm_grad_k(const NormGradArgs &a, dim3 grid, size_t smem, cudaStream_t s) {
  auto kern = rms_norm_backward_kernel<T, WT, VEC, V>;
  static PerDeviceOnce once;  // 512 threads x V vectors of fp32 sums: up to 64 KB
  const cudaError_t err = once.run([&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kNormThreads * V * VEC * 4);
  });
  if (err != cudaSuccess) return err;
  return launch_dependent(kern, grid, dim3((unsigned)(grad_threads(V) / a.G * a.G)), smem, s, a);
}

template <typename T, typename WT, int VEC>
cudaError_t norm_grad_v(const NormGradArgs &a, int V, dim3 grid, size_t smem, cudaStream_t s) {
  switch (V) {
    case 1: return norm_grad_k<T, WT, VEC, 1>(a, grid, smem, s);
    case 2: return norm_grad_k<T, WT, VEC, 2>(a, grid, smem, s);
    case 3: return norm_grad_k<T, WT, VEC, 3>(a, grid, smem, s);
    default: return norm_grad_k<T, WT, VEC, 4>(a, grid, smem, s);
  }
}

constexpr int kPartRows = 2 * 152;  // blocks of the backward pass, and rows of their sums

template <typename T, typename WT>
cudaError_t norm_grad_t(NormGradArgs a, int w_dtype, void *d_weight, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  const bool wide = a.H % VEC == 0 && on16(a.x) && on16(a.d_y) && on16(a.weight) &&
                    on16(a.d_sum) && on16(a.d_x);
  const RowShape r = row_shape(a.n, wide ? a.H / VEC : a.H, NORM_GRAD_TARGET, 4, grad_threads(2));
  int P;
  cudaError_t err;
  if (r.V == 0) {
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
    err = wide ? norm_grad_v<T, WT, VEC>(a, r.V, dim3((unsigned)P), smem, s)
               : norm_grad_v<T, WT, 1>(a, r.V, dim3((unsigned)P), smem, s);
  }
  if (err != cudaSuccess || !d_weight) return err;
  return launch_column_join(a.part, P, a.H, w_dtype, d_weight, s);
}

}  // namespace

cudaError_t launch_rms_norm(const void *x, const void *residual, const void *weight, int w_dtype,
                            int64_t n, int H, int dtype, float eps, void *y, void *sum,
                            uint8_t *codes, uint8_t *scales, cudaStream_t s) {
  const NormArgs a{x, residual, weight, y, sum, codes, scales, n, H, 0, eps, 1.0f / (float)H};
  const bool w32 = weight && w_dtype == MOE_FP32;
  switch (dtype) {
    case MOE_BF16: return w32 ? norm_w<__nv_bfloat16, float>(a, s) : norm_w<__nv_bfloat16, __nv_bfloat16>(a, s);
    case MOE_FP16: return w32 ? norm_w<__half, float>(a, s) : norm_w<__half, __half>(a, s);
    default: return norm_w<float, float>(a, s);
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
