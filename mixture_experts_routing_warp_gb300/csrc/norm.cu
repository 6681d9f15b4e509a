// norm.cu -- the root-mean-square norm in front of a layer, with the
// residual's addition and an 8-bit output (its gradients: norm_backward.cu).
//
//   s = x + residual (rounded to the rows' type: what the residual stream
//       keeps, and what the backward pass sees again)
//   r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//   backward, v = s r:  d_s = r (d w - v mean(d w v)) + d_sum,  d_w = sum d v
//
// Bound by HBM: each row crosses it once, and waits in registers between its
// sum of squares and its result. A row belongs to a group of G threads (a warp
// up to the whole block of 512) with V vectors of 16 bytes each, as they lie in
// memory; a block's groups take rows independently and meet at barriers of
// their own. V = 3 for many rows (16384 x 2880 bf16 with residual, V = 1 / 2 /
// 3 / 4 / 6 / 12: 71 / 72 / 57 / 57 / 74 / 74 us; 56 us is the HBM copy rate;
// in 8 bits 57 us, its floor 49), V = 1 for few. Rows of a length that is no whole
// number of vectors are cut where memory is (load_span: 16384 x 1001 100 -> 41 us);
// arrays that do not start on 16 bytes, and rows too long for the registers,
// take a kernel that goes element by element and reads a row twice. All sums
// are fp32; no atomics: the bits depend on inputs and sizes alone.
#include "norm.cuh"

namespace moe {
namespace {

using namespace norm;

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

template <typename T, typename WT, bool SHIFT, int V, bool MX>
__global__ void __launch_bounds__(kNormThreads, norm_blocks(V))
rms_norm_kernel(const NormArgs a) {
  constexpr int VEC = 16 / sizeof(T);
  __shared__ float scratch[2][kNormThreads / 32][1];
  pdl_launch_dependents();
  pdl_wait();
  const int G = a.G, group = threadIdx.x / G, t = threadIdx.x % G;
  const int per_block = (int)blockDim.x / G;
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * per_block + group; row < a.n;
       row += (int64_t)gridDim.x * per_block, slot ^= 1) {
    const int64_t at = row * a.H;
    const int shift = row_shift<SHIFT, VEC>(row, a.H);
    auto column = [&](int v) { return (t + v * G) * VEC - shift; };
    Raw<T, VEC> s[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      load_span<SHIFT>(static_cast<const T *>(a.x) + at, column(v), a.H, s[v]);
    if (a.residual) {
      Raw<T, VEC> d[V];
#pragma unroll
      for (int v = 0; v < V; ++v)
        load_span<SHIFT>(static_cast<const T *>(a.residual) + at, column(v), a.H, d[v]);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f[VEC], g[VEC];
        s[v].get(f);
        d[v].get(g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] += g[i];
        s[v].set(f);
        if (a.sum) store_span<SHIFT>(static_cast<T *>(a.sum) + at, column(v), a.H, s[v]);
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
      const int c = column(v);
      const bool live = c < a.H;
      float f[VEC], w[VEC];
      s[v].get(f);
      if (live) load_weight<WT, VEC, SHIFT>(a.weight, c, w, a.H);
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = live ? f[i] * r * w[i] : 0.f;
      if constexpr (MX) {
        store_mx8<VEC>(a, row, c, live, f);
      } else if (live) {
        Raw<T, VEC> y;
        y.set(f);
        store_span<SHIFT>(static_cast<T *>(a.y) + at, c, a.H, y);
      }
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

template <typename T, typename WT, bool SHIFT, bool MX>
cudaError_t norm_v(const NormArgs &a, int V, dim3 grid, cudaStream_t s) {
  const dim3 block((unsigned)(kNormThreads / a.G * a.G));  // whole groups
  switch (V) {
    case 1: return launch_dependent(rms_norm_kernel<T, WT, SHIFT, 1, MX>, grid, block, 0, s, a);
    case 2: return launch_dependent(rms_norm_kernel<T, WT, SHIFT, 2, MX>, grid, block, 0, s, a);
    case 3: return launch_dependent(rms_norm_kernel<T, WT, SHIFT, 3, MX>, grid, block, 0, s, a);
    case 4: return launch_dependent(rms_norm_kernel<T, WT, SHIFT, 4, MX>, grid, block, 0, s, a);
    default: return launch_dependent(rms_norm_kernel<T, WT, SHIFT, 8, MX>, grid, block, 0, s, a);
  }
}


template <typename T, typename WT, bool MX>
cudaError_t norm_t(NormArgs a, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  const bool based = on16(a.x) && on16(a.residual) && on16(a.weight) && on16(a.y) && on16(a.sum);
  const bool shift = a.H % VEC != 0;  // then a row is cut by one vector more
  const RowShape r = row_shape(a.n, (a.H + VEC - 1) / VEC + shift, 3, 8);
  const int64_t cap = (int64_t)device_sm_count() * 4 * 16;
  if (!based || r.V == 0) {
    const dim3 grid((unsigned)(a.n < cap ? a.n : cap));
    return launch_dependent(rms_norm_long_kernel<T, WT, MX>, grid, dim3(kNormThreads), 0, s, a);
  }
  a.G = r.G;
  const int per_block = kNormThreads / r.G;
  int64_t blocks = (a.n + per_block - 1) / per_block;
  if (blocks > cap) blocks = cap;
  const dim3 grid((unsigned)blocks);
  if constexpr (!MX)  // 8-bit rows are whole groups of 32
    if (shift) return norm_v<T, WT, true, MX>(a, r.V, grid, s);
  return norm_v<T, WT, false, MX>(a, r.V, grid, s);
}

template <typename T, typename WT>
cudaError_t norm_w(const NormArgs &a, cudaStream_t s) {
  return a.codes ? norm_t<T, WT, true>(a, s) : norm_t<T, WT, false>(a, s);
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

}  // namespace moe
