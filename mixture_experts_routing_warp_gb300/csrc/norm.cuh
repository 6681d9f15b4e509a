// norm.cuh -- what the norm and its gradients share (norm.cu,
// norm_backward.cu): rows as vectors in registers, weights, sums over the
// threads of a row, and the shape of a row's threads.
#pragma once

#include <type_traits>

#include "dense.cuh"

namespace moe {
namespace norm {

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
// Where the rows' length is not a multiple of a vector (bases on 16 bytes), row
// r starts s = (r H) mod VEC elements into a vector, alike in every array:
// vector j of the row then covers its elements [j VEC - s, (j + 1) VEC - s),
// the first and last of them in part, element by element.
template <bool SHIFT, typename T, int VEC>
__device__ __forceinline__ void load_span(const T *row, int c, int H, Raw<T, VEC> &r) {
  if constexpr (!SHIFT) {
    if (c < H) r.load(row + c);
    else r.zero();
  } else if (c >= 0 && c + VEC <= H) {
    r.load(row + c);
  } else {
    float f[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = c + i >= 0 && c + i < H ? to_float(row[c + i]) : 0.f;
    r.set(f);
  }
}
template <bool SHIFT, typename T, int VEC>
__device__ __forceinline__ void store_span(T *row, int c, int H, const Raw<T, VEC> &r) {
  if constexpr (!SHIFT) {
    if (c < H) r.store(row + c);
  } else if (c >= 0 && c + VEC <= H) {
    r.store(row + c);
  } else {
    float f[VEC];
    r.get(f);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c + i >= 0 && c + i < H) row[c + i] = from_float<T>(f[i]);
  }
}
template <bool SHIFT, int VEC>
__device__ __forceinline__ int row_shift(int64_t row, int H) {
  return SHIFT ? (int)((row * H) % VEC) : 0;
}

template <typename T, int VEC>
__device__ __forceinline__ void load_pack(const T *p, float (&f)[VEC]) {
  Raw<T, VEC> r;
  r.load(p);
  r.get(f);
}
// VEC weights of WT (the rows' type or fp32); ones where there are none. Shifted
// rows take them one by one, from L1.
template <typename WT, int VEC, bool SHIFT = false>
__device__ __forceinline__ void load_weight(const void *w, int c, float (&f)[VEC], int H = 0) {
  const WT *p = static_cast<const WT *>(w) + c;
  if (!w) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = 1.f;
  } else if constexpr (SHIFT) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = c + i >= 0 && c + i < H ? to_float(p[i]) : 0.f;
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

// ------------------------------------------------------------------- host --
// Threads per row (whole warps, at most 512) and vectors per thread, at most
// `most`; V = 0: the row does not stay in registers. Few rows take one vector
// per thread, for latency.
struct RowShape {
  int G, V;
};
inline RowShape row_shape(int64_t n, int64_t vectors, int target, int most, int two = kNormThreads) {
  if (n <= 2 * 152) target = 1;
  const int64_t fit = (vectors + kNormThreads - 1) / kNormThreads;
  int V = (int)(fit > target ? fit : target);
  if (V == 2 && vectors > 2 * two) V = 3;
  if (fit > most) return {kNormThreads, 0};
  if (vectors < 32 * V) V = (int)((vectors + 31) / 32);
  const int64_t per = (vectors + V - 1) / V;
  return {(int)((per + 31) / 32 * 32), V};
}

inline bool on16(const void *p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace norm
}  // namespace moe
