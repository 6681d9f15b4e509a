// dense.cuh -- shared pieces of the dense products beside the experts
// (moe_linear, moe_gated_linear and their gradients): what becomes of the
// fp32 sums, the row types, and the launchers' interface.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <string.h>

#include "operators.cuh"

namespace moe {

// What is done with the sums a[row, col] of a product.
enum DenseKind {
  EPI_LINEAR = 0,    // out = act(a + bias) + add
  EPI_DACT = 1,      // out = add * act'(a + bias): add is the gradient of act's result. 16 bits,
                     // since the gradients' products take 16-bit operands; as EPI_DGATED
  EPI_GATED = 2,     // a holds (gate, up) pairs: out = h
  EPI_GATED_MX = 3,  // the same, h as E4M3 codes with a scale per 32
  EPI_DGATED = 4,    // (gate, up) pairs and add = d_h: out = (d_gate, d_up) in w13's row order
  EPI_PARTIAL = 5,   // fp32 parts of a split sum, whose joining kernel has the epilogue
  EPI_GRAD = 6,      // out = a (of two products at a time), or the same parts
  EPI_COLUMNS = 7    // EPI_LINEAR where rows do not start on 16 bytes
};

struct DenseEpi {
  int64_t rows;        // rows of out
  int cols;            // columns of the sums
  int half;            // 16-bit values are fp16, else bf16
  int act;             // moe_linear_act
  ActParams gate;      // gated kinds
  const void *bias;    // [cols] or null
  const void *add;     // [rows, cols] (EPI_DGATED: [rows, cols / 2]) or null
  void *out;           // [rows, cols] (EPI_GATED: [rows, cols / 2])
  uint8_t *codes, *scales;  // EPI_GATED_MX
  float *column_part;  // EPI_DACT: sums over 32 rows each of out before its rounding, or null
  int vec;             // every row of bias, add and out starts on 16 bytes
};

// ------------------------------------------------------------ 16-bit rows --
__device__ __forceinline__ float from16(uint16_t b, int half) {
  return half ? __half2float(__ushort_as_half(b)) : bf16_bits_to_float(b);
}
__device__ __forceinline__ uint16_t to16(float f, int half) {
  return half ? __half_as_ushort(__float2half_rn(f)) : float_to_bf16_bits(f);
}

__device__ __forceinline__ void unpack8(const uint4 &q, int half, float *f) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (half) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 h;
      memcpy(&h, &w[i], 4);
      const float2 d = __half22float2(h);
      f[2 * i] = d.x;
      f[2 * i + 1] = d.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ uint4 pack8(const float *f, int half) {
  uint32_t w[4];
  if (half) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      memcpy(&w[i], &h, 4);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      memcpy(&w[i], &h, 4);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// W 16-bit values at element `at` as floats; with `vec` the address is a
// multiple of 16 bytes. Values from `left` on are not read (0).
template <int W>
__device__ __forceinline__ void load_row(const void *base, int64_t at, bool vec, int left,
                                         int half, float (&f)[W]) {
  const uint16_t *p = static_cast<const uint16_t *>(base) + at;
  if (vec && left >= W) {
    uint4 q[W / 8];
#pragma unroll
    for (int i = 0; i < W / 8; ++i) q[i] = *reinterpret_cast<const uint4 *>(p + 8 * i);
#pragma unroll
    for (int i = 0; i < W / 8; ++i) unpack8(q[i], half, f + 8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = i < left ? from16(p[i], half) : 0.f;
  }
}

// One 32-byte store: a thread of an epilogue writes its own row, and L2 takes
// whole sectors at half the transactions of 16-byte pieces.
__device__ __forceinline__ void store32(void *p, const uint4 &a, const uint4 &b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

template <int W>
__device__ __forceinline__ void store_row(void *base, int64_t at, bool vec, int left, int half,
                                          const float (&f)[W]) {
  uint16_t *p = static_cast<uint16_t *>(base) + at;
  if (vec && left >= W) {
    bool done = false;
    if constexpr (W % 16 == 0) {
      if (((uintptr_t)p & 31) == 0) {  // whole sectors
        done = true;
#pragma unroll
        for (int i = 0; i < W; i += 16) store32(p + i, pack8(f + i, half), pack8(f + i + 8, half));
      }
    }
    if (!done) {
#pragma unroll
      for (int i = 0; i < W / 8; ++i)
        *reinterpret_cast<uint4 *>(p + 8 * i) = pack8(f + 8 * i, half);
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < left) p[i] = to16(f[i], half);
  }
}

// ------------------------------------------------------------------ MXFP8 --
// Scale byte of a group whose largest magnitude has the bits `top`: the least
// power of two 2^(b - 127) under which it is at most 448, E4M3's largest
// (1.75 * 2^8, so the mantissa decides between two exponents); 255, which
// reads as NaN, where a value of the group is infinite or NaN.
__device__ __forceinline__ uint32_t mx8_scale(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;
  const int b = (int)(top >> 23) - ((top & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return b < 0 ? 0u : (uint32_t)b;
}
// 2^(127 - b): what a value is multiplied with before it is rounded to a code
__device__ __forceinline__ float mx8_inverse(uint32_t b) {
  return __uint_as_float((254u - (b > 253u ? 253u : b)) << 23);
}
__device__ __forceinline__ uint32_t mx8_codes4(const float *f, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0] * inv, f[1] * inv),
                                               __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2] * inv, f[3] * inv),
                                               __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// ------------------------------------------------------------ activations --
// exp(-v^2 / 2); 0 below 2^-126 (|v| > 13.2)
__device__ __forceinline__ float gauss(float v) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * v * -0.72134752044448170f));
  return e;
}
// The normal distribution (1 + erf(v / sqrt 2)) / 2 for e = gauss(v). Below zero 1 + erf
// cancels (a tenth of the value is lost at -5, all of it from -5.6 on), so the tail is computed
// itself: at -|v| it is e t P(t), t = 1 / (1 + 0.3 |v|), where t P(t) is half of
// exp(v^2 / 2) erfc(|v| / sqrt 2), a smooth function. P is the polynomial of degree 7 with the least
// largest relative error on |v| <= 15 (1.8e-7; fitted to scipy's erfcx by Lawson's weights).
// In fp32 the value is off by 2^-20 of itself above -4 and, through e's argument, by 2^-17 at -12.
__device__ __forceinline__ float normal_below(float v, float e) {
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.3f, fabsf(v), 1.0f)));
  float p = 0.03517841175f;
  p = fmaf(p, t, -0.15514108539f);
  p = fmaf(p, t, 0.20281428099f);
  p = fmaf(p, t, -0.05044236779f);
  p = fmaf(p, t, 0.12685777247f);
  p = fmaf(p, t, 0.10042563826f);
  p = fmaf(p, t, 0.12067272514f);
  p = fmaf(p, t, 0.11963453144f);
  const float tail = p * t * e;
  return v < 0.f ? tail : 1.0f - tail;
}

__device__ __forceinline__ float linear_act(float v, int act) {
  if (act == MOE_LINEAR_SILU) return v * sigmoid_fast(v);
  if (act == MOE_LINEAR_GELU) return v * normal_below(v, gauss(v));
  if (act == MOE_LINEAR_RELU2) {
    const float r = v < 0.f ? 0.f : v;  // NaN stays
    return r * r;
  }
  return v;
}

__device__ __forceinline__ float linear_slope(float v, int act) {
  if (act == MOE_LINEAR_SILU) {
    const float s = sigmoid_fast(v);
    return s * (1.0f + v * (1.0f - s));
  }
  if (act == MOE_LINEAR_GELU) {
    const float e = gauss(v);
    return normal_below(v, e) + v * (e * 0.39894228040143268f);
  }
  if (act == MOE_LINEAR_RELU2) return 2.f * (v < 0.f ? 0.f : v);
  return 1.f;
}

// h of a (gate, up) pair, as activate() but NaN passes the clamps.
__device__ __forceinline__ float gated(float g, float u, const ActParams &p) {
  if (p.limit < INFINITY) {
    g = g > p.limit ? p.limit : g;
    u = u > p.limit ? p.limit : (u < -p.limit ? -p.limit : u);
  }
  return (g * sigmoid_fast(p.alpha * g)) * (u + p.beta);
}

// The gradients of gated() for d = d_h; a clamped value has none (a value at
// the limit is not clamped).
__device__ __forceinline__ void gated_backward(float g, float u, float d, const ActParams &p,
                                               float &d_g, float &d_u) {
  const float gc = g > p.limit ? p.limit : g;
  const float uc = u > p.limit ? p.limit : (u < -p.limit ? -p.limit : u);
  const float s = sigmoid_fast(p.alpha * gc);
  d_g = g > p.limit ? 0.f : d * (uc + p.beta) * s * (1.f + p.alpha * gc * (1.f - s));
  d_u = u > p.limit || u < -p.limit ? 0.f : d * gc * s;
}

// --------------------------------------------------------------- epilogue --
// Loads that stay where they are written.
__device__ __forceinline__ uint4 load_now(const uint4 *p) {
  uint4 q;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "l"(p));
  return q;
}
__device__ __forceinline__ uint2 load_now(const uint2 *p) {
  uint2 q;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "l"(p));
  return q;
}
__device__ __forceinline__ uint16_t load_now(const uint16_t *p) {
  uint16_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
// f on all of v, eight at a time in one copy of its code: unrolled over 32
// values a tile's epilogue waits for its own instructions (4000 x 1000 x 1000 with GELU, then
// by erff, 30 KB of them: 23 us for 19).
template <int W, typename F>
__device__ __forceinline__ void by_eights(float (&v)[W], F f) {
  if constexpr (W <= 8) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = f(v[i]);
  } else {
#pragma unroll 1
    for (int g = 0; g < W / 8; ++g) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = f(v[i]);
#pragma unroll
      for (int i = 0; i < W - 8; ++i) v[i] = v[i + 8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[W - 8 + i] = t[i];
    }
  }
}
// Columns [c, c + W) of a row's sums to where they go, by one thread (the
// gated results of a tile, and joined parts). c is a multiple of W and c <
// e.cols, row < e.rows.
template <int EPI, int W>
__device__ __forceinline__ void dense_epilogue(const DenseEpi &e, int64_t row, int c,
                                               float (&v)[W]) {
  const int left = e.cols - c;
  if constexpr (EPI == EPI_LINEAR || EPI == EPI_DACT) {
    if (e.bias) {
      float b[W];
      load_row<W>(e.bias, c, e.vec, left, e.half, b);
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] += b[i];
    }
    if constexpr (EPI == EPI_LINEAR) {
      if (e.act != MOE_LINEAR_NONE) by_eights(v, [&](float f) { return linear_act(f, e.act); });
      if (e.add) {
        float r[W];
        load_row<W>(e.add, row * e.cols + c, e.vec, left, e.half, r);
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] += r[i];
      }
    } else {
      by_eights(v, [&](float f) { return linear_slope(f, e.act); });
      float d[W];
      load_row<W>(e.add, row * e.cols + c, e.vec, left, e.half, d);
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] *= d[i];
    }
    store_row<W>(e.out, row * e.cols + c, e.vec, left, e.half, v);
  } else if constexpr (EPI == EPI_GATED) {
    float h[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) h[i] = gated(v[2 * i], v[2 * i + 1], e.gate);
    store_row<W / 2>(e.out, row * (e.cols / 2) + c / 2, e.vec, left / 2, e.half, h);
  } else if constexpr (EPI == EPI_GATED_MX) {
    static_assert(EPI != EPI_GATED_MX || W == 64, "one group of 32 at a time");
    float h[W / 2];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      h[i] = gated(v[2 * i], v[2 * i + 1], e.gate);
      top = max(top, __float_as_uint(h[i]) & 0x7fffffffu);
    }
    const uint32_t b = mx8_scale(top);
    const float inv = mx8_inverse(b);
    const int64_t at = row * (e.cols / 2) + c / 2;
    uint32_t q[W / 8];
#pragma unroll
    for (int i = 0; i < W / 8; ++i) q[i] = mx8_codes4(h + 4 * i, inv);
    uint4 *dst = reinterpret_cast<uint4 *>(e.codes + at);
    const uint4 lo = make_uint4(q[0], q[1], q[2], q[3]), hi = make_uint4(q[4], q[5], q[6], q[7]);
    if (((uintptr_t)dst & 31) == 0) {
      store32(dst, lo, hi);
    } else {
      dst[0] = lo;
      dst[1] = hi;
    }
    e.scales[at / 32] = (uint8_t)b;
  } else if constexpr (EPI == EPI_DGATED) {
    const int I = e.cols / 2;
    float d[W / 2];
    load_row<W / 2>(e.add, row * I + c / 2, e.vec, left / 2, e.half, d);
    if (e.gate.layout == MOE_W13_PACKED) {
      float g[W / 2], u[W / 2];
#pragma unroll
      for (int i = 0; i < W / 2; ++i)
        gated_backward(v[2 * i], v[2 * i + 1], d[i], e.gate, g[i], u[i]);
      store_row<W / 2>(e.out, row * e.cols + c / 2, e.vec, left / 2, e.half, g);
      store_row<W / 2>(e.out, row * e.cols + I + c / 2, e.vec, left / 2, e.half, u);
    } else {
#pragma unroll
      for (int i = 0; i < W / 2; ++i)
        gated_backward(v[2 * i], v[2 * i + 1], d[i], e.gate, v[2 * i], v[2 * i + 1]);
      store_row<W>(e.out, row * e.cols + c, e.vec, left, e.half, v);
    }
  }
}

// Columns of a row of fp32 partial sums: whole chunks of 64, so that parts are
// written and read in vectors.
__host__ __device__ __forceinline__ int64_t part_columns(int cols) { return (cols + 63) / 64 * 64; }

// ----------------------------------------------------------- warp roles --
// The producer and MMA roles run as whole warps whose every value is the same
// in all lanes, and one elected lane issues: addresses and descriptors then
// stay in uniform registers. (With the loop in lane 0 alone an MMA took 60
// cycles to issue and a K step 570, whatever its width.)
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// --------------------------------------------------------------- products --
// D[m, n] = sum_k A(m, k) B(n, k). K-major operands are stored [rows, K] row
// by row, the others [K, rows].
struct DenseOperand {
  const void *p;
  const uint8_t *scales;  // MXFP8: [rows, K / 32], else null
  int k_major;
  int pairs;              // rows 2i, 2i + 1 are rows i and i + rows / 2 of p (a packed w13)
};

struct DensePlan {
  int tn, tn_last;  // columns per tile, and of the last one of a row of tiles
  int m_tiles, n_tiles, splits;
  size_t partial;  // bytes of fp32 partial sums (0: one part)
  size_t blocks;   // bytes of the MXFP8 scales in the tensor core's layout
};

struct DenseProduct {
  DenseOperand a, b;
  int64_t M, N, K;
  int kind;       // DenseKind, EPI_PARTIAL excepted
  DenseEpi epi;
  uint64_t starve_ns;  // non-zero: every wait for operands runs out after so long (self-test)
};

DensePlan dense_plan(int64_t M, int64_t N, int64_t K, int kind, bool mx);
// blocks and partial: scratch of plan.blocks and plan.partial bytes. status null:
// the current device's own word, which read_wait_status copies to the host.
cudaError_t launch_dense(const DenseProduct &p, const DensePlan &plan, uint8_t *blocks,
                         float *partial, int32_t *status, cudaStream_t s);
cudaError_t read_wait_status(int32_t *out, bool reset, cudaStream_t s);
// A product of few rows, where dense_skinny says so (dense_skinny.cu). No
// scratch.
bool dense_skinny(int64_t n, int64_t out, int64_t in, int kind, bool mx);
cudaError_t launch_dense_skinny(const DenseProduct &p, cudaStream_t s);

// Plans of two gradients that go in one launch.
void dense_plan_two(int64_t M0, int64_t N0, int64_t K0, int64_t M1, int64_t N1, int64_t K1,
                    DensePlan *plan0, DensePlan *plan1);
// One or two gradients (EPI_LINEAR without bias, activation or addend; B
// stored along its rows) in one launch, which with column_out also adds up the
// rows of column_part [column_rows, columns].
cudaError_t launch_dense_gradients(const DenseProduct *const *p, const DensePlan *const *plan,
                                   float *const *partial, int count, const float *column_part,
                                   int column_rows, int columns, int half, void *column_out,
                                   int32_t *status, cudaStream_t s);

}  // namespace moe
