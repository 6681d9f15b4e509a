// q4_matvec.cu -- products of few token rows with 4-bit weights
// (moe_linear_q4, moe_grouped_ffn_q4): y[p, r] = sum_c W_e[r, c] * x[p, c],
// W_e[r, c] = E2M1 code * group scale, for each expert's slots p.
//
// At decode sizes every weight is read once per step and used for a handful
// of tokens: bound by the weight bytes, 4.25 (MXFP4) or 4.5 (NVFP4) bits
// each, as long as a weight costs under about 2.7 issue slots (6.8 TB/s is
// ~47 weights per SM and clock against 128 lanes).
//
//  - The products run on mma.sync m16n8k16 (fp16 inputs, fp32 sums): 16
//    weight rows x 8 tokens, so 1 to 8 tokens cost the same, and a lane's
//    share of a row is any k-subset as long as both operands agree on it.
//    Each lane therefore takes 16 contiguous bytes (32 codes) of row g and of
//    row g + 8, straight from the checkpoint's row-major layout: 128 columns
//    (a "slab") per warp step, no repacking. (tcgen05's E2M1 kinds want 8- or
//    4-bit activations.)
//  - One conversion instruction makes two fp16 values of a byte of codes
//    (exact). The group scale is folded in before the product, because the
//    four lanes of a row hold four different groups: an E4M3 scale times an
//    E2M1 value has 6 significant bits and fits fp16's range, so the product
//    is exact. E8M0 scales span 2^-127 .. 2^127: a slab's scales are taken
//    relative to the row's largest of the slab, 2^(s - max) >= 2^-23 exact in
//    fp16, and the slab's sum is scaled by 2^max in fp32. A slab whose scales
//    lie further apart (no quantiser makes one) runs group by group.
//  - Activations become fp16 once per CTA, each token's row scaled by a power
//    of two so that its largest magnitude lies in [2^14, 2^15): bf16's 8 (or
//    fp16's 11) significant bits stay exact down to 2^-28 of the row's
//    maximum (fp32 h: 11 bits, half an fp16 step), values below 2^-39 of it
//    vanish. The sum is scaled back in fp32.
#include "moe_internal.cuh"

#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int kQ4Threads = 256;
constexpr int kQ4Warps = kQ4Threads / 32;
constexpr int kSlab = 128;       // columns per warp step: 32 per lane of a quad
constexpr int kRing = 4;         // warp steps in flight in registers
constexpr int kSlabXBytes = 2048;  // fp16 fragments of 8 tokens x 128 columns
constexpr int kMaxSlabsX = 48;   // slabs of activations resident at once (x 8-token blocks)

// Which row of x a slot reads, and where its result goes.
enum Q4Mode {
  Q4_DENSE = 0,  // slot p: row p of x, row p of out
  Q4_W13 = 1,    // slot p: row col_sorted[p] / k of x, fp32 row p of h (activated)
  Q4_W2 = 2      // slot p: fp32 row p of h, row p of out; rows past the slots zero
};

struct Q4Args {
  const uint8_t *codes, *scales;
  const float *mscale;        // [E] or null (1)
  const int32_t *offs;        // [E + 1]; null: one matrix, slots [0, N)
  const int32_t *col_sorted;  // Q4_W13
  const void *x;
  void *out;
  int64_t N;                  // slots at most (rows of out)
  int E, k, R, C;             // matrices of R rows, C columns
  int x_dtype, out_dtype;     // moe_dtype
  int mode;
  int act;                    // Q4_W13: moe_activation, layout in `ap`
  int slabs, spw, kw;         // slabs of a row; per warp; warps along a row
  int chunk;                  // warp steps whose activations are resident at once
  int tile_groups;            // groups of (kQ4Warps / kw) row tiles
  ActParams ap;
};

// Eight E2M1 codes (two per byte, the even column low) as four fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t word, uint32_t *h) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(word));
}

__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t pair) {
  uint32_t h;
  asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}"
      : "=r"(h) : "r"(pair));
  return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  __half2 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  const __half2 z = __hmul2(x, y);
  uint32_t r;
  memcpy(&r, &z, 4);
  return r;
}

__device__ __forceinline__ void mma16816(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Weights are read once: keep them out of L1.
__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Eight consecutive activations (16-byte aligned) as floats.
__device__ __forceinline__ void load_x8(const void *x, int dtype, int64_t i, float *f) {
  if (dtype == MOE_FP32) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
    const float4 u = p[0], v = p[1];
    f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
    f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
    return;
  }
  const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + i);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (dtype == MOE_FP16) {
      __half2 h;
      memcpy(&h, &w[j], 4);
      f[2 * j] = __low2float(h);
      f[2 * j + 1] = __high2float(h);
    } else {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

// 2^e as a float, e in [-127, 127].
__device__ __forceinline__ float exp2i(int e) {
  return e == -127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(e + 127) << 23);
}

// Where a warp stands in its CTA's run of units; one unit is a group of row
// tiles of one expert against one block of its tokens.
struct Q4Cursor {
  int64_t unit;
  int e, tb, tg;  // expert, token block, tile group
};

template <int NB>
struct Q4Shared {
  alignas(16) float red[2][kQ4Warps][NB][32][4];  // partial sums, read and written as float4
  int cnt[kMaxExperts + 1];    // first slot of each expert (offs)
  int blk[kMaxExperts + 1];    // exclusive prefix of the experts' token blocks
  uint32_t amax[8 * NB];
  float inv[8 * NB];
};

template <int FMT, int NB>
__global__ void __launch_bounds__(kQ4Threads, 2) q4_kernel(const Q4Args a) {
  constexpr int TB = 8 * NB;                       // tokens per block
  constexpr int G = FMT == MOE_Q4_MXFP4 ? 32 : 16;  // columns per scale
  extern __shared__ __align__(16) unsigned char smem_x[];
  __shared__ Q4Shared<NB> sh;
  __shared__ int s_warp[kQ4Warps];
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int kw = wid % a.kw, rw = wid / a.kw, rws = kQ4Warps / a.kw;

  // offs may come from the kernel before this one (Q4_W13); before Q4_W2 lies
  // the Q4_W13 launch, which passed its own wait before triggering this one,
  // so what offs holds is complete and the weights can be fetched ahead.
  if (a.mode != Q4_W2) {
    pdl_wait();
    pdl_launch_dependents();
  }
  // token blocks of each expert and their prefix
  {
    int lo = 0, nb = 0;
    if (a.offs == nullptr) {
      if (tid == 0) nb = (int)((a.N + TB - 1) / TB);
      if (tid <= 1) sh.cnt[tid] = tid == 0 ? 0 : (int)a.N;
    } else if (tid < a.E) {
      // sizes of a caller's own making stay inside [0, N]
      lo = min(max(__ldg(a.offs + tid), 0), (int)a.N);
      const int hi = min(max(__ldg(a.offs + tid + 1), lo), (int)a.N);
      nb = (hi - lo + TB - 1) / TB;
      sh.cnt[tid] = lo;
      if (tid == a.E - 1) sh.cnt[a.E] = hi;
    }
    int inc = nb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s_warp[wid] = inc;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < wid; ++w) base += s_warp[w];
    if (tid < a.E) {
      sh.blk[tid] = base + inc - nb;
      if (tid == a.E - 1) sh.blk[a.E] = base + inc;
    }
    __syncthreads();
  }
  const int64_t units = (int64_t)sh.blk[a.E] * a.tile_groups;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;

  auto seek = [&](int64_t unit) {
    Q4Cursor q;
    q.unit = unit;
    const int b = (int)(unit / a.tile_groups);
    q.tg = (int)(unit - (int64_t)b * a.tile_groups);
    int lo = 0, hi = a.E;  // the last expert whose prefix is <= b: it has a block there
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sh.blk[mid] <= b) lo = mid; else hi = mid;
    }
    q.e = lo;
    q.tb = b - sh.blk[lo];
    return q;
  };
  auto next = [&](Q4Cursor &q) {
    ++q.unit;
    if (++q.tg < a.tile_groups) return;
    q.tg = 0;
    ++q.tb;
    while (q.e < a.E - 1 && sh.blk[q.e] + q.tb >= sh.blk[q.e + 1]) {
      ++q.e;
      q.tb = 0;
    }
  };
  // the lane's two weight rows of a unit: gate and up of one h column for a
  // gated w13, rows g and g + 8 of the tile otherwise. Rows past the end read
  // the last row; their results are dropped.
  const bool gated = a.mode == Q4_W13 && a.act != MOE_ACT_RELU2;
  auto rows_of = [&](const Q4Cursor &q, int &r0, int &r1) {
    const int tile = q.tg * rws + rw;
    if (!gated) {
      r0 = tile * 16 + g;
      r1 = r0 + 8;
    } else if (a.ap.layout == MOE_W13_INTERLEAVED) {
      r0 = tile * 16 + 2 * g;
      r1 = r0 + 1;
    } else {
      r0 = tile * 8 + g;
      r1 = (a.R >> 1) + r0;
    }
    r0 = min(r0, a.R - 1);
    r1 = min(r1, a.R - 1);
  };

  // ---- the ring of weight steps in flight
  uint4 wv[kRing][2];
  uint32_t sv[kRing][2];
  Q4Cursor pf = seek(u0 < u1 ? u0 : 0);
  int pf_step = 0;
  const uint8_t *pw0 = nullptr, *pw1 = nullptr, *ps0 = nullptr, *ps1 = nullptr;
  const int64_t items = (u1 - u0) * a.spw;
  auto point = [&]() {
    int r0, r1;
    rows_of(pf, r0, r1);
    const int64_t b0 = (int64_t)pf.e * a.R + r0, b1 = (int64_t)pf.e * a.R + r1;
    pw0 = a.codes + b0 * (a.C / 2);
    pw1 = a.codes + b1 * (a.C / 2);
    ps0 = a.scales + b0 * (a.C / G);
    ps1 = a.scales + b1 * (a.C / G);
  };
  auto fetch = [&](uint4 *w, uint32_t *s) {
    const int col = (kw + a.kw * pf_step) * kSlab + 32 * c;
    if (col < a.C) {
      w[0] = ld_stream(pw0 + col / 2);
      w[1] = ld_stream(pw1 + col / 2);
      if (FMT == MOE_Q4_MXFP4) {
        s[0] = __ldg(ps0 + col / 32);
        s[1] = __ldg(ps1 + col / 32);
      } else {
        s[0] = __ldg(reinterpret_cast<const uint16_t *>(ps0 + col / 16));
        s[1] = __ldg(reinterpret_cast<const uint16_t *>(ps1 + col / 16));
      }
    } else {
      w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u);
      s[0] = s[1] = 0u;
    }
    if (++pf_step == a.spw) {
      pf_step = 0;
      next(pf);
      if (pf.unit < u1) point();
    }
  };
  if (items > 0) point();
#pragma unroll
  for (int d = 0; d < kRing; ++d)
    if (d < items) fetch(wv[d], sv[d]);

  if (a.mode == Q4_W2) {
    pdl_wait();
    pdl_launch_dependents();
  }

  // ---- activations of a token block as fp16 B fragments: for slab s, quarter
  // q and token block b, lane (g, c) finds columns 128 s + 32 c + 8 q .. + 7 of
  // token 8 b + g in its 16 bytes.
  auto token_row = [&](int p) -> int64_t {
    if (a.mode != Q4_W13) return p;
    return min(max(__ldg(a.col_sorted + p), 0), (int)a.N - 1) / a.k;  // in range whatever it holds
  };
  auto load_x_chunk = [&](const Q4Cursor &q, int step0, bool fresh) {
    const int p0 = sh.cnt[q.e] + q.tb * TB;
    const int nt = min(TB, sh.cnt[q.e + 1] - p0);
    const int chunks = a.C / 8;
    __syncthreads();  // the previous block's fragments and scales are no longer read
    if (fresh) {
      if (tid < TB) sh.amax[tid] = 0u;
      __syncthreads();
      for (int i = tid; i < nt * chunks; i += kQ4Threads) {
        const int t = i / chunks, ch = i - t * chunks;
        const int64_t at = token_row(p0 + t) * a.C + ch * 8;
        float v[8];
        load_x8(a.x, a.x_dtype, at, v);
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
        atomicMax(&sh.amax[t], m);
      }
      __syncthreads();
    }
    // columns [c_lo, c_hi) belong to the steps [step0, step0 + chunk)
    const int c_lo = step0 * a.kw * kSlab;
    const int c_hi = min(a.slabs, (step0 + a.chunk) * a.kw) * kSlab;
    const int per = (c_hi - c_lo) / 8;
    for (int i = tid; i < nt * per; i += kQ4Threads) {
      const int t = i / per, ch = i - t * per, col = c_lo + ch * 8;
      // scale exponent: the row's largest magnitude into [2^14, 2^15); a row
      // of zeros, or one that is not finite, keeps its values
      const uint32_t m = sh.amax[t];
      const int ex = (int)(m >> 23);
      const int sc = m == 0u || ex == 255 ? 0 : min(14 + 127 - ex, 126);
      const float f = exp2i(sc);
      if (ch == 0) sh.inv[t] = exp2i(-sc);
      __half h[8];
      float x[8] = {};
      if (col < a.C) load_x8(a.x, a.x_dtype, token_row(p0 + t) * a.C + col, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float w = x[j] * f;
        // finite values of a row that holds an infinity stay finite
        h[j] = fabsf(w) < INFINITY && fabsf(w) > 65504.f ? __float2half_rn(copysignf(65504.f, w))
                                                        : __float2half_rn(w);
      }
      const int s = ch / 16, lc = (ch / 4) % 4, quarter = ch % 4;
      uint4 v;
      memcpy(&v, h, 16);
      *reinterpret_cast<uint4 *>(
          smem_x + ((((size_t)s * 4 + quarter) * NB + t / 8) * 32 + (t % 8) * 4 + lc) * 16) = v;
    }
    __syncthreads();
  };

  float acc[NB][4] = {};
  Q4Cursor cur = seek(u0 < u1 ? u0 : 0);
  int64_t x_block = -1;  // token block and step that the fragments belong to
  int x_step = -1, step = 0, buf = 0, nt = 0;

  auto compute = [&](const uint4 *w, const uint32_t *s) {
    const int xb = sh.blk[cur.e] + cur.tb, xs = step / a.chunk * a.chunk;
    if (xb != x_block || xs != x_step) {
      load_x_chunk(cur, xs, xb != x_block);
      x_block = xb;
      x_step = xs;
      nt = min(TB, sh.cnt[cur.e + 1] - (sh.cnt[cur.e] + cur.tb * TB));
    }
    const int slab = (kw + a.kw * step) - x_step * a.kw;
    const uint4 *frag =
        reinterpret_cast<const uint4 *>(smem_x) + (size_t)slab * 4 * NB * 32 + lane;
    const bool here = kw + a.kw * step < a.slabs;
    if (here) {
      const uint32_t words[2][4] = {{w[0].x, w[0].y, w[0].z, w[0].w},
                                    {w[1].x, w[1].y, w[1].z, w[1].w}};
      // one pass over the slab with the lane's weights times m0 / m1 (two
      // half-pairs each: columns 0..15 and 16..31 of the lane's 32)
      auto pass = [&](float (*d)[4], const uint32_t *m0, const uint32_t *m1) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t v0[4], v1[4], A[2][4];
          e2m1x8_to_half2(words[0][q], v0);
          e2m1x8_to_half2(words[1][q], v1);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              A[i][2 * h] = hmul2(v0[2 * i + h], m0[q >> 1]);
              A[i][2 * h + 1] = hmul2(v1[2 * i + h], m1[q >> 1]);
            }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (b * 8 + g < nt) x = frag[(q * NB + b) * 32];
            mma16816(d[b], A[0], x.x, x.y);
            mma16816(d[b], A[1], x.z, x.w);
          }
        }
      };
      if (FMT == MOE_Q4_NVFP4) {
        const uint32_t h0 = e4m3x2_to_half2(s[0]), h1 = e4m3x2_to_half2(s[1]);
        const uint32_t m0[2] = {__byte_perm(h0, h0, 0x1010), __byte_perm(h0, h0, 0x3232)};
        const uint32_t m1[2] = {__byte_perm(h1, h1, 0x1010), __byte_perm(h1, h1, 0x3232)};
        pass(acc, m0, m1);
      } else {
        uint32_t b0 = s[0], b1 = s[1];
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          b0 = max(b0, __shfl_xor_sync(0xffffffffu, b0, o));
          b1 = max(b1, __shfl_xor_sync(0xffffffffu, b1, o));
        }
        // columns past C read scale 0: their activations are zero, and only
        // their distance to the maximum must not force the slow way
        const bool real = (kw + a.kw * step) * kSlab + 32 * c < a.C;
        const bool far = real && (b0 - s[0] > 23u || b1 - s[1] > 23u || b0 == 255u || b1 == 255u);
        const bool slow = __any_sync(0xffffffffu, far);
        const int passes = slow ? 4 : 1;
#pragma unroll 1
        for (int j = 0; j < passes; ++j) {
          uint32_t m[2];
          uint32_t t0 = b0, t1 = b1;
          if (slow) {
            t0 = __shfl_sync(0xffffffffu, s[0], (lane & ~3) + j);
            t1 = __shfl_sync(0xffffffffu, s[1], (lane & ~3) + j);
            m[0] = m[1] = c == j ? 0x3c003c00u : 0u;
          } else {
            const __half f0 = __float2half_rn(exp2i(-(int)min(b0 - s[0], 126u)));
            const __half f1 = __float2half_rn(exp2i(-(int)min(b1 - s[1], 126u)));
            m[0] = (uint32_t)__half_as_ushort(f0) * 0x10001u;
            m[1] = (uint32_t)__half_as_ushort(f1) * 0x10001u;
          }
          const uint32_t m0[2] = {m[0], m[0]}, m1[2] = {m[1], m[1]};
          float d[NB][4] = {};
          pass(d, m0, m1);
          const float f0 = t0 == 255u ? NAN : exp2i((int)t0 - 127);
          const float f1 = t1 == 255u ? NAN : exp2i((int)t1 - 127);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            acc[b][0] = fmaf(d[b][0], f0, acc[b][0]);
            acc[b][1] = fmaf(d[b][1], f0, acc[b][1]);
            acc[b][2] = fmaf(d[b][2], f1, acc[b][2]);
            acc[b][3] = fmaf(d[b][3], f1, acc[b][3]);
          }
        }
      }
    }
    if (++step < a.spw) return;
    // ---- the unit's end: join the warps along the row, finish, store
    step = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      *reinterpret_cast<float4 *>(sh.red[buf][wid][b][lane]) =
          make_float4(acc[b][0], acc[b][1], acc[b][2], acc[b][3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[b][i] = 0.f;
    }
    __syncthreads();  // the other buffer's readers passed this barrier a unit ago
    for (int i = tid; i < rws * NB * 32; i += kQ4Threads) {
      const int l = i & 31, b = (i >> 5) % NB, r = (i >> 5) / NB;
      float v[4] = {};
      for (int w = 0; w < a.kw; ++w) {
        const float4 t = *reinterpret_cast<const float4 *>(sh.red[buf][r * a.kw + w][b][l]);
        v[0] += t.x;
        v[1] += t.y;
        v[2] += t.z;
        v[3] += t.w;
      }
      const int tile = cur.tg * rws + r, lg = l >> 2;
      const float ms = a.mscale ? __ldg(a.mscale + cur.e) : 1.f;
      const int p0 = sh.cnt[cur.e] + cur.tb * TB;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = b * 8 + (l & 3) * 2 + j;
        if (t >= nt) continue;
        const float s = sh.inv[t];
        const float lo = v[j] * ms * s, hi = v[2 + j] * ms * s;
        const int64_t p = p0 + t;
        if (a.mode == Q4_W13) {
          float *h = static_cast<float *>(a.out);
          if (gated) {
            const int I = a.R >> 1, col = tile * 8 + lg;
            if (col < I) h[p * I + col] = activate(lo, hi, a.ap);
          } else {
            const int row = tile * 16 + lg;
            if (row < a.R) h[p * a.R + row] = relu2(lo);
            if (row + 8 < a.R) h[p * a.R + row + 8] = relu2(hi);
          }
        } else {
          const int row = tile * 16 + lg;
          uint16_t *o = static_cast<uint16_t *>(a.out) + p * a.R;
          const bool half = a.out_dtype == MOE_FP16;
          if (row < a.R)
            o[row] = half ? __half_as_ushort(__float2half_rn(lo)) : float_to_bf16_bits(lo);
          if (row + 8 < a.R)
            o[row + 8] = half ? __half_as_ushort(__float2half_rn(hi)) : float_to_bf16_bits(hi);
        }
      }
    }
    buf ^= 1;
    next(cur);
  };

  for (int64_t t = 0; t < items; t += kRing) {
#pragma unroll
    for (int d = 0; d < kRing; ++d)
      if (t + d < items) {
        const uint4 w[2] = {wv[d][0], wv[d][1]};
        const uint32_t s[2] = {sv[d][0], sv[d][1]};
        if (t + d + kRing < items) fetch(wv[d], sv[d]);
        compute(w, s);
      }
  }

  if (a.mode == Q4_W2) {  // rows of no kept slot
    const int64_t words = (a.N - sh.cnt[a.E]) * a.R / 2;  // R is even: 4-byte words
    uint32_t *z = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) +
                                               (int64_t)sh.cnt[a.E] * a.R);
    for (int64_t i = (int64_t)blockIdx.x * kQ4Threads + tid; i < words;
         i += (int64_t)gridDim.x * kQ4Threads)
      z[i] = 0u;
  }
}

template <int FMT, int NB>
cudaError_t launch(Q4Args &a, cudaStream_t s) {
  a.slabs = (a.C + kSlab - 1) / kSlab;
  // Warps along a row: the more, the sooner a unit ends and the finer the
  // work splits; but a short row must not leave warps without slabs. The
  // largest count whose rounded-up share wastes at most an eighth.
  a.kw = 1;
  for (int kw = kQ4Warps; kw >= 1; kw /= 2) {
    const int padded = (a.slabs + kw - 1) / kw * kw;
    if (kw == 1 || (padded - a.slabs) * 8 <= a.slabs) {
      a.kw = kw;
      break;
    }
  }
  a.spw = (a.slabs + a.kw - 1) / a.kw;
  a.chunk = kMaxSlabsX / NB / a.kw < 1 ? 1 : kMaxSlabsX / NB / a.kw;
  if (a.chunk > a.spw) a.chunk = a.spw;
  const int rws = kQ4Warps / a.kw;
  const int tiles = (a.R + 15) / 16;
  a.tile_groups = (tiles + rws - 1) / rws;
  const int resident = a.chunk * a.kw < a.slabs ? a.chunk * a.kw : a.slabs;
  const size_t smem = (size_t)resident * NB * kSlabXBytes;
  static PerDeviceOnce configured;
  cudaError_t err = configured.run([] {
    cudaError_t e = uniform_carveout(q4_kernel<FMT, NB>);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(q4_kernel<FMT, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kMaxSlabsX * kSlabXBytes);
  });
  if (err != cudaSuccess) return err;
  // token blocks there can be: every expert's last one may be partial
  const int64_t full = (a.N + 8 * NB - 1) / (8 * NB);
  const int64_t blocks = a.offs ? (a.N < full + a.E ? a.N : full + a.E) : full;
  int64_t grid = (int64_t)device_sm_count() * 2;
  if (grid > blocks * a.tile_groups) grid = blocks * a.tile_groups;
  err = launch_dependent(q4_kernel<FMT, NB>, dim3((unsigned)grid), dim3(kQ4Threads), smem, s, a);
  return err == cudaSuccess ? cudaGetLastError() : err;
}

cudaError_t launch_format(Q4Args &a, int format, cudaStream_t s) {
  const bool two = a.N > 8 * (int64_t)(a.offs ? a.E / 2 : 1);
  if (format == MOE_Q4_MXFP4) return two ? launch<MOE_Q4_MXFP4, 2>(a, s) : launch<MOE_Q4_MXFP4, 1>(a, s);
  return two ? launch<MOE_Q4_NVFP4, 2>(a, s) : launch<MOE_Q4_NVFP4, 1>(a, s);
}

}  // namespace

cudaError_t launch_linear_q4(const void *x, const moe_q4_matrix &w, int64_t n, int R, int C,
                             int dtype, void *y, cudaStream_t s) {
  Q4Args a = {};
  a.codes = w.codes;
  a.scales = w.scales;
  a.mscale = w.matrix_scale;
  a.x = x;
  a.out = y;
  a.N = n;
  a.E = 1;
  a.k = 1;
  a.R = R;
  a.C = C;
  a.x_dtype = a.out_dtype = dtype;
  a.mode = Q4_DENSE;
  return launch_format(a, w.format, s);
}

cudaError_t launch_ffn_q4(const void *x, const moe_routing_meta &m, const moe_q4_matrix &w13,
                          const moe_q4_matrix &w2, int64_t N, int E, int k, int H, int I,
                          const ActParams &act, int dtype, float *h, void *y_sorted,
                          cudaStream_t s) {
  Q4Args a = {};
  a.codes = w13.codes;
  a.scales = w13.scales;
  a.mscale = w13.matrix_scale;
  a.offs = m.offs;
  a.col_sorted = m.col_sorted;
  a.x = x;
  a.out = h;
  a.N = N;
  a.E = E;
  a.k = k;
  a.R = w13_rows(act, I);
  a.C = H;
  a.x_dtype = dtype;
  a.out_dtype = MOE_FP32;
  a.mode = Q4_W13;
  a.act = act.act;
  a.ap = act;
  cudaError_t err = launch_format(a, w13.format, s);
  if (err != cudaSuccess) return err;
  Q4Args b = a;
  b.codes = w2.codes;
  b.scales = w2.scales;
  b.mscale = w2.matrix_scale;
  b.x = h;
  b.out = y_sorted;
  b.R = H;
  b.C = I;
  b.x_dtype = MOE_FP32;
  b.out_dtype = dtype;
  b.mode = Q4_W2;
  return launch_format(b, w2.format, s);
}

}  // namespace moe
