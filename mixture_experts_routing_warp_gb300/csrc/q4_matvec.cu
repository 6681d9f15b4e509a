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
//    four lanes of a row hold different groups: an E4M3 scale times an E2M1
//    value has 6 significant bits and fits fp16's range, so the product is
//    exact. E8M0 scales span 2^-127 .. 2^127: each row takes its scales
//    relative to one reference 2^(r - 127), its own first scale, and 2^(s - r)
//    is exact in fp16 for -14 <= s - r <= 12; the row's sum is scaled by the
//    reference in fp32. Steps with a scale outside that run group by group.
//  - Activations become fp16 once per CTA, each token's row scaled by a power
//    of two so that its largest magnitude lies in [2^14, 2^15): bf16's 8 (or
//    fp16's 11) significant bits stay exact down to 2^-28 of the row's
//    maximum (fp32 h: 11 bits, half an fp16 step), values below 2^-39 of it
//    vanish. The sum is scaled back in fp32.
#include "moe_internal.cuh"

#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int kQ4Threads = 512;  // one CTA per SM
constexpr int kQ4Warps = kQ4Threads / 32;
constexpr int kSlab = 128;         // columns per warp step: 32 per lane of a quad
constexpr int kRing = 4;           // steps of weights in flight per warp
constexpr int kSlabXBytes = 2048;  // fp16 fragments of 8 tokens x 128 columns
constexpr int kMaxSlabsX = 96;     // slabs x 8-token blocks of activations resident at once

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
  int slabs;                  // slabs of a row
  int chunk, chunks;          // slabs whose activations are resident at once; how many such
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

// A unit: a group of row tiles of one expert against one block of its tokens.
struct Q4Unit {
  int e, tb, tg;  // expert, token block, tile group
};

template <int NB>
struct Q4Shared {
  alignas(16) float red[2][kQ4Warps][NB][32][4];  // partial sums, read and written as float4
  int cnt[kMaxExperts + 1];  // first slot of each expert (offs)
  int blk[kMaxExperts + 1];  // exclusive prefix of the experts' token blocks
  int warp_sum[kQ4Warps];
  int row[8 * NB];           // the block's rows of x
  uint32_t amax[8 * NB];     // largest magnitude of each (bits)
  float inv[8 * NB];         // what undoes their scaling
};

// A warp step's share of a lane: 32 codes of two rows and their scales.
struct Q4Step {
  uint4 w0, w1;
  uint32_t s0, s1;
};

// FMT: moe_q4_format; NB: blocks of 8 tokens per unit.
template <int FMT, int NB>
__global__ void __launch_bounds__(kQ4Threads, 1) q4_kernel(const Q4Args a) {
  constexpr int TB = 8 * NB;                        // tokens per unit
  constexpr int G = FMT == MOE_Q4_MXFP4 ? 32 : 16;  // columns per scale
  extern __shared__ __align__(16) unsigned char smem_x[];
  __shared__ Q4Shared<NB> sh;
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;

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
      // offsets of a caller's own making stay inside [0, N]
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
    if (lane == 31) sh.warp_sum[wid] = inc;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < wid; ++w) base += sh.warp_sum[w];
    if (tid < a.E) {
      sh.blk[tid] = base + inc - nb;
      if (tid == a.E - 1) sh.blk[a.E] = base + inc;
    }
    __syncthreads();
  }

  // Warps along a row (kw): one needs no join, but a unit is then 16 row
  // tiles, and units are dealt out whole. The fewest that leave a CTA 12
  // units or more, so that the last round idles little; at most 8, and no
  // more than the row has slabs.
  const int blocks = sh.blk[a.E], tiles = (a.R + 15) / 16;
  int kw = 1, tile_groups = (tiles + kQ4Warps - 1) / kQ4Warps;
  while (kw < 8 && kw * 2 <= min(a.slabs, a.chunk) &&
         (int64_t)blocks * tile_groups < 12 * (int64_t)gridDim.x) {
    kw *= 2;
    tile_groups = (tiles * kw + kQ4Warps - 1) / kQ4Warps;
  }
  const int rws = kQ4Warps / kw, kpart = wid % kw, rw = wid / kw;
  const int share = (min(a.slabs, a.chunk) + kw - 1) / kw;  // slabs per warp and chunk
  const int rounds = (share + kRing - 1) / kRing;

  const int64_t units = (int64_t)blocks * tile_groups;
  const int64_t first = units * blockIdx.x / gridDim.x;
  int64_t left = units * (blockIdx.x + 1) / gridDim.x - first;  // units this CTA still has

  Q4Unit cur;
  {
    const int b = (int)(first / tile_groups);
    cur.tg = (int)(first - (int64_t)b * tile_groups);
    int lo = 0, hi = a.E;  // the last expert whose prefix is <= b: it has a block there
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sh.blk[mid] <= b) lo = mid; else hi = mid;
    }
    cur.e = lo;
    cur.tb = b - sh.blk[lo];
  }

  // ---- the ring of weights: `rem` columns are left from this lane's next
  // step on (none when <= 0), its pointers stand there.
  const bool gated = a.mode == Q4_W13 && a.act != MOE_ACT_RELU2;
  const uint8_t *pw0, *pw1, *ps0, *ps1;
  int rem;
  // the lane's two weight rows of a unit: gate and up of one h column for a
  // gated w13, rows g and g + 8 of the tile otherwise. Rows past the end read
  // the last row; their results are dropped.
  auto point = [&](const Q4Unit &q, int ch) {
    const int tile = q.tg * rws + rw;
    int r0, r1;
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
    const int col = (ch * a.chunk + kpart * share) * kSlab + 32 * c;
    const int end = min(min((kpart + 1) * share, a.chunk) + ch * a.chunk, a.slabs) * kSlab;
    rem = min(end, a.C) - col;
    const int64_t at = (int64_t)q.e * a.R;
    const int64_t b0 = at + min(r0, a.R - 1), b1 = at + min(r1, a.R - 1);
    pw0 = a.codes + b0 * (a.C / 2) + col / 2;
    pw1 = a.codes + b1 * (a.C / 2) + col / 2;
    ps0 = a.scales + b0 * (a.C / G) + col / G;
    ps1 = a.scales + b1 * (a.C / G) + col / G;
  };
  auto fetch = [&](Q4Step &st, int d) {
    if (rem > d * kSlab) {
      st.w0 = ld_stream(pw0 + d * (kSlab / 2));
      st.w1 = ld_stream(pw1 + d * (kSlab / 2));
      if (FMT == MOE_Q4_MXFP4) {
        st.s0 = __ldg(ps0 + d * (kSlab / G));
        st.s1 = __ldg(ps1 + d * (kSlab / G));
      } else {
        st.s0 = __ldg(reinterpret_cast<const uint16_t *>(ps0 + d * (kSlab / G)));
        st.s1 = __ldg(reinterpret_cast<const uint16_t *>(ps1 + d * (kSlab / G)));
      }
    } else {
      st.w0 = st.w1 = make_uint4(0u, 0u, 0u, 0u);
      st.s0 = st.s1 = FMT == MOE_Q4_MXFP4 ? 127u : 0u;
    }
  };
  auto advance = [&]() {
    rem -= kRing * kSlab;
    pw0 += kRing * (kSlab / 2);
    pw1 += kRing * (kSlab / 2);
    ps0 += kRing * (kSlab / G);
    ps1 += kRing * (kSlab / G);
  };
  Q4Step ring[kRing];
  if (left > 0) {
    point(cur, 0);
#pragma unroll
    for (int d = 0; d < kRing; ++d) fetch(ring[d], d);
    advance();
  }

  if (a.mode == Q4_W2) {
    pdl_wait();
    pdl_launch_dependents();
  }

  // ---- activations of a token block as fp16 B fragments: for slab s, quarter
  // q and token block b, lane (g, c) finds columns 128 s + 32 c + 8 q .. + 7 of
  // token 8 b + g in its 16 bytes.
  int nt = 0;
  auto load_x = [&](const Q4Unit &q, int ch, bool fresh) {
    const int p0 = sh.cnt[q.e] + q.tb * TB;
    nt = max(min(TB, sh.cnt[q.e + 1] - p0), 0);
    __syncthreads();  // the previous block's fragments and scales are no longer read
    if (fresh) {
      if (tid < TB) {
        sh.amax[tid] = 0u;
        if (tid < nt)  // a row in range whatever col_sorted holds
          sh.row[tid] = a.mode != Q4_W13
                            ? p0 + tid
                            : min(max(__ldg(a.col_sorted + p0 + tid), 0), (int)a.N - 1) / a.k;
      }
      __syncthreads();
      const int segs = (a.C / 8 + 31) / 32;  // a warp takes 32 x 8 columns of one token
      for (int i = wid; i < nt * segs; i += kQ4Warps) {
        const int t = i / segs, at = (i - t * segs) * 256 + lane * 8;
        uint32_t m = 0u;
        if (at < a.C) {
          float v[8];
          load_x8(a.x, a.x_dtype, (int64_t)sh.row[t] * a.C + at, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) atomicMax(&sh.amax[t], m);
      }
      __syncthreads();
    }
    const int c_lo = ch * a.chunk * kSlab;
    const int per = (min(a.slabs, (ch + 1) * a.chunk) * kSlab - c_lo) / 8;
    for (int i = tid; i < nt * per; i += kQ4Threads) {
      const int t = i / per, at = i - t * per, col = c_lo + at * 8;
      // scale exponent: the row's largest magnitude into [2^14, 2^15); a row
      // of zeros, or one that is not finite, keeps its values
      const uint32_t m = sh.amax[t];
      const int ex = (int)(m >> 23);
      const int sc = m == 0u || ex == 255 ? 0 : min(14 + 127 - ex, 126);
      const float f = exp2i(sc);
      if (at == 0) sh.inv[t] = exp2i(-sc);
      float x[8] = {};
      if (col < a.C) load_x8(a.x, a.x_dtype, (int64_t)sh.row[t] * a.C + col, x);
      if (ex == 255) {  // finite values of a row that holds an infinity stay finite
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (fabsf(x[j]) < INFINITY) x[j] = fminf(fmaxf(x[j], -65504.f), 65504.f);
      }
      __half2 h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(x[2 * j] * f, x[2 * j + 1] * f);
      uint4 v;
      memcpy(&v, h, 16);
      // at = 16 s + 4 c + q
      reinterpret_cast<uint4 *>(
          smem_x)[(((at >> 4) * 4 + (at & 3)) * NB + (t >> 3)) * 32 + (t & 7) * 4 + ((at >> 2) & 3)] = v;
    }
    __syncthreads();
  };

  // Sums of the unit. With one token block the two products of a quarter go
  // to sums of their own, which halves the chain of dependent instructions.
  constexpr int NS = NB == 1 ? 2 : NB;
  float acc[NS][4] = {};
  uint32_t ref0 = 127u, ref1 = 127u;  // MXFP4: the rows' reference scales

  // one step's products into d: the lane's codes times m0 / m1 (a half-pair
  // each for columns 0..15 and 16..31 of its 32)
  auto products = [&](float (*d)[4], const Q4Step &st, const uint4 *frag, const uint32_t *m0,
                      const uint32_t *m1) {
    const uint32_t w0[4] = {st.w0.x, st.w0.y, st.w0.z, st.w0.w};
    const uint32_t w1[4] = {st.w1.x, st.w1.y, st.w1.z, st.w1.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t v0[4], v1[4], A[2][4];
      e2m1x8_to_half2(w0[q], v0);
      e2m1x8_to_half2(w1[q], v1);
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
        mma16816(d[NB == 1 ? 1 : b], A[1], x.z, x.w);
      }
    }
  };
  auto compute = [&](const Q4Step &st, const uint4 *frag) {
    if (FMT == MOE_Q4_NVFP4) {
      const uint32_t h0 = e4m3x2_to_half2(st.s0), h1 = e4m3x2_to_half2(st.s1);
      const uint32_t m0[2] = {__byte_perm(h0, h0, 0x1010), __byte_perm(h0, h0, 0x3232)};
      const uint32_t m1[2] = {__byte_perm(h1, h1, 0x1010), __byte_perm(h1, h1, 0x3232)};
      products(acc, st, frag, m0, m1);
      return;
    }
    const int d0 = (int)st.s0 - (int)ref0, d1 = (int)st.s1 - (int)ref1;
    const bool far = (uint32_t)(d0 + 14) > 26u || (uint32_t)(d1 + 14) > 26u || st.s0 == 255u ||
                     st.s1 == 255u;
    uint32_t e0 = (uint32_t)(d0 + 15) * 0x04000400u, e1 = (uint32_t)(d1 + 15) * 0x04000400u;
    if (!__any_sync(0xffffffffu, far)) {
      const uint32_t m0[2] = {e0, e0}, m1[2] = {e1, e1};
      products(acc, st, frag, m0, m1);
      return;
    }
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {  // the lanes c = j of every row: one group per row
      const uint32_t t0 = __shfl_sync(0xffffffffu, st.s0, (lane & ~3) + j);
      const uint32_t t1 = __shfl_sync(0xffffffffu, st.s1, (lane & ~3) + j);
      const uint32_t one = c == j ? 0x3c003c00u : 0u;
      const uint32_t m[2] = {one, one};
      float d[NS][4] = {};
      products(d, st, frag, m, m);
      // 2^(t - ref) in two factors, each in range
      const int h0 = ((int)t0 - (int)ref0) / 2, h1 = ((int)t1 - (int)ref1) / 2;
      const float a0 = t0 == 255u ? NAN : exp2i(h0), b0 = exp2i((int)t0 - (int)ref0 - h0);
      const float a1 = t1 == 255u ? NAN : exp2i(h1), b1 = exp2i((int)t1 - (int)ref1 - h1);
#pragma unroll
      for (int b = 0; b < NS; ++b) {
        acc[b][0] = fmaf(d[b][0] * a0, b0, acc[b][0]);
        acc[b][1] = fmaf(d[b][1] * a0, b0, acc[b][1]);
        acc[b][2] = fmaf(d[b][2] * a1, b1, acc[b][2]);
        acc[b][3] = fmaf(d[b][3] * a1, b1, acc[b][3]);
      }
    }
  };
  // the finished sums v of one row tile and token block: rows g, g + 8 (or
  // gate, up) of tokens 2 c and 2 c + 1
  auto store = [&](const float *v, int tile, int b) {
    const float ms = a.mscale ? __ldg(a.mscale + cur.e) : 1.f;
    const int64_t p0 = sh.cnt[cur.e] + cur.tb * TB;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = b * 8 + c * 2 + j;
      if (t >= nt) continue;
      const float s = sh.inv[t];
      const float lo = v[j] * ms * s, hi = v[2 + j] * ms * s;
      const int64_t p = p0 + t;
      const int row = tile * 16 + g;
      if (a.mode == Q4_W13) {
        float *h = static_cast<float *>(a.out);
        if (gated) {
          const int I = a.R >> 1, col = tile * 8 + g;
          if (col < I) h[p * I + col] = activate(lo, hi, a.ap);
        } else {
          if (row < a.R) h[p * a.R + row] = relu2(lo);
          if (row + 8 < a.R) h[p * a.R + row + 8] = relu2(hi);
        }
      } else {
        uint16_t *o = static_cast<uint16_t *>(a.out) + p * a.R;
        const bool half = a.out_dtype == MOE_FP16;
        if (row < a.R)
          o[row] = half ? __half_as_ushort(__float2half_rn(lo)) : float_to_bf16_bits(lo);
        if (row + 8 < a.R)
          o[row + 8] = half ? __half_as_ushort(__float2half_rn(hi)) : float_to_bf16_bits(hi);
      }
    }
  };

  bool new_block = true;
  int turn = 0, ch = 0, round = 0, x_chunk = -1;
  while (left > 0) {
    if (new_block || ch != x_chunk) {
      load_x(cur, ch, new_block);
      x_chunk = ch;
      new_block = false;
    }
    if (FMT == MOE_Q4_MXFP4 && round == 0 && ch == 0) {
      // each row's first scale, kept where 2^(s - ref) of any s has room
      ref0 = __shfl_sync(0xffffffffu, ring[0].s0, lane & ~3);
      ref1 = __shfl_sync(0xffffffffu, ring[0].s1, lane & ~3);
      ref0 = min(max(ref0, 96u), 158u);
      ref1 = min(max(ref1, 96u), 158u);
    }
    // what the ring takes up next: the next round, chunk or unit
    Q4Unit nxt = cur;
    bool next_block = false, more = true;
    const bool round_last = round + 1 == rounds, unit_last = round_last && ch + 1 == a.chunks;
    if (unit_last) {
      more = left > 1;
      if (++nxt.tg == tile_groups) {
        nxt.tg = 0;
        ++nxt.tb;
        next_block = true;
        while (nxt.e < a.E - 1 && sh.blk[nxt.e] + nxt.tb >= sh.blk[nxt.e + 1]) {
          ++nxt.e;
          nxt.tb = 0;
        }
      }
      if (more) point(nxt, 0);
    } else if (round_last) {
      point(cur, ch + 1);
    }
    // this round's slabs inside the chunk: s0 .. s0 + steps - 1
    const int s0 = kpart * share + round * kRing;
    const int steps = min(min((kpart + 1) * share, a.chunk), a.slabs - ch * a.chunk) - s0;
    const uint4 *frag = reinterpret_cast<const uint4 *>(smem_x) + s0 * (4 * NB * 32) + lane;
#pragma unroll
    for (int d = 0; d < kRing; ++d) {
      if (d < steps) compute(ring[d], frag + d * (4 * NB * 32));
      if (more) fetch(ring[d], d);
    }
    if (more) advance();
    if (!unit_last) {
      if (round_last) ++ch;
      round = round_last ? 0 : round + 1;
      continue;
    }
    // ---- the unit's end
    if (NB == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[0][i] += acc[NS - 1][i];
    }
    if (FMT == MOE_Q4_MXFP4) {
      const float f0 = exp2i((int)ref0 - 127), f1 = exp2i((int)ref1 - 127);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        acc[b][0] *= f0;
        acc[b][1] *= f0;
        acc[b][2] *= f1;
        acc[b][3] *= f1;
      }
    }
    if (kw == 1) {
#pragma unroll
      for (int b = 0; b < NB; ++b) store(acc[b], cur.tg * rws + rw, b);
    } else {
      // join the warps along the row; another warp finishes a tile each unit
      const int buf = turn & 1;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        *reinterpret_cast<float4 *>(sh.red[buf][wid][b][lane]) =
            make_float4(acc[b][0], acc[b][1], acc[b][2], acc[b][3]);
      __syncthreads();  // the other buffer's readers passed this barrier a unit ago
      for (int i = (wid + turn * rws * NB) & (kQ4Warps - 1); i < rws * NB; i += kQ4Warps) {
        const int b = i % NB, r = i / NB;
        float v[4] = {};
        for (int w = 0; w < kw; ++w) {
          const float4 t = *reinterpret_cast<const float4 *>(sh.red[buf][r * kw + w][b][lane]);
          v[0] += t.x;
          v[1] += t.y;
          v[2] += t.z;
          v[3] += t.w;
        }
        store(v, cur.tg * rws + r, b);
      }
      ++turn;
    }
#pragma unroll
    for (int b = 0; b < NS; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[b][i] = 0.f;
    cur = nxt;
    new_block = next_block;
    --left;
    ch = round = 0;
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
  a.chunk = a.slabs < kMaxSlabsX / NB ? a.slabs : kMaxSlabsX / NB;
  a.chunks = (a.slabs + a.chunk - 1) / a.chunk;
  static PerDeviceOnce configured;
  cudaError_t err = configured.run([] {
    cudaError_t e = uniform_carveout(q4_kernel<FMT, NB>);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(q4_kernel<FMT, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kMaxSlabsX * kSlabXBytes);
  });
  if (err != cudaSuccess) return err;
  err = launch_dependent(q4_kernel<FMT, NB>, dim3((unsigned)device_sm_count()), dim3(kQ4Threads),
                         (size_t)a.chunk * NB * kSlabXBytes, s, a);
  return err == cudaSuccess ? cudaGetLastError() : err;
}

cudaError_t launch_format(Q4Args &a, int format, cudaStream_t s) {
  const bool two = a.N > 8 * (int64_t)(a.offs ? a.E / 2 : 1);
  if (format == MOE_Q4_MXFP4)
    return two ? launch<MOE_Q4_MXFP4, 2>(a, s) : launch<MOE_Q4_MXFP4, 1>(a, s);
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
