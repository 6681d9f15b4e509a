// q4_matvec.cu -- products of few token rows with 4-bit weights
// (moe_linear_q4, moe_grouped_ffn_q4): y[p, r] = sum_c W_e[r, c] * x[p, c],
// W_e[r, c] = E2M1 code * group scale, for each expert's slots p.
//
// At decode sizes every weight is read once per step and used for a handful
// of tokens: the floor is the weight bytes, 4.25 (MXFP4) or 4.5 (NVFP4) bits
// each, as long as a weight costs under about 2.9 issue slots (6.8 TB/s is
// ~44 weights per SM and clock against 128 lanes). It costs 2.8 (NVFP4) to 3.6
// (MXFP4), and with 4 warps per scheduler about half the slots stay empty on the
// latency of dependent instructions: GPT-OSS experts for 64 tokens 157 and 170 us
// against floors of 66 and 63, for one token 26.5 and 28.5 against 8.3 and 7.8.
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
//    relative to one reference 2^(r - 127), the largest of its first slab, and
//    2^(s - r) is exact in fp16 for -14 <= s - r <= 12; the row's sum is scaled
//    by the reference in fp32. Steps with a scale outside that, in a group that
//    is not all zeros, run group by group.
//  - Activations become fp16 once per CTA, each token's row scaled by a power
//    of two so that its largest magnitude lies in [2^14, 2^15): bf16's 8 (or
//    fp16's 11) significant bits stay exact down to 2^-28 of the row's
//    maximum, values below 2^-39 of it vanish. The sum is scaled back in fp32.
//  - The fp32 h of the experts takes two of the 8 token columns, its fp16 value
//    and what that leaves, 22 bits in all (with one term, 11 bits, the error of
//    an fp16 result was that of h). So w2's units hold half as many tokens as
//    w13's. Up to 4 slots per expert that costs nothing; beyond it w2's codes
//    are converted once per 8 tokens and not per 16 (GPT-OSS experts, 64 tokens,
//    one term and two: NVFP4 143 and 156 us, MXFP4 155 and 163).
#include <cuda_fp16.h>

#include <type_traits>

#include "operators.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kQ4Threads = 512;  // one CTA per SM
constexpr int kQ4Warps = kQ4Threads / 32;
constexpr int kSlab = 128;         // columns per warp step: 32 per lane of a quad
constexpr int kSlabXBytes = 2048;  // fp16 fragments of 8 tokens x 128 columns
constexpr int kSmemMax = 226 * 1024;  // dynamic and static shared memory of a CTA

// Slabs per step. Two halve the waits and the ring's bookkeeping: NVFP4, 64
// tokens of the GPT-OSS experts, 170 -> 158 us. MXFP4 gains nothing (156 us
// either way: its checks of the scales are per slab), so it takes one.
__host__ __device__ constexpr int step_slabs(int fmt) { return fmt == MOE_Q4_MXFP4 ? 1 : 2; }
// Shared memory of one step: the lanes' codes of two rows each, 16 bytes a
// lane, row and slab, then the 16 rows' scales (4 bytes; 16) as whole 4-byte
// words, one word more than they fill where they start inside one.
__host__ __device__ constexpr int scale_words(int fmt) { return fmt == MOE_Q4_MXFP4 ? 2 : 5; }
__host__ __device__ constexpr int step_bytes(int fmt) {
  return 1024 * step_slabs(fmt) + 64 * scale_words(fmt);
}
// Steps of weights on their way per warp: four slabs, 70 KB per SM in all. More
// only make the first copies wait for one another: eight took the experts of
// one token (GPT-OSS, MXFP4) from 30.3 us to 31.5.
__host__ __device__ constexpr int ring_steps(int fmt) { return 4 / step_slabs(fmt); }
// Units whose partial sums may be on their way to the warps that join them.
__host__ __device__ constexpr int red_slots(int nb) { return nb == 1 ? 3 : 2; }

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
  int act;                    // Q4_W13: moe_activation, layout in `ap`
  int slabs;                  // slabs of a row
  int chunk, chunks;          // slabs whose activations are resident at once; how many such
  int64_t scale_bytes;        // of all matrices
  uint32_t *ctrl;             // control block for the status of the bounded waits, or null
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

// Asynchronous copies to shared memory, AT and FROM bytes past the addresses
// (of a word, `bytes` are read and the rest filled with zeros); one group per
// warp step.
template <int AT, int FROM>
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(AT),
               "n"(FROM)
               : "memory");
}
template <int AT, int FROM>
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0 + %2], [%1 + %3], 4;" ::"r"(dst), "l"(src), "n"(AT),
               "n"(FROM)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Wait for a phase of an mbarrier, at most kWaitTimeoutNs; a wait that gives
// up is recorded and the kernel goes on to its end (its result is void).
__device__ __forceinline__ void wait_phase(uint32_t bar, uint32_t parity, uint32_t *ctrl) {
  if (tc::mbar_try_wait(bar, parity)) return;
  const long long deadline = wait_deadline(kWaitTimeoutNs);
  while (!tc::mbar_try_wait(bar, parity))
    if (clock64() > deadline) {
      record_status(ctrl, MOE_ERR_TIMEOUT);
      return;
    }
}

// 2^e as a float, e in [-127, 127].
__device__ __forceinline__ float exp2i(int e) {
  return e == -127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(e + 127) << 23);
}

// Tokens per unit: 8 token columns a block, two of them for one of h.
__host__ __device__ constexpr int block_tokens(int mode) { return mode == Q4_W2 ? 4 : 8; }

// BOTH: the launch runs both products of the experts.
template <int NB, bool BOTH>
struct Q4Shared {
  unsigned long long full[2][red_slots(NB)], empty[2][red_slots(NB)];  // mbarriers, by product
  int4 info[red_slots(NB)];  // unit in a slot: expert, first token slot, tokens, first tile
  int tile_end[red_slots(NB)];  // tiles from here on are not the unit's
  int part[red_slots(NB)];   // and its part of amax
  int cnt[kMaxExperts + 1];  // first slot of each expert (offs)
  int blk[BOTH + 1][kMaxExperts + 1];  // exclusive prefix of the experts' units, by product
  int warp_sum[BOTH + 1][kQ4Warps];
  int64_t t0, t1;            // the CTA's row tiles
  int row[8 * NB];           // the block's rows of x
  uint32_t amax[4][8 * NB];  // largest magnitude of each token's row (bits), by block
};

// Scale exponent of a row: its largest magnitude comes into [2^14, 2^15); a
// row of zeros, or one that is not finite, keeps its values.
__device__ __forceinline__ int row_exponent(uint32_t amax) {
  const int ex = (int)(amax >> 23);
  return amax == 0u || ex == 255 ? 0 : min(14 + 127 - ex, 126);
}

// Sums of a unit. With one token block the two products of a quarter go to
// sums of their own, which halves the chain of dependent instructions.
template <int NB>
struct Q4Sums {
  static constexpr int N = NB == 1 ? 2 : NB;
  float v[N][4];
};

// One slab's products into d: the lane's codes of two rows times m0 / m1 (a
// half-pair each for columns 0..15 and 16..31 of its 32).
template <int NB>
__device__ __forceinline__ void products(Q4Sums<NB> &d, const uint4 &c0, const uint4 &c1,
                                         const uint4 *x, const uint32_t *m0, const uint32_t *m1) {
  const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w};
  const uint32_t w1[4] = {c1.x, c1.y, c1.z, c1.w};
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
      const uint4 f = x[(q * NB + b) * 32];
      mma16816(d.v[b], A[0], f.x, f.y);
      mma16816(d.v[NB == 1 ? 1 : b], A[1], f.z, f.w);
    }
  }
}

// Whether a lane's 32 codes are all zeros, of either sign.
__device__ __forceinline__ bool all_zeros(const uint4 &c) {
  return ((c.x | c.y | c.z | c.w) & 0x77777777u) == 0u;
}

// A row's reference from its first slab (scale s and codes c of this lane's
// group): the largest scale but those of groups of zeros, which quantisers give
// a scale far below the others', and NaN; about a trained weight's where all
// four are such.
__device__ __forceinline__ uint32_t row_reference(uint32_t s, const uint4 &c) {
  uint32_t top = s == 255u || all_zeros(c) ? 0u : s;
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  return top == 0u ? 120u : min(max(top, 96u), 158u);
}

// An MXFP4 slab whose scales do not fit one reference: one group per row at a
// time, the lanes c = j; the other lanes' activations count as zeros (their
// weights may not: an infinity would meet a zero there). Rare, so it is kept
// small: a quarter at a time, codes read where they are used.
template <int NB>
__device__ __forceinline__ void products_far(Q4Sums<NB> &acc, const unsigned char *codes,
                                             const uint4 *x, uint32_t s0, uint32_t s1,
                                             uint32_t ref0, uint32_t ref1) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int j = 0; j < 4; ++j) {
    const uint32_t mine = (lane & 3) == j ? 0xffffffffu : 0u;
    float d[NB][4] = {};
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      uint32_t v0[4], v1[4];
      e2m1x8_to_half2(*reinterpret_cast<const uint32_t *>(codes + 4 * q), v0);
      e2m1x8_to_half2(*reinterpret_cast<const uint32_t *>(codes + 512 + 4 * q), v1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t A[4] = {v0[2 * i], v1[2 * i], v0[2 * i + 1], v1[2 * i + 1]};
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint4 f = x[(q * NB + b) * 32];
          mma16816(d[b], A, (i ? f.z : f.x) & mine, (i ? f.w : f.y) & mine);
        }
      }
    }
    // 2^(t - ref) in two factors, each in range
    const uint32_t t0 = __shfl_sync(0xffffffffu, s0, (lane & ~3) + j);
    const uint32_t t1 = __shfl_sync(0xffffffffu, s1, (lane & ~3) + j);
    const int h0 = ((int)t0 - (int)ref0) / 2, h1 = ((int)t1 - (int)ref1) / 2;
    const float a0 = t0 == 255u ? NAN : exp2i(h0), b0 = exp2i((int)t0 - (int)ref0 - h0);
    const float a1 = t1 == 255u ? NAN : exp2i(h1), b1 = exp2i((int)t1 - (int)ref1 - h1);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      acc.v[b][0] = fmaf(d[b][0] * a0, b0, acc.v[b][0]);
      acc.v[b][1] = fmaf(d[b][1] * a0, b0, acc.v[b][1]);
      acc.v[b][2] = fmaf(d[b][2] * a1, b1, acc.v[b][2]);
      acc.v[b][3] = fmaf(d[b][3] * a1, b1, acc.v[b][3]);
    }
  }
}

// The activations with NaN passed on: the layer's own take minima and maxima,
// which drop it, and a corrupt token or scale would go on as a finite number.
__device__ __forceinline__ float activate_or_nan(float g, float u, const ActParams &p) {
  const float h = activate(g, u, p);
  return isnan(g) || isnan(u) ? NAN : h;
}
__device__ __forceinline__ float relu2_or_nan(float a) { return isnan(a) ? a : relu2(a); }

// One product. FMT: moe_q4_format; NB: blocks of 8 tokens per unit; CHUNKS:
// rows may be too long for all their activations to be resident; SECOND: after
// a Q4_W13 in the same launch, whose h is complete when the grid barrier that
// this CTA arrived at (`arrived`) opens.
template <int FMT, int NB, bool CHUNKS, int MODE, bool SECOND, bool BOTH>
__device__ __forceinline__ void q4_run(const Q4Args &a, Q4Shared<NB, BOTH> &sh, uint32_t arrived) {
  constexpr int TB = block_tokens(MODE) * NB;       // tokens per unit
  constexpr int G = FMT == MOE_Q4_MXFP4 ? 32 : 16;  // columns per scale
  constexpr int SW = scale_words(FMT), RS = red_slots(NB), STEP = step_bytes(FMT);
  constexpr int SL = step_slabs(FMT), RING = ring_steps(FMT);
  const int chunks = CHUNKS ? a.chunks : 1;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  float4 *red = reinterpret_cast<float4 *>(smem);  // [RS][kQ4Warps][NB][32]
  unsigned char *ring = smem + RS * kQ4Warps * NB * 512 + wid * (RING * STEP);
  uint4 *xs = reinterpret_cast<uint4 *>(smem + RS * kQ4Warps * NB * 512 + kQ4Warps * RING * STEP);
  const uint32_t full_at = tc::smem_u32(sh.full[SECOND]),
                 empty_at = tc::smem_u32(sh.empty[SECOND]);

  if (tid < 4 * TB) (&sh.amax[0][0])[tid] = 0u;
  // offs may come from the kernel before this one (Q4_W13); before Q4_W2 lies
  // the Q4_W13 launch, which passed its own wait before triggering this one,
  // so what offs holds is complete and the weights can be fetched ahead.
  if (MODE != Q4_W2) {
    pdl_wait();
    pdl_launch_dependents();
  }
  // units of tokens of each expert and their prefix, for the second product too
  const auto &blk = sh.blk[SECOND];
  if (!SECOND) {
    constexpr int TB2 = block_tokens(Q4_W2) * NB;
    int lo = 0, nb = 0, nb2 = 0;
    if (a.offs == nullptr) {
      if (tid == 0) nb = (int)((a.N + TB - 1) / TB);
      if (tid <= 1) sh.cnt[tid] = tid == 0 ? 0 : (int)a.N;
    } else if (tid < a.E) {
      // offsets of a caller's own making stay inside [0, N]
      lo = min(max(__ldg(a.offs + tid), 0), (int)a.N);
      const int hi = min(max(__ldg(a.offs + tid + 1), lo), (int)a.N);
      nb = (hi - lo + TB - 1) / TB;
      if (BOTH) nb2 = (hi - lo + TB2 - 1) / TB2;
      sh.cnt[tid] = lo;
      if (tid == a.E - 1) sh.cnt[a.E] = hi;
    }
    int inc = nb, inc2 = nb2;
    if (a.E > 1) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
        if (BOTH) {
          const int v2 = __shfl_up_sync(0xffffffffu, inc2, o);
          if (lane >= o) inc2 += v2;
        }
      }
      if (lane == 31) {
        sh.warp_sum[0][wid] = inc;
        if (BOTH) sh.warp_sum[BOTH][wid] = inc2;
      }
      __syncthreads();
      for (int w = 0; w < wid && w < kMaxExperts / 32; ++w) {
        inc += sh.warp_sum[0][w];
        if (BOTH) inc2 += sh.warp_sum[BOTH][w];
      }
    }
    if (tid < a.E) {
      sh.blk[0][tid] = inc - nb;
      if (BOTH) sh.blk[BOTH][tid] = inc2 - nb2;
      if (tid == a.E - 1) {
        sh.blk[0][a.E] = inc;
        if (BOTH) sh.blk[BOTH][a.E] = inc2;
      }
    }
    __syncthreads();
  }

  // Row tiles (16 rows) of all token blocks are dealt out evenly, in order, to
  // the CTAs. A unit is what a CTA works on at a time: kQ4Warps / kw tiles of
  // one block, kw warps along each row. More warps along a row leave fewer
  // idle at the end of the CTA's tiles, but cost a join and, for each unit,
  // about the time of two steps.
  const int blocks = blk[a.E], tiles = (a.R + 15) / 16, in_row = min(a.slabs, a.chunk);
  int kw = 1;
  const int64_t all = (int64_t)blocks * tiles;
  const int64_t share = all >> 32 ? all / gridDim.x : (uint32_t)all / gridDim.x;
  const int rest = (int)(all - share * gridDim.x);  // CTAs with one tile more
  {
    int64_t best = INT64_MAX;
    for (int w = 0; w <= 3 && 1 << w <= in_row; ++w) {
      const int64_t n = (((share + 1) << w) + kQ4Warps - 1) / kQ4Warps;
      const int64_t cost = n * (((in_row + (1 << w) - 1) >> w) + 2);
      if (cost < best) {
        best = cost;
        kw = 1 << w;
      }
    }
  }
  const int rws = kQ4Warps / kw, kpart = wid & (kw - 1), rw = wid / kw;
  const int items = rws * NB;  // joins per unit
  if (tid == 0) {
    for (int i = 0; i < RS; ++i) {
      tc::mbar_init(full_at + 8 * i, kQ4Warps);
      tc::mbar_init(empty_at + 8 * i, items);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const int64_t t0 = share * blockIdx.x + min((int)blockIdx.x, rest);
  const int64_t t1 = t0 + share + ((int)blockIdx.x < rest ? 1 : 0);
  // the CTA's tiles [lo, hi) of a block
  if (tid == 0) {
    sh.t0 = t0;
    sh.t1 = t1;
  }
  __syncthreads();
  auto tiles_of = [&](int b, int &lo, int &hi) {
    const int64_t at = (int64_t)b * tiles;
    lo = (int)max(sh.t0 - at, (int64_t)0);
    hi = (int)min(sh.t1 - at, (int64_t)tiles);
  };
  const int b0 = (int)(t0 >> 32 ? t0 / tiles : (uint32_t)t0 / (uint32_t)tiles);
  const int b1 = t1 == t0 ? b0 - 1
                          : b0 + (int)((uint32_t)(t1 - 1 - (int64_t)b0 * tiles) / (uint32_t)tiles);
  // block b is the tb-th of expert e, the last one whose prefix is <= b
  auto where = [&](int b, int &e, int &tb) {
    int lo = 0, hi = a.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (blk[mid] <= b) lo = mid; else hi = mid;
    }
    e = lo;
    tb = b - blk[lo];
  };
  // this warp's slabs of a chunk: n of them from lo
  auto slabs_of = [&](int ch, int &lo, int &n) {
    const int m = min(a.chunk, a.slabs - ch * a.chunk), at = m * kpart / kw;
    lo = ch * a.chunk + at;
    n = m * (kpart + 1) / kw - at;
  };
  int s_lo, s_n;  // with a single chunk, for good
  slabs_of(0, s_lo, s_n);

  // ---- weights on their way: step after step, RING steps ahead of the
  // products, by an iterator over (block, tile, chunk, slab)
  const bool gated = MODE == Q4_W13 && a.act != MOE_ACT_RELU2;
  const bool split = gated && a.ap.layout == MOE_W13_PACKED;  // up rows I below the gate rows
  // Row r (0..15) of a tile. Fragment rows g and g + 8 are gate and up of one
  // column of h for a gated w13. Rows past the end read the last row; their
  // results are dropped.
  auto tile_row = [&](int tile, int r) {
    const int row = !split ? tile * 16 + r
                           : tile * 8 + (r & 7) + (r & 8 ? a.R >> 1 : 0);
    return min(row, a.R - 1);
  };
  const int frag0 = gated && !split ? 2 * g : g, frag1 = gated && !split ? 2 * g + 1 : g + 8;
  int p_b = b0, p_tile = 0, p_end = 0, p_ch = 0;
  int p_n = 0, p_left = 0;  // slabs to issue; columns left from the lane's next one
  // the block's matrix, and in it the lane's two code rows (in 16 bytes; a
  // matrix has 2^36 codes at most) and its scale words (in bytes)
  const uint8_t *p_codes = a.codes, *p_scales = a.scales;
  uint32_t pw0 = 0, pw1 = 0, ps = 0;
  uint32_t p_safe = 0;  // scale words from here on may pass the array's end
  auto point = [&]() {
    int lo = s_lo;
    p_n = s_n;
    if (chunks > 1) slabs_of(p_ch, lo, p_n);
    const uint32_t row16 = (uint32_t)a.C / 32, col16 = (uint32_t)lo * 4 + c;
    pw0 = (uint32_t)tile_row(p_tile, frag0) * row16 + col16;
    pw1 = (uint32_t)tile_row(p_tile, frag1) * row16 + col16;
    p_left = a.C - lo * kSlab - 32 * c;
    // whole words around the row's bytes of the slab, two lanes per row
    ps = ((uint32_t)tile_row(p_tile, lane >> 1) * (uint32_t)(a.C / G) & ~3u) + lo * (kSlab / G) +
         4 * (lane & 1);
  };
  auto enter = [&]() {  // the first tile of block p_b for this warp
    int e, tb, lo;
    where(p_b, e, tb);
    tiles_of(p_b, lo, p_end);
    p_tile = lo + rw;
    p_codes = a.codes + (int64_t)e * a.R * (a.C / 2);
    const int64_t at = (int64_t)e * a.R * (a.C / G);  // a multiple of 4 where e > 0
    p_scales = a.scales + at;
    p_safe = (uint32_t)min(max(a.scale_bytes - at - (4 * SW - 1), (int64_t)0),
                           (int64_t)UINT32_MAX);
  };
  // bytes before the array's end of a word that may pass it
  const uint32_t lane_at = tc::smem_u32(ring) + lane * 16;
  const uint32_t scales_at =
      tc::smem_u32(ring) + 1024 * SL + (lane >> 1) * (4 * SW) + (lane & 1) * 4;
  auto copy_edge = [&](uint32_t dst, const uint8_t *src) {
    const int64_t left = a.scales + a.scale_bytes - src;
    copy4(dst, left > 0 ? src : a.scales, left >= 4 ? 4 : left > 0 ? (int)left : 0);
  };
  const bool words_fit = FMT == MOE_Q4_MXFP4 || a.C % 64 == 0;  // in SW - 1 words, or in two
  auto fetch = [&](uint32_t slot) {
    if (p_n <= 0 && p_b <= b1) {  // on to the next chunk, the next tile, the next block
      do {
        if (p_tile >= p_end || ++p_ch == chunks) {
          p_ch = 0;
          if (p_tile < p_end) p_tile += rws;
          if (p_tile >= p_end) {
            if (++p_b > b1) break;
            enter();
            if (p_tile >= p_end) continue;
          }
        }
        point();
      } while (p_n <= 0);
    }
    if (p_n > 0) {
      // (places that are not filled keep older codes: finite, against zero activations)
      const uint32_t dst = lane_at + slot;
      const uint8_t *w0 = p_codes + (uint64_t)pw0 * 16, *w1 = p_codes + (uint64_t)pw1 * 16;
      if (p_left > 0) {
        copy16<0, 0>(dst, w0);
        copy16<512, 0>(dst, w1);
      }
      if (SL == 2 && p_n > 1 && p_left > kSlab) {
        copy16<1024, kSlab / 2>(dst, w0);
        copy16<1536, kSlab / 2>(dst, w1);
      }
      const uint32_t sdst = scales_at + slot;
      const uint8_t *src = p_scales + ps;
      if (ps < p_safe) {
        copy4<0, 0>(sdst, src);
        if (SW == 5) copy4<8, 8>(sdst, src);
        if (!words_fit && (lane & 1) == 0) copy4<4 * (SW - 1), 4 * (SW - 1)>(sdst, src);
      } else {
        copy_edge(sdst, src);
        if (SW == 5) copy_edge(sdst + 8, src + 8);
        if (!words_fit && (lane & 1) == 0) copy_edge(sdst + 4 * (SW - 1), src + 4 * (SW - 1));
      }
      pw0 += SL * kSlab / 32;
      pw1 += SL * kSlab / 32;
      ps += SL * kSlab / G;
      p_left -= SL * kSlab;
      p_n -= SL;
    }
    copies_commit();  // a group per step, also past the end: the waits count groups
  };
  // where the lane's scales lie in a step: fixed, as tiles are 8 or 16 rows
  // apart and several matrices have a multiple of 64 rows
  const int s_at0 =
      1024 * SL + frag0 * (4 * SW) + ((uint32_t)tile_row(rw, frag0) * (a.C / G) & 3) + c * (32 / G);
  const int s_at1 =
      1024 * SL + frag1 * (4 * SW) + ((uint32_t)tile_row(rw, frag1) * (a.C / G) & 3) + c * (32 / G);

  // ---- activations of a unit's tokens as fp16 B fragments: for slab s, quarter
  // q and block b, lane (g, c) finds columns 128 s + 32 c + 8 q .. + 7 of
  // token 8 b + g in its 16 bytes; of h, token 4 b + g / 2, the fp16 value where
  // g is even and what it leaves where g is odd. What lies there for tokens
  // past the unit's end reaches only sums that are dropped.
  int nt = 0, part = 3, cur_e = 0, cur_p0 = 0;  // tokens of the block; its part of sh.amax
  int cur_b = b0;
  // BYTES of an activation: 4 warps (fp32; 2 for 16 bits) take a token's row
  // together, 3 (6) times 8 columns per lane in flight. A row that fits is
  // read once, its values held until the row's largest magnitude is known.
  auto load_rows = [&](auto bytes, int ch, bool fresh) {
    constexpr int WPT = decltype(bytes)::value, BATCH = 12 / WPT, PER = BATCH * 32 * WPT;
    constexpr int RAW = WPT / 2;  // 16-byte words of 8 columns
    const int c_lo = ch * a.chunk * kSlab;
    const int pieces = min(a.chunk, a.slabs - ch * a.chunk) * (kSlab / 8);
    const bool once = fresh && chunks == 1 && pieces <= PER;
#pragma unroll 1
    for (int t0 = 0; t0 < nt; t0 += kQ4Warps / WPT) {
      const int t = t0 + wid / WPT, q0 = wid % WPT * 32 + lane;
      const uint4 *row = reinterpret_cast<const uint4 *>(
          static_cast<const char *>(a.x) + (t < nt ? (int64_t)sh.row[t] * a.C * WPT : 0));
      uint4 raw[BATCH][RAW];
      auto load = [&](int col0, int from) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int at = from + k * 32 * WPT + q0;
#pragma unroll
          for (int i = 0; i < RAW; ++i) {
            raw[k][i] = make_uint4(0u, 0u, 0u, 0u);
            if (t < nt && col0 + at * 8 < a.C) raw[k][i] = row[(col0 / 8 + at) * RAW + i];
          }
        }
      };
      auto floats = [&](const uint4 *r, float *f) {
        const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
        if constexpr (WPT == 4) {
          const uint32_t v[4] = {r[RAW - 1].x, r[RAW - 1].y, r[RAW - 1].z, r[RAW - 1].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[j] = __uint_as_float(w[j]);
            f[4 + j] = __uint_as_float(v[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (a.x_dtype == MOE_FP16) {
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
      };
      if (fresh) {
        uint32_t m = 0u;
#pragma unroll 1
        for (int from = 0; from < a.slabs * (kSlab / 8); from += PER) {
          load(0, from);
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            float v[8];
            floats(raw[k], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
          }
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0 && t < nt) atomicMax(&sh.amax[part][t], m);
        __syncthreads();
      }
      const uint32_t m = t < nt ? sh.amax[part][t] : 0u;
      const float f = exp2i(row_exponent(m));
#pragma unroll 1
      for (int from = 0; from < pieces; from += PER) {
        if (!once) load(c_lo, from);
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int at = from + k * 32 * WPT + q0;
          if (t >= nt || at >= pieces) continue;
          float x[8];
          floats(raw[k], x);
          if ((m >> 23) == 255u) {  // finite values beside an infinity stay finite
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (fabsf(x[j]) < INFINITY) x[j] = fminf(fmaxf(x[j], -65504.f), 65504.f);
          }
          __half2 h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(x[2 * j] * f, x[2 * j + 1] * f);
          uint4 v;
          memcpy(&v, h, 16);
          // at = 16 slab + 4 c + quarter
          constexpr int BT = block_tokens(MODE), COLS = 8 / BT;
          uint4 *to = xs + (((at >> 4) * 4 + (at & 3)) * NB + (uint32_t)t / BT) * 32 +
                      (t & (BT - 1)) * (4 * COLS) + ((at >> 2) & 3);
          to[0] = v;
          if constexpr (MODE == Q4_W2) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 d = __half22float2(h[j]);
              // an infinity or NaN leaves nothing (inf - inf would be NaN)
              const float lo = fabsf(d.x) < INFINITY ? x[2 * j] * f - d.x : 0.f;
              const float hi = fabsf(d.y) < INFINITY ? x[2 * j + 1] * f - d.y : 0.f;
              h[j] = __floats2half2_rn(lo, hi);
            }
            memcpy(&v, h, 16);
            to[4] = v;
          }
        }
      }
    }
  };
  auto load_x = [&](int ch, bool fresh) {
    if (fresh) {
      int tb;
      where(cur_b, cur_e, tb);
      cur_p0 = sh.cnt[cur_e] + tb * TB;
      nt = max(min(TB, sh.cnt[cur_e + 1] - cur_p0), 0);
      part = (part + 1) & 3;
      if (tid < nt)  // a row in range whatever col_sorted holds
        sh.row[tid] = MODE != Q4_W13
                          ? cur_p0 + tid
                          : min(max(__ldg(a.col_sorted + cur_p0 + tid), 0), (int)a.N - 1) / a.k;
    }
    __syncthreads();  // the previous fragments are no longer read
    load_rows(std::integral_constant<int, MODE == Q4_W2 ? 4 : 2>{}, ch, fresh);
    __syncthreads();
    // the block before the last has been stored by every warp: its part of
    // amax is free for the block after the next, past another barrier
    if (fresh && tid < TB) sh.amax[(part + 2) & 3][tid] = 0u;
  };

  // The first block's activations come before the weights, whose copies would
  // keep them waiting; but Q4_W2 may only fetch weights until Q4_W13 is done.
  if (b0 <= b1) {
    if (MODE != Q4_W2) load_x(0, true);
    enter();
    if (p_tile < p_end) point();
  }
#pragma unroll 1
  for (int d = 0; d < RING; ++d) fetch(d * STEP);
  if (SECOND) {
    if (!grid_wait(a.ctrl, arrived, kWaitTimeoutNs)) {  // every thread of the CTA: no result
      copies_wait<0>();
      return;
    }
  } else if (MODE == Q4_W2) {
    pdl_wait();
    pdl_launch_dependents();
  }
  if (MODE == Q4_W2 && b0 <= b1) load_x(0, true);

  constexpr int NS = Q4Sums<NB>::N;
  Q4Sums<NB> acc = {};
  uint32_t ref0 = 127u, ref1 = 127u;  // MXFP4: the rows' reference scales

  // A step, `left` columns before the row's end for this lane (columns past it
  // have no codes and scales of their own, and activations of zero: any finite
  // weight will do); `two`: its second slab is not past the warp's share. Its
  // place takes the step RING ahead as soon as it is read by all lanes.
  auto compute = [&](int slot, const uint4 *x, bool fresh, int left, bool two) {
    const unsigned char *st = ring + slot, *codes = st + lane * 16;
    auto code = [&](int h, int row) {
      return *reinterpret_cast<const uint4 *>(codes + h * 1024 + row * 512);
    };
    auto refill = [&] {
      __syncwarp();
      fetch(slot);
    };
    if constexpr (FMT == MOE_Q4_NVFP4) {
      auto slab = [&](int h, auto then) {
        uint32_t s0 = *reinterpret_cast<const uint16_t *>(st + s_at0 + h * 8);
        uint32_t s1 = *reinterpret_cast<const uint16_t *>(st + s_at1 + h * 8);
        if (left <= h * kSlab) s0 = s1 = 0u;
        const uint32_t h0 = e4m3x2_to_half2(s0), h1 = e4m3x2_to_half2(s1);
        const uint32_t m0[2] = {__byte_perm(h0, h0, 0x1010), __byte_perm(h0, h0, 0x3232)};
        const uint32_t m1[2] = {__byte_perm(h1, h1, 0x1010), __byte_perm(h1, h1, 0x3232)};
        const uint4 c0 = code(h, 0), c1 = code(h, 1);
        then();
        products<NB>(acc, c0, c1, x + h * (4 * NB * 32), m0, m1);
      };
      if (two) {
        slab(0, [] {});
        slab(1, refill);
      } else {
        slab(0, refill);
      }
    } else {
      uint32_t s0 = st[s_at0], s1 = st[s_at1];
      if (left <= 0) s0 = s1 = 0u;  // (of stale codes: no part of a reference)
      if (fresh) {  // the unit's first step
        ref0 = row_reference(s0, code(0, 0));
        ref1 = row_reference(s1, code(0, 1));
      }
      if (left <= 0) {
        s0 = ref0;
        s1 = ref1;
      }
      auto apart = [&] {
        return __any_sync(0xffffffffu, s0 - ref0 + 14u > 26u || s1 - ref1 + 14u > 26u);
      };
      bool far = false;
      if (apart()) {
        // groups of zeros take any scale but NaN; what is still apart takes the
        // place of the products below, whose zero weights would meet infinities.
        // With one block the step ends here, a second copy of the refill: a test
        // after the first one keeps the products from overlapping it (GPT-OSS
        // experts, 8 tokens: 95 us, 87 so); with two blocks the copy costs spills
        // (64 tokens: 168 us, 175 with it).
        if (s0 != 255u && all_zeros(code(0, 0))) s0 = ref0;
        if (s1 != 255u && all_zeros(code(0, 1))) s1 = ref1;
        far = apart();
        if (far) products_far<NB>(acc, codes, x, s0, s1, ref0, ref1);
        if (NB == 1 && far) {
          refill();
          return;
        }
      }
      const uint32_t e0 = (s0 - ref0 + 15u) * 0x04000400u, e1 = (s1 - ref1 + 15u) * 0x04000400u;
      const uint32_t m0[2] = {e0, e0}, m1[2] = {e1, e1};
      const uint4 c0 = code(0, 0), c1 = code(0, 1);
      refill();
      if (NB == 1 || !far) products<NB>(acc, c0, c1, x, m0, m1);
    }
  };
  // The finished sums v of one row tile and token block: fragment rows g and
  // g + 8 of columns 2 c and 2 c + 1, two tokens or the two terms of one.
  auto store = [&](const float *v, int e, int p0, int q_nt, int q_part, int tile, int b) {
    const float ms = a.mscale ? __ldg(a.mscale + e) : 1.f;
#pragma unroll
    for (int j = 0; j < (MODE == Q4_W2 ? 1 : 2); ++j) {
      const int t = MODE == Q4_W2 ? b * 4 + c : b * 8 + c * 2 + j;
      if (t >= q_nt) continue;
      const float s = exp2i(-row_exponent(sh.amax[q_part][t]));
      const float lo = (MODE == Q4_W2 ? v[0] + v[1] : v[j]) * ms * s;
      const float hi = (MODE == Q4_W2 ? v[2] + v[3] : v[2 + j]) * ms * s;
      const int64_t p = (int64_t)p0 + t;
      const int row = tile * 16 + g;
      if (MODE == Q4_W13) {
        float *h = static_cast<float *>(a.out);
        if (gated) {
          const int I = a.R >> 1, col = tile * 8 + g;
          if (col < I) h[p * I + col] = activate_or_nan(lo, hi, a.ap);
        } else {
          if (row < a.R) h[p * a.R + row] = relu2_or_nan(lo);
          if (row + 8 < a.R) h[p * a.R + row + 8] = relu2_or_nan(hi);
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
  // Joins a unit's partial sums along the row; other warps take it each unit.
  auto join = [&](int u, int rs, uint32_t phase) {
    for (int i = (wid - u * items) & (kQ4Warps - 1); i < items; i += kQ4Warps) {
      const int b = i % NB, r = i / NB;
      wait_phase(full_at + 8 * rs, phase, a.ctrl);
      const int4 q = sh.info[rs];
      const int q_part = sh.part[rs], tile = q.w + r;
      const bool real = tile < sh.tile_end[rs];
      float v[4] = {};
      if (real)
        for (int w = 0; w < kw; ++w) {
          const float4 t = red[((rs * kQ4Warps + r * kw + w) * NB + b) * 32 + lane];
          v[0] += t.x;
          v[1] += t.y;
          v[2] += t.z;
          v[3] += t.w;
        }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty_at + 8 * rs);
      if (real) store(v, q.x, q.y, q.z, q_part, tile, b);
    }
  };

  int rs = 0, slot = 0, u = 0;
  uint32_t rs_phase = 0;  // the slot of red; how often it came round, modulo 2
  for (; cur_b <= b1; ++cur_b) {
    int t_lo, t_hi;
    tiles_of(cur_b, t_lo, t_hi);
    if (cur_b > b0) load_x(0, true);
    for (int tile0 = t_lo; tile0 < t_hi; tile0 += rws) {
      const bool busy = tile0 + rw < t_hi;
      for (int ch = 0; ch < chunks; ++ch) {
        int lo = s_lo, n = s_n;
        if (chunks > 1) {
          if (ch > 0 || tile0 > t_lo) load_x(ch, false);
          slabs_of(ch, lo, n);
        }
        if (!busy) n = 0;
        const uint4 *x = xs + (lo - ch * a.chunk) * (4 * NB * 32) + lane;
        int left = a.C - lo * kSlab - 32 * c;
#pragma unroll 1
        for (int d = 0; d < n; d += SL) {
          copies_wait<RING - 1>();
          __syncwarp();  // the lanes' copies are in, for all lanes
          compute(slot, x, ch == 0 && d == 0, left, SL == 2 && d + 1 < n);
          slot = slot == (RING - 1) * STEP ? 0 : slot + STEP;
          x += SL * 4 * NB * 32;
          left -= SL * kSlab;
        }
      }
      if (NB == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc.v[0][i] += acc.v[NS - 1][i];
      }
      if (FMT == MOE_Q4_MXFP4) {
        const float f0 = exp2i((int)ref0 - 127), f1 = exp2i((int)ref1 - 127);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          acc.v[b][0] *= f0;
          acc.v[b][1] *= f0;
          acc.v[b][2] *= f1;
          acc.v[b][3] *= f1;
        }
      }
      if (kw == 1) {
        if (busy)
#pragma unroll
          for (int b = 0; b < NB; ++b) store(acc.v[b], cur_e, cur_p0, nt, part, tile0 + rw, b);
      } else {
        wait_phase(empty_at + 8 * rs, rs_phase ^ 1u, a.ctrl);
#pragma unroll
        for (int b = 0; b < NB; ++b)
          red[((rs * kQ4Warps + wid) * NB + b) * 32 + lane] =
              make_float4(acc.v[b][0], acc.v[b][1], acc.v[b][2], acc.v[b][3]);
        if (tid == 0) {
          sh.info[rs] = make_int4(cur_e, cur_p0, nt, tile0);
          sh.tile_end[rs] = t_hi;
          sh.part[rs] = part;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(full_at + 8 * rs);
        // one unit late, so that the other warps' sums are there
        if (u > 0) join(u - 1, rs == 0 ? RS - 1 : rs - 1, rs == 0 ? rs_phase ^ 1u : rs_phase);
        if (++rs == RS) {
          rs = 0;
          rs_phase ^= 1u;
        }
      }
#pragma unroll
      for (int b = 0; b < NS; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc.v[b][i] = 0.f;
      ++u;
    }
  }
  if (kw > 1 && u > 0)
    join(u - 1, rs == 0 ? RS - 1 : rs - 1, rs == 0 ? rs_phase ^ 1u : rs_phase);
  copies_wait<0>();

  if (MODE == Q4_W2) {  // rows of no kept slot
    const int64_t words = (a.N - sh.cnt[a.E]) * a.R / 2;  // R is even: 4-byte words
    uint32_t *z = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) +
                                               (int64_t)sh.cnt[a.E] * a.R);
    for (int64_t i = (int64_t)blockIdx.x * kQ4Threads + tid; i < words;
         i += (int64_t)gridDim.x * kQ4Threads)
      z[i] = 0u;
  }
}

template <int FMT, int NB, bool CHUNKS, int MODE>
__global__ void __launch_bounds__(kQ4Threads, 1) q4_kernel(const Q4Args a) {
  __shared__ Q4Shared<NB, false> sh;
  q4_run<FMT, NB, CHUNKS, MODE, false>(a, sh, 0u);
}

// Both products of the experts in one launch: a CTA that is done with its
// share of w13 fetches its first w2 weights while the others finish. The grid
// barrier needs all CTAs resident (one per SM); it is bounded like every wait.
template <int FMT, int NB>
__global__ void __launch_bounds__(kQ4Threads, 1) q4_ffn_kernel(const Q4Args a, const Q4Args b) {
  __shared__ Q4Shared<NB, true> sh;
  q4_run<FMT, NB, false, Q4_W13, false>(a, sh, 0u);
  const uint32_t arrived = grid_arrive(a.ctrl);
  q4_run<FMT, NB, false, Q4_W2, true>(b, sh, arrived);
}

// Slabs whose activations fit beside the ring and the partial sums.
template <int FMT, int NB>
constexpr int slabs_that_fit() {
  return (kSmemMax - (int)sizeof(Q4Shared<NB, true>) -
          kQ4Warps * (ring_steps(FMT) * step_bytes(FMT) + red_slots(NB) * NB * 512)) /
         (NB * kSlabXBytes);
}

template <int FMT, int NB>
constexpr int fixed_smem() {
  return kQ4Warps * (ring_steps(FMT) * step_bytes(FMT) + red_slots(NB) * NB * 512);
}

// Fills in what follows from the sizes; returns the dynamic shared memory.
template <int FMT, int NB>
size_t plan(Q4Args &a) {
  constexpr int fit = slabs_that_fit<FMT, NB>();
  a.chunk = a.slabs < fit ? a.slabs : fit;
  a.chunks = (a.slabs + a.chunk - 1) / a.chunk;
  a.scale_bytes = (int64_t)a.E * a.R * (a.C / (FMT == MOE_Q4_MXFP4 ? 32 : 16));
  return fixed_smem<FMT, NB>() + (size_t)a.chunk * NB * kSlabXBytes;
}

// The kernel of both products waits for all its CTAs: a cooperative launch has
// them resident together or not at all, whatever other streams run.
template <int FMT, int NB, auto Kern, typename... Args>
cudaError_t go(size_t smem, cudaStream_t s, const Args &...args) {
  constexpr bool cooperative = sizeof...(Args) == 2;
  static PerDeviceOnce configured;
  cudaError_t err = configured.run([] {
    cudaError_t e = uniform_carveout(Kern);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                fixed_smem<FMT, NB>() +
                                    slabs_that_fit<FMT, NB>() * NB * kSlabXBytes);
  });
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)device_sm_count()), block(kQ4Threads);
  if constexpr (cooperative) {
    void *params[] = {const_cast<Args *>(&args)...};
    err = cudaLaunchCooperativeKernel(Kern, grid, block, params, smem, s);
  } else {
    err = launch_dependent(Kern, grid, block, smem, s, args...);
  }
  return err == cudaSuccess ? cudaGetLastError() : err;
}

// Two token blocks per unit for more than 8 tokens of one matrix, and for
// experts of 7 or more on average, if a row's activations then stay resident.
// One and two blocks in us, MXFP4 / NVFP4:
//   one matrix 16384 x 2880, 8 tokens     13.4 14.9 / 12.3 14.5
//                            9            23.8 15.9 / 20.4 15.6
//   GPT-OSS experts, average of 5         138.9 153.2 / 136.4 141.4
//                               6         151.9 153.5 / 152.4 143.7
//                               8         180.0 170.5 / 173.0 157.8
//   8 experts of 2880 x 2880,   6         54.5 59.1 / 47.4 54.5
//                               8         65.3 65.5 / 55.0 58.3
//                               10        75.4 68.5 / 64.3 64.3
// A single expert does not mind the second reading of its weights: 15.4 and
// 17.1 for one token, 22.7 and 22.8 for 16. The average counts dropped slots too,
// as the host does not know how many a rank keeps: with 4 of 32 experts and 8
// tokens that takes 30.5 us for 27.3 (the layer). The layer does know what to
// expect, but its rows would then not be moe_grouped_ffn_q4's bit for bit.
template <int FMT>
bool two_blocks(const Q4Args &a) {
  return (a.offs ? a.N >= 7 * (int64_t)a.E : a.N > 8) && a.slabs <= slabs_that_fit<FMT, 2>();
}

template <int FMT, int MODE>
cudaError_t launch(Q4Args &a, cudaStream_t s) {
  a.slabs = (a.C + kSlab - 1) / kSlab;
  if (two_blocks<FMT>(a)) {
    const size_t smem = plan<FMT, 2>(a);
    return go<FMT, 2, q4_kernel<FMT, 2, false, MODE>>(smem, s, a);
  }
  const size_t smem = plan<FMT, 1>(a);
  if (a.chunks > 1) return go<FMT, 1, q4_kernel<FMT, 1, true, MODE>>(smem, s, a);
  return go<FMT, 1, q4_kernel<FMT, 1, false, MODE>>(smem, s, a);
}

template <int MODE>
cudaError_t launch(Q4Args &a, int format, cudaStream_t s) {
  return format == MOE_Q4_MXFP4 ? launch<MOE_Q4_MXFP4, MODE>(a, s)
                                : launch<MOE_Q4_NVFP4, MODE>(a, s);
}

cudaError_t launch_dense(Q4Args &a, int format, cudaStream_t s) {
  return launch<Q4_DENSE>(a, format, s);
}

// w13 and w2 in one launch, where both take the same variant without chunks;
// *done says whether.
template <int FMT>
cudaError_t launch_both(Q4Args &a, Q4Args &b, cudaStream_t s, bool *done) {
  a.slabs = (a.C + kSlab - 1) / kSlab;
  b.slabs = (b.C + kSlab - 1) / kSlab;
  *done = true;
  if (two_blocks<FMT>(a) && two_blocks<FMT>(b)) {
    const size_t sa = plan<FMT, 2>(a), sb = plan<FMT, 2>(b);
    return go<FMT, 2, q4_ffn_kernel<FMT, 2>>(sa > sb ? sa : sb, s, a, b);
  }
  if (!two_blocks<FMT>(a) && !two_blocks<FMT>(b)) {
    const size_t sa = plan<FMT, 1>(a), sb = plan<FMT, 1>(b);
    if (a.chunks == 1 && b.chunks == 1)
      return go<FMT, 1, q4_ffn_kernel<FMT, 1>>(sa > sb ? sa : sb, s, a, b);
  }
  *done = false;
  return cudaSuccess;
}

cudaError_t launch_experts(Q4Args &a, Q4Args &b, int format13, int format2, cudaStream_t s) {
  if (format13 == format2) {
    bool done = false;
    const cudaError_t err = format13 == MOE_Q4_MXFP4 ? launch_both<MOE_Q4_MXFP4>(a, b, s, &done)
                                                     : launch_both<MOE_Q4_NVFP4>(a, b, s, &done);
    if (done) return err;
  }
  const cudaError_t err = launch<Q4_W13>(a, format13, s);
  return err == cudaSuccess ? launch<Q4_W2>(b, format2, s) : err;
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
  return launch_dense(a, w.format, s);
}

cudaError_t launch_ffn_q4(const void *x, const moe_routing_meta &m, const moe_q4_matrix &w13,
                          const moe_q4_matrix &w2, int64_t N, int E, int k, int H, int I,
                          const ActParams &act, int dtype, float *h, void *y_sorted,
                          uint32_t *ctrl, cudaStream_t s) {
  Q4Args a = {};
  a.ctrl = ctrl;
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
  a.act = act.act;
  a.ap = act;
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
  return launch_experts(a, b, w13.format, w2.format, s);
}

}  // namespace moe
