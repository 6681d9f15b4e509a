// dense_api.cu -- the extern "C" entry points of the dense blocks beside the
// experts (norm, linear, gated linear and their gradients): argument checks,
// workspace carving and the launch sequence on the caller's stream.
#include <math.h>

#include "dense.cuh"

using namespace moe;

namespace {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline moe_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

constexpr int kMaxFeatures = 65536;
constexpr int64_t kMaxElements = (int64_t)1 << 38;  // of one matrix: 512 GB of 16-bit values

bool rows_ok(int64_t n, int64_t cols) {
  return n >= 0 && n < (int64_t)INT32_MAX && n * cols < kMaxElements;
}
bool dtype16(int dtype) { return dtype == MOE_BF16 || dtype == MOE_FP16; }

// A product's sizes: `in` features per row of x (whole 16-byte pieces of a
// row, groups of 32 in 8 bits), `out` of the result.
moe_status check_product(int64_t n, int64_t out, int64_t in, int dtype, bool mx) {
  if (in < 1 || in > kMaxFeatures || in % (mx ? 32 : 8) != 0) return MOE_ERR_INVALID_ARG;
  if (out < 1 || out > 2 * kMaxFeatures) return MOE_ERR_INVALID_ARG;
  if (!rows_ok(n, in > out ? in : out)) return MOE_ERR_INVALID_ARG;
  return dtype16(dtype) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

moe_status check_gated(int64_t n, int H, int I, int dtype, const moe_params *params, bool mx,
                       ActParams &act) {
  if (I < 8 || I > kMaxFeatures || I % 8 != 0) return MOE_ERR_INVALID_ARG;
  moe_status st = check_product(n, 2 * (int64_t)I, H, dtype, mx);
  if (st != MOE_OK || (st = resolve_params(params, act, nullptr)) != MOE_OK) return st;
  return act.act == MOE_ACT_RELU2 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_mx8(const moe_mx8_rows *m) {
  if (!m || !m->codes || !m->scales) return MOE_ERR_INVALID_ARG;
  return aligned(m->codes, 16) ? MOE_OK : MOE_ERR_MISALIGNED;
}

bool act_ok(int act) { return act >= MOE_LINEAR_NONE && act <= MOE_LINEAR_RELU2; }

moe_status check_workspace(const void *ws, size_t have, size_t need) {
  if (need == 0) return MOE_OK;
  if (!ws) return have < need ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_ERR_INVALID_ARG;
  if (!aligned(ws, kAlign)) return MOE_ERR_MISALIGNED;
  return have < need ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

char *at(void *ws, size_t off) { return static_cast<char *>(ws) + off; }

// --------------------------------------------------------------- products --
// How a forward product runs: few rows without a workspace, else by a
// plan, with the 8-bit scales in the tensor core's layout and the parts of a
// split sum in the workspace.
struct ForwardPlan {
  bool skinny;
  DensePlan plan;
  size_t bytes;
};
ForwardPlan forward_plan(int64_t n, int64_t out, int64_t in, int kind, bool mx) {
  ForwardPlan f{};
  f.skinny = dense_skinny(n, out, in, kind, mx);
  if (f.skinny) return f;
  f.plan = dense_plan(n, out, in, kind, mx);
  f.bytes = align_up(f.plan.blocks, kAlign) + align_up(f.plan.partial, kAlign);
  return f;
}

moe_status run_forward(const DenseProduct &p, void *workspace, size_t workspace_bytes,
                       int32_t *status, moe_stream stream) {
  const ForwardPlan f = forward_plan(p.M, p.N, p.K, p.kind, p.a.scales != nullptr);
  const moe_status st = check_workspace(workspace, workspace_bytes, f.bytes);
  if (st != MOE_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (f.skinny) return from_cuda(launch_dense_skinny(p, s));
  return from_cuda(
      launch_dense(p, f.plan, static_cast<uint8_t *>(workspace),
                   reinterpret_cast<float *>(at(workspace, align_up(f.plan.blocks, kAlign))),
                   status, s));
}

DenseProduct forward_product(const void *x, const void *w, int64_t n, int64_t out, int64_t in,
                             int kind) {
  DenseProduct p{};
  p.a = {x, nullptr, 1, 0};
  p.b = {w, nullptr, 1, 0};
  p.M = n;
  p.N = out;
  p.K = in;
  p.kind = kind;
  p.epi.rows = n;
  p.epi.cols = (int)out;
  return p;
}

// d_x [n, in] = d [n, out] w [out, in]
DenseProduct input_gradient(const void *d, const void *w, int64_t n, int64_t out, int64_t in,
                            int half, void *d_x) {
  DenseProduct p{};
  p.a = {d, nullptr, 1, 0};
  p.b = {w, nullptr, 0, 0};
  p.M = n;
  p.N = in;
  p.K = out;
  p.kind = EPI_LINEAR;
  p.epi.rows = n;
  p.epi.cols = (int)in;
  p.epi.half = half;
  p.epi.out = d_x;
  p.epi.vec = 1;
  return p;
}

// d_w [out, in] = d^T x
DenseProduct weight_gradient(const void *d, const void *x, int64_t n, int64_t out, int64_t in,
                             int half, void *d_w) {
  DenseProduct p{};
  p.a = {d, nullptr, 0, 0};
  p.b = {x, nullptr, 0, 0};
  p.M = out;
  p.N = in;
  p.K = n;
  p.kind = EPI_LINEAR;
  p.epi.rows = out;
  p.epi.cols = (int)in;
  p.epi.half = half;
  p.epi.out = d_w;
  p.epi.vec = 1;
  return p;
}

// The backward passes' workspace: the gradient of the sums (where it is not
// the caller's), the parts of split sums, the column sums' scratch.
struct GradLayout {
  bool skinny;               // the recomputed sums take few rows
  DensePlan sums, d_x, d_w;  // of the recomputed sums and of both gradients
  size_t d, partial, partial_w, columns, total;
};
GradLayout grad_layout(int64_t n, int64_t out, int64_t in, int kind, bool own_d, bool columns) {
  GradLayout g{};
  g.skinny = dense_skinny(n, out, in, kind, false);
  if (own_d && !g.skinny) g.sums = dense_plan(n, out, in, kind, false);
  dense_plan_two(n, in, out, out, in, n, &g.d_x, &g.d_w);
  g.partial = own_d ? align_up((size_t)n * out * 2, kAlign) : 0;
  g.partial_w = g.partial + align_up(g.d_x.partial, kAlign);
  const size_t both = g.partial_w + align_up(g.d_w.partial, kAlign);
  const size_t first = g.partial + align_up(g.sums.partial, kAlign);
  g.columns = both > first ? both : first;
  const int64_t rows = (n + 31) / 32;
  const size_t sums = (size_t)rows * out * 4, other = column_sum_scratch((int)out);
  g.total = g.columns + (columns ? align_up(sums > other ? sums : other, kAlign) : 0);
  return g;
}

cudaError_t run_sums(const DenseProduct &p, const GradLayout &g, void *workspace, int32_t *status,
                     cudaStream_t s) {
  if (g.skinny) return launch_dense_skinny(p, s);
  return launch_dense(p, g.sums, nullptr, reinterpret_cast<float *>(at(workspace, g.partial)),
                      status, s);
}

// d_x and d_w of d, each where it is wanted; with column_rows, d_bias from
// the column sums that d's epilogue left, in the same launch.
cudaError_t run_gradients(const void *d, const void *x, const void *w, int64_t n, int64_t out,
                          int64_t in, int half, void *d_x, void *d_w, const GradLayout &g,
                          void *workspace, int column_rows, void *d_bias, int32_t *status,
                          cudaStream_t s) {
  const DenseProduct px = input_gradient(d, w, n, out, in, half, d_x);
  const DenseProduct pw = weight_gradient(d, x, n, out, in, half, d_w);
  const DenseProduct *p[2];
  const DensePlan *plan[2];
  float *part[2];
  int count = 0;
  if (d_x) {
    p[count] = &px;
    plan[count] = &g.d_x;
    part[count++] = reinterpret_cast<float *>(at(workspace, g.partial));
  }
  if (d_w) {
    p[count] = &pw;
    plan[count] = &g.d_w;
    part[count++] = reinterpret_cast<float *>(at(workspace, g.partial_w));
  }
  const float *columns = reinterpret_cast<const float *>(at(workspace, g.columns));
  void *joined = column_rows ? d_bias : nullptr;
  if (count == 0)
    return joined ? launch_column_join(columns, column_rows, (int)out, half ? MOE_FP16 : MOE_BF16,
                                       joined, s)
                  : cudaSuccess;
  return launch_dense_gradients(p, plan, part, count, columns, column_rows, (int)out, half, joined,
                                status, s);
}

moe_status run_linear(const void *x, const uint8_t *x_scales, const void *w,
                      const uint8_t *w_scales, const void *bias, const void *residual, int64_t n,
                      int32_t R, int32_t C, int32_t dtype, int32_t act, void *y, void *workspace,
                      size_t workspace_bytes, int32_t *status, moe_stream stream) {
  if (!y) return MOE_ERR_INVALID_ARG;
  if (!aligned(bias, 2) || !aligned(residual, 2) || !aligned(y, 2) || !aligned(status, 4))
    return MOE_ERR_MISALIGNED;
  DenseProduct p = forward_product(x, w, n, R, C, EPI_LINEAR);
  p.a.scales = x_scales;
  p.b.scales = w_scales;
  p.epi.half = dtype == MOE_FP16;
  p.epi.act = act;
  p.epi.bias = bias;
  p.epi.add = residual;
  p.epi.out = y;
  p.epi.vec = R % 8 == 0 && aligned(bias, 16) && aligned(residual, 16) && aligned(y, 16);
  return run_forward(p, workspace, workspace_bytes, status, stream);
}

moe_status run_gated(const void *x, const uint8_t *x_scales, const void *w13,
                     const uint8_t *w13_scales, int64_t n, int32_t H, int32_t I, int32_t dtype,
                     const ActParams &act, void *h, const moe_mx8_rows *h_mx8, void *workspace,
                     size_t workspace_bytes, int32_t *status, moe_stream stream) {
  if ((h == nullptr) == (h_mx8 == nullptr)) return MOE_ERR_INVALID_ARG;
  if (h_mx8) {
    const moe_status st = check_mx8(h_mx8);
    if (st != MOE_OK) return st;
    if (I % 32 != 0) return MOE_ERR_INVALID_ARG;
  }
  if (!aligned(h, 2) || !aligned(status, 4)) return MOE_ERR_MISALIGNED;
  const int kind = h_mx8 ? EPI_GATED_MX : EPI_GATED;
  DenseProduct p = forward_product(x, w13, n, 2 * (int64_t)I, H, kind);
  p.a.scales = x_scales;
  p.b.scales = w13_scales;
  p.b.pairs = act.layout == MOE_W13_PACKED;
  p.epi.half = dtype == MOE_FP16;
  p.epi.gate = act;
  p.epi.out = h;
  if (h_mx8) {
    p.epi.codes = h_mx8->codes;
    p.epi.scales = h_mx8->scales;
  }
  p.epi.vec = aligned(h, 16);
  return run_forward(p, workspace, workspace_bytes, status, stream);
}

}  // namespace

extern "C" {

// -------------------------------------------------------------------- norm --
moe_status moe_rms_norm(const void *x, const void *residual, const void *weight,
                        int32_t weight_dtype, int64_t n, int32_t H, int32_t dtype, float eps,
                        void *y, const moe_mx8_rows *y_mx8, void *sum, moe_stream stream) {
  if (H < 1 || H > kMaxFeatures || !rows_ok(n, H)) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_BF16 && dtype != MOE_FP16 && dtype != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (weight_dtype != dtype && weight_dtype != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || isinf(eps)) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!x || (y == nullptr) == (y_mx8 == nullptr)) return MOE_ERR_INVALID_ARG;
  if (sum && !residual) return MOE_ERR_INVALID_ARG;
  if (y_mx8) {
    const moe_status st = check_mx8(y_mx8);
    if (st != MOE_OK) return st;
    if (H % 32 != 0) return MOE_ERR_INVALID_ARG;
  }
  const size_t a = dtype == MOE_FP32 ? 4 : 2;
  if (!aligned(x, a) || !aligned(residual, a) || !aligned(y, a) || !aligned(sum, a) ||
      !aligned(weight, weight_dtype == MOE_FP32 ? 4 : 2))
    return MOE_ERR_MISALIGNED;
  return from_cuda(launch_rms_norm(x, residual, weight, weight_dtype, n, H, dtype, eps, y, sum,
                                   y_mx8 ? y_mx8->codes : nullptr,
                                   y_mx8 ? y_mx8->scales : nullptr, (cudaStream_t)stream));
}

size_t moe_rms_norm_backward_workspace_size(int64_t n, int32_t H) {
  if (H < 1 || H > kMaxFeatures || !rows_ok(n, H)) return 0;
  return align_up(rms_norm_backward_scratch(n, H), kAlign);
}

moe_status moe_rms_norm_backward(const void *d_y, const void *x, const void *weight,
                                 int32_t weight_dtype, const void *d_sum, int64_t n, int32_t H,
                                 int32_t dtype, float eps, void *d_x, void *d_weight,
                                 void *workspace, size_t workspace_bytes, moe_stream stream) {
  if (H < 1 || H > kMaxFeatures || !rows_ok(n, H)) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_BF16 && dtype != MOE_FP16 && dtype != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (weight_dtype != dtype && weight_dtype != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || isinf(eps)) return MOE_ERR_INVALID_ARG;
  const size_t wa = weight_dtype == MOE_FP32 ? 4 : 2;
  if (!aligned(d_weight, wa)) return MOE_ERR_MISALIGNED;
  if (n == 0)  // an empty sum is zero
    return d_weight ? from_cuda(cudaMemsetAsync(d_weight, 0, (size_t)H * wa, (cudaStream_t)stream))
                    : MOE_OK;
  if (!d_y || !x || !d_x) return MOE_ERR_INVALID_ARG;
  const size_t a = dtype == MOE_FP32 ? 4 : 2;
  if (!aligned(d_y, a) || !aligned(x, a) || !aligned(d_sum, a) || !aligned(d_x, a) ||
      !aligned(weight, wa))
    return MOE_ERR_MISALIGNED;
  const moe_status st =
      check_workspace(workspace, workspace_bytes,
                      d_weight ? moe_rms_norm_backward_workspace_size(n, H) : 0);
  if (st != MOE_OK) return st;
  return from_cuda(launch_rms_norm_backward(d_y, x, weight, weight_dtype, d_sum, n, H, dtype, eps,
                                            d_x, d_weight, static_cast<float *>(workspace),
                                            (cudaStream_t)stream));
}

// ------------------------------------------------------------------ linear --
size_t moe_linear_workspace_size(int64_t n, int32_t R, int32_t C, int32_t mx8) {
  if (check_product(n, R, C, MOE_BF16, mx8) != MOE_OK) return 0;
  return forward_plan(n, R, C, EPI_LINEAR, mx8).bytes;
}

moe_status moe_linear(const void *x, const void *w, const void *bias, const void *residual,
                      int64_t n, int32_t R, int32_t C, int32_t dtype, int32_t act, void *y,
                      void *workspace, size_t workspace_bytes, int32_t *status,
                      moe_stream stream) {
  const moe_status st = check_product(n, R, C, dtype, false);
  if (st != MOE_OK) return st;
  if (!act_ok(act)) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!x || !w) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16)) return MOE_ERR_MISALIGNED;
  return run_linear(x, nullptr, w, nullptr, bias, residual, n, R, C, dtype, act, y, workspace,
                    workspace_bytes, status, stream);
}

moe_status moe_linear_mx8(const moe_mx8_rows *x, const moe_mx8_rows *w, const void *bias,
                          const void *residual, int64_t n, int32_t R, int32_t C, int32_t dtype,
                          int32_t act, void *y, void *workspace, size_t workspace_bytes,
                          int32_t *status, moe_stream stream) {
  moe_status st = check_product(n, R, C, dtype, true);
  if (st != MOE_OK) return st;
  if (!act_ok(act)) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if ((st = check_mx8(x)) != MOE_OK || (st = check_mx8(w)) != MOE_OK) return st;
  return run_linear(x->codes, x->scales, w->codes, w->scales, bias, residual, n, R, C, dtype, act,
                    y, workspace, workspace_bytes, status, stream);
}

moe_status moe_read_dense_status(int32_t reset, moe_stream stream) {
  int32_t word = 0;
  if (read_wait_status(&word, reset != 0, (cudaStream_t)stream) != cudaSuccess) return MOE_ERR_CUDA;
  return (moe_status)word;
}

moe_status moe_selftest_linear_timeout(const void *x, const void *w, int64_t n, int32_t R,
                                       int32_t C, int32_t dtype, void *y, void *workspace,
                                       size_t workspace_bytes, uint64_t timeout_ns,
                                       int32_t *status, moe_stream stream) {
  const moe_status st = check_product(n, R, C, dtype, false);
  if (st != MOE_OK) return st;
  if (timeout_ns == 0 || timeout_ns > kWaitTimeoutNs) return MOE_ERR_INVALID_ARG;
  if (!x || !w || !y || n == 0 || dense_skinny(n, R, C, EPI_LINEAR, false))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 2) || !aligned(status, 4))
    return MOE_ERR_MISALIGNED;
  DenseProduct p = forward_product(x, w, n, R, C, EPI_LINEAR);
  p.epi.half = dtype == MOE_FP16;
  p.epi.out = y;
  p.epi.vec = R % 8 == 0 && aligned(y, 16);
  p.starve_ns = timeout_ns;
  return run_forward(p, workspace, workspace_bytes, status, stream);
}

size_t moe_linear_backward_workspace_size(int64_t n, int32_t R, int32_t C, int32_t act) {
  if (check_product(n, R, C, MOE_BF16, false) != MOE_OK || R % 8 != 0 || !act_ok(act)) return 0;
  return grad_layout(n, R, C, EPI_DACT, act != MOE_LINEAR_NONE, true).total;
}

moe_status moe_linear_backward(const void *d_y, const void *x, const void *w, const void *bias,
                               int64_t n, int32_t R, int32_t C, int32_t dtype, int32_t act,
                               void *d_x, void *d_w, void *d_bias, void *workspace,
                               size_t workspace_bytes, int32_t *status, moe_stream stream) {
  moe_status st = check_product(n, R, C, dtype, false);
  if (st != MOE_OK) return st;
  if (R % 8 != 0 || !act_ok(act)) return MOE_ERR_INVALID_ARG;
  if (!aligned(d_w, 16) || !aligned(d_bias, 2)) return MOE_ERR_MISALIGNED;
  cudaStream_t s = (cudaStream_t)stream;
  if (n == 0) {  // empty sums are zero
    cudaError_t e = cudaSuccess;
    if (d_w) e = cudaMemsetAsync(d_w, 0, (size_t)R * C * 2, s);
    if (e == cudaSuccess && d_bias) e = cudaMemsetAsync(d_bias, 0, (size_t)R * 2, s);
    return from_cuda(e);
  }
  const bool own_d = act != MOE_LINEAR_NONE;
  if (!d_y || !x || !w) return MOE_ERR_INVALID_ARG;
  if (!aligned(d_y, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 2) ||
      !aligned(d_x, 16) || !aligned(status, 4))
    return MOE_ERR_MISALIGNED;
  const GradLayout g = grad_layout(n, R, C, EPI_DACT, own_d, true);
  if ((st = check_workspace(workspace, workspace_bytes, g.total)) != MOE_OK) return st;
  const int half = dtype == MOE_FP16;
  const void *d = d_y;
  int column_rows = 0;
  cudaError_t e = cudaSuccess;
  if (own_d) {
    DenseProduct p = forward_product(x, w, n, R, C, EPI_DACT);
    p.epi.half = half;
    p.epi.act = act;
    p.epi.bias = bias;
    p.epi.add = d_y;
    p.epi.out = at(workspace, g.d);
    p.epi.vec = aligned(bias, 16);
    if (d_bias && g.sums.splits <= 1) {
      p.epi.column_part = reinterpret_cast<float *>(at(workspace, g.columns));
      column_rows = (int)((n + 31) / 32);
    }
    e = run_sums(p, g, workspace, status, s);
    d = p.epi.out;
  }
  if (e == cudaSuccess && d_bias && !column_rows)
    e = launch_column_sum(d, n, R, dtype, d_bias,
                          reinterpret_cast<float *>(at(workspace, g.columns)), s);
  if (e == cudaSuccess)
    e = run_gradients(d, x, w, n, R, C, half, d_x, d_w, g, workspace, column_rows, d_bias, status,
                      s);
  return from_cuda(e);
}

// ------------------------------------------------------------ gated linear --
size_t moe_gated_linear_workspace_size(int64_t n, int32_t H, int32_t I, int32_t mx8,
                                       int32_t h_mx8) {
  if (I < 8 || I > kMaxFeatures || I % 8 != 0 || (h_mx8 && I % 32 != 0) ||
      check_product(n, 2 * (int64_t)I, H, MOE_BF16, mx8) != MOE_OK)
    return 0;
  return forward_plan(n, 2 * (int64_t)I, H, h_mx8 ? EPI_GATED_MX : EPI_GATED, mx8).bytes;
}

moe_status moe_gated_linear(const void *x, const void *w13, int64_t n, int32_t H, int32_t I,
                            const moe_params *params, int32_t dtype, void *h,
                            const moe_mx8_rows *h_mx8, void *workspace, size_t workspace_bytes,
                            int32_t *status, moe_stream stream) {
  ActParams act;
  const moe_status st = check_gated(n, H, I, dtype, params, false, act);
  if (st != MOE_OK) return st;
  if (n == 0) return MOE_OK;
  if (!x || !w13) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w13, 16)) return MOE_ERR_MISALIGNED;
  return run_gated(x, nullptr, w13, nullptr, n, H, I, dtype, act, h, h_mx8, workspace,
                   workspace_bytes, status, stream);
}

moe_status moe_gated_linear_mx8(const moe_mx8_rows *x, const moe_mx8_rows *w13, int64_t n,
                                int32_t H, int32_t I, const moe_params *params, int32_t dtype,
                                void *h, const moe_mx8_rows *h_mx8, void *workspace,
                                size_t workspace_bytes, int32_t *status, moe_stream stream) {
  ActParams act;
  moe_status st = check_gated(n, H, I, dtype, params, true, act);
  if (st != MOE_OK) return st;
  if (n == 0) return MOE_OK;
  if ((st = check_mx8(x)) != MOE_OK || (st = check_mx8(w13)) != MOE_OK) return st;
  return run_gated(x->codes, x->scales, w13->codes, w13->scales, n, H, I, dtype, act, h, h_mx8,
                   workspace, workspace_bytes, status, stream);
}

size_t moe_gated_linear_backward_workspace_size(int64_t n, int32_t H, int32_t I) {
  if (I < 8 || I > kMaxFeatures || I % 8 != 0 ||
      check_product(n, 2 * (int64_t)I, H, MOE_BF16, false) != MOE_OK)
    return 0;
  return grad_layout(n, 2 * (int64_t)I, H, EPI_DGATED, true, false).total;
}

moe_status moe_gated_linear_backward(const void *d_h, const void *x, const void *w13, int64_t n,
                                     int32_t H, int32_t I, const moe_params *params,
                                     int32_t dtype, void *d_x, void *d_w13, void *workspace,
                                     size_t workspace_bytes, int32_t *status,
                                     moe_stream stream) {
  ActParams act;
  moe_status st = check_gated(n, H, I, dtype, params, false, act);
  if (st != MOE_OK) return st;
  if (!aligned(d_w13, 16)) return MOE_ERR_MISALIGNED;
  cudaStream_t s = (cudaStream_t)stream;
  if (n == 0)
    return d_w13 ? from_cuda(cudaMemsetAsync(d_w13, 0, (size_t)2 * I * H * 2, s)) : MOE_OK;
  if (!d_h || !x || !w13) return MOE_ERR_INVALID_ARG;
  if (!aligned(d_h, 2) || !aligned(x, 16) || !aligned(w13, 16) || !aligned(d_x, 16) ||
      !aligned(status, 4))
    return MOE_ERR_MISALIGNED;
  const int64_t out = 2 * (int64_t)I;
  const GradLayout g = grad_layout(n, out, H, EPI_DGATED, true, false);
  if ((st = check_workspace(workspace, workspace_bytes, g.total)) != MOE_OK) return st;
  const int half = dtype == MOE_FP16;
  DenseProduct p = forward_product(x, w13, n, out, H, EPI_DGATED);
  p.b.pairs = act.layout == MOE_W13_PACKED;
  p.epi.half = half;
  p.epi.gate = act;
  p.epi.add = d_h;
  p.epi.out = at(workspace, g.d);
  p.epi.vec = aligned(d_h, 16);
  if (!d_x && !d_w13) return MOE_OK;
  cudaError_t e = run_sums(p, g, workspace, status, s);
  if (e == cudaSuccess)
    e = run_gradients(p.epi.out, x, w13, n, out, H, half, d_x, d_w13, g, workspace, 0, nullptr,
                      status, s);
  return from_cuda(e);
}

}  // extern "C"
