// operators.cuh -- launchers of the operators around the layer, apart from
// moe_internal.cuh so that the layer's kernels, and the figures measured on
// their sources, do not change with them.
#pragma once

#include "moe_internal.cuh"

namespace moe {

// The rows' way to expert-sorted order and back, with gradients (permute.cu).
cudaError_t launch_dispatch(const void *x, const int32_t *row_sorted, const int32_t *n_kept,
                            int64_t n, int k, int H, int dtype, void *x_sorted, cudaStream_t s);
// weights null: every weight 1 (moe_dispatch_backward)
cudaError_t launch_combine_weighted(const void *y_sorted, const int32_t *row_sorted,
                                    const void *weights, int w_dtype, int64_t n, int k, int H,
                                    int dtype, void *out, cudaStream_t s);
cudaError_t launch_combine_backward(const void *d_out, const void *y_sorted,
                                    const int32_t *row_sorted, const void *weights, int w_dtype,
                                    const int32_t *n_kept, int64_t n, int k, int H, int dtype,
                                    void *d_sorted, float *d_weights, cudaStream_t s);
cudaError_t launch_route_backward(const float *logits, const int32_t *topk_indx,
                                  const float *d_vals, int64_t n, int E, int k, int gating,
                                  float *d_logits, cudaStream_t s);

// Products with 4-bit weights (q4_matvec.cu). h: fp32 [N, I] scratch.
cudaError_t launch_linear_q4(const void *x, const moe_q4_matrix &w, int64_t n, int R, int C,
                             int dtype, void *y, cudaStream_t s);
cudaError_t launch_ffn_q4(const void *x, const moe_routing_meta &m, const moe_q4_matrix &w13,
                          const moe_q4_matrix &w2, int64_t N, int E, int k, int H, int I,
                          const ActParams &act, int dtype, float *h, void *y_sorted,
                          uint32_t *ctrl, cudaStream_t s);

}  // namespace moe
