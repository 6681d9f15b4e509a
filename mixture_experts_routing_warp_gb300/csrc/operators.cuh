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

// moe_params checked and resolved (moe_api.cu).
moe_status resolve_params(const moe_params *p, ActParams &out, int *gating);

// The norm in front of a layer (norm.cu), its gradients and column sums
// (norm_backward.cu). codes null: y, else codes and scales. Scratch sizes in bytes.
cudaError_t launch_rms_norm(const void *x, const void *residual, const void *weight, int w_dtype,
                            int64_t n, int H, int dtype, float eps, void *y, void *sum,
                            uint8_t *codes, uint8_t *scales, cudaStream_t s);
size_t rms_norm_backward_scratch(int64_t n, int H);
cudaError_t launch_rms_norm_backward(const void *d_y, const void *x, const void *weight,
                                     int w_dtype, const void *d_sum, int64_t n, int H, int dtype,
                                     float eps, void *d_x, void *d_weight, float *scratch,
                                     cudaStream_t s);
cudaError_t launch_column_join(const float *part, int rows, int cols, int dtype, void *out,
                               cudaStream_t s);
size_t column_sum_scratch(int cols);
cudaError_t launch_column_sum(const void *d, int64_t n, int cols, int dtype, void *out,
                              float *scratch, cudaStream_t s);

}  // namespace moe
