"""GB300-native (sm_103a) Mixture-of-Experts layer forward.

route -> routing metadata -> grouped SwiGLU / SwiGLU-OAI / ReLU2 expert FFN
-> gate-weighted combine, every stage a CUDA kernel in libmoe_gb300.so
behind the C ABI of include/moe.h. This package is the thin Python binding
(argument marshalling over torch tensors) and nothing else; the seeded
synthetic inputs that tests and the benchmark use live in the top-level
`moe_inputs` module, outside the product.
"""
from ._binding import (ACT, DTYPE, FFN_KERNEL, GATING, LAYOUT, MoEError, MoeParams, Q4Weight,
                       Q4_FORMAT, RoutingMeta, STAGES, build_metadata, combine, combine_weighted,
                       combine_weighted_backward, dispatch, dispatch_backward, empty_meta,
                       ffn_plan, forward, forward_gate, forward_launch_count, forward_q4,
                       forward_timed, grouped_ffn, grouped_ffn_q4, lib, library_path, linear_q4,
                       make_params, read_status, route, route_backward, route_gemm,
                       route_metadata, selftest_wait_timeout, status_string, workspace,
                       workspace_q4, workspace_q4_size, workspace_regions, workspace_size)

__all__ = ["ACT", "DTYPE", "FFN_KERNEL", "GATING", "LAYOUT", "MoEError", "MoeParams", "Q4Weight",
           "Q4_FORMAT", "RoutingMeta", "STAGES", "build_metadata", "combine", "combine_weighted",
           "combine_weighted_backward", "dispatch", "dispatch_backward", "empty_meta", "ffn_plan",
           "forward", "forward_gate", "forward_launch_count", "forward_q4", "forward_timed",
           "grouped_ffn", "grouped_ffn_q4", "lib", "library_path", "linear_q4", "make_params",
           "read_status", "route", "route_backward", "route_gemm", "route_metadata",
           "selftest_wait_timeout", "status_string", "workspace", "workspace_q4",
           "workspace_q4_size", "workspace_regions", "workspace_size"]
