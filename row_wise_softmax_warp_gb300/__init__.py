"""rowops on GB300: row-wise normalise-and-reduce ops (softmax and its backward,
scaled causal attention softmax, hard-masked softmax, logsumexp, fused softmax
cross-entropy, LayerNorm forward/backward, top-k kept mask) and the
mixture-of-experts layer behind the router (plan, gather, combine, the experts'
matrix products) as hand-written sm_103a CUDA kernels behind a C ABI
(include/rowops.h).  Between two sublayers' products it has dropout, and the
residual's addition with a root-mean-square norm whose answer may be quantised rows.

The functions below are the ctypes binding of that ABI; ``inputs`` holds the
seeded synthetic workloads and ``build`` compiles the library.
"""
from .binding import (  # noqa: F401
    RowopsError,
    library,
    rowops_add_rmsnorm_bwd,
    rowops_add_rmsnorm_bwd_workspace,
    rowops_add_rmsnorm_fwd,
    rowops_argmax_onehot,
    rowops_attn_softmax_bwd,
    rowops_attn_softmax_fwd,
    rowops_column_sums,
    rowops_dropout,
    rowops_expert_combine,
    rowops_expert_combine_bwd,
    rowops_expert_gather,
    rowops_expert_matmul,
    rowops_expert_matmul_fp8,
    rowops_expert_matmul_fp8_workspace,
    rowops_expert_matmul_mx4,
    rowops_expert_matmul_mx4_workspace,
    rowops_expert_matmul_wgrad,
    rowops_expert_matmul_wgrad_workspace,
    rowops_expert_matmul_workspace,
    rowops_expert_plan,
    rowops_expert_plan_workspace,
    rowops_kernel_launches,
    rowops_layernorm_bwd,
    rowops_layernorm_bwd_workspace,
    rowops_layernorm_fwd,
    rowops_logsumexp,
    rowops_lrp_softmax_rows,
    rowops_masked_softmax,
    rowops_masked_softmax_fmask,
    rowops_quantize_blocks,
    rowops_quantize_mx4,
    rowops_rmsnorm_bwd,
    rowops_rmsnorm_fwd,
    rowops_router_masked_topk,
    rowops_softmax_bwd,
    rowops_softmax_ce,
    rowops_soft_ce,
    rowops_softmax_fwd,
    rowops_teacher_ce,
    rowops_top_k_rows,
    rowops_topk_kept,
)
