"""Lossless BF16 exponent coding on AMD MI355X (gfx950).

The codec of ZipCCL ("Key idea and contribution", technique 1) as HIP kernels
behind the C ABI in include/zc.h; ``Plan`` is the thin ctypes binding.
``workloads`` draws the seeded synthetic inputs.

Around a MoE's compressed all-to-all (include/zc_experts.h): ``Router`` chooses
each token's experts and takes the loss that balances them, ``ExpertPlan`` sorts
tokens by expert and brings them back, ``expert_product`` and
``expert_weight_grad`` are the experts' products of 8-bit blocks,
``orthogonalize`` makes updates of their weights.
"""
from .binding import (EXPORTS, LIB_PATH, Plan, ZcError, check_buffer, lib, prefer_compressed,
                      reduce_native)
from .experts import (EXPERT_EXPORTS, Choice, ExpertPlan, Fp8Blocks, Fp8Columns, Router, Routing,
                      empty_fp8_columns, empty_fp8_rows, empty_fp8_weights, expert_product, expert_weight_grad,
                      expert_weight_grad_workspace_bytes, orthogonalize, orthogonalize_workspace_bytes,
                      quantize_columns, quantize_rows, quantize_weights)

__all__ = ["EXPORTS", "LIB_PATH", "Plan", "ZcError", "check_buffer", "lib", "prefer_compressed",
           "reduce_native",
           "EXPERT_EXPORTS", "Choice", "ExpertPlan", "Fp8Blocks", "Fp8Columns", "Router", "Routing", "empty_fp8_columns",
           "empty_fp8_rows", "empty_fp8_weights", "expert_product", "expert_weight_grad",
           "expert_weight_grad_workspace_bytes", "orthogonalize", "orthogonalize_workspace_bytes",
           "quantize_columns", "quantize_rows", "quantize_weights"]
