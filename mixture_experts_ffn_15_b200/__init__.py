"""Fused mixture-of-experts FFN layer (com.microsoft::MoE with standard SwiGLU) for B200.

The layer runs in the CUDA kernels of libmoe_b200.so (sm_100a), behind the C ABI
declared in include/moe_b200.h; this package is the thin Python binding.
"""
from ._abi import MoEError, load as load_library  # noqa: F401
from .ops import (alloc_workspace, balance_loss, balance_loss_backward, combine,  # noqa: F401
                  convert_chunked_to_interleaved, expert_ffn, expert_ffn_q8, expert_ffn_w8a8,
                  expert_ffn_w8a8_workspace_size, forward, forward_q8, forward_w8a8, get_error,
                  matmul_q8, permute, quantize_rows, rmsnorm, route, set_stage_events,
                  w8a8_workspace_size, workspace_error_word, workspace_size)

__all__ = ["forward", "forward_q8", "rmsnorm", "route", "permute", "expert_ffn", "expert_ffn_q8",
           "combine", "quantize_rows", "matmul_q8", "expert_ffn_w8a8",
           "expert_ffn_w8a8_workspace_size", "forward_w8a8", "w8a8_workspace_size",
           "balance_loss", "balance_loss_backward",
           "convert_chunked_to_interleaved", "get_error", "set_stage_events",
           "workspace_size", "alloc_workspace", "workspace_error_word", "load_library",
           "MoEError"]
