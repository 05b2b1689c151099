"""Sparse Mixture-of-Experts layer (Nemotron 3 MoE and LatentMoE) for MI355X / gfx950: the
forward pass, the backward pass of the bf16 layer, and the operators around it (token rows in
expert order, the residual block's norms, gradient clipping).

The layer runs in hand-written HIP kernels behind the C ABI declared in include/moe.h
(libmoe_mi355x.so, built in-tree by ``python -m sparse_moe_layer_05_amd.build``). This package
is its thin Python binding: torch provides device memory and streams.
"""
from .binding import (Backward, Layer, MoeError, alloc_routing, backward_from, bias_update,
                      dispatch, layer_forward, layer_from, lib, mx_dequantize, mx_gemm,
                      mx_quantize, route, status_str, to_device, workspace_size)
from .block import (Block, GradClip, block_norm, block_norm_backward, block_residual,
                    block_residual_backward, clip_grad_norm, sort_tokens, sort_tokens_backward,
                    unsort_tokens, unsort_tokens_backward)

__all__ = ["Backward", "Block", "GradClip", "Layer", "MoeError", "alloc_routing", "backward_from",
           "bias_update", "block_norm", "block_norm_backward", "block_residual",
           "block_residual_backward", "clip_grad_norm", "dispatch", "layer_forward", "layer_from",
           "lib", "mx_dequantize", "mx_gemm", "mx_quantize", "route", "sort_tokens",
           "sort_tokens_backward", "status_str", "to_device", "unsort_tokens",
           "unsort_tokens_backward", "workspace_size"]
