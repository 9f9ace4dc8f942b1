"""B200-native (sm_100a) routed Mixture-of-Experts FFN layer.

The public calls mirror the C ABI of include/moe.h:

    ids, weights = route(x, w_router, k, bias=None, renorm=True)
    y            = forward(x, w_router, w_gate, w_up, w_down, k, bias=None, renorm=True)
    g            = ForwardGraph(x, w_router, w_gate, w_up, w_down, k); y = g.replay()
    y_dense      = dense_ffn(x, w_gate_d, w_up_d, w_down_d)   # the dense MLP beside the MoE

and, for batches of at most 16 tokens, the same with 4-bit weights (group scales, bf16
activations):

    q            = w4_quantize(w, group=64)         # or w4_pack(codes, scales, zeros) of a checkpoint
    w            = w4_dequantize(q)                 # bf16 again, for larger batches
    y            = linear_w4(x, q)                  # one projection (fp32=True: logits)
    y_dense      = dense_ffn_w4(x, q_gate, q_up, q_down)
    y            = forward_w4(x, w_router, q_gate, q_up, q_down, k)

x, weights and outputs are CUDA tensors (bf16 operands, int32 ids, fp32 routing weights);
all arithmetic runs in libmoe_b200.so.  ``workloads`` (seeded synthetic inputs) can be
imported without a GPU.
"""
from ._abi import (ForwardGraph, MoEError, W4Weights, dense_ffn, dense_ffn_w4,  # noqa: F401
                   ffn_kernel_name, forward, forward_w4, last_kernel_count, last_stage_times,
                   linear_w4, load, route, router_stats, status_string, sync_status, w4_dequantize,
                   w4_pack, w4_quantize)

__all__ = ["route", "forward", "dense_ffn", "ForwardGraph", "sync_status", "last_stage_times",
           "load", "router_stats", "status_string", "MoEError", "last_kernel_count",
           "ffn_kernel_name", "W4Weights", "w4_pack", "w4_quantize", "w4_dequantize", "linear_w4",
           "dense_ffn_w4", "forward_w4"]
