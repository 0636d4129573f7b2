"""MI355X-native MoE expert-parallel dispatch / combine (DeepEP-style token exchange).

The hot path -- dispatch layout, dispatch (with fused BF16->FP8 e4m3 pack),
combine (fp32 weighted gather-reduce to BF16) and the backward pair -- runs in
hand-written HIP kernels for gfx950 behind the C ABI declared in include/ep.h.

Submodules:
  ep         ctypes binding of libep.so (same names as the C ABI) plus a small
             torch-tensor convenience wrapper (argument marshalling only)
  workloads  seeded synthetic inputs (routing, activations, gradients)
  build      compiles libep.so with hipcc for gfx950

Nothing is loaded at import time; ``ep.load()`` raises if libep.so is missing.

Usage (torch tensors on the GPU; every call is asynchronous on torch's
current stream, and the outputs are caller-owned tensors)::

    from combine_get_dispatch_amd import ep
    buf = ep.Buffer(num_tokens, hidden, num_topk, num_experts, num_ranks, cap_rows)
    # x [T, H] bf16, topk_idx [T, k] int32 (-1 = no expert), topk_w [T, k] fp32
    layout, recv_x, recv_scales, recv_w, handle = buf.dispatch_with_layout(
        x, topk_idx, topk_w, use_fp8=True)
    # ... the experts turn rank d's rows [d*cap_rows, d*cap_rows + rank_rows[d])
    #     of recv_x / recv_scales into expert_out [R*cap_rows, H] bf16 ...
    y = buf.combine(expert_out, handle, topk_w)            # [T, H] bf16
    grad_rows = buf.combine_backward(grad_y, handle)       # backward of combine
    grad_x = buf.dispatch_backward(grad_expert_in, handle, topk_w)
    assert buf.status() == 0                               # sticky device status

The experts' own computation on the received rows (FP8 rows and weights here;
bf16 and MXFP4 likewise, and the bf16 gradients)::

    g = buf.groups(layout)                                 # low-latency: buf.groups_low_latency(recv_count)
    h = ep.expert_gemm(recv_x, w13, g, row_scales=recv_scales, weight_scales=s13)   # [rows, 2I] bf16
    a, a_scales = ep.swiglu(h, g, kind="fp8")
    expert_out = ep.expert_gemm(a, w2, g, row_scales=a_scales, weight_scales=s2)

The router before the dispatch, the same layer in 8-bit integers, and training
that keeps its activations in 8 bits::

    r = ep.Router(num_experts, num_topk, score="sigmoid", num_groups=8, topk_groups=4, scale=2.5)
    topk_idx, topk_w = ep.route(logits, r, bias=bias)      # ready for the dispatch calls
    grad_logits = ep.route_backward(grad_w, logits, topk_idx, r)

    q, s = ep.quantize_int8(rows, g)                       # weights once: ep.quantize_int8(w13)
    h = ep.expert_gemm(q, w13, g, row_scales=s, weight_scales=s13)
    a, a_scales = ep.swiglu(h, g, kind="int8")
    expert_out = ep.expert_gemm(a, w2, g, row_scales=a_scales, weight_scales=s2)

    x_kept, x_scales = ep.quantize_mxint8(rows, g)         # rows need not be held
    a, h_kept, h_scales = ep.swiglu_checkpoint(h, g)       # nor h, nor a
    grad_h, a = ep.swiglu_checkpoint_backward(grad_a, h_kept, h_scales, g)
    grad_w13 = ep.expert_gemm_wgrad(grad_h, x_kept, g, row_scales=x_scales)

The rank-deduplicated exchange (``dispatch_dedup_with_layout``: one row per
(token, destination rank) with the row's local expert indices and weights)
and the low-latency form (``dispatch_low_latency``: fixed per-(expert,
source) regions, one launch, graph-capturable) return handles that
``combine`` and the backward pair take the same way.
"""
__all__ = ["ep", "workloads", "build"]
