"""The experts' operators on arrays that lie back to back in one allocation:
not refused, and the same bits as on arrays of their own."""
import numpy as np
import pytest
import torch

import experts_helpers as xh
from combine_get_dispatch_amd import ep

pytestmark = pytest.mark.gpu


def back_to_back(*tensors):
    """Copies of the tensors, one right behind the other (their sizes are multiples of 16 bytes)."""
    sizes = [t.numel() * t.element_size() for t in tensors]
    assert all(s % 16 == 0 for s in sizes)
    whole = torch.empty(sum(sizes), dtype=torch.uint8, device="cuda")
    parts = [p.view(t.dtype).view(t.shape) for p, t in zip(whole.split(sizes), tensors)]
    for p, t in zip(parts, tensors):
        p.copy_(t)
    return parts


@pytest.mark.parametrize("order", [1, -1])
def test_adjacent_arrays(order):
    rng = np.random.default_rng(41)
    off, cap, _ = xh.packed_groups([20, 0, 1, 27], 1, slack=0)
    g = ep.Groups(torch.tensor([20, 0, 1, 27], dtype=torch.int32).cuda(), torch.from_numpy(off).cuda(), num_experts=4,
                  num_ranks=1, cap_rows=cap)
    K, N = 256, 128
    zeros = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731

    def same(call, inputs, outs):
        """`call(inputs, outs)` on separate arrays and on adjacent ones, in this order of inputs and outputs."""
        inputs, own = [t.cuda() for t in inputs], [o.clone() for o in outs]
        call(inputs, own)
        placed = back_to_back(*(inputs + outs)[::order])[::order]
        call(placed[:len(inputs)], placed[len(inputs):])
        for a, b in zip(own, placed[len(inputs):]):
            assert torch.equal(a, b)
        for a, b in zip(inputs, placed):
            assert torch.equal(a, b)  # inputs are as they were

    for form in ("bf16", "fp8", "mxfp4"):
        x, xs = xh.make_operand(rng, (cap, K), form)
        w, ws = xh.make_operand(rng, (4, N, K), form, weights=True)
        scales = [] if xs is None else [xs, ws]
        same(lambda i, o: ep.expert_gemm(i[0], i[1], g, *(i[2:] or (None, None)), out=o[0]), [x, w] + scales,
             [zeros(cap, N)])
    x, w, d = xh.bf16(rng, (cap, K)), xh.bf16(rng, (4, N, K)), xh.bf16(rng, (cap, N))
    same(lambda i, o: ep.expert_gemm_dgrad(*i, g, out=o[0]), [d, w], [zeros(cap, K)])
    for dtype in (torch.float32, torch.bfloat16):
        same(lambda i, o: ep.expert_gemm_wgrad(*i, g, out=o[0]), [d, x], [zeros(4, N, K, dtype=dtype)])
    gu, gd, u8 = xh.bf16(rng, (cap, 2 * K)), xh.bf16(rng, (cap, K)), torch.uint8
    same(lambda i, o: ep.swiglu(i[0], g, out=o[0]), [gu], [zeros(cap, K)])
    same(lambda i, o: ep.swiglu(i[0], g, "fp8", out=o), [gu], [zeros(cap, K, dtype=u8), zeros(cap, 2, dtype=torch.float32)])
    same(lambda i, o: ep.swiglu(i[0], g, "mxfp4", out=o), [gu], [zeros(cap, K // 2, dtype=u8), zeros(cap, 8, dtype=u8)])
    same(lambda i, o: ep.swiglu_backward(*i, g, out=o[0]), [gd, gu], [zeros(cap, 2 * K)])
    same(lambda i, o: ep.quantize_mxfp4(i[0], g, out=o), [x], [zeros(cap, K // 2, dtype=u8), zeros(cap, 8, dtype=u8)])
    q, s = xh.make_operand(rng, (cap, K), "mxfp4")
    same(lambda i, o: ep.dequantize_mxfp4(*i, g, out=o[0]), [q, s], [zeros(cap, K)])


def test_empty_rows_share_no_memory():
    """No receive rows: the weight gradients are zeros, whatever the row arrays' pointers are."""
    counts = torch.zeros(4, dtype=torch.int32).cuda()
    g = ep.Groups(counts, counts, num_experts=4, num_ranks=2, cap_rows=0).c()
    out = torch.full((4, 24, 40), 7.0, device="cuda")
    inside = out.data_ptr() + 64
    ep.ep_expert_gemm_wgrad(g, inside, inside, 40, 24, out.data_ptr(), True, False, torch.cuda.current_stream().cuda_stream)
    assert bool((out == 0).all())
