"""Captured calls of the experts' operators whose counts change between the
replays, down to none, in sizes of the 256-channel tiles; two replays at once."""
import numpy as np
import pytest
import torch

import experts_helpers as xh
from combine_get_dispatch_amd import ep

pytestmark = pytest.mark.gpu

E, R, H, I, CAP = 16, 2, 512, 2056, 1800
COUNTS = [
    [130, 0, 257, 1, 400, 64, 33, 700, 90, 129, 200, 5, 0, 1000, 256, 100],
    [0] * E,
    [0, 0, 0, 1800, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 0],
    [1] * E,
    [225] * E,
    [1800, 1, 0, 0, 0, 0, 0, 0, 17, 300, 0, 64, 65, 0, 128, 1],  # past the first rank's rows: the last is left out
]


def layout(counts):
    per = np.asarray(counts).reshape(R, E // R)
    return torch.tensor(counts, dtype=torch.int32), torch.from_numpy((np.cumsum(per, 1) - per).reshape(-1).astype(np.int32))


class Step:
    """One expert layer, forward and backward, on its own buffers."""

    def __init__(self, seed, hint):
        rng = np.random.default_rng(seed)
        self.counts, self.offsets = (t.cuda() for t in layout(COUNTS[0]))
        self.groups = ep.Groups(self.counts, self.offsets, num_experts=E, num_ranks=R, cap_rows=CAP, rows_hint=hint)
        self.x = xh.bf16(rng, (R * CAP, H)).cuda()
        self.w = xh.bf16(rng, (E, 2 * I, H), 0.05).cuda()
        self.w8, self.s8 = (t.cuda() for t in xh.make_operand(rng, (E, 2 * I, H), "fp8", weights=True))
        self.x8, self.xs8 = (t.cuda() for t in xh.make_operand(rng, (R * CAP, H), "fp8"))
        n, bf = R * CAP, torch.bfloat16
        self.outs = [torch.zeros(s, dtype=t, device="cuda") for s, t in (
            ((n, 2 * I), bf), ((n, I), bf), ((n, 2 * I), bf), ((n, H), bf), ((E, 2 * I, H), torch.float32), ((n, 2 * I), bf),
            ((n, H // 2), torch.uint8), ((n, H // 32), torch.uint8), ((n, H), bf))]

    def run(self):
        g, (h, a, gh, gx, gw, y, q, s, back) = self.groups, self.outs
        ep.expert_gemm(self.x, self.w, g, out=h)
        ep.swiglu(h, g, out=a)
        ep.swiglu_backward(a, h, g, out=gh)
        ep.expert_gemm_dgrad(gh, self.w, g, out=gx)
        ep.expert_gemm_wgrad(gh, self.x, g, out=gw)
        ep.expert_gemm(self.x8, self.w8, g, row_scales=self.xs8, weight_scales=self.s8, out=y)
        ep.quantize_mxfp4(gx, g, out=(q, s))
        ep.dequantize_mxfp4(q, s, g, out=back)

    def set(self, counts):
        for t, v in zip((self.counts, self.offsets), layout(counts)):
            t.copy_(v)
        for o in self.outs:
            o.fill_(3)


@pytest.mark.parametrize("hint", [0, 1, 3000])
def test_replays_with_other_counts(hint):
    steps = [Step(51, hint), Step(52, hint)]
    want = []
    for counts in COUNTS:
        for s in steps:
            s.set(counts)
            s.run()
        torch.cuda.synchronize()
        want.append([[o.clone() for o in s.outs] for s in steps])
        for s in steps:
            # rows no expert has, and experts without rows
            c, off = layout(counts)
            used = torch.zeros(R * CAP, dtype=torch.bool)
            for e in range(E):
                first = e // (E // R) * CAP
                used[first + min(int(off[e]), CAP):first + min(int(off[e] + c[e]), CAP)] = True
            for i, o in enumerate(s.outs):
                if i == 4:
                    assert bool((o[c.cuda() == 0] == 0).all())
                else:
                    assert bool((o[~used.cuda()] == 3).all())
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in steps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.run()
    for turn in range(2):
        for i in (list(range(len(COUNTS))) if turn == 0 else [4, 1, 0, 5, 2, 3]):
            for s in steps:
                s.set(COUNTS[i])
            torch.cuda.synchronize()
            for g, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    g.replay()
            torch.cuda.synchronize()
            for s, outs in zip(steps, want[i]):
                for k, (a, b) in enumerate(zip(s.outs, outs)):
                    assert torch.equal(a, b), f"turn {turn}, counts {i}, output {k}"
