"""The routed cases of operators.py with their rows spread over the experts as
its comments say, and cases that it does not have. (Its own routing keys are
all NaN, as the clamp in `_routing` acts on log u and not on its negative, so
that every token takes the same k experts: T rows each, the others none.)

    python3 perf/spread_rows.py [case ...]

For each case: the time of a pass (HIP events around 50 ms of passes back to
back, 20 at least, alternating between two sets of inputs; the median of five
such runs, after one that is not counted), the
bytes and operations of `work` over it, and how far the result is from the
64-bit form (root mean square over root mean square).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from perf import operators  # noqa: E402

MORE = [
    # a training step of 16 experts on bf16 rows, forward: 16384 ragged rows
    dict(name="bf16_prefill_up", op="product", form="bf16", layout="packed", T=4096, k=4, E=16, R=4, K=7168, N=4096, skew=0.5),
    # the training share of grad_rank with fp32 weight gradients
    dict(name="grad_rank_fp32", op="gradient", layout="packed", T=32768, k=1, E=8, R=1, K=7168, N=4096, skew=0.1, acc="fp32"),
    # the gradients of 256 tokens, top-8 of 64 experts, in the low-latency layout and packed
    dict(name="grad_regions", op="gradient", layout="low_latency", T=256, k=8, E=64, R=8, K=2048, N=4096, skew=0.2, acc="fp32"),
    dict(name="grad_few_rows", op="gradient", layout="packed", T=256, k=8, E=64, R=8, K=2048, N=4096, skew=0.2, acc="fp32"),
    # SwiGLU in the forms that operators.py does not list, 32768 rows
    dict(name="swiglu_bf16", op="swiglu", out="bf16", layout="packed", T=4096, k=8, E=64, R=8, I=2048, skew=0.5),
]


def routing(case, g):
    T, k, E, R = (case[n] for n in ("T", "k", "E", "R"))
    popularity = torch.log_softmax(case["skew"] * torch.randn(E, generator=g, device="cuda"), 0)
    u = torch.rand((T, E), generator=g, device="cuda").clamp_min(1e-30)
    idx = (popularity - torch.log((-torch.log(u)).clamp_min(1e-30))).topk(k, dim=1).indices
    if case["layout"] == "low_latency":
        src = torch.arange(T, device="cuda")[:, None] // (T // R)
        counts = torch.bincount((idx * R + src).view(-1), minlength=E * R).view(E, R).to(torch.int32)
        return dict(offsets=None, counts=counts, cap=E * T // R, region=T // R, widest=int(counts.max()))
    counts = torch.bincount(idx.view(-1), minlength=E)
    per_rank = counts.view(R, E // R)
    return dict(offsets=(per_rank.cumsum(1) - per_rank).view(E).to(torch.int32), counts=counts.to(torch.int32),
                cap=int(per_rank.sum(1).max()) + 3, region=0, widest=int(counts.max()))


def burst(states, passes):
    """Seconds a pass, of so many back to back."""
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    for i in range(passes):
        operators.run(states[i % len(states)])
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) * 1e-3 / passes


def timed(states, runs=5):
    burst(states, 2 * len(states))
    passes = max(20, int(0.05 / burst(states, 4)))
    burst(states, passes)  # the clocks settle
    return sorted(burst(states, passes) for _ in range(runs))[runs // 2]


def distance(got, want):
    """Largest over the outputs (those with a 64-bit form) of rms(got - want) / rms(want)."""
    got, want = ((t,) if torch.is_tensor(t) else t for t in (got, want))
    return max(float((a.double() - b.double()).square().mean().sqrt() / b.double().square().mean().sqrt().clamp_min(1e-300))
               for a, b in zip(got, want) if b is not None)


def main():
    operators.own, operators._routing = True, routing
    cases = [c for c in operators.listed() if c["op"] != "mxfp4"] + MORE
    names = sys.argv[1:] or [c["name"] for c in cases]
    for case in cases:
        if case["name"] not in names:
            continue
        states = [operators.prepare(case, seed) for seed in (1, 2)]
        t, w = timed(states), operators.work(case)
        got = operators.run(states[0])
        want = operators.exact(case, 1)
        far = "-" if want is None else f"{distance(got, want):.2e}"
        print(f"{case['name']:20s} {t * 1e6:9.1f} us {w['bytes'] / t / 1e9:8.0f} GB/s {w['flops'] / t / 1e12:8.1f} TFLOP/s  "
              f"from 64 bits {far}", flush=True)
        del states, got, want
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
