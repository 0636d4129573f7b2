"""SwiGLU and its gradient at the largest gates: finite ones whose product with
log2(e) passes the fp32 range, and infinities."""
import numpy as np
import pytest
import torch

import experts_helpers as xh
from combine_get_dispatch_amd import ep

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8         # a rounding's largest relative error
SILU = 16 * 2.0 ** -24   # silu's own error in fp32: exponential, 1 + x, reciprocal and products, a step or two each

# the largest fp32 number over log2(e) is 2.3587e38: the bf16 numbers beside it, some further off, the largest one
BORDER = [2.2994e38, 2.3527e38, 2.3660e38, 2.4058e38, 3.0e38, 3.3895314e38]
FINITE = torch.tensor(BORDER + [-v for v in BORDER]).to(torch.bfloat16)
INFINITE = torch.tensor([float("inf"), -float("inf"), float("nan")], dtype=torch.bfloat16)
UPS = (0.0, 1e-30, -1e-38, 0.5)   # silu(gate) * up stays finite


def silu(g):
    """By its definition, g / (1 + exp(-g)), in 64 bits."""
    return g / (1 + torch.exp(-g))


def check(got, ref, tol, what):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN places differ: {got} {ref}"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    keep = torch.isfinite(ref)
    diff = (got[keep] - ref[keep]).abs()
    assert bool((diff <= tol[keep]).all()), f"{what}: off by {float((diff - tol[keep]).max())} more than allowed"


def test_border_is_crossed():
    """Finite gates on both sides of the largest fp32 number over log2(e)."""
    t = FINITE.float() * np.float32(1.4426950408889634)
    assert torch.isfinite(t).any() and torch.isinf(t).any() and torch.isfinite(FINITE.float()).all()


@pytest.mark.parametrize("up", UPS)
@pytest.mark.parametrize("infinite", [False, True])
def test_swiglu_bf16_and_gradient_at_large_gates(infinite, up):
    special = INFINITE if infinite else FINITE
    I, rows = 16, len(special)
    rng = np.random.default_rng(31)
    gate, u = xh.bf16(rng, (rows, I)), torch.full((rows, I), up).to(torch.bfloat16)
    gate[:, 5] = special
    gu, d = torch.cat((gate, u), 1), torch.full((rows, I), 0.25).to(torch.bfloat16)
    g, u, dd = gate.double(), u.double(), d.double()
    ref = silu(g) * u
    check(ep.swiglu(gu.cuda()), ref, ref.abs() * (BF16 + SILU) + 2.0 ** -126, "swiglu")
    s = 1 / (1 + torch.exp(-g))
    slope, gs = s * (1 + g * (1 - s)), g * s
    ref = torch.cat((dd * u * slope, dd * gs), 1)
    # the slope's terms may cancel for ordinary gates: the error is theirs
    parts = torch.cat((dd * u * (s + (gs * (1 - s)).abs()), dd * gs), 1).abs()
    check(ep.swiglu_backward(d.cuda(), gu.cuda()), ref, ref.abs() * BF16 + 2 * SILU * parts + 2.0 ** -126, "gradient")


@pytest.mark.parametrize("kind", ["fp8", "mxfp4"])
@pytest.mark.parametrize("at", range(len(FINITE)))
def test_quantized_swiglu_at_large_gates(kind, at):
    """One large gate of a scale group, with an up value that keeps h finite: the scales are those of the definition."""
    I, size = 256, 128 if kind == "fp8" else 32
    rng = np.random.default_rng(32)
    gu = xh.bf16(rng, (2, 2 * I))
    gu[1, 70] = FINITE[at]
    gu[1, I + 70] = 1e-36
    q, s = (t.cpu() for t in ep.swiglu(gu.cuda(), kind=kind))
    h = (silu(gu[:, :I].double()) * gu[:, I:].double()).unflatten(1, (-1, size))
    amax = h.abs().amax(2)
    if kind == "fp8":
        scale = amax.clamp_min(1e-4) / 448
        check(s, scale, scale * (SILU + 4 * 2.0 ** -24), "scales")
        # half a step of e4m3, 2^-10 among its subnormals, and what h, scale and product are off by before it
        y = (h / scale.unsqueeze(2)).flatten(1)
        check(q.view(torch.float8_e4m3fn), y, y.abs() * (2.0 ** -4 + 2 * SILU + 2.0 ** -21) + 2.0 ** -10, "codes")
    else:
        e = torch.frexp(amax).exponent - 3 + 127
        lo, hi = (torch.frexp(amax * (1 + sign * SILU)).exponent - 3 + 127 for sign in (-1, 1))
        assert bool(((s.int() >= lo) & (s.int() <= hi)).all()), (s, e)


@pytest.mark.parametrize("gate", [float("inf"), -float("inf"), float("nan")])
def test_quantized_swiglu_of_infinite_gates(gate):
    """The group that holds the value is a NaN group, the others are not."""
    I = 256
    gu = xh.bf16(np.random.default_rng(33), (2, 2 * I))
    gu[1, 70] = gate
    q, s = (t.cpu() for t in ep.swiglu(gu.cuda(), kind="fp8"))
    assert torch.isnan(s).tolist() == [[False, False], [True, False]] and bool((q[1, :128] == 0x7F).all())
    q, s = (t.cpu() for t in ep.swiglu(gu.cuda(), kind="mxfp4"))
    assert (s == 255).nonzero().tolist() == [[1, 2]] and bool((q[1, 32:48] == 0).all())
