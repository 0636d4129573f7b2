"""The router on the GPU against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import router_helpers as rh
from combine_get_dispatch_amd import ep

pytestmark = pytest.mark.gpu

INF = float("inf")
LOWEST = float(torch.finfo(torch.bfloat16).min)


def drawn(rng, T, E, dtype, scale=2.0):
    return torch.from_numpy(rng.standard_normal((T, E), dtype=np.float32) * np.float32(scale)).to(dtype)


def tolerance(logits, w):
    """Exponents' arguments are rounded differences of logits (at most `span` here), each exponential, quotient and sum of at
    most 1024 positive terms in a tree adds a few roundings; results below 2^-126 may be 0."""
    l = np.nan_to_num(logits.double().numpy(), nan=0.0, posinf=0.0, neginf=0.0)
    l = np.where(np.abs(l) > 1e30, 0.0, l)
    span = np.minimum(l.max(1) - l.min(1), 100.0)[:, None]
    return np.abs(w) * (64 + 4 * span) * 2.0 ** -24 + 2.0 ** -120


def check(logits, r, bias=None, tol=None):
    idx, w = ep.route(logits.cuda(), r, bias=None if bias is None else bias.cuda())
    want, ref = rh.route(logits.double().numpy(), r, None if bias is None else bias.double().numpy())
    got = idx.cpu().numpy()
    bad = np.flatnonzero((got != want).any(1))
    assert not len(bad), f"token {bad[0]}: {got[bad[0]]}, not {want[bad[0]]}"
    w = w.double().cpu().numpy()
    assert np.array_equal(np.isnan(w), np.isnan(ref))
    off = np.abs(w - ref) - (tolerance(logits, ref) if tol is None else tol)
    assert not (np.nan_to_num(off, nan=0.0) > 0).any(), f"weights off by {np.nanmax(off)} more than allowed"
    return idx, w


SHAPES = [  # E, k, groups, kept, group_top
    (1, 1, 1, 1, 2), (8, 8, 1, 1, 2), (37, 3, 1, 1, 2), (48, 2, 1, 1, 2), (60, 4, 4, 2, 2), (64, 6, 8, 3, 1),
    (160, 6, 8, 3, 1), (160, 6, 8, 3, 2), (256, 8, 1, 1, 2), (256, 8, 8, 4, 2), (256, 8, 8, 8, 2), (250, 10, 5, 2, 2),
    (256, 16, 16, 9, 2), (384, 10, 3, 2, 1), (1020, 32, 5, 2, 2), (1024, 32, 64, 17, 2), (1024, 1, 1, 1, 2), (33, 32, 1, 1, 2),
    (34, 5, 17, 5, 2), (63, 4, 21, 4, 2), (1023, 8, 33, 7, 2),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("score,bias,renorm", [("softmax", False, True), ("softmax", False, False), ("softmax", True, False),
                                               ("sigmoid", True, True), ("sigmoid", False, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_route(shape, score, bias, renorm, dtype):
    E, k, G, kept, top = shape
    r = ep.Router(E, k, score=score, renormalize=renorm, scale=2.5, num_groups=G, topk_groups=kept, group_top=top)
    rng = np.random.default_rng([E, k, G, int(bias)])
    b = torch.from_numpy(rng.standard_normal(E, dtype=np.float32) * np.float32(0.1)) if bias else None
    for T in (1, 7, 70):
        check(drawn(rng, T, E, dtype), r, b)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] <= 384], ids=str)
@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", True)])
def test_route_of_many_tokens(shape, score, bias):
    """A batch that fills the chip gives every token what it gets alone (and alone is checked above)."""
    E, k, G, kept, top = shape
    r = ep.Router(E, k, score=score, num_groups=G, topk_groups=kept, group_top=top)
    rng = np.random.default_rng([E, k, 5])
    b = torch.from_numpy(rng.standard_normal(E, dtype=np.float32) * np.float32(0.1)).cuda() if bias else None
    logits = drawn(rng, 4099, E, torch.bfloat16).cuda()
    logits[100:140] = logits[100:140].round()  # ties
    idx, w = ep.route(logits, r, bias=b)
    for at in (0, 97, 2040, 4029):
        few, fw = ep.route(logits[at:at + 70].contiguous(), r, bias=b)
        assert torch.equal(few, idx[at:at + 70])
        assert bool(((fw - w[at:at + 70]).abs() <= 64 * 2.0 ** -24 * fw).all())


@pytest.mark.parametrize("T", [50, 4100])
@pytest.mark.parametrize("score,bias,groups", [("softmax", None, False), ("sigmoid", 0.0, False), ("sigmoid", None, True),
                                               ("softmax", 0.0, True), ("sigmoid", 0.25, True)])
def test_ties_go_to_the_lowest_index(T, score, bias, groups):
    E, k = 64, 6
    r = ep.Router(E, k, score=score, num_groups=8 if groups else 1, topk_groups=3 if groups else 1)
    rng = np.random.default_rng([T, 1])
    logits = torch.from_numpy(rng.integers(-1, 2, (50, E)).astype(np.float32))
    logits[0] = 0.0
    b = None if bias is None else torch.full((E,), bias)
    logits = logits.to(torch.bfloat16)
    if T > 50:
        many = logits[torch.arange(T) % 50]
        idx, w = ep.route(many.cuda(), r, bias=None if b is None else b.cuda())
        few, fw = check(logits, r, b)
        assert torch.equal(idx, few[(torch.arange(T) % 50).cuda()])
    else:
        check(logits, r, b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("groups", [1, 8])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masks_and_ends(score, renorm, groups, with_bias):
    E, k = 64, 6
    r = ep.Router(E, k, score=score, renormalize=renorm, num_groups=groups, topk_groups=max(1, groups // 2))
    rng = np.random.default_rng([groups, int(with_bias), 2])
    logits = drawn(rng, 12, E, torch.float32)
    logits[0] = -INF                                   # nothing open
    logits[1, 3:] = -INF                               # three open, of one group
    logits[2, ::2] = -INF
    logits[3, 4:] = LOWEST                             # four that matter, the others at the type's lowest value
    logits[4] = LOWEST                                 # all equal, and open
    logits[5, [5, 40]] = INF
    logits[6, 7] = float("nan")
    logits[7] = float("nan")
    logits[8, 1:] = -INF                               # one expert
    logits[9] = torch.from_numpy(rng.standard_normal(E)) * 0.01 - 60.0  # sigmoids near 2^-87
    logits[10] = 30.0 + torch.from_numpy(rng.standard_normal(E).astype(np.float32))
    logits[11, :8], logits[11, 8:] = 0.25, -INF        # one group's experts, all equal
    b = None
    if with_bias:
        b = torch.from_numpy(rng.standard_normal(E, dtype=np.float32) * np.float32(0.1))
        b[9], b[10], b[33], b[34] = -INF, float("nan"), 50.0, -50.0
    idx, w = check(logits, r, b)
    assert bool((idx[0] == -1).all()) and not w[0].any()
    if not with_bias:  # the lower index of two that agree in all that counts
        assert idx[4].tolist() == list(range(k))
    if with_bias:
        assert not torch.isin(idx, torch.tensor([9, 10], dtype=torch.int32, device="cuda")).any()


@pytest.mark.parametrize("T", [2050, 4100])
@pytest.mark.parametrize("score,groups,with_bias", [("softmax", 1, False), ("softmax", 8, False), ("sigmoid", 1, True),
                                                    ("sigmoid", 8, True), ("sigmoid", 8, False), ("softmax", 8, True)])
def test_masks_and_ends_of_many_tokens(T, score, groups, with_bias):
    """Masked, infinite, equal and NaN logits among the tokens of a batch that fills the chip: as in a small one."""
    E, k = 64, 6
    r = ep.Router(E, k, score=score, renormalize=groups == 1, num_groups=groups, topk_groups=max(1, groups // 2))
    rng = np.random.default_rng([groups, int(with_bias), 7])
    logits = drawn(rng, 16, E, torch.float32)
    logits[0] = -INF
    logits[1, 3:] = -INF
    logits[2, ::2] = -INF
    logits[3, 4:] = LOWEST
    logits[4] = LOWEST
    logits[5, [5, 40]] = INF
    logits[6, 7] = float("nan")
    logits[7] = float("nan")
    logits[8, 1:] = -INF
    logits[9] = 50.0 + torch.from_numpy(rng.standard_normal(E).astype(np.float32))  # sigmoids that are 1 in 32 bits
    logits[10] = INF
    logits[11, :8], logits[11, 8:] = 0.25, -INF
    logits[12] = logits[12].round()
    logits[13] = -200.0 + torch.from_numpy(rng.standard_normal(E).astype(np.float32))
    b = None
    if with_bias:
        b = torch.from_numpy(rng.standard_normal(E, dtype=np.float32) * np.float32(0.1))
        b[9], b[10], b[33], b[34], b[35] = -INF, float("nan"), 50.0, -50.0, 1e30
    few, fw = check(logits, r, b)
    at = torch.arange(T) % 16
    idx, w = ep.route(logits[at].cuda(), r, bias=None if b is None else b.cuda())
    assert torch.equal(idx, few[at.cuda()])
    fw = torch.from_numpy(fw)[at].cuda()
    assert torch.equal(w.isnan(), fw.isnan())
    assert bool(((w - fw).abs().nan_to_num(0.0) <= 64 * 2.0 ** -24 * fw.nan_to_num(0.0) + 2.0 ** -120).all())


@pytest.mark.parametrize("value", [-1e4, -200.0, 200.0, 1e4, LOWEST])
def test_renormalized_weights_of_far_logits(value):
    """Scores that underflow (or are all 1) still give weights that sum to the scale."""
    for score in ("softmax", "sigmoid"):
        r = ep.Router(16, 4, score=score, scale=2.0)
        _, w = ep.route(torch.full((3, 16), value).cuda(), r)
        assert bool(((w - 0.5).abs() <= 2.0 ** -22).all())


def test_choice_by_exact_scores():
    """Sums of score and bias that are one 32-bit number but not one real number: the larger is chosen."""
    rng = np.random.default_rng(3)
    E, found = 32, 0
    for turn in range(40):
        l = rng.standard_normal(E).astype(np.float32)
        s = rh.scores(l, "sigmoid")
        b = (np.float64(1.0) - s).astype(np.float32)  # sums within 2^-25 of 1
        r = ep.Router(E, 4, score="sigmoid")
        check(torch.from_numpy(l)[None], r, torch.from_numpy(b))
        found += len(np.unique(s.astype(np.float32) + b)) < E
    assert found == 40


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (7, 37, 3), (70, 256, 8), (33, 300, 20), (5, 1024, 32), (9, 16, 16), (3, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_gradient(score, renorm, T, E, k, dtype):
    rng = np.random.default_rng([T, E, k])
    r = ep.Router(E, k, score=score, renormalize=renorm, scale=2.5)
    logits = drawn(rng, T, E, dtype)
    idx = torch.from_numpy(np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32))
    if T > 4:
        idx[0] = -1
        idx[1, 0] = -1
        idx[2, -1], idx[3, -1] = E, -7      # no experts: left out
        idx[4, 1:] = idx[4, 0].clone()      # one expert again and again: once
    d = torch.from_numpy(rng.standard_normal((T, k), dtype=np.float32))
    out = torch.full((T + 1, E), 77.0, dtype=dtype, device="cuda")
    got = ep.route_backward(d.cuda(), logits.cuda(), idx.cuda(), r, out=out[:T])
    assert bool((out[T] == 77.0).all())
    ref, size = rh.gradient(d.numpy(), logits.double().numpy(), idx.numpy(), r)
    step = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24
    span = logits.double().amax(1) - logits.double().amin(1)
    # scores as in the weights' tolerance, twice (score and slope); a sum over k, and the difference's magnitudes
    tol = size * (128 + 8 * span.numpy()[:, None]) * 2.0 ** -24
    tol = tol + step * (np.abs(ref) + tol) + 2.0 ** -120
    off = np.abs(got.double().cpu().numpy() - ref) - tol
    assert (off <= 0).all(), f"off by {off.max()} more than allowed"


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_against_differences(score, renorm):
    """<gradient, direction> against central differences of the 64-bit weights of the same choice."""
    rng = np.random.default_rng(4)
    T, E, k = 20, 48, 4
    r = ep.Router(E, k, score=score, renormalize=renorm)
    logits = drawn(rng, T, E, torch.float32)
    idx, _ = ep.route(logits.cuda(), r)
    d = torch.from_numpy(rng.standard_normal((T, k), dtype=np.float32))
    g = ep.route_backward(d.cuda(), logits.cuda(), idx, r).double().cpu().numpy()
    picked, l = idx.cpu().numpy(), logits.double().numpy()

    def loss(x):
        return sum(float(d[t].double().numpy() @ rh.weights(x[t], picked[t], r)) for t in range(T))

    for _ in range(3):
        u, eps = rng.standard_normal((T, E)), 1e-4
        want = (loss(l + eps * u) - loss(l - eps * u)) / (2 * eps)
        # third derivatives of order 1 over T tokens: eps^2 each; 64-bit rounding / eps; the kernel's own 2^-17 of every term
        assert abs((g * u).sum() - want) <= 2.0 ** -17 * np.abs(g * u).sum() + T * 100 * eps ** 2 + 1e-9


def test_lengths_and_memory_around():
    """No token; a call writes what is its own."""
    r = ep.Router(64, 4)
    idx, w = ep.route(torch.zeros(0, 64).cuda(), r)
    assert idx.shape == w.shape == (0, 4)
    assert ep.route_backward(w, torch.zeros(0, 64).cuda(), idx, r).shape == (0, 64)
    for T in (1, 3, 4097):
        idx = torch.full((T + 2, 4), 77, dtype=torch.int32, device="cuda")
        w = torch.full((T + 2, 4), 77.0, device="cuda")
        ep.route(torch.randn(T, 64, device="cuda"), r, out=(idx[1:T + 1], w[1:T + 1]))
        assert bool((idx[[0, T + 1]] == 77).all()) and bool((w[[0, T + 1]] == 77.0).all())
        assert bool((idx[1:T + 1] < 64).all()) and bool((idx[1:T + 1] >= 0).all())


def test_routed_layer_with_its_gradient():
    """Logits to combined output and back to the logits' gradient, through the exchange, in a graph that is replayed with other
    logits; the weights' gradient is <expert_out row, grad_combined row>."""
    rng = np.random.default_rng(6)
    T, H, E, R, k = 96, 256, 32, 4, 4
    r = ep.Router(E, k, score="sigmoid", num_groups=4, topk_groups=2, scale=1.5)
    bias = torch.from_numpy(rng.standard_normal(E, dtype=np.float32) * np.float32(0.1)).cuda()
    x = torch.from_numpy(rng.standard_normal((T, H), dtype=np.float32)).to(torch.bfloat16).cuda()
    gy = torch.from_numpy(rng.standard_normal((T, H), dtype=np.float32)).to(torch.bfloat16).cuda()
    wt = torch.from_numpy(rng.standard_normal((E, H, H), dtype=np.float32) * np.float32(0.06)).to(torch.bfloat16).cuda()
    buf = ep.Buffer(T, H, k, E, R, T * k)

    def step(logits):
        idx, w = ep.route(logits, r, bias=bias)
        lay, rx, _, _, h = buf.dispatch_with_layout(x, idx, w, False)
        y = ep.expert_gemm(rx, wt, buf.groups(lay))
        out = buf.combine(y, h, w)
        pos = h.pos.clamp_min(0).long()
        dw = torch.where(h.pos >= 0, (y[pos].float() * gy[:, None].float()).sum(2), 0.0)
        return idx, w, out, dw, ep.route_backward(dw, logits, idx, r), pos, y

    inputs = [drawn(rng, T, E, torch.float32).cuda() for _ in range(3)]
    inputs[1][5] = -INF
    eager = [[t.clone() for t in step(l)] for l in inputs]
    assert buf.status() == 0
    for l, (idx, w, out, dw, g, pos, y) in zip(inputs, eager):
        want, ref = rh.route(l.double().cpu().numpy(), r, bias.double().cpu().numpy())
        assert np.array_equal(idx.cpu().numpy(), want)
        taken = torch.where((idx >= 0)[..., None], y[pos].double() * w[..., None].double(), 0.0)
        tol = taken.sum(1).abs() * 2.0 ** -8 + 2 * k * 2.0 ** -23 * taken.abs().sum(1)
        assert bool(((out.double() - taken.sum(1)).abs() <= tol).all())
        ref, size = rh.gradient(dw.cpu().numpy(), l.double().cpu().numpy(), want, r)
        assert (np.abs(g.double().cpu().numpy() - ref) <= size * 256 * 2.0 ** -24 + 2.0 ** -120).all()
    logits = inputs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(logits)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(logits)
    for turn in range(2):
        for l, want in zip(inputs, eager):
            logits.copy_(l)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(captured[:5], want[:5]):
                assert torch.equal(a, b)
            step(l)  # eager work between the replays
    assert buf.status() == 0
