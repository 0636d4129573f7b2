"""The experts' operators as a program uses them: between dispatch and combine,
forward and backward, captured in graphs, on several streams, at far offsets."""
import numpy as np
import pytest
import torch

import experts_helpers as xh
from combine_get_dispatch_amd import ep

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8  # a rounding's largest relative error
SILU = 16 * 2.0 ** -24


def near(got, ref, tol, what):
    diff = (got.double().cpu() - ref).abs()
    assert not torch.isnan(diff).any(), what
    assert bool((diff <= tol).all()), f"{what}: off by {float((diff - tol).max())} more than allowed"


def routed(rng, T, E, k):
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    idx[0, 1:] = -1          # a token with one expert, and one with none
    idx[1, :] = -1
    w = rng.random((T, k), dtype=np.float32)
    return torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda()


def expert_rows(pos, idx, E):
    """Rows of each expert, from the handle's positions and the routing."""
    pos, idx = pos.cpu(), idx.cpu()
    return [pos[(idx == e) & (pos >= 0)].long() for e in range(E)]


def product_ref(x, w, rows, form):
    """64-bit product of the given rows and what the fp32 one may be off (see test_experts_gpu.py)."""
    ref, tol = {}, {}
    for e, r in enumerate(rows):
        a, b = x[r], w[e].t()
        ref[e] = a @ b
        t = (a.shape[1] + 8) * 2.0 ** -23 * (a.abs() @ b.abs())
        if form == "fp8":
            t = t + 128 * 2.0 ** -14 * (a.abs().unflatten(1, (-1, 128)).amax(2) @ b.abs().unflatten(0, (-1, 128)).amax(1))
        tol[e] = t + BF16 * (ref[e].abs() + t)
    return ref, tol


def check_product(out, x, w, rows, form, what):
    ref, tol = product_ref(x, w, rows, form)
    for e, r in enumerate(rows):
        near(out[r.cuda()], ref[e], tol[e], f"{what}, expert {e}")


@pytest.mark.parametrize("layout", ["packed", "low_latency"])
@pytest.mark.parametrize("form", ["bf16", "fp8", "mxfp4"])
def test_expert_layer(form, layout):
    """Dispatch, gate and up product, SwiGLU, down product, combine: every step
    against its 64-bit form on what the step before left."""
    rng = np.random.default_rng(11)
    T, H, I, E, R, k = 96, 512, 256, 8, 4, 3
    idx, w = routed(rng, T, E, k)
    x = xh.bf16(rng, (T, H)).cuda()
    cap = ep.ll_cap_rows(T, E, R) if layout == "low_latency" else T * k
    buf = ep.Buffer(T, H, k, E, R, cap)
    fp8 = form == "fp8"
    if layout == "low_latency":
        rx, rs, rw, count, handle = buf.dispatch_low_latency(x, idx, w, fp8)
        g = buf.groups_low_latency(count)
    else:
        lay, rx, rs, rw, handle = buf.dispatch_with_layout(x, idx, w, fp8)
        g = buf.groups(lay)
    rows = expert_rows(handle.pos, idx, E)
    w1, s1 = xh.make_operand(rng, (E, 2 * I, H), form if form != "mxfp4" else "bf16", weights=True)
    w2, s2 = xh.make_operand(rng, (E, H, I), form if form != "mxfp4" else "bf16", weights=True)
    w1, w2 = w1.cuda(), w2.cuda()
    s1, s2 = (None if s is None else s.cuda() for s in (s1, s2))
    if form == "mxfp4":
        (w1, s1), (w2, s2) = ep.quantize_mxfp4(w1), ep.quantize_mxfp4(w2)
        rx, rs = ep.quantize_mxfp4(rx, g)
    host = lambda t: None if t is None else t.cpu()  # noqa: E731
    h = ep.expert_gemm(rx, w1, g, row_scales=rs, weight_scales=s1)
    check_product(h, xh.operand(host(rx), host(rs), form), xh.operand(host(w1), host(s1), form, True), rows, form, "up")
    a = ep.swiglu(h, g, kind=form)
    a, sa = a if form != "bf16" else (a, None)
    y = ep.expert_gemm(a, w2, g, row_scales=sa, weight_scales=s2)
    check_product(y, xh.operand(host(a), host(sa), form), xh.operand(host(w2), host(s2), form, True), rows, form, "down")
    # what SwiGLU left is its 64-bit form up to the rounding of the form: half a step, of e2m1 below its smallest too
    used = torch.cat(rows)
    hv = h.double().cpu()[used]
    ref = hv[:, :I] * torch.sigmoid(hv[:, :I]) * hv[:, I:]
    av = xh.operand(host(a), host(sa), form)[used]
    if form == "bf16":
        tol = ref.abs() * (BF16 + SILU)
    elif form == "fp8":
        tol = ref.abs() * (2.0 ** -4 + 2.0 ** -20) + xh.operand(torch.full_like(host(a), 0x38), host(sa), form)[used] * 2.0 ** -10
    else:  # steps of 1/4 below 2, 1/2 below 4, 1 below 6, up to 2 where it is cut, in units of the scale
        unit = torch.ldexp(torch.ones(()).double(), host(sa)[used].int() - 127).repeat_interleave(32, 1)
        r = ref.abs() / unit
        tol = unit * torch.where(r < 2, 0.25, torch.where(r < 4, 0.5, torch.where(r <= 6, 1.0, 2.0))) + ref.abs() * SILU
    near(av, ref, tol + 2.0 ** -100, "swiglu")
    out = buf.combine(y, handle, w)
    yv, pos, wv = y.double().cpu(), handle.pos.cpu().long(), w.double().cpu()
    taken = torch.where((pos >= 0)[..., None], yv[pos.clamp_min(0)] * wv[..., None], 0.0)
    ref = taken.sum(1)
    near(out, ref, ref.abs() * BF16 + 2 * k * 2.0 ** -23 * taken.abs().sum(1), "combine")
    assert buf.status() == 0
    assert bool((out[1] == 0).all())  # the token without experts


def test_layouts_agree():
    """The same tokens through packed rows and through regions: the same output bits."""
    rng = np.random.default_rng(12)
    T, H, E, R, k = 64, 384, 16, 2, 2
    idx, w = routed(rng, T, E, k)
    x, w1 = xh.bf16(rng, (T, H)).cuda(), xh.bf16(rng, (E, 200, H)).cuda()
    w2 = xh.bf16(rng, (E, H, 200)).cuda()
    outs = []
    for ll in (False, True):
        buf = ep.Buffer(T, H, k, E, R, ep.ll_cap_rows(T, E, R))
        if ll:
            rx, _, _, count, handle = buf.dispatch_low_latency(x, idx, w, False)
            g = buf.groups_low_latency(count)
        else:
            lay, rx, _, _, handle = buf.dispatch_with_layout(x, idx, w, False)
            g = buf.groups(lay)
        y = ep.expert_gemm(ep.expert_gemm(rx, w1, g), w2, g)
        outs.append(buf.combine(y, handle, w))
    assert torch.equal(*outs)


def test_training_step():
    """Forward and backward through the experts, each gradient against its formula in 64 bits on the same inputs."""
    rng = np.random.default_rng(13)
    T, H, I, E, R, k = 80, 264, 136, 8, 2, 2
    idx, w = routed(rng, T, E, k)
    x = xh.bf16(rng, (T, H)).cuda()
    w1, w2 = xh.bf16(rng, (E, 2 * I, H), 0.1).cuda(), xh.bf16(rng, (E, H, I), 0.1).cuda()
    buf = ep.Buffer(T, H, k, E, R, T * k)
    lay, rx, _, rw, handle = buf.dispatch_with_layout(x, idx, w, False)
    g, rows = buf.groups(lay), expert_rows(handle.pos, idx, E)
    h = ep.expert_gemm(rx, w1, g)
    a = ep.swiglu(h, g)
    y = ep.expert_gemm(a, w2, g)
    buf.combine(y, handle, w)
    gy = xh.bf16(rng, (T, H)).cuda()
    d = buf.combine_backward(gy, handle) * rw.to(torch.bfloat16)[:, None]
    ga, gw2 = ep.expert_gemm_dgrad(d, w2, g), ep.expert_gemm_wgrad(d, a, g)
    gh = ep.swiglu_backward(ga, h, g)
    gx, gw1 = ep.expert_gemm_dgrad(gh, w1, g), ep.expert_gemm_wgrad(gh, rx, g, dtype=torch.bfloat16)
    grad_x = buf.dispatch_backward(gx, handle)
    assert gw2.dtype == torch.float32 and gw1.dtype == torch.bfloat16 and buf.status() == 0
    v = {n: t.double().cpu() for n, t in dict(rx=rx, h=h, a=a, d=d, ga=ga, gh=gh, w1=w1, w2=w2).items()}
    for e, r in enumerate(rows):
        for got, up, wt, n in ((ga, "d", "w2", H), (gx, "gh", "w1", 2 * I)):
            ref, mag = v[up][r] @ v[wt][e], v[up][r].abs() @ v[wt][e].abs()
            t = (n + 8) * 2.0 ** -23 * mag
            near(got[r.cuda()], ref, t + BF16 * (ref.abs() + t), f"dgrad {wt}")
        for got, up, inp, step in ((gw2, "d", "a", 2.0 ** -24), (gw1, "gh", "rx", BF16)):
            ref, mag = v[up][r].t() @ v[inp][r], v[up][r].abs().t() @ v[inp][r].abs()
            t = (len(r) + 8) * 2.0 ** -23 * mag
            near(got[e], ref, t + step * (ref.abs() + t), f"wgrad of {inp}")
    used = torch.cat(rows)
    gate, up, dd = v["h"][used][:, :I], v["h"][used][:, I:], v["ga"][used]
    s = torch.sigmoid(gate)
    ref = torch.cat((dd * up * s * (1 + gate * (1 - s)), dd * gate * s), 1)
    mag = torch.cat((dd * up * s * (1 + gate.abs()), dd * gate * s), 1).abs()
    near(gh[used.cuda()], ref, ref.abs() * BF16 + 2 * SILU * mag, "swiglu_backward")
    assert torch.isfinite(grad_x).all()


def test_gradients_against_differences():
    """<gradient, direction> against central differences of the 64-bit forward form."""
    rng = np.random.default_rng(14)
    E, K, N = 4, 72, 40
    counts, off = [9, 0, 1, 33], [0, 9, 0, 1]
    g = ep.Groups(torch.tensor(counts, dtype=torch.int32).cuda(), torch.tensor(off, dtype=torch.int32).cuda(),
                  num_experts=E, num_ranks=2, cap_rows=40)
    rows = [list(range(e // 2 * 40 + off[e], e // 2 * 40 + off[e] + counts[e])) for e in range(E)]
    x, w, d = xh.bf16(rng, (80, K)), xh.bf16(rng, (E, N, K)), xh.bf16(rng, (80, N))
    gx = ep.expert_gemm_dgrad(d.cuda(), w.cuda(), g, out=torch.zeros(80, K, dtype=torch.bfloat16, device="cuda"))
    gw = ep.expert_gemm_wgrad(d.cuda(), x.cuda(), g)

    def loss(x, w):
        return sum(float((d[r].double() * (x[r] @ w[e].t())).sum()) for e, r in enumerate(rows))

    x, w = x.double(), w.double()
    for _ in range(3):
        dx = torch.from_numpy(rng.standard_normal(x.shape))
        dw = torch.from_numpy(rng.standard_normal(w.shape))
        # the loss is linear in each: the difference is exact up to 64-bit rounding; the gradient's error is a rounding of
        # each value and fp32 sums of up to N (rows) products of magnitudes about 1
        want = (loss(x + dx, w) - loss(x - dx, w)) / 2
        got, size = float((gx.double().cpu() * dx).sum()), float((gx.double().cpu() * dx).abs().sum())
        assert abs(got - want) <= size * BF16 + dx.abs().sum() * N * N * 2.0 ** -23 * 16
        want = (loss(x, w + dw) - loss(x, w - dw)) / 2
        got, size = float((gw.double().cpu() * dw).sum()), float((gw.double().cpu() * dw).abs().sum())
        assert abs(got - want) <= size * 2.0 ** -24 + dw.abs().sum() * 33 * 33 * 2.0 ** -23 * 16
    I = 64
    gu, dd = xh.bf16(rng, (20, 2 * I), 2.0), xh.bf16(rng, (20, I))
    gg = ep.swiglu_backward(dd.cuda(), gu.cuda()).double().cpu()

    def swiglu_loss(t):
        return float((dd.double() * t[:, :I] * torch.sigmoid(t[:, :I]) * t[:, I:]).sum())

    for _ in range(3):
        dt = torch.from_numpy(rng.standard_normal(gu.shape))
        eps = 1e-5  # third derivatives of order 1: the difference is off by some eps^2 a value, and 64-bit rounding / eps
        want = (swiglu_loss(gu.double() + eps * dt) - swiglu_loss(gu.double() - eps * dt)) / (2 * eps)
        got, size = float((gg * dt).sum()), float((gg * dt).abs().sum())
        assert abs(got - want) <= size * (BF16 + 64 * SILU) + 1e-5 * float(dt.abs().pow(3).sum()) + 1e-4


def test_graphs_and_streams():
    """A captured expert layer replayed with new inputs, eager work on another
    stream between the replays; two streams at once; every time the same bits."""
    rng = np.random.default_rng(15)
    E, H, I, n = 8, 512, 256, 300
    off, cap, rows = xh.packed_groups([40, 0, 1, 129, 64, 7, 30, 20], 1, slack=9)
    counts = torch.tensor([len(r) for r in rows], dtype=torch.int32).cuda()
    g = ep.Groups(counts, torch.from_numpy(off).cuda(), num_experts=E, num_ranks=1, cap_rows=cap)
    w1, s1 = (t.cuda() for t in xh.make_operand(rng, (E, 2 * I, H), "fp8", weights=True))
    w2, s2 = (t.cuda() for t in xh.make_operand(rng, (E, H, I), "fp8", weights=True))

    def layer(x, xs, y):
        h = ep.expert_gemm(x, w1, g, row_scales=xs, weight_scales=s1)
        a, sa = ep.swiglu(h, g, kind="fp8")
        ep.expert_gemm(a, w2, g, row_scales=sa, weight_scales=s2, out=y)
        gw = ep.expert_gemm_wgrad(y, y, g)
        q, qs = ep.quantize_mxfp4(y, g)
        ep.dequantize_mxfp4(q, qs, g, out=y)
        return gw

    inputs = [tuple(t.cuda() for t in xh.make_operand(rng, (cap, H), "fp8")) for _ in range(4)]
    fresh = lambda: torch.zeros((cap, H), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    eager = []
    for x, xs in inputs:
        y = fresh()
        eager.append((y, layer(x, xs, y)))
    x, xs, y = inputs[0][0].clone(), inputs[0][1].clone(), fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, xs, y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gw = layer(x, xs, y)
    for turn in range(2):
        for (a, b), (want, want_w) in zip(inputs, eager):
            x.copy_(a), xs.copy_(b)
            y.zero_()
            torch.cuda.synchronize()
            other = fresh()
            graph.replay()
            with torch.cuda.stream(side):  # beside the replay
                side_w = layer(*inputs[3], other)
            torch.cuda.synchronize()
            assert torch.equal(y, want) and torch.equal(gw, want_w)
            assert torch.equal(other, eager[3][0]) and torch.equal(side_w, eager[3][1])


def test_not_a_number_stays_in_its_row():
    rng = np.random.default_rng(16)
    off, cap, rows = xh.packed_groups([20, 70], 1)
    g = ep.Groups(torch.tensor([20, 70], dtype=torch.int32).cuda(), torch.from_numpy(off).cuda(), num_experts=2,
                  num_ranks=1, cap_rows=cap)
    x, w = xh.bf16(rng, (cap, 96)), xh.bf16(rng, (2, 64, 96))
    clean = ep.expert_gemm(x.cuda(), w.cuda(), g)
    bad = x.clone()
    bad[3, 95], bad[50, 0], bad[51, 7] = float("nan"), float("inf"), -float("inf")
    got = ep.expert_gemm(bad.cuda(), w.cuda(), g)
    assert torch.isnan(got[3]).all()
    sign = torch.sign(w[1, :, 0].float()).cuda()
    assert torch.equal(got[50].float(), sign * float("inf"))
    keep = torch.tensor([r for e in rows for r in e if r not in (3, 50, 51)]).cuda()
    assert torch.equal(got[keep], clean[keep])
    gu = xh.bf16(rng, (4, 512))
    gu[1, 5], gu[2, 300] = float("nan"), float("inf")
    q, s = ep.swiglu(gu.cuda(), kind="fp8")
    nan = torch.isnan(s.cpu())
    want = torch.zeros(4, 2, dtype=torch.bool)
    want[1, 0] = want[2, 0] = True  # channel 5 is in group 0, as is the up value of channel 44
    assert torch.equal(nan, want)
    assert (q.cpu()[1, :128] == 0x7F).all() and (q.cpu()[0] != 0x7F).all()
    q, s = ep.swiglu(gu.cuda(), kind="mxfp4")
    assert (s.cpu() == 255).sum() == 2 and s.cpu()[1, 0] == 255 and s.cpu()[2, 1] == 255


def test_bad_counts_stay_inside():
    """Counts and offsets outside the rows are cut: nothing past a rank's rows is written."""
    rng = np.random.default_rng(17)
    counts, off = [5, 1 << 30, -7, 4], [0, 5, 3, 62]
    g = ep.Groups(torch.tensor(counts, dtype=torch.int32).cuda(), torch.tensor(off, dtype=torch.int32).cuda(),
                  num_experts=4, num_ranks=2, cap_rows=64)
    rows = [list(range(5)), list(range(5, 64)), [], [126, 127]]
    x, w = xh.bf16(rng, (128, 64)), xh.bf16(rng, (4, 40, 64))
    guard = torch.full((128 + 64, 40), -5.0, dtype=torch.bfloat16, device="cuda")
    out = ep.expert_gemm(x.cuda(), w.cuda(), g, out=guard[:128])
    used = torch.zeros(192, dtype=torch.bool)
    used[[r for e in rows for r in e]] = True
    assert bool((guard.cpu()[~used] == -5.0).all())
    check_product(out, x.double(), w.double(), [torch.tensor(r, dtype=torch.long) for r in rows], "bf16", "cut")
    region = ep.Groups(torch.tensor([[9, -1], [3, 1 << 30]], dtype=torch.int32).cuda(), None, num_experts=2, num_ranks=2,
                       cap_rows=16, region_rows=8)
    y = torch.full((32, 32), -5.0, dtype=torch.bfloat16, device="cuda")
    ep.swiglu(xh.bf16(rng, (32, 64)).cuda(), region, out=y)
    same = (y.cpu() == -5.0).all(1)
    assert same.tolist() == [False] * 8 + [True] * 8 + [False] * 3 + [True] * 5 + [False] * 8


@pytest.mark.parametrize("form", ["bf16", "fp8", "mxfp4"])
def test_far_offsets(form):
    """Rows, weights and results past 4 GiB: the last expert's, at the end of the arrays."""
    rng = np.random.default_rng(18)
    K, N, n = 16384, 2048, 37
    width = {"bf16": 2 * K, "fp8": K, "mxfp4": K // 2}[form]
    E = (5 << 30) // (N * width) + 1
    cap = (5 << 30) // width + n
    out_rows = torch.empty((cap, N), dtype=torch.bfloat16, device="cuda")
    x, xs = xh.make_operand(rng, (n, K), form)
    w, ws = xh.make_operand(rng, (1, N, K), form, weights=True)

    def at_end(t, shape):
        if t is None:
            return None
        big = torch.empty(shape, dtype=t.dtype, device="cuda")
        big[-t.shape[0]:] = t.cuda()
        return big

    big = [at_end(x, (cap,) + tuple(x.shape[1:])), at_end(w, (E,) + tuple(w.shape[1:])),
           at_end(xs, (cap,) + tuple(xs.shape[1:])) if xs is not None else None,
           at_end(ws, (E,) + tuple(ws.shape[1:])) if ws is not None else None]
    counts, off = torch.zeros(E, dtype=torch.int32), torch.zeros(E, dtype=torch.int32)
    counts[-1], off[-1] = n, cap - n
    g = ep.Groups(counts.cuda(), off.cuda(), num_experts=E, num_ranks=1, cap_rows=cap, rows_hint=n)
    ep.expert_gemm(big[0], big[1], g, row_scales=big[2], weight_scales=big[3], out=out_rows)
    check_product(out_rows[-n:], xh.operand(x, xs, form), xh.operand(w, ws, form, True), [torch.arange(n)], form, "far")


@pytest.mark.parametrize("E", [1, 1024])
def test_expert_counts(E):
    """One expert, and as many as there may be, on 64 ranks."""
    rng = np.random.default_rng(19)
    R, K, N = (64, 32, 16) if E == 1024 else (1, 40, 24)
    counts = rng.integers(0, 4, E).astype(np.int32)
    counts[-1] = 3
    off, cap, rows = xh.packed_groups(list(counts), R, slack=1)
    g = ep.Groups(torch.from_numpy(counts).cuda(), torch.from_numpy(off).cuda(), num_experts=E, num_ranks=R, cap_rows=cap)
    x, w = xh.bf16(rng, (R * cap, K)), xh.bf16(rng, (E, N, K))
    out = torch.full((R * cap, N), -3.0, dtype=torch.bfloat16, device="cuda")
    ep.expert_gemm(x.cuda(), w.cuda(), g, out=out)
    check_product(out, x.double(), w.double(), [torch.tensor(r, dtype=torch.long) for r in rows], "bf16", "product")
    gw = ep.expert_gemm_wgrad(out, x.cuda(), g)
    ov = out.double().cpu()
    for e in range(0, E, max(1, E // 7)):
        ref = ov[rows[e]].t() @ x.double()[rows[e]]
        mag = ov[rows[e]].abs().t() @ x.double()[rows[e]].abs()
        near(gw[e], ref, 12 * 2.0 ** -23 * mag + 2.0 ** -24 * ref.abs(), "wgrad")


@pytest.mark.parametrize("form", ["bf16", "fp8", "mxfp4"])
def test_same_bits_again_and_on_few_compute_units(form):
    """A call repeated, and made on a stream that may use 32 compute units, gives the same bits; any hint the right result."""
    rng = np.random.default_rng(20)
    E, K, N = 8, 1024, 640
    off, cap, rows = xh.packed_groups([300, 0, 17, 256, 90, 1, 513, 64], 2)
    counts = torch.tensor([len(r) for r in rows], dtype=torch.int32).cuda()
    x, xs = (t if t is None else t.cuda() for t in xh.make_operand(rng, (2 * cap, K), form))
    w, ws = (t if t is None else t.cuda() for t in xh.make_operand(rng, (E, N, K), form, weights=True))

    def call(hint):
        g = ep.Groups(counts, torch.from_numpy(off).cuda(), num_experts=E, num_ranks=2, cap_rows=cap, rows_hint=hint)
        out = torch.zeros((2 * cap, N), dtype=torch.bfloat16, device="cuda")
        return ep.expert_gemm(x, w, g, row_scales=xs, weight_scales=ws, out=out)

    first = call(0)
    assert torch.equal(call(0), first)
    torch.cuda.synchronize()
    with ep.CuStream(32) as s, torch.cuda.stream(s.torch_stream):
        capped = call(0)
        s.torch_stream.synchronize()
    assert torch.equal(capped, first)
    for hint in (1, 8 * 40, 1 << 20):
        check_product(call(hint), xh.operand(*(t if t is None else t.cpu() for t in (x, xs)), form),
                      xh.operand(*(t if t is None else t.cpu() for t in (w, ws)), form, True),
                      [torch.tensor(r, dtype=torch.long) for r in rows], form, f"hint {hint}")
