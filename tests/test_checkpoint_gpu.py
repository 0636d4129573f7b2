"""8-bit activation checkpoints on the GPU, and their use in the backward pass."""
import numpy as np
import pytest
import torch

import experts_helpers as xh
from combine_get_dispatch_amd import ep
from test_experts_gpu import COUNTS, SENTINEL, check, groups_of, poisoned

pytestmark = pytest.mark.gpu


def kept_of(x):
    """(codes, scale bytes) of bf16 values [.., 32 n] by the rule, in 64 bits."""
    b = x.double().unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad.unsqueeze(-1), 0.0, b)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1, -127).clamp_min(-127)
    q = torch.ldexp(b, (6 - e).unsqueeze(-1)).round().clamp(-127, 127)
    return q.flatten(-2).to(torch.int8), torch.where(bad, 255, e + 127).to(torch.uint8)


def values_of(q, s):
    unit = torch.ldexp(torch.ones(s.shape, dtype=torch.float64), s.to(torch.int32) - 133)
    unit[s == 255] = float("nan")
    return (q.double().unflatten(-1, (-1, 32)) * unit.unsqueeze(-1)).flatten(-2)


def bits(t):
    return t.contiguous().view(torch.int16).cpu()


def same_bits(a, b):
    """The same bf16 numbers (NaN of any kind)."""
    nan = a.isnan()
    return torch.equal(nan, b.isnan()) and torch.equal(bits(a)[~nan.cpu()], bits(b)[~nan.cpu()])


@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (37, 2080), (300, 512), (2, 5, 64), (11, 65536)])
def test_rows(shape):
    rng = np.random.default_rng(shape[-1])
    x = xh.bf16(rng, shape)
    spread = np.exp2(rng.integers(-30, 30, shape[:-1] + (shape[-1] // 32, 1))).astype(np.float32)
    x = (x.float().unflatten(-1, (-1, 32)) * torch.from_numpy(spread)).flatten(-2).to(torch.bfloat16)
    flat = x.view(-1)
    flat[:4] = torch.tensor([1.9921875, -1.9921875, 1.0, 2.0 ** -7])  # 127.5 steps: 127; half a step: 0
    flat[4:32] = 0.0078125 * torch.arange(28)
    if x.numel() > 32 * 8:
        flat[32:64] = 0
        flat[64:96] = 2.0 ** -133 * torch.arange(32)               # subnormals
        flat[96:128] = 2.0 ** -126
        flat[128:160] = torch.finfo(torch.bfloat16).max
        flat[161] = float("inf")
        flat[200] = float("nan")
        flat[224:256] = -0.0
    q, s = ep.quantize_mxint8(x.cuda())
    want, ws = kept_of(x)
    assert q.shape == x.shape and torch.equal(s.cpu(), ws) and torch.equal(q.cpu(), want)
    back = ep.dequantize_mxint8(q, s)
    v = values_of(want, ws)
    assert torch.equal(back.double().cpu().nan_to_num(nan=7.0), v.nan_to_num(nan=7.0))
    fine = torch.isfinite(v)
    half = torch.ldexp(torch.ones(ws.shape, dtype=torch.float64), ws.to(torch.int32) - 134).repeat_interleave(32, -1)
    assert bool(((back.double().cpu() - x.double()).abs() <= half)[fine].all())


def test_every_code_and_scale_back():
    """All 256 codes under all 256 scale bytes."""
    q = torch.arange(-128, 128, dtype=torch.int16).to(torch.int8).repeat(256, 1)
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    back = ep.dequantize_mxint8(q.cuda(), s.cuda()).double().cpu()
    v = values_of(q, s)
    v = torch.where(v.abs() == 2.0 ** 128, v.sign() * float("inf"), v)  # -128 under the largest scale is past bf16
    assert torch.equal(back.nan_to_num(nan=7.0), v.nan_to_num(nan=7.0))


@pytest.mark.parametrize("layout", ["packed", "low_latency"])
def test_rows_of_groups(layout):
    rng = np.random.default_rng(1)
    g, rows = groups_of(rng, 8, 2, COUNTS["some"], layout)
    x, used = poisoned(xh.bf16(rng, (g.num_rows, 96)), rows, float("nan"))
    q = torch.full((g.num_rows, 96), 99, dtype=torch.int8, device="cuda")
    s = torch.full((g.num_rows, 3), 9, dtype=torch.uint8, device="cuda")
    ep.quantize_mxint8(x.cuda(), g, out=(q, s))
    want, ws = kept_of(x)
    assert torch.equal(q.cpu()[used], want[used]) and torch.equal(s.cpu()[used], ws[used])
    assert bool((q.cpu()[~used] == 99).all()) and bool((s.cpu()[~used] == 9).all())
    back = torch.full((g.num_rows, 96), SENTINEL, dtype=torch.bfloat16, device="cuda")
    ep.dequantize_mxint8(q, s, g, out=back)
    assert torch.equal(back.double().cpu()[used], values_of(want, ws)[used]) and bool((back.cpu()[~used] == SENTINEL).all())


@pytest.mark.parametrize("layout", ["packed", "low_latency", None])
@pytest.mark.parametrize("I", [32, 96, 512, 672, 2048])
def test_swiglu(I, layout):
    """Bit for bit what swiglu, quantize_mxint8 and, of the kept values, swiglu_backward and swiglu give."""
    rng = np.random.default_rng([I, 2])
    g, rows = groups_of(rng, 8, 2, COUNTS["few"], layout) if layout else (None, [list(range(41))])
    n = g.num_rows if g else 41
    x, d = xh.bf16(rng, (n, 2 * I), 2.0), xh.bf16(rng, (n, I))
    r = [r for e in rows for r in e]
    x[r[0], 1], x[r[1], I + 3], x[r[2], 5], x[r[3]] = float("nan"), float("inf"), 3e38, 0.0
    x, d = x.cuda(), d.cuda()
    full = lambda cols, dtype=torch.bfloat16, v=SENTINEL: torch.full((n, cols), v, dtype=dtype, device="cuda")  # noqa: E731
    h, q, s = ep.swiglu_checkpoint(x, g, out=full(I), kept=(full(2 * I, torch.int8, 99), full(I // 16, torch.uint8, 9)))
    assert same_bits(h, ep.swiglu(x, g, out=full(I)))
    wq, ws = ep.quantize_mxint8(x, g, out=(full(2 * I, torch.int8, 99), full(I // 16, torch.uint8, 9)))
    assert torch.equal(q, wq) and torch.equal(s, ws)
    back = ep.dequantize_mxint8(q, s, g, out=full(2 * I))
    grad, again = ep.swiglu_checkpoint_backward(d, q, s, g, out=(full(2 * I), full(I)))
    assert same_bits(grad, ep.swiglu_backward(d, back, g, out=full(2 * I)))
    assert same_bits(again, ep.swiglu(back, g, out=full(I)))
    assert same_bits(ep.swiglu_checkpoint_backward(d, q, s, g, out=full(2 * I), again=False), grad)
    # and the gradient against its formula of the values that are kept
    used = torch.tensor(r)
    v = values_of(q.cpu()[used], s.cpu()[used])
    gate, up, dd = v[:, :I], v[:, I:], d.double().cpu()[used]
    sg = torch.sigmoid(gate)
    ref = torch.cat((dd * up * sg * (1 + gate * (1 - sg)), dd * gate * sg), 1)
    mag = torch.cat((dd * up * sg * (1 + gate.abs()), dd * gate * sg), 1).abs()
    fine = torch.isfinite(ref) & (ref.abs() < 1e38)
    off = (grad.double().cpu()[used] - ref).abs() - ref.abs() * 2.0 ** -8 - 32 * 2.0 ** -24 * mag - 2.0 ** -120
    assert bool((off[fine] <= 0).all())


def rows_kept(rng, n, K, rows):
    x = xh.bf16(rng, (n, K))
    x = (x.float().unflatten(-1, (-1, 32)) * torch.from_numpy(np.exp2(rng.integers(-3, 4, (n, K // 32, 1))).astype(np.float32)))
    q, s = kept_of(x.flatten(-2).to(torch.bfloat16))
    q, _ = poisoned(q, rows, 77)
    s, _ = poisoned(s, rows, 255)
    return q, s


@pytest.mark.parametrize("layout", ["packed", "low_latency"])
@pytest.mark.parametrize("K,N,E", [(32, 8, 8), (64, 64, 8), (160, 200, 8), (544, 328, 8), (288, 136, 256)])
@pytest.mark.parametrize("kind", list(COUNTS))
@pytest.mark.parametrize("mode", ["fp32", "bf16", "accumulate"])
def test_weight_gradient(K, N, E, kind, layout, mode):
    rng = np.random.default_rng([K, N, 3])
    R = 4
    counts = (COUNTS[kind] * (E // 8))[:E]
    if E > 8:
        counts = [c // 8 for c in counts]
    g, rows = groups_of(rng, E, R, counts, layout)
    d, _ = poisoned(xh.bf16(rng, (g.num_rows, N)), rows, float("nan"))
    q, s = rows_kept(rng, g.num_rows, K, rows)
    dtype = torch.bfloat16 if mode == "bf16" else torch.float32
    start = torch.from_numpy(rng.standard_normal((E, N, K), dtype=np.float32)).to(dtype).cuda()
    out = start.clone()
    ep.expert_gemm_wgrad(d.cuda(), q.cuda(), g, out=out, accumulate=mode == "accumulate", row_scales=s.cuda())
    # the same bits as of the bf16 rows that are kept
    same = start.clone()
    ep.expert_gemm_wgrad(d.cuda(), values_of(q, s).to(torch.bfloat16).cuda(), g, out=same, accumulate=mode == "accumulate")
    assert torch.equal(out, same)
    v = values_of(q, s)
    ref = start.double().cpu() if mode == "accumulate" else torch.zeros(E, N, K, dtype=torch.float64)
    tol = torch.zeros(E, N, K, dtype=torch.float64)
    for e in range(E):
        a, b = d[rows[e]].double().t(), v[rows[e]]
        t = (len(rows[e]) + 8) * 2.0 ** -23 * (a.abs() @ b.abs() + ref[e].abs())
        ref[e] += a @ b
        tol[e] = t + (2.0 ** -8 if mode == "bf16" else 2.0 ** -24) * (ref[e].abs() + t)
    check(out, ref, tol, f"{K}x{N} {kind} {layout} {mode}")


@pytest.mark.parametrize("counts", [[0, 1, 64, 63, 65, 127, 128, 300], [700, 129, 192, 0, 1, 512, 640, 66]])
def test_weight_gradient_in_wide_tiles(counts):
    """256 x 256 tiles, which rows and channels enough take: ragged channels on both sides; poisoned unused rows; NaN kept in
    one expert's rows stays there."""
    rng = np.random.default_rng(len(counts) + counts[0])
    E, R, K, N = 8, 2, 1312, 1608
    off, cap, rows = xh.packed_groups(counts, R, slack=3)
    g = ep.Groups(*(torch.from_numpy(np.asarray(v, np.int32)).cuda() for v in (counts, off)), num_experts=E, num_ranks=R,
                  cap_rows=cap, rows_hint=100000)
    d, _ = poisoned(xh.bf16(rng, (g.num_rows, N)), rows, float("nan"))
    q, s = rows_kept(rng, g.num_rows, K, rows)
    s[rows[5][0], 7] = 255
    out = ep.expert_gemm_wgrad(d.cuda(), q.cuda(), g, row_scales=s.cuda())
    v = values_of(q, s)
    same = ep.expert_gemm_wgrad(d.cuda(), v.to(torch.bfloat16).cuda(), g)
    assert torch.equal(out.isnan(), same.isnan()) and torch.equal(out.nan_to_num(), same.nan_to_num())
    assert bool(out[5, :, 7 * 32:8 * 32].isnan().all()) and int(out.isnan().sum()) == 32 * N
    for e in (1, 3, 7):
        a, b = d[rows[e]].double().t(), v[rows[e]]
        t = (len(rows[e]) + 8) * 2.0 ** -23 * (a.abs() @ b.abs())
        assert bool(((out[e].double().cpu() - a @ b).abs() <= t + 2.0 ** -24 * (a @ b).abs()).all())


def test_rows_past_32_bits():
    """Rows whose places in the codes, and in the scales' and gradients' arrays, pass 32 bits."""
    K, N, cap = 7168, 64, 700000
    counts, off = [40, 70], [cap - 200000, cap - 90]
    g = ep.Groups(*(torch.tensor(v, dtype=torch.int32).cuda() for v in (counts, off)), num_experts=2, num_ranks=1, cap_rows=cap)
    rng = np.random.default_rng(8)
    q = torch.empty((cap, K), dtype=torch.int8, device="cuda")
    s = torch.empty((cap, K // 32), dtype=torch.uint8, device="cuda")
    d = torch.empty((cap, N), dtype=torch.bfloat16, device="cuda")
    gu = torch.empty((cap, 2 * 2048), dtype=torch.bfloat16, device="cuda")
    h, kq, ks = (torch.empty((cap, c), dtype=t, device="cuda")
                 for c, t in ((2048, torch.bfloat16), (4096, torch.int8), (128, torch.uint8)))
    near = ep.Groups(g.counts, torch.tensor([0, 40], dtype=torch.int32).cuda(), num_experts=2, num_ranks=1, cap_rows=110)
    at = torch.cat([torch.arange(o, o + c) for o, c in zip(off, counts)]).cuda()
    x, dd, gg = (xh.bf16(rng, (110, c)).cuda() for c in (K, N, 4096))
    nq, ns = ep.quantize_mxint8(x)
    q[at], s[at], d[at], gu[at] = nq, ns, dd, gg
    assert torch.equal(ep.expert_gemm_wgrad(d, q, g, row_scales=s), ep.expert_gemm_wgrad(dd, nq, near, row_scales=ns))
    ep.swiglu_checkpoint(gu, g, out=h, kept=(kq, ks))
    for a, b in zip((h, kq, ks), ep.swiglu_checkpoint(gg)):
        assert torch.equal(a[at], b)


def test_training_step():
    """Forward keeping 8-bit checkpoints, backward from them alone, each result against its formula in 64 bits on what the
    step before left; in a graph as well, replayed with other inputs."""
    rng = np.random.default_rng(9)
    T, H, I, E, R, k = 80, 288, 160, 8, 2, 2
    idx = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)).cuda()
    idx[3] = -1
    wr = torch.from_numpy(rng.random((T, k), dtype=np.float32)).cuda()
    w1, w2 = xh.bf16(rng, (E, 2 * I, H), 0.1).cuda(), xh.bf16(rng, (E, H, I), 0.1).cuda()
    buf = ep.Buffer(T, H, k, E, R, T * k)

    def step(x, gy):
        lay, rx, _, rw, handle = buf.dispatch_with_layout(x, idx, wr, False)
        g = buf.groups(lay)
        gu = ep.expert_gemm(rx, w1, g)
        xq, xs = ep.quantize_mxint8(rx, g)
        h, q, s = ep.swiglu_checkpoint(gu, g)
        out = buf.combine(ep.expert_gemm(h, w2, g), handle, wr)
        # backward: rx, gu and h are no more
        d = buf.combine_backward(gy, handle) * rw.to(torch.bfloat16)[:, None]
        ga = ep.expert_gemm_dgrad(d, w2, g)
        ggu, again = ep.swiglu_checkpoint_backward(ga, q, s, g)
        gw2 = ep.expert_gemm_wgrad(d, again, g)
        gw1 = ep.expert_gemm_wgrad(ggu, xq, g, row_scales=xs)
        gx = buf.dispatch_backward(ep.expert_gemm_dgrad(ggu, w1, g), handle)
        return out, gw1, gw2, gx, ggu, xq, xs, d, again, handle.pos

    inputs = [(xh.bf16(rng, (T, H)).cuda(), xh.bf16(rng, (T, H)).cuda()) for _ in range(3)]
    eager = [[t.clone() for t in step(*i)] for i in inputs]
    assert buf.status() == 0
    for out, gw1, gw2, gx, ggu, xq, xs, d, again, pos in eager:
        ih, ph = idx.cpu(), pos.cpu()
        for e in range(E):
            r = ph[(ih == e) & (ph >= 0)].long()
            for got, a, b in ((gw1[e], ggu, values_of(xq.cpu(), xs.cpu())), (gw2[e], d, again.double().cpu())):
                a, b = a.double().cpu()[r].t(), b[r]
                t = (len(r) + 8) * 2.0 ** -23 * (a.abs() @ b.abs())
                assert bool(((got.double().cpu() - a @ b).abs() <= t + 2.0 ** -24 * (a @ b).abs()).all())
        assert torch.isfinite(gx).all() and torch.isfinite(out).all()
    x, gy = (t.clone() for t in inputs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, gy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(x, gy)
    for turn in range(2):
        for i, want in zip(inputs, eager):
            x.copy_(i[0]), gy.copy_(i[1])
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(captured[:4], want[:4]):
                assert torch.equal(a, b)
            step(*i)
    assert buf.status() == 0
