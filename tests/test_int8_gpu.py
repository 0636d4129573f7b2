"""8-bit integer rows and products on the GPU against plain forms."""
import numpy as np
import pytest
import torch

import experts_helpers as xh
from combine_get_dispatch_amd import ep
from test_experts_gpu import COUNTS, HALF, SENTINEL, check, groups_of, poisoned

pytestmark = pytest.mark.gpu


def codes_of(x):
    """(codes, scales) of fp32 rows by the rule, each step in 32 bits."""
    x = np.asarray(x, np.float32)
    bad = ~np.isfinite(x).all(-1)
    a = np.maximum(np.abs(np.where(bad[..., None], 0, x)).max(-1), np.float32(1e-30))
    inv = np.float32(127) / a
    q = np.rint(np.where(bad[..., None], 0, x) * inv[..., None]).astype(np.int8)
    return torch.from_numpy(q), torch.from_numpy(np.where(bad, np.float32("nan"), a / np.float32(127)))


def same(a, b):
    return torch.equal(a.cpu().nan_to_num(nan=-1.0), b.nan_to_num(nan=-1.0))


@pytest.mark.parametrize("cols", [16, 48, 512, 1008, 2048, 2064, 4096, 7168, 8192, 8208, 20000, 65536])
def test_quantize(cols):
    rng = np.random.default_rng(cols)
    n = 37
    x = xh.bf16(rng, (n, cols))
    x = (x.float() * torch.from_numpy(np.exp2(rng.integers(-20, 20, (n, 1))).astype(np.float32))).to(torch.bfloat16)
    x[0] = 0
    x[1], x[1, 3] = 0, -1e-38                     # below the smallest magnitude that a scale is made for
    x[2, 5] = float("inf")
    x[3, cols - 1] = float("nan")
    x[4] = torch.finfo(torch.bfloat16).max
    x[5, :8] = torch.tensor([127, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -127.0])  # halves, ties to even
    x[5, 8:] = 0
    q, s = ep.quantize_int8(x.cuda())
    want, ws = codes_of(x.float().numpy())
    assert q.dtype == torch.int8 and s.shape == (n,)
    assert torch.equal(q.cpu(), want) and same(s, ws)
    assert q[5, :8].tolist() == [127, 0, 2, 2, 0, -2, 126, -127]


@pytest.mark.parametrize("layout", ["packed", "low_latency"])
def test_quantize_groups(layout):
    rng = np.random.default_rng(1)
    g, rows = groups_of(rng, 8, 2, COUNTS["some"], layout)
    x = xh.bf16(rng, (g.num_rows, 176))
    q = torch.full((g.num_rows, 176), 99, dtype=torch.int8, device="cuda")
    s = torch.full((g.num_rows,), 99.0, device="cuda")
    ep.quantize_int8(x.cuda(), g, out=(q, s))
    used = torch.zeros(g.num_rows, dtype=torch.bool)
    used[[r for e in rows for r in e]] = True
    want, ws = codes_of(x.float().numpy())
    assert torch.equal(q.cpu()[used], want[used]) and same(s.cpu()[used], ws[used])
    assert bool((q.cpu()[~used] == 99).all()) and bool((s.cpu()[~used] == 99).all())


def test_quantize_weights():
    rng = np.random.default_rng(2)
    w = xh.bf16(rng, (5, 24, 80), 0.1)
    q, s = ep.quantize_int8(w.cuda())
    want, ws = codes_of(w.float().numpy())
    assert q.shape == w.shape and s.shape == (5, 24) and torch.equal(q.cpu(), want) and same(s, ws)


@pytest.mark.parametrize("layout", ["packed", "low_latency"])
@pytest.mark.parametrize("K,N", [(16, 8), (64, 64), (208, 136), (336, 520), (640, 264), (1040, 256)])
@pytest.mark.parametrize("kind", list(COUNTS))
@pytest.mark.parametrize("per", [1, 20, 10000])
def test_product(K, N, kind, layout, per):
    rng = np.random.default_rng([K, N, per, 3])
    E, R = 8, 2
    g, rows = groups_of(rng, E, R, COUNTS[kind], layout, slack=400 if per > 1000 else 5, hint=per * E)
    n = g.num_rows
    x = torch.from_numpy(rng.integers(-128, 128, (n, K), dtype=np.int8))
    w = torch.from_numpy(rng.integers(-128, 128, (E, N, K), dtype=np.int8))
    xs = torch.from_numpy(np.exp2(rng.uniform(-9, -5, n)).astype(np.float32))
    ws = torch.from_numpy(np.exp2(rng.uniform(-9, -5, (E, N))).astype(np.float32))
    xs, _ = poisoned(xs, rows, float("nan"))
    out = torch.full((n, N), SENTINEL, dtype=torch.bfloat16, device="cuda")
    got = ep.expert_gemm(x.cuda(), w.cuda(), g, row_scales=xs.cuda(), weight_scales=ws.cuda(), out=out)
    assert got is out
    ref = torch.full((n, N), SENTINEL, dtype=torch.float64)
    tol = torch.zeros((n, N), dtype=torch.float64)
    for e in range(E):
        if rows[e]:
            v = (x[rows[e]].double() @ w[e].double().t()) * xs[rows[e]].double()[:, None] * ws[e].double()
            ref[rows[e]] = v
            t = 3 * 2.0 ** -24 * v.abs()  # the sum's conversion and two products
            tol[rows[e]] = t + HALF[torch.bfloat16] * (v.abs() + t)
    check(out, ref, tol, f"int8 {K}x{N} {kind} {layout}")


def test_largest_sums():
    """Codes of -128 over the longest reduction: 2^30."""
    K = 65536
    g = ep.Groups(*(torch.tensor([v], dtype=torch.int32).cuda() for v in (3, 0)), num_experts=1, num_ranks=1, cap_rows=3)
    x, w = torch.full((3, K), -128, dtype=torch.int8).cuda(), torch.full((1, 8, K), -128, dtype=torch.int8).cuda()
    one = torch.ones(3, device="cuda")
    out = ep.expert_gemm(x, w, g, row_scales=one, weight_scales=torch.ones(1, 8, device="cuda"))
    assert bool((out.float() == 2.0 ** 30).all())


def test_ends_of_scales():
    """Rows of NaN scales are NaN, infinite scales infinite, zero scales zero; other rows are not touched by them."""
    rng = np.random.default_rng(4)
    g = ep.Groups(*(torch.tensor([v], dtype=torch.int32).cuda() for v in (20, 0)), num_experts=1, num_ranks=1, cap_rows=20)
    x, w = (torch.from_numpy(rng.integers(1, 128, s, dtype=np.int8)).cuda() for s in ((20, 64), (1, 40, 64)))
    xs, ws = torch.ones(20, device="cuda"), torch.ones(1, 40, device="cuda")
    plain = ep.expert_gemm(x, w, g, row_scales=xs, weight_scales=ws)
    xs[3], xs[5], xs[7] = float("nan"), float("inf"), 0.0
    out = ep.expert_gemm(x, w, g, row_scales=xs, weight_scales=ws)
    assert bool(out[3].isnan().all()) and bool(out[5].isposinf().all()) and bool((out[7] == 0).all())
    rest = [i for i in range(20) if i not in (3, 5, 7)]
    assert torch.equal(out[rest], plain[rest])


@pytest.mark.parametrize("layout", ["packed", "low_latency", None])
@pytest.mark.parametrize("I", [16, 272, 512, 1024, 2048, 4096, 4112, 9000 // 8 * 8])
def test_swiglu(I, layout):
    rng = np.random.default_rng([I, 5])
    g, rows = groups_of(rng, 8, 2, COUNTS["few"], layout) if layout else (None, [list(range(41))])
    n = g.num_rows if g else 41
    if I % 16:
        with pytest.raises(ep.EpError):
            ep.swiglu(torch.zeros(n, 2 * I, dtype=torch.bfloat16, device="cuda"), g, kind="int8")
        return
    x = xh.bf16(rng, (n, 2 * I), 2.0)
    first = rows[0] or rows[1]
    x[first[0], 0] = 40.0 if len(first) == 1 else float("nan")
    q = torch.full((n, I), 99, dtype=torch.int8, device="cuda")
    s = torch.full((n,), 99.0, device="cuda")
    ep.swiglu(x.cuda(), g, kind="int8", out=(q, s))
    used = torch.zeros(n, dtype=torch.bool)
    used[[r for e in rows for r in e]] = True
    assert bool((q.cpu()[~used] == 99).all()) and bool((s.cpu()[~used] == 99).all())
    xv = x[used].double()
    h = xv[:, :I] * torch.sigmoid(xv[:, :I]) * xv[:, I:]
    q, s = q.cpu()[used].double(), s.cpu()[used].double()
    bad = h.isnan().any(1)
    assert torch.equal(s.isnan(), bad) and not q[bad].any()
    h, q, s = h[~bad], q[~bad], s[~bad]
    # h in fp32 is off by 16 of its roundings (as in its other forms); the scale by that and one of its own; a code is a
    # nearest whole number of a value that is off by that, of at most 127 steps
    off = 16 * 2.0 ** -24
    scale = h.abs().amax(1).clamp_min(1e-30) / 127
    assert bool(((s - scale).abs() <= scale * (off + 2.0 ** -23)).all())
    assert bool(((q - h / scale[:, None]).abs() <= 0.5 + 127 * (2 * off + 3 * 2.0 ** -24)).all())


def test_layer():
    """Rows to int8, gate and up product, SwiGLU to int8, down product, between dispatch and combine; twice, on two streams."""
    rng = np.random.default_rng(7)
    T, H, I, E, R, k = 96, 512, 272, 8, 4, 3
    idx = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)).cuda()
    idx[1] = -1
    w = torch.from_numpy(rng.random((T, k), dtype=np.float32)).cuda()
    x = xh.bf16(rng, (T, H)).cuda()
    w1, s1 = ep.quantize_int8(xh.bf16(rng, (E, 2 * I, H), 0.05).cuda())
    w2, s2 = ep.quantize_int8(xh.bf16(rng, (E, H, I), 0.05).cuda())
    outs = []
    for ll in (False, True):
        buf = ep.Buffer(T, H, k, E, R, ep.ll_cap_rows(T, E, R) if ll else T * k)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            if ll:
                rx, _, _, count, h = buf.dispatch_low_latency(x, idx, w, False)
                g = buf.groups_low_latency(count)
            else:
                lay, rx, _, _, h = buf.dispatch_with_layout(x, idx, w, False)
                g = buf.groups(lay)
            q, qs = ep.quantize_int8(rx, g)
            gu = ep.expert_gemm(q, w1, g, row_scales=qs, weight_scales=s1)
            a, sa = ep.swiglu(gu, g, kind="int8")
            y = ep.expert_gemm(a, w2, g, row_scales=sa, weight_scales=s2)
            outs.append(buf.combine(y, h, w))
        side.synchronize()
        assert buf.status() == 0
    assert torch.equal(*outs) and bool((outs[0][1] == 0).all())
    # the layer against 64 bits without any quantization: a code is half a step of the row's largest off, some 0.3% of the
    # rows' size for normal rows of these lengths, in each of four operands; the whole below 3%
    v1, v2 = w1.double() * s1.double()[..., None], w2.double() * s2.double()[..., None]
    ref = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            if e >= 0:
                gu = v1[e] @ x[t].double()
                ref[t] += float(w[t, j]) * (v2[e] @ (gu[:I] * torch.sigmoid(gu[:I]) * gu[I:]))
    assert float((outs[0].double() - ref).norm() / ref.norm()) < 0.03


def test_rows_past_32_bits():
    """Rows whose places in the arrays pass 32 bits: as the same rows near the start."""
    K, N, cap = 7168, 4096, 700000
    counts, off = [40, 70], [cap - 200000, cap - 90]
    g = ep.Groups(*(torch.tensor(v, dtype=torch.int32).cuda() for v in (counts, off)), num_experts=2, num_ranks=1, cap_rows=cap)
    near = ep.Groups(g.counts, torch.tensor([0, 40], dtype=torch.int32).cuda(), num_experts=2, num_ranks=1, cap_rows=110)
    rng = np.random.default_rng(10)
    at = torch.cat([torch.arange(o, o + c) for o, c in zip(off, counts)]).cuda()
    few = xh.bf16(rng, (110, K)).cuda()
    x, out, a = (torch.empty((cap, c), dtype=torch.bfloat16, device="cuda") for c in (K, N, N // 2))
    q, aq = (torch.empty((cap, c), dtype=torch.int8, device="cuda") for c in (K, N // 2))
    s, s2 = (torch.empty(cap, device="cuda") for _ in range(2))
    w, ws = ep.quantize_int8(xh.bf16(rng, (2, N, K), 0.05).cuda())
    x[at] = few
    ep.quantize_int8(x, g, out=(q, s))
    ep.expert_gemm(q, w, g, row_scales=s, weight_scales=ws, out=out)
    ep.swiglu(out, g, kind="int8", out=(aq, s2))
    nq, ns = ep.quantize_int8(few)
    h = ep.expert_gemm(nq, w, near, row_scales=ns, weight_scales=ws)
    for far, want in zip((q, s, out, aq, s2), (nq, ns, h) + ep.swiglu(h, kind="int8")):
        assert torch.equal(far[at], want)


def test_calls_at_once():
    """The layer and the router on four streams at once: each the result it has alone."""
    rng = np.random.default_rng(11)
    E, K, I = 8, 1024, 512
    w1, w2 = (ep.quantize_int8(xh.bf16(rng, s, 0.05).cuda()) for s in ((E, 2 * I, K), (E, K, I)))
    r = ep.Router(64, 6, score="sigmoid", num_groups=8, topk_groups=4)

    def work(x, g, logits):
        idx, wt = ep.route(logits, r)
        q, s = ep.quantize_int8(x, g)
        a, t = ep.swiglu(ep.expert_gemm(q, w1[0], g, row_scales=s, weight_scales=w1[1]), g, kind="int8")
        y = ep.expert_gemm(a, w2[0], g, row_scales=t, weight_scales=w2[1])
        k, ks = ep.quantize_mxint8(x, g)
        return idx, wt, ep.route_backward(wt, logits, idx, r), y, ep.expert_gemm_wgrad(y, k, g, row_scales=ks)

    cases = []
    for i in range(4):
        counts = [int(n) for n in rng.integers(0, 200, E)]
        off = [sum(counts[:e]) for e in range(E)]
        g = ep.Groups(*(torch.tensor(v, dtype=torch.int32).cuda() for v in (counts, off)), num_experts=E, num_ranks=1,
                      cap_rows=sum(counts))
        cases.append((xh.bf16(rng, (sum(counts), K)).cuda(), g,
                      torch.from_numpy(rng.standard_normal((300 + 3000 * i, 64), dtype=np.float32)).cuda()))
    alone = [work(*c) for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], []
    for s, c in zip(streams, cases):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(work(*c))
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        for u, v in zip(a, b):
            assert torch.equal(u, v)
