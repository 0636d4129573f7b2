"""The experts' side of the exchange, as measurable cases: what a rank computes
between the dispatch that fills its receive rows and the combine that takes the
experts' outputs back.

  product      out[p] = W[e(p)] . row[p] for every received row p of expert e:
               bf16 rows and weights; the dispatch's FP8 rows (one fp32 scale
               per 128 channels) with e4m3 weights (one fp32 scale per 128 x 128
               block); MXFP4 rows and weights (one power of two per 32 values)
  gradient     of the bf16 product: grad_row[p] = W[e(p)]^T . grad_out[p] and
               grad_W[e] = sum over e's rows of grad_out[p] (x) row[p]
  swiglu       h = silu(gate) * up on the received rows, to bf16 or to FP8 with
               scales, and its gradient
  mxfp4        quantization to 4-bit values with a power of two per 32 of them,
               and back

Receive rows come in the dispatch's two layouts: packed (expert e's rows start
at offsets[e] of its rank's cap_rows rows) and low-latency (expert e owns one
region of T/R rows for each of the R sources). Rows that no expert has are
left as they were: the outputs' buffers start as zeros here.
"""
import math

import torch

own = False

FP8_MAX = 448.0
MOST_EXACT_FLOPS = 3e14  # 64-bit products beyond this take too long


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # 64 tokens of hidden 256 on 16 small experts: a call as short as calls get, its latency is all that counts
        dict(name="bf16_tiny", op="product", form="bf16", layout="packed", T=64, k=2, E=16, R=4, K=256, N=512, skew=0.0),
        # one rank's decode share of 128 tokens x 8 ranks, top-8 of 256 experts: 32 local experts, about 32 rows each, down product
        dict(name="bf16_decode_down", op="product", form="bf16", layout="packed", T=1024, k=1, E=32, R=1, K=2048, N=7168,
             skew=0.0),
        # a decode batch of 128 tokens over all 256 experts in the low-latency layout: the weights' bytes are the time
        dict(name="fp8_decode_up", op="product", form="fp8", layout="low_latency", T=128, k=8, E=256, R=8, K=7168, N=4096,
             skew=0.3),
        # 4096 tokens, top-8 of 64 experts of uneven popularity: 32768 ragged rows, gate and up products in one
        dict(name="fp8_prefill_up", op="product", form="fp8", layout="packed", T=4096, k=8, E=64, R=8, K=7168, N=4096,
             skew=0.5),
        # decode on 4-bit weights: one rank's 32 experts, some 8 rows each
        dict(name="mxfp4_decode_up", op="product", form="mxfp4", layout="packed", T=256, k=1, E=32, R=1, K=7168, N=4096,
             skew=0.5),
        # a prefill rank share on 4-bit rows and weights: 8 local experts, 2048 rows each
        dict(name="mxfp4_prefill_up", op="product", form="mxfp4", layout="packed", T=16384, k=1, E=8, R=1, K=7168, N=4096,
             skew=0.1),
        # small training step with odd sizes: empty and one-row experts among 48, fp32 weight gradient
        dict(name="grad_odd", op="gradient", layout="packed", T=173, k=2, E=48, R=1, K=1016, N=648, skew=2.0, acc="fp32"),
        # a training rank share: 8 local experts, 4096 rows each, both gradients of the gate and up product
        dict(name="grad_rank", op="gradient", layout="packed", T=32768, k=1, E=8, R=1, K=7168, N=4096, skew=0.1, acc="bf16"),
        # between the two products of an FP8 prefill: 32768 rows to e4m3 with scales
        dict(name="swiglu_fp8_prefill", op="swiglu", out="fp8", layout="packed", T=4096, k=8, E=64, R=8, I=2048, skew=0.5),
        # its gradient in training on 16384 tokens
        dict(name="swiglu_gradient", op="swiglu_gradient", layout="packed", T=16384, k=4, E=64, R=8, I=2048, skew=0.2),
        # a prefill batch's rows to 4 bits and back
        dict(name="mxfp4_rows", op="mxfp4", rows=16384, cols=7168),
        # one rank's decode rows, an odd count of narrow ones
        dict(name="mxfp4_rows_odd", op="mxfp4", rows=1021, cols=2080),
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, even over the logarithm, a multiple of step."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["product"] * 5 + ["gradient"] * 2 + ["swiglu", "swiglu_gradient", "mxfp4"])
    if op == "mxfp4":
        cols = _log(rng, 32, 8192, 32)
        return dict(op=op, rows=_log(rng, 1, max(1, 16384 * 7168 // cols)), cols=cols)
    E, skew = rng.choice([4, 8, 16, 24, 32, 48, 64]), rng.choice([0.0, 0.2, 0.5, 1.0])
    R = rng.choice([r for r in (1, 2, 4, 8) if E % r == 0])
    k = rng.choice([1, 2, 4])
    case = dict(op=op, layout="packed", k=k, E=E, R=R, skew=skew)
    if op in ("swiglu", "swiglu_gradient"):
        out = rng.choice(["bf16", "fp8"])
        I = _log(rng, 128, 4096, 128 if out == "fp8" else 8)
        T = R * _log(rng, 1, max(1, min(16384, 65536 * 2048 // (k * I)) // R))
        return dict(case, T=T, I=I, out=out) if op == "swiglu" else dict(case, T=T, I=I)
    form = rng.choice(["bf16", "fp8", "mxfp4"]) if op == "product" else "bf16"
    K, N = _log(rng, 128, 7168, 8 if form == "bf16" else 128), _log(rng, 64, 7168, 8)
    if op == "gradient":  # the weight gradient is as large as the weights
        K, N = (K, N) if E * K * N <= 5e8 else (_log(rng, 128, 2048, 8), _log(rng, 64, 2048, 8))
    most = max(1, int(min(16384, 1.5e12 / (2.0 * K * N * k))) // R)
    if op == "product" and rng.random() < 0.3:
        case["layout"], most = "low_latency", min(most, 256)
    case.update(T=R * _log(rng, 1, most), K=K, N=N)
    return dict(case, form=form) if op == "product" else dict(case, acc=rng.choice(["fp32", "bf16"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g, scale=1.0, dtype=torch.bfloat16):
    """N(0, scale) values, drawn in pieces so that no fp32 copy of a large tensor is held."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for part in flat.split(1 << 28):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * scale)
    return out


def _routing(case, g):
    """Row groups of a routed batch: T tokens choose k of E experts, the experts' popularity a softmax of skew * N(0, 1)."""
    T, k, E, R = (case[n] for n in ("T", "k", "E", "R"))
    pop = torch.log_softmax(case["skew"] * torch.randn(E, generator=g, device="cuda"), 0)
    u = torch.rand((T, E), generator=g, device="cuda").clamp_min(1e-30)
    idx = (pop - torch.log(-torch.log(u).clamp_min(1e-30))).topk(k, dim=1).indices  # k distinct experts, by popularity
    if case["layout"] == "low_latency":
        src = torch.arange(T, device="cuda")[:, None] // (T // R)
        cnt = torch.bincount((idx * R + src).view(-1), minlength=E * R).view(E, R).to(torch.int32)
        return dict(offsets=None, counts=cnt, cap=E * T // R, region=T // R, widest=int(cnt.max()))
    cnt = torch.bincount(idx.view(-1), minlength=E)
    per_rank = cnt.view(R, E // R)
    off = (per_rank.cumsum(1) - per_rank).view(E)
    return dict(offsets=off.to(torch.int32), counts=cnt.to(torch.int32), cap=int(per_rank.sum(1).max()) + 3, region=0,
                widest=int(cnt.max()))


def _fp8_rows(rows, cols, g):
    """Rows as the dispatch leaves them: e4m3 values and one scale per 128 channels, 1% of the rows 100 times as large."""
    q = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, cols // 128), dtype=torch.float32, device="cuda")
    for at in range(0, rows, 65536):
        n = min(65536, rows - at)
        x = torch.randn((n, cols // 128, 128), generator=g, device="cuda")
        x *= torch.where(torch.rand((n, 1, 1), generator=g, device="cuda") < 0.01, 100.0, 1.0)
        a = x.abs().amax(2, keepdim=True).clamp_min(1e-4)
        q[at:at + n] = (x * (FP8_MAX / a)).to(torch.float8_e4m3fn).view(n, cols).view(torch.uint8)
        scales[at:at + n] = (a / FP8_MAX).view(n, -1)
    return q, scales


def _fp8_weights(E, N, K, g):
    q = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
    for part in q.view(-1).split(1 << 28):
        x = torch.randn(part.shape, generator=g, device="cuda").mul_(100.0).clamp_(-FP8_MAX, FP8_MAX)
        part.copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
    scales = (0.5 + torch.rand((E, (N + 127) // 128, K // 128), generator=g, device="cuda")) / (100.0 * math.sqrt(K))
    return q, scales


def _mx_rows(shape, g, scale=1.0):
    x = _normal(shape, g, scale)
    q = torch.empty(tuple(shape[:-1]) + (shape[-1] // 2,), dtype=torch.uint8, device="cuda")
    s = torch.empty(tuple(shape[:-1]) + (shape[-1] // 32,), dtype=torch.uint8, device="cuda")
    for a, b, c in zip(x.view(-1, shape[-1]).split(8192), q.view(-1, shape[-1] // 2).split(8192),
                       s.view(-1, shape[-1] // 32).split(8192)):
        code, e = _mx_codes(a.float())
        b.copy_(code[:, 0::2] | (code[:, 1::2] << 4))
        c.copy_(e)
    return q, s


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    if case["op"] == "mxfp4":
        x = _normal((case["rows"], case["cols"]), g)
        spread = torch.exp2(torch.randint(-6, 7, (case["rows"], 1), generator=g, device="cuda").float())
        s["x"] = (x.float() * spread).to(torch.bfloat16)
        return s
    s.update(_routing(case, g))
    rows = case["R"] * s["cap"]
    E = case["E"]
    if case["op"] in ("swiglu", "swiglu_gradient"):
        I = case["I"]
        s["gate_up"] = _normal((rows, 2 * I), g, 1.5)
        if case["op"] == "swiglu_gradient":
            s["grad"] = _normal((rows, I), g)
            s["out"] = torch.zeros((rows, 2 * I), dtype=torch.bfloat16, device="cuda")
        elif case["out"] == "fp8":
            s["out"] = torch.zeros((rows, I), dtype=torch.uint8, device="cuda")
            s["out_scales"] = torch.zeros((rows, I // 128), dtype=torch.float32, device="cuda")
        else:
            s["out"] = torch.zeros((rows, I), dtype=torch.bfloat16, device="cuda")
        return s
    K, N = case["K"], case["N"]
    if case["op"] == "gradient":
        s["w"] = _normal((E, N, K), g, 1.0 / math.sqrt(K))
        s["x"] = _normal((rows, K), g)
        s["grad"] = _normal((rows, N), g)
        s["out"] = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
        s["out_w"] = torch.zeros((E, N, K), dtype=torch.float32 if case["acc"] == "fp32" else torch.bfloat16, device="cuda")
        return s
    s["x_scales"] = s["w_scales"] = None
    if case["form"] == "bf16":
        s["w"], s["x"] = _normal((E, N, K), g, 1.0 / math.sqrt(K)), _normal((rows, K), g)
    elif case["form"] == "fp8":
        s["w"], s["w_scales"] = _fp8_weights(E, N, K, g)
        s["x"], s["x_scales"] = _fp8_rows(rows, K, g)
    else:
        s["w"], s["w_scales"] = _mx_rows((E, N, K), g, 1.0 / math.sqrt(K))
        s["x"], s["x_scales"] = _mx_rows((rows, K), g)
    s["out"] = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _pow2(n):
    """2^n as fp32 by its bits, for integers -126 <= n <= 127."""
    return ((n.to(torch.int32) + 127) << 23).view(torch.float32)


def _mx_codes(x):
    """E2M1 codes [rows, cols] and E8M0 scale bytes [rows, cols/32] of fp32 rows: per 32 values the scale is
    2^(floor(log2(largest magnitude)) - 2), each value is divided by it and rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6
    (ties to the even code), at most 6."""
    b = x.view(x.shape[0], -1, 32)
    amax = b.abs().amax(2)
    e = torch.frexp(amax).exponent - 1 - 2                       # amax = m 2^exponent with m in [1/2, 1)
    e = torch.where(amax > 0, e, -127).clamp(-127, 125)
    v = (b * _pow2(-e[:, :, None])).abs()
    # codes 0..7 by the borders between neighbours; a border belongs to the even code
    code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0))
    code = code | (torch.signbit(b).to(torch.uint8) << 3)
    return code.view(x.shape).to(torch.uint8), (e + 127).to(torch.uint8)


def _mx_values(code, e):
    """The values that codes [.., cols] and scale bytes [.., cols/32] stand for: the power of two in two factors, as 2^-127 has
    no normal fp32 number."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=code.device)
    half = (e >> 1).to(torch.int32)
    v = table[code.to(torch.int32)].view(*e.shape, 32) * _pow2(half - 63)[..., None]
    return (v * _pow2(e.to(torch.int32) - half - 64)[..., None]).view(code.shape)


def _mx_unpacked(q, e):
    return _mx_values(torch.stack((q & 15, q >> 4), -1).view(*q.shape[:-1], 2 * q.shape[-1]), e)


def _rows_of(s):
    """Every expert's rows as an index [E, most rows] into the receive rows, and which entries are rows."""
    case, cnt = s["case"], s["counts"].long()
    E, R = case["E"], case["R"]
    r = torch.arange(s["widest"], device="cuda")
    if s["region"]:
        start = torch.arange(E * R, device="cuda").view(E, R) * s["region"]
        idx, valid = start[:, :, None] + r, r < cnt[:, :, None]
        idx, valid = idx.view(E, -1), valid.view(E, -1)
    else:
        start = torch.arange(E, device="cuda") // (E // R) * s["cap"] + s["offsets"].long()
        idx, valid = start[:, None] + r, r < cnt[:, None]
    return torch.where(valid, idx, 0), valid


def _written(out, idx, valid, values):
    """`out` with values[e, i] in row idx[e, i] of the valid entries: one more row takes the others."""
    rows = out.shape[0]
    more = torch.zeros((rows + 1,) + tuple(out.shape[1:]), dtype=out.dtype, device="cuda")
    more[torch.where(valid, idx, rows)] = values.to(out.dtype)
    return more[:rows]


def _taken(t, idx):
    return t[idx.view(-1)].view(tuple(idx.shape) + tuple(t.shape[1:]))


def _fp8_w(q, scales, N, dtype):
    v = q.view(torch.float8_e4m3fn).to(dtype)
    return v * scales.to(dtype).repeat_interleave(128, -1).repeat_interleave(128, -2)[..., :N, :]


def _fp8_x(q, scales, dtype):
    v = q.view(torch.float8_e4m3fn).to(dtype)
    return (v.view(*scales.shape, 128) * scales.to(dtype)[..., None]).view(q.shape)


def _plain(s):
    case = s["case"]
    if case["op"] == "mxfp4":
        code, e = _mx_codes(s["x"].float())
        return _mx_values(code, e).to(torch.bfloat16), e.view(torch.float8_e8m0fnu)
    idx, valid = _rows_of(s)
    if case["op"] in ("swiglu", "swiglu_gradient"):
        I, rows = case["I"], s["gate_up"].shape[0]
        used = torch.zeros(rows + 1, dtype=torch.bool, device="cuda")
        used[torch.where(valid, idx, rows)] = True
        used = used[:rows, None]
        gate, up = s["gate_up"][:, :I].float(), s["gate_up"][:, I:].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        if case["op"] == "swiglu_gradient":
            d = s["grad"].float()
            slope = sig * (1.0 + gate * (1.0 - sig))
            return torch.where(used, torch.cat((d * up * slope, d * (gate * sig)), 1), 0.0).to(torch.bfloat16)
        h = gate * sig * up
        if case["out"] == "bf16":
            return torch.where(used, h, 0.0).to(torch.bfloat16)
        h = h.view(rows, I // 128, 128)
        a = h.abs().amax(-1).clamp_min(1e-4)
        q = torch.where(used, (h * (FP8_MAX / a)[..., None]).clamp(-FP8_MAX, FP8_MAX).view(rows, I), 0.0)
        return q.to(torch.float8_e4m3fn), torch.where(used, a / FP8_MAX, 0.0)
    if case["op"] == "gradient":
        live = valid[..., None].float()
        d = _taken(s["grad"], idx).float() * live
        x = _taken(s["x"], idx).float() * live
        grad_rows = _written(s["out"], idx, valid, torch.bmm(d, s["w"].float()))
        return grad_rows, torch.bmm(d.transpose(1, 2), x).to(s["out_w"].dtype)
    if case["form"] == "bf16":
        x, w = _taken(s["x"], idx).float(), s["w"].float()
    elif case["form"] == "fp8":
        x = _fp8_x(_taken(s["x"], idx), _taken(s["x_scales"], idx), torch.float32)
        w = _fp8_w(s["w"], s["w_scales"], case["N"], torch.float32)
    else:
        x = _mx_unpacked(_taken(s["x"], idx), _taken(s["x_scales"], idx))
        w = _mx_unpacked(s["w"], s["w_scales"])
    return _written(s["out"], idx, valid, torch.bmm(x, w.transpose(1, 2)))


def run(state):
    if not own:
        return _plain(state)
    from combine_get_dispatch_amd import ep
    s, case = state, state["case"]
    if case["op"] == "mxfp4":
        q, scales = ep.quantize_mxfp4(s["x"])
        return ep.dequantize_mxfp4(q, scales), scales.view(torch.float8_e8m0fnu)
    groups = ep.Groups(s["counts"], s["offsets"], num_experts=case["E"], num_ranks=case["R"], cap_rows=s["cap"],
                       region_rows=s["region"], rows_hint=case["T"] * case["k"])
    if case["op"] == "swiglu":
        if case["out"] == "bf16":
            return ep.swiglu(s["gate_up"], groups, out=s["out"])
        q, scales = ep.swiglu(s["gate_up"], groups, kind="fp8", out=(s["out"], s["out_scales"]))
        return q.view(torch.float8_e4m3fn), scales
    if case["op"] == "swiglu_gradient":
        return ep.swiglu_backward(s["grad"], s["gate_up"], groups, out=s["out"])
    if case["op"] == "gradient":
        return (ep.expert_gemm_dgrad(s["grad"], s["w"], groups, out=s["out"]),
                ep.expert_gemm_wgrad(s["grad"], s["x"], groups, out=s["out_w"]))
    return ep.expert_gemm(s["x"], s["w"], groups, row_scales=s["x_scales"], weight_scales=s["w_scales"], out=s["out"])


# ---------------------------------------------------------------------------
# the work of one pass, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "mxfp4":
        n = case["rows"] * case["cols"]  # read bf16; written: 4-bit values, scales, bf16 values
        return {"bytes": n * (2 + 0.5 + 1 / 32 + 2), "flops": 4.0 * n}
    slots, E = case["T"] * case["k"], case["E"]
    if case["op"] == "swiglu":
        n = slots * case["I"]
        return {"bytes": n * (4 + (2 if case["out"] == "bf16" else 1 + 4 / 128)), "flops": 8.0 * n}
    if case["op"] == "swiglu_gradient":
        return {"bytes": slots * case["I"] * 10, "flops": 16.0 * slots * case["I"]}
    K, N = case["K"], case["N"]
    hit = E * (1.0 - (1.0 - 1.0 / E) ** slots)  # experts with a row, were all as popular
    if case["op"] == "gradient":
        return {"bytes": slots * (K + N + K) * 2 + hit * N * K * 2 + E * N * K * (4 if case["acc"] == "fp32" else 2),
                "flops": 4.0 * slots * N * K}
    each = {"bf16": 2.0, "fp8": 1.0, "mxfp4": 0.5 + 1 / 32}[case["form"]]
    return {"bytes": slots * (K * each + N * 2) + hit * N * K * each, "flops": 2.0 * slots * N * K}


def _exact_groups(s):
    """[(expert, its rows)] of the experts that have some, from the layout's definition."""
    case, cnt = s["case"], s["counts"].cpu()
    E, R, found = case["E"], case["R"], []
    for e in range(E):
        if s["region"]:
            rows = [(e * R + r) * s["region"] + i for r in range(R) for i in range(int(cnt[e, r]))]
        else:
            at = (e // (E // R)) * s["cap"] + int(s["offsets"][e])
            rows = list(range(at, at + int(cnt[e])))
        if rows:
            found.append((e, torch.tensor(rows, device="cuda")))
    return found


def _e2m1(q):
    """Values of packed 4-bit codes, low half first: sign, two exponent bits of bias 1, one bit of mantissa."""
    code = torch.empty(tuple(q.shape[:-1]) + (q.shape[-1], 2), dtype=torch.int64, device="cuda")
    code[..., 0], code[..., 1] = q & 15, q >> 4
    code = code.flatten(-2)
    exponent, mantissa = (code >> 1) & 3, (code & 1).double()
    size = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * torch.pow(2.0, exponent.double() - 1))
    return torch.where(code >= 8, -size, size)


def _exact_operand(q, scales, form, weights):
    if form == "bf16":
        return q.double()
    if form == "mxfp4":
        v = _e2m1(q)
        return (v.unflatten(-1, (-1, 32)) * torch.pow(2.0, scales.double() - 127).unsqueeze(-1)).flatten(-2)
    v = q.view(torch.float8_e4m3fn).double()
    if weights:
        n, c = torch.arange(v.shape[-2], device="cuda") // 128, torch.arange(v.shape[-1], device="cuda") // 128
        return v * scales.double()[n][:, c]
    return (v.unflatten(-1, (-1, 128)) * scales.double().unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    if case["op"] in ("product", "gradient") and work(case)["flops"] > MOST_EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    if case["op"] == "mxfp4":
        b = s["x"].double().unflatten(-1, (-1, 32))
        # floor(log2) of the largest magnitude is its exponent field, and 2^e a number with that field alone
        e = (b.abs().amax(-1, keepdim=True).view(torch.int64) >> 52) - 1023 - 2
        scale = ((e + 1023) << 52).view(torch.float64)
        v = b / scale
        # spacing of the 4-bit values: 1/2 below 2, 1 below 4, 2 above; torch.round takes ties to even
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
        v = (torch.round(v / step) * step).clamp(-6, 6) * scale
        return v.flatten(-2), scale.squeeze(-1)
    rows = case["R"] * s["cap"]
    groups = _exact_groups(s)
    if case["op"] in ("swiglu", "swiglu_gradient"):
        I = case["I"]
        used = torch.cat([r for _, r in groups])
        fp8 = case["op"] == "swiglu" and case["out"] == "fp8"
        out = torch.zeros((rows, 2 * I if case["op"] == "swiglu_gradient" else I), dtype=torch.float64, device="cuda")
        scales = torch.zeros((rows, I // 128), dtype=torch.float64, device="cuda") if fp8 else None
        for at in used.split(4096):
            gate, up = s["gate_up"][at].double().split(I, 1)
            silu = gate * torch.sigmoid(gate)
            if case["op"] == "swiglu_gradient":
                d = s["grad"][at].double()
                slope = torch.sigmoid(gate) + silu * (1 - torch.sigmoid(gate))
                out[at] = torch.cat((d * up * slope, d * silu), 1)
            elif fp8:
                h = (silu * up).unflatten(1, (-1, 128))
                scale = h.abs().amax(2).clamp_min(1e-4) / FP8_MAX
                out[at], scales[at] = (h / scale.unsqueeze(2)).flatten(1), scale
            else:
                out[at] = silu * up
        return (out, scales) if fp8 else out
    K, N = case["K"], case["N"]
    if case["op"] == "gradient":
        grad_rows = torch.zeros((rows, K), dtype=torch.float64, device="cuda")
        grad_w = torch.zeros((case["E"], N, K), dtype=torch.float64, device="cuda")
        for e, at in groups:
            d = s["grad"][at].double()
            grad_rows[at] = d @ s["w"][e].double()
            grad_w[e] = d.t().contiguous() @ s["x"][at].double()
        return grad_rows, grad_w
    out = torch.zeros((rows, N), dtype=torch.float64, device="cuda")
    for e, at in groups:
        x = _exact_operand(s["x"][at], None if s["x_scales"] is None else s["x_scales"][at], case["form"], False)
        w = _exact_operand(s["w"][e], None if s["w_scales"] is None else s["w_scales"][e], case["form"], True)
        out[at] = x @ w.t().contiguous()
    return out
