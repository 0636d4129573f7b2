"""The router before the exchange, the experts' 8-bit integer layer and 8-bit
activation checkpoints, as measurable cases.

  route        logits [T, E] -> the k experts of each token and their weights:
               softmax or sigmoid scores, a bias that takes part in the choice
               alone, groups of experts of which the best are kept, weights
               renormalised over the chosen ones or not
  route_gradient  of the weights in the logits
  int8_layer   an expert layer in 8-bit integers: rows to int8 with one scale
               each, product with int8 weights of one scale per channel, SwiGLU
               to int8 rows, second product
  rows         rows to MXINT8 (a power of two per 32 values, 8-bit integers) and
               back: what a checkpoint of activations keeps
  swiglu       SwiGLU that keeps its input in MXINT8, and its gradient from what
               was kept, with the forward result computed again
  weights      rows kept in MXINT8, and the weight gradient of a product from them

Receive rows come in the dispatch's two layouts, as in operators.py: packed and
low-latency. Rows that no expert has are left as they were: the outputs' buffers
start as zeros here.
"""
import math

import torch

own = False

MOST_EXACT_FLOPS = 3e14  # 64-bit products beyond this take too long
SMALLEST = 1e-30         # of a row's largest magnitude, for its int8 scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a decode step's router: 128 tokens (some of them padding) over 256 experts, one call of the many between small kernels
        dict(name="route_decode", op="route", T=128, E=256, k=8, score="softmax", bias=False, groups=1, kept=1, top=1,
             renorm=True, scale=1.0, dtype="bf16"),
        # a prefill batch or a training step of 16384 tokens: sigmoid scores, a balance bias, 4 of 8 groups by their best two
        dict(name="route_prefill", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4, top=2,
             renorm=True, scale=2.5, dtype="fp32"),
        # a small training step with odd counts: plain softmax scores as weights, whose gradient reaches every expert
        dict(name="route_gradient_odd", op="route_gradient", T=173, E=48, k=2, score="softmax", renorm=False, scale=1.0,
             dtype="bf16"),
        # the backward pass of route_prefill
        dict(name="route_gradient", op="route_gradient", T=16384, E=256, k=8, score="sigmoid", renorm=True, scale=2.5,
             dtype="fp32"),
        # a decode batch of 128 tokens over all 256 experts in the low-latency layout: the weights' bytes are the time
        dict(name="int8_layer_decode", op="int8_layer", layout="low_latency", T=128, k=8, E=256, R=8, K=7168, I=2048, skew=0.3),
        # 4096 tokens, top-8 of 64 experts of uneven popularity: 32768 ragged rows
        dict(name="int8_layer_prefill", op="int8_layer", layout="packed", T=4096, k=8, E=64, R=8, K=7168, I=2048, skew=0.5),
        # rows of a small batch, an odd count of narrow ones
        dict(name="checkpoint_rows_odd", op="rows", rows=1021, cols=2080),
        # a training batch's received rows
        dict(name="checkpoint_rows", op="rows", rows=16384, cols=7168),
        # SwiGLU of a small training step with odd sizes: empty and one-row experts among 48
        dict(name="checkpoint_swiglu_odd", op="swiglu", layout="packed", T=173, k=2, E=48, R=1, I=672, skew=2.0),
        # SwiGLU in training on 16384 tokens, four experts each
        dict(name="checkpoint_swiglu", op="swiglu", layout="packed", T=16384, k=4, E=64, R=8, I=2048, skew=0.2),
        # weight gradient of the small training step, in fp32
        dict(name="checkpoint_weights_odd", op="weights", layout="packed", T=173, k=2, E=48, R=1, K=1056, N=648, skew=2.0,
             acc="fp32"),
        # a training rank share: 8 local experts, some 4096 rows each, of the gate and up product
        dict(name="checkpoint_weights", op="weights", layout="packed", T=32768, k=1, E=8, R=1, K=7168, N=4096, skew=0.1,
             acc="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, even over the logarithm, a multiple of step."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["route"] * 2 + ["route_gradient"] + ["int8_layer"] * 2 + ["rows", "swiglu", "weights"])
    if op == "rows":
        cols = _log(rng, 32, 8192, 32)
        return dict(op=op, rows=_log(rng, 1, max(1, 16384 * 7168 // cols)), cols=cols)
    if op in ("route", "route_gradient"):
        E = rng.choice([8, 16, 48, 60, 64, 96, 128, 160, 256, 384, 512])
        case = dict(op=op, T=_log(rng, 1, 16384 * 256 // max(E, 256)), E=E, k=rng.choice([k for k in (1, 2, 4, 6, 8, 10) if k <= E // 2]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 2.5, 16.0]),
                    dtype=rng.choice(["bf16", "fp32"]))
        if op == "route_gradient":
            return case
        groups = rng.choice([1, 1] + [g for g in (2, 4, 8) if E % g == 0 and E // g >= 4])
        kept = rng.choice([n for n in range(1, groups + 1) if n * (E // groups) >= case["k"]])
        return dict(case, bias=rng.random() < 0.5, groups=groups, kept=kept, top=rng.choice([1, 2]))
    E, skew = rng.choice([4, 8, 16, 24, 32, 48, 64]), rng.choice([0.0, 0.2, 0.5, 1.0])
    R = rng.choice([r for r in (1, 2, 4, 8) if E % r == 0])
    k = rng.choice([1, 2, 4])
    case = dict(op=op, layout="packed", k=k, E=E, R=R, skew=skew)
    if op == "swiglu":
        I = _log(rng, 32, 4096, 32)
        return dict(case, T=R * _log(rng, 1, max(1, min(16384, 65536 * 2048 // (k * I)) // R)), I=I)
    if op == "weights":
        K, N = _log(rng, 128, 7168, 32), _log(rng, 64, 7168, 8)
        if E * K * N > 5e8:  # the gradient is as large as the weights
            K, N = _log(rng, 128, 2048, 32), _log(rng, 64, 2048, 8)
        return dict(case, T=R * _log(rng, 1, max(1, int(min(16384, 1.5e12 / (2.0 * K * N * k))) // R)), K=K, N=N,
                    acc=rng.choice(["fp32", "bf16"]))
    K, I = _log(rng, 128, 7168, 16), _log(rng, 64, 3584, 16)
    most = max(1, int(min(16384, 1.5e12 / (6.0 * K * I * k))) // R)
    if rng.random() < 0.3:
        case["layout"], most = "low_latency", min(most, 256)
    return dict(case, T=R * _log(rng, 1, most), K=K, I=I)


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
    for part in out.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * scale)
    return out


def _picks(case, g):
    """[T, k] distinct experts of T tokens, by popularity: a softmax of skew * N(0, 1), the same for all seeds."""
    pop = case["skew"] * torch.randn(case["E"], generator=_generator(case["E"]), device="cuda")
    u = torch.rand((case["T"], case["E"]), generator=g, device="cuda").clamp(1e-30, 1.0 - 1e-7)
    return (pop - torch.log(-torch.log(u))).topk(case["k"], dim=1).indices


def _routing(case, g):
    """Row groups of a routed batch. The packed layout's rows per rank, fixed in advance as a program's buffer is, hold a tenth
    more than another batch needed; what a rank gets past them is dropped."""
    T, k, E, R = (case[n] for n in ("T", "k", "E", "R"))
    idx = _picks(case, g)
    if case["layout"] == "low_latency":
        src = torch.arange(T, device="cuda")[:, None] // (T // R)
        cnt = torch.bincount((idx * R + src).view(-1), minlength=E * R).view(E, R).to(torch.int32)
        return dict(offsets=None, counts=cnt, cap=E * T // R, region=T // R, widest=int(cnt.max()))
    cnt, other = (torch.bincount(i.view(-1), minlength=E).view(R, E // R) for i in (idx, _picks(case, _generator(1))))
    cap = min(int(1.1 * int(other.sum(1).max())) + 64, T * min(k, E // R) + 3)
    off = (cnt.cumsum(1) - cnt).clamp_max(cap)
    cnt = torch.minimum(cnt, cap - off)
    return dict(offsets=off.view(E).to(torch.int32), counts=cnt.view(E).to(torch.int32), cap=cap, region=0,
                widest=int(cnt.max()))


def _int8_weights(E, N, K, g):
    """Weights N(0, 1/K) as int8 with one scale per channel, the channels of different sizes."""
    q = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
    for part in q.view(-1).split(1 << 28):
        part.copy_((torch.randn(part.shape, generator=g, device="cuda") * 40.0).round_().clamp_(-127, 127))
    return q, (0.5 + torch.rand((E, N), generator=g, device="cuda")) / (40.0 * math.sqrt(K))


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "rows":
        spread = torch.exp2(torch.randint(-6, 7, (case["rows"], 1), generator=g, device="cuda").float())
        s["x"] = (_normal((case["rows"], case["cols"]), g).float() * spread).to(torch.bfloat16)
        return s
    if op in ("route", "route_gradient"):
        T, E, k = case["T"], case["E"], case["k"]
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["logits"] = _normal((T, E), g, 1.5, dtype)
        if op == "route":
            s["logits"][T - T // 32:] = -math.inf  # padding at the batch's end: no expert is open to it
            s["bias"] = 0.05 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        else:
            s["idx"] = s["logits"].float().topk(k, dim=1).indices.to(torch.int32)
            s["grad"] = torch.randn((T, k), generator=g, device="cuda")
        return s
    s.update(_routing(case, g))
    rows, E = case["R"] * s["cap"], case["E"]
    if op == "swiglu":
        I = case["I"]
        s["gate_up"], s["grad"] = _normal((rows, 2 * I), g, 1.5), _normal((rows, I), g)
        s["out"], s["again"] = (torch.zeros((rows, I), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        s["grad_out"] = torch.zeros((rows, 2 * I), dtype=torch.bfloat16, device="cuda")
    elif op == "weights":
        s["x"], s["grad"] = _normal((rows, case["K"]), g), _normal((rows, case["N"]), g)
        s["out"] = torch.zeros((E, case["N"], case["K"]), dtype=torch.float32 if case["acc"] == "fp32" else torch.bfloat16,
                               device="cuda")
    else:
        K, I = case["K"], case["I"]
        loud = torch.where(torch.rand((rows, 1), generator=g, device="cuda") < 0.01, 100.0, 1.0)
        s["x"] = _normal((rows, K), g).mul_(loud)
        s["w1"], s["s1"] = _int8_weights(E, 2 * I, K, g)
        s["w2"], s["s2"] = _int8_weights(E, K, I, g)
        s["out"] = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _scores(logits, score):
    """Scores [T, E] of 64-bit logits. (A token without any open expert has none: NaN where softmax divides by its sum.)"""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    """In 64 bits: the choice depends on which of two neighbouring scores is larger."""
    case = s["case"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    logits = s["logits"].double()
    scores = _scores(logits, case["score"])
    choice = scores if s["bias"] is None else scores + s["bias"].double()
    choice = torch.where(logits > -math.inf, choice, -math.inf)
    if G > 1:
        best = choice.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :case["top"]]
        best = torch.where(best > -math.inf, best, 0.0).sum(2) + torch.where(best[:, :, 0] > -math.inf, 0.0, -math.inf)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        open_ = torch.zeros((T, G), dtype=torch.bool, device="cuda").scatter_(1, order, True)
        choice = torch.where(open_.repeat_interleave(E // G, 1), choice, -math.inf)
    best = choice.sort(dim=1, descending=True, stable=True)
    idx, found = best.indices[:, :k], best.values[:, :k] > -math.inf
    w = torch.where(found, scores.gather(1, idx), 0.0)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return torch.where(found, idx, -1).to(torch.int32), (w * case["scale"]).float()


def _plain_route_gradient(s):
    case = s["case"]
    logits, idx = s["logits"].float(), s["idx"].long()
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-logits))
        chosen = p.gather(1, idx)
        slope = chosen * (1.0 - chosen)
    else:
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        chosen = p.gather(1, idx)
        slope = chosen
    d = s["grad"] * case["scale"]
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True)
        d = (d - (d * chosen).sum(1, keepdim=True) / total) / total
    out = torch.zeros_like(logits).scatter_(1, idx, d * slope)
    if case["score"] == "softmax" and not case["renorm"]:
        out = out - p * (d * chosen).sum(1, keepdim=True)
    return out.to(s["logits"].dtype)


def _pow2(n):
    """2^n as fp32 by its bits, for integers -126 <= n <= 127."""
    return ((n.to(torch.int32) + 127) << 23).view(torch.float32)


def _mx_codes(x):
    """MXINT8 codes (as fp32 whole numbers) and scale bytes [rows, cols/32] of fp32 rows: per 32 values 2^e is the power of two of
    the largest magnitude, codes are multiples of 2^(e-6), at most 127, ties to even."""
    b = x.view(x.shape[0], -1, 32)
    amax = b.abs().amax(2)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1, -127).clamp(-120, 127)
    codes = torch.round(b * _pow2(6 - e)[:, :, None]).clamp(-127, 127)
    return codes.view(x.shape), torch.where(amax > 0, e + 127, 0).to(torch.uint8)


def _mx_values(codes, e):
    return (codes.view(*e.shape, 32) * _pow2(e.to(torch.int32).clamp_min(7) - 133)[..., None]).view(codes.shape)


def _int8_rows(x):
    """int8 codes (as fp32 whole numbers) and one scale of each row."""
    a = x.abs().amax(-1, keepdim=True).clamp_min(SMALLEST)
    return torch.round(x * torch.full_like(a, 127.0).div(a)), a / 127.0


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


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "route":
        return _plain_route(s)
    if op == "route_gradient":
        return _plain_route_gradient(s)
    if op == "rows":
        codes, e = _mx_codes(s["x"].float())
        return _mx_values(codes, e).to(torch.bfloat16), e.view(torch.float8_e8m0fnu)
    idx, valid = _rows_of(s)
    if op == "weights":
        live = valid[..., None].float()
        d = _taken(s["grad"], idx).float() * live
        x = _mx_values(*_mx_codes(s["x"].float()))
        return torch.bmm(d.transpose(1, 2), _taken(x, idx) * live).to(s["out"].dtype)
    I = case["I"]
    if op == "swiglu":
        rows = s["gate_up"].shape[0]
        used = torch.zeros(rows + 1, dtype=torch.bool, device="cuda")
        used[torch.where(valid, idx, rows)] = True
        used = used[:rows, None]
        x = s["gate_up"].float()
        h = x[:, :I] / (1.0 + torch.exp(-x[:, :I])) * x[:, I:]
        x = _mx_values(*_mx_codes(x))
        gate, up, d = x[:, :I], x[:, I:], s["grad"].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        back = torch.cat((d * up * (sig * (1.0 + gate * (1.0 - sig))), d * (gate * sig)), 1)
        return tuple(torch.where(used, t, 0.0).to(torch.bfloat16) for t in (h, back, gate * sig * up))
    q, scale = _int8_rows(_taken(s["x"], idx).float())
    h = torch.bmm(q, s["w1"].float().transpose(1, 2)) * (scale * s["s1"][:, None, :])
    h = h.to(torch.bfloat16).float()
    q, scale = _int8_rows(h[..., :I] / (1.0 + torch.exp(-h[..., :I])) * h[..., I:])
    y = torch.bmm(q, s["w2"].float().transpose(1, 2)) * (scale * s["s2"][:, None, :])
    return _written(s["out"], idx, valid, y)


def run(state):
    if not own:
        return _plain(state)
    from combine_get_dispatch_amd import ep
    s, case = state, state["case"]
    op = case["op"]
    if op == "rows":
        q, scales = ep.quantize_mxint8(s["x"])
        return ep.dequantize_mxint8(q, scales), scales.view(torch.float8_e8m0fnu)
    if op == "route":
        router = ep.Router(case["E"], case["k"], score=case["score"], renormalize=case["renorm"], scale=case["scale"],
                           num_groups=case["groups"], topk_groups=case["kept"], group_top=case["top"])
        return ep.route(s["logits"], router, bias=s["bias"])
    if op == "route_gradient":
        router = ep.Router(case["E"], case["k"], score=case["score"], renormalize=case["renorm"], scale=case["scale"])
        return ep.route_backward(s["grad"], s["logits"], s["idx"], router)
    groups = ep.Groups(s["counts"], s["offsets"], num_experts=case["E"], num_ranks=case["R"], cap_rows=s["cap"],
                       region_rows=s["region"], rows_hint=case["T"] * case["k"])
    if op == "weights":
        q, scales = ep.quantize_mxint8(s["x"], groups)
        return ep.expert_gemm_wgrad(s["grad"], q, groups, out=s["out"], row_scales=scales)
    if op == "swiglu":
        h, q, scales = ep.swiglu_checkpoint(s["gate_up"], groups, out=s["out"])
        back, again = ep.swiglu_checkpoint_backward(s["grad"], q, scales, groups, out=(s["grad_out"], s["again"]))
        return h, back, again
    q, scale = ep.quantize_int8(s["x"], groups)
    h = ep.expert_gemm(q, s["w1"], groups, row_scales=scale, weight_scales=s["s1"])
    q, scale = ep.swiglu(h, groups, kind="int8")
    return ep.expert_gemm(q, s["w2"], groups, row_scales=scale, weight_scales=s["s2"], out=s["out"])


# ---------------------------------------------------------------------------
# the work of one pass, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    mx = 1 + 1 / 32  # bytes of a value in MXINT8: written by one call, read by the other
    if op == "rows":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (4 + 2 * mx), "flops": 4.0 * n}
    if op in ("route", "route_gradient"):
        n, picks = case["T"] * case["E"], case["T"] * case["k"]
        each = 2 if case["dtype"] == "bf16" else 4
        if op == "route":
            return {"bytes": n * each + picks * 8, "flops": 4.0 * n}
        dense = case["score"] == "softmax" and not case["renorm"]  # else the chosen logits alone are read
        return {"bytes": n * each + (n if dense else picks) * each + picks * 8, "flops": (6.0 if dense else 1.0) * n}
    slots, E = case["T"] * case["k"], case["E"]
    if op == "swiglu":
        n = slots * case["I"]
        return {"bytes": n * (14 + 4 * mx), "flops": 24.0 * n}
    if op == "weights":
        K, N = case["K"], case["N"]
        return {"bytes": slots * (K * (2 + 2 * mx) + N * 2) + E * N * K * (4 if case["acc"] == "fp32" else 2),
                "flops": 2.0 * slots * N * K}
    K, I = case["K"], case["I"]
    hit = E * (1.0 - (1.0 - 1.0 / E) ** slots)  # experts with a row, were all as popular
    return {"bytes": slots * K * 4 + hit * (3 * K * I + (2 * I + K) * 4), "flops": 6.0 * slots * K * I}


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


def _exact_kept(x):
    """What MXINT8 keeps of 64-bit rows, and the groups' powers of two."""
    b = x.unflatten(-1, (-1, 32))
    power = (b.abs().amax(-1, keepdim=True).view(torch.int64) >> 52 << 52).view(torch.float64)  # the exponent field alone
    return ((b / (power / 64)).round().clamp(-127, 127) * (power / 64)).flatten(-2), power.squeeze(-1)


def _exact_int8(x):
    """The codes are by definition those of 127 / a and of its product with x, each rounded to 32 bits: bf16 values often lie
    halfway between two codes."""
    a = x.abs().amax(-1, keepdim=True).clamp_min(SMALLEST)
    return (x * (127 / a).float().double()).float().double().round(), a / 127


def _exact_choice(case, logits, bias):
    """Row by row of the definition: chosen experts in order, -1 where none is left."""
    T, E, G = case["T"], case["E"], case["groups"]
    shut = logits == -math.inf
    s = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits.masked_fill(shut.all(1, keepdim=True), 0), 1)
    c = (s if bias is None else s + bias.double()).masked_fill(shut, -math.inf)
    if G > 1:
        g = c.unflatten(1, (G, -1)).clone()
        value = torch.zeros((T, G), dtype=torch.float64, device="cuda")
        for turn in range(case["top"]):
            m = g.max(2)
            value += m.values if turn == 0 else m.values.clamp_min(0).where(m.values == -math.inf, m.values)
            g.scatter_(2, m.indices[..., None], -math.inf)
        index = torch.arange(G, device="cuda")
        ahead = (value[:, None, :] > value[:, :, None]) | ((value[:, None, :] == value[:, :, None]) & (index[None, :] < index[:, None]))
        c = c.masked_fill((ahead.sum(2) >= case["kept"]).repeat_interleave(E // G, 1), -math.inf)
    picked, weights = [], []
    index = torch.arange(E, device="cuda").expand(T, E)
    for _ in range(case["k"]):
        m = c.amax(1, keepdim=True)
        i = torch.where(c == m, index, E).amin(1, keepdim=True)  # the lowest of those that tie
        none = m == -math.inf
        picked.append(torch.where(none, -1, i))
        weights.append(s.gather(1, i).masked_fill(none, 0))
        c = c.scatter(1, i, -math.inf)
    return torch.cat(picked, 1), torch.cat(weights, 1), s


def exact(case, seed):
    op = case["op"]
    if op in ("int8_layer", "weights") and work(case)["flops"] > MOST_EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    if op == "route":
        idx, w, _ = _exact_choice(case, s["logits"].double(), s["bias"])
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True).masked_fill(idx[:, :1] < 0, 1)
        return idx.to(torch.int32), w * case["scale"]
    if op == "route_gradient":
        # differentiated by torch, in 64 bits
        with torch.enable_grad():
            l = s["logits"].double().requires_grad_()
            p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
            w = p.gather(1, s["idx"].long())
            if case["renorm"]:
                w = w / w.sum(1, keepdim=True)
            return torch.autograd.grad((w * s["grad"].double()).sum() * case["scale"], l)[0]
    if op == "rows":
        return _exact_kept(s["x"].double())
    groups = _exact_groups(s)
    if op == "weights":
        out = torch.zeros(tuple(s["out"].shape), dtype=torch.float64, device="cuda")
        for e, at in groups:
            out[e] = s["grad"][at].double().t().contiguous() @ _exact_kept(s["x"][at].double())[0]
        return out
    if op == "swiglu":
        I = case["I"]
        out = [torch.zeros(tuple(s[n].shape), dtype=torch.float64, device="cuda") for n in ("out", "grad_out", "again")]
        for at in torch.cat([r for _, r in groups]).split(4096):
            gate, up = s["gate_up"][at].double().split(I, 1)
            out[0][at] = gate * torch.sigmoid(gate) * up
            gate, up = _exact_kept(s["gate_up"][at].double())[0].split(I, 1)
            sig, d = torch.sigmoid(gate), s["grad"][at].double()
            out[1][at] = torch.cat((d * up * (sig + gate * sig * (1 - sig)), d * gate * sig), 1)
            out[2][at] = gate * sig * up
        return tuple(out)
    I = case["I"]
    out = torch.zeros(tuple(s["out"].shape), dtype=torch.float64, device="cuda")
    for e, at in groups:
        q, scale = _exact_int8(s["x"][at].double())
        h = (q @ s["w1"][e].double().t().contiguous()) * scale * s["s1"][e].double()
        gate, up = h.to(torch.bfloat16).double().split(I, 1)  # the first product's result is a bf16 tensor
        q, scale = _exact_int8(gate * torch.sigmoid(gate) * up)
        out[at] = (q @ s["w2"][e].double().t().contiguous()) * scale * s["s2"][e].double()
    return out
