"""What the router's, the 8-bit integer rows' and the checkpoints' calls refuse
before anything is launched, in sizes and tensors that no GPU is needed for."""
import ctypes
import os

import pytest
import torch

from combine_get_dispatch_amd import build as epbuild
from combine_get_dispatch_amd import ep
from test_experts_arguments import as_if_on_gpu, code_of, groups, overlapping, wrong  # noqa: F401

P16, P8, P4, P2, P1 = ((1 << 20) + v for v in (0, 8, 4, 2, 1))
FAR = (1 << 32) + 256  # as a 32-bit int: 256
ROWS, E, K, N = 128, 8, 256, 64
BASE = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def library():
    if not os.path.exists(ep.LIB_PATH):
        epbuild.build()
    return ep.load()


# every call by name, of a dict of its arguments' places and sizes; and arrays {argument: bytes}, outputs, alignment
def place(**kw):
    v = dict(g=groups(), rows=ROWS, K=K, N=N, T=ROWS, form=ep.EP_FORM_INT8, f32=True, accumulate=False, bias=None, x=None, q=None,
             s=None, d=None, out=None, w=None, ws=None, grad=None, idx=None, again=None)
    v.update(kw)
    return v


def router(**kw):
    v = dict(num_experts=64, num_topk=4, score=1, renormalize=1, num_groups=8, topk_groups=3, group_top=2, scale=1.0)
    v.update(kw)
    return ep.EpRouter(*[v[n] for n, _ in ep.EpRouter._fields_])


CALLS = {
    "gemm": (lambda v: ep.ep_expert_gemm(v["g"], v["form"], v["q"], v["s"], v["w"], v["ws"], v["K"], v["N"], v["out"], 0),
             dict(q=ROWS * K, s=ROWS * 4, w=E * N * K, ws=E * N * 4, out=ROWS * N * 2), ["out"], dict(q=16, w=16, out=16, s=4, ws=16)),
    "swiglu": (lambda v: ep.ep_swiglu(v["g"], v["x"], v["rows"], v["K"], v["form"], v["q"], v["s"], 0),
               dict(x=ROWS * K * 4, q=ROWS * K, s=ROWS * 4), ["q", "s"], dict(x=16, q=16, s=4)),
    "int8": (lambda v: ep.ep_quantize_int8(v["g"], v["x"], v["rows"], v["K"], v["q"], v["s"], 0),
             dict(x=ROWS * K * 2, q=ROWS * K, s=ROWS * 4), ["q", "s"], dict(x=16, q=16, s=4)),
    "mxint8": (lambda v: ep.ep_quantize_mxint8(v["g"], v["x"], v["rows"], v["K"], v["q"], v["s"], 0),
               dict(x=ROWS * K * 2, q=ROWS * K, s=ROWS * K // 32), ["q", "s"], dict(x=16, q=16)),
    "back": (lambda v: ep.ep_dequantize_mxint8(v["g"], v["q"], v["s"], v["rows"], v["K"], v["x"], 0),
             dict(x=ROWS * K * 2, q=ROWS * K, s=ROWS * K // 32), ["x"], dict(x=16, q=16)),
    "keep": (lambda v: ep.ep_swiglu_checkpoint(v["g"], v["x"], v["rows"], v["K"], v["out"], v["q"], v["s"], 0),
             dict(x=ROWS * K * 4, out=ROWS * K * 2, q=ROWS * K * 2, s=ROWS * K // 16), ["out", "q", "s"], dict(x=16, out=16, q=16)),
    "kept": (lambda v: ep.ep_swiglu_checkpoint_backward(v["g"], v["d"], v["q"], v["s"], v["rows"], v["K"], v["grad"], v["again"], 0),
             dict(d=ROWS * K * 2, q=ROWS * K * 2, s=ROWS * K // 16, grad=ROWS * K * 4, again=ROWS * K * 2), ["grad", "again"],
             dict(d=16, q=16, grad=16, again=16)),
    "wgrad": (lambda v: ep.ep_expert_gemm_wgrad_mxint8(v["g"], v["d"], v["q"], v["s"], v["K"], v["N"], v["out"], v["f32"],
                                                       v["accumulate"], 0),
              dict(d=ROWS * N * 2, q=ROWS * K, s=ROWS * K // 32, out=E * N * K * 4), ["out"], dict(d=16, q=16, out=16)),
}
ROW_CALLS = ["swiglu", "int8", "mxint8", "back", "keep", "kept"]
ROUTES = {
    "route": (lambda v: ep.ep_route(v.get("r", router()), v["x"], v["f32"], v["bias"], v["T"], v["idx"], v["w"], 0),
              dict(x=ROWS * 64 * 4, bias=64 * 4, idx=ROWS * 16, w=ROWS * 16), ["idx", "w"], dict(x=4, bias=4, idx=4, w=4)),
    "route_backward": (lambda v: ep.ep_route_backward(v.get("r", router()), v["x"], v["f32"], v["idx"], v["d"], v["T"], v["grad"], 0),
                       dict(x=ROWS * 64 * 4, idx=ROWS * 16, d=ROWS * 16, grad=ROWS * 64 * 4), ["grad"],
                       dict(x=4, idx=4, d=4, grad=4)),
}
ALL = dict(CALLS, **ROUTES)


def apart(name, **kw):
    """Arguments with every array in a place of its own."""
    return place(**{n: BASE + (i << 30) for i, n in enumerate(ALL[name][1])}, **kw)


@pytest.mark.parametrize("name", list(ALL))
def test_arrays_missing_misaligned_or_overlapping(name):
    call, arrays, outputs, align = ALL[name]
    for a in arrays:
        if a not in ("bias", "again"):  # (these may be NULL)
            assert code_of(call, dict(apart(name), **{a: None})) == ep.EP_ERR_ARG, a
    for a, n in align.items():
        bad = dict(apart(name))
        bad[a] += n // 2
        assert code_of(call, bad) == ep.EP_ERR_ALIGN, a
    for what, at in overlapping(arrays, outputs):
        assert code_of(call, place(**at)) == ep.EP_ERR_ARG, what
    if name in ROUTES:  # bf16: half the bytes; arrays one after another are apart
        bad = apart(name, f32=False)
        bad["x"] += 1
        assert code_of(call, bad) == ep.EP_ERR_ALIGN


@pytest.mark.parametrize("name", list(CALLS))
def test_groups_of_every_call(name):
    call = CALLS[name][0]
    for bad in (dict(num_experts=0), dict(num_experts=1025, num_ranks=1), dict(num_ranks=3), dict(cap_rows=-1),
                dict(cap_rows=1 << 62), dict(region_rows=8), dict(counts=None), dict(offsets=None), dict(rows_hint=-1)):
        g = groups(**bad)
        rows = max(0, min(g.num_ranks * g.cap_rows, 1 << 40))
        assert code_of(call, dict(apart(name), g=g, rows=rows)) == ep.EP_ERR_ARG, bad
    assert code_of(call, dict(apart(name), g=groups(counts=(1 << 20) + 2))) == ep.EP_ERR_ALIGN
    if name in ROW_CALLS:
        assert code_of(call, dict(apart(name), rows=ROWS - 1)) == ep.EP_ERR_ARG
        assert code_of(call, dict(apart(name), g=None, rows=-1)) == ep.EP_ERR_ARG
        assert code_of(call, dict(apart(name), g=None, rows=1 << 31)) == ep.EP_ERR_ARG
    else:
        assert code_of(call, dict(apart(name), g=None)) == ep.EP_ERR_ARG
    empty = dict(apart(name), g=groups(cap_rows=0), rows=0, x=None, q=None, s=None, d=None)
    if name != "wgrad":  # (whose result is zeros then)
        call(empty)


@pytest.mark.parametrize("size", [0, 8, -16, 65552, FAR, -FAR])
def test_channels(size):
    for name in CALLS:
        assert code_of(CALLS[name][0], dict(apart(name), K=size)) == ep.EP_ERR_ARG, name
    for name in ("gemm", "wgrad"):
        if size != 8:
            assert code_of(CALLS[name][0], dict(apart(name), N=size)) == ep.EP_ERR_ARG, name
        assert code_of(CALLS[name][0], dict(apart(name), N=12)) == ep.EP_ERR_ARG, name
    for name in ("mxint8", "back", "keep", "kept", "wgrad"):
        assert code_of(CALLS[name][0], dict(apart(name), K=48)) == ep.EP_ERR_ARG, name


def test_forms():
    gemm, swiglu = CALLS["gemm"][0], CALLS["swiglu"][0]
    for form in (3, 5, -1):
        assert code_of(gemm, dict(apart("gemm"), form=form)) == ep.EP_ERR_ARG
        assert code_of(swiglu, dict(apart("swiglu"), form=form)) == ep.EP_ERR_ARG
    far = groups(offsets=None, region_rows=1 << 15, cap_rows=8 << 15)  # an expert's regions over 4 GiB of rows
    assert code_of(gemm, dict(apart("gemm"), g=far, K=65536)) == ep.EP_ERR_ARG
    assert code_of(CALLS["wgrad"][0], dict(apart("wgrad"), f32=False, accumulate=True)) == ep.EP_ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(num_experts=0), dict(num_experts=1025, num_groups=1, topk_groups=1), dict(num_experts=-64), dict(num_topk=0),
    dict(num_topk=33), dict(num_topk=25), dict(score=2), dict(score=-1), dict(renormalize=2), dict(num_groups=0),
    dict(num_groups=7), dict(num_groups=128, num_experts=256), dict(topk_groups=0), dict(topk_groups=9), dict(group_top=0),
    dict(group_top=3), dict(scale=float("inf")), dict(scale=float("nan")),
])
def test_routers(bad):
    for name, (call, *_) in ROUTES.items():
        assert code_of(call, dict(apart(name), r=router(**bad))) == ep.EP_ERR_ARG
        call(dict(apart(name), T=0))  # nothing to do
        for T in (-1, (1 << 24) + 1, FAR):
            assert code_of(call, dict(apart(name), T=T)) == ep.EP_ERR_ARG


def test_logits_types():
    lib = ep.load()
    r = router()
    for f32 in (2, -1):
        assert lib.ep_route(ctypes.byref(r), P16, f32, None, 4, P16, P16, None) == ep.EP_ERR_ARG
        assert lib.ep_route_backward(ctypes.byref(r), P16, f32, P16, P16, 4, P16, None) == ep.EP_ERR_ARG
    assert lib.ep_route(None, P16, 1, None, 4, P16, P16, None) == ep.EP_ERR_ARG
    assert lib.ep_route_backward(None, P16, 1, P16, P16, 4, P16, None) == ep.EP_ERR_ARG


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------

def binding_calls():
    i32, bf, u8, i8, f32 = torch.int32, torch.bfloat16, torch.uint8, torch.int8, torch.float32
    t = lambda dtype, *shape: torch.zeros(shape, dtype=dtype)  # noqa: E731
    E, R, cap, K, N, T, k = 4, 2, 8, 256, 136, 16, 2
    n = R * cap
    g = dict(counts=t(i32, E), offsets=t(i32, E))
    mk = lambda d: ep.Groups(d.pop("counts"), d.pop("offsets"), num_experts=E, num_ranks=R, cap_rows=cap)  # noqa: E731
    pair = lambda d, a="out", b="scales": (d.pop(a), d.pop(b))  # noqa: E731
    r = ep.Router(8, k)
    return {
        "expert_gemm": (lambda d: ep.expert_gemm(groups=mk(d), **d),
                        dict(g, rows=t(i8, n, K), weights=t(i8, E, N, K), row_scales=t(f32, n), weight_scales=t(f32, E, N),
                             out=t(bf, n, N))),
        "swiglu": (lambda d: ep.swiglu(d.pop("gate_up"), mk(d), "int8", out=pair(d)),
                   dict(g, gate_up=t(bf, n, 2 * K), out=t(i8, n, K), scales=t(f32, n))),
        "quantize_int8": (lambda d: ep.quantize_int8(d.pop("x"), mk(d), out=pair(d)),
                          dict(g, x=t(bf, n, K), out=t(i8, n, K), scales=t(f32, n))),
        "quantize_mxint8": (lambda d: ep.quantize_mxint8(d.pop("x"), mk(d), out=pair(d)),
                            dict(g, x=t(bf, n, K), out=t(i8, n, K), scales=t(u8, n, 8))),
        "dequantize_mxint8": (lambda d: ep.dequantize_mxint8(d.pop("q"), d.pop("scales"), mk(d), **d),
                              dict(g, q=t(i8, n, K), scales=t(u8, n, 8), out=t(bf, n, K))),
        "swiglu_checkpoint": (lambda d: ep.swiglu_checkpoint(d.pop("gate_up"), mk(d), out=d.pop("out"), kept=pair(d, "q")),
                              dict(g, gate_up=t(bf, n, 2 * K), out=t(bf, n, K), q=t(i8, n, 2 * K), scales=t(u8, n, 16))),
        "swiglu_checkpoint_backward": (
            lambda d: ep.swiglu_checkpoint_backward(d.pop("grad_out"), d.pop("q"), d.pop("scales"), mk(d),
                                                    out=pair(d, "grad", "again")),
            dict(g, grad_out=t(bf, n, K), q=t(i8, n, 2 * K), scales=t(u8, n, 16), grad=t(bf, n, 2 * K), again=t(bf, n, K))),
        "expert_gemm_wgrad_mxint8": (
            lambda d: ep.expert_gemm_wgrad(d.pop("grad_out"), d.pop("rows"), mk(d), dtype=f32, **d),
            dict(g, grad_out=t(bf, n, N), rows=t(i8, n, K), row_scales=t(u8, n, 8), out=t(f32, E, N, K))),
        "route": (lambda d: ep.route(d.pop("logits"), r, d.pop("bias"), out=pair(d, "idx", "w")),
                  dict(logits=t(bf, T, 8), bias=t(f32, 8), idx=t(i32, T, k), w=t(f32, T, k))),
        "route_backward": (lambda d: ep.route_backward(d.pop("grad"), d.pop("logits"), d.pop("idx"), r, out=d.pop("out")),
                           dict(grad=t(f32, T, k), logits=t(f32, T, 8), idx=t(i32, T, k), out=t(f32, T, 8))),
    }


@pytest.mark.parametrize("name", list(binding_calls()))
def test_binding_refuses_each_tensor(as_if_on_gpu, name):  # noqa: F811
    call, tensors = binding_calls()[name]
    call(dict(tensors))
    assert [c for c, _ in as_if_on_gpu] == ["ep_" + name]  # as it should be: it reaches the C call, once
    as_if_on_gpu.clear()
    for arg, t in tensors.items():
        for what, b in wrong(t if t.dtype is not torch.int8 else t.view(torch.uint8)):
            if t.dtype is torch.int8:  # (`wrong` of bytes, as 8-bit integers but for the wrong type)
                b = t.view(torch.uint8) if what == "type" else b.view(torch.int8)
            try:
                call(dict(tensors, **{arg: b}))
            except ep.EpError as e:
                assert e.code == ep.EP_ERR_ARG
            assert not as_if_on_gpu, f"{arg} of wrong {what}"


def test_binding_refuses_other_devices(monkeypatch):
    """Every tensor is another device's in turn."""
    monkeypatch.setattr(ep, "_torch", torch)
    monkeypatch.setattr(ep, "_device", lambda: 0)
    monkeypatch.setattr(ep, "_raw_stream", lambda dev: 0)
    for name, (call, tensors) in binding_calls().items():
        for arg in tensors:
            places = {t.data_ptr(): 0 for t in tensors.values()}
            places[tensors[arg].data_ptr()] = 1
            monkeypatch.setattr(torch.Tensor, "get_device", lambda t: places[t.data_ptr()])
            assert code_of(call, dict(tensors)) == ep.EP_ERR_ARG, (name, arg)


def test_binding_without_a_gpu():
    """CPU tensors, and what is no router."""
    x = torch.zeros(4, 64)
    if not torch.cuda.is_available():
        assert code_of(ep.route, x, ep.Router(64, 4)) == ep.EP_ERR_ARG
        assert code_of(ep.quantize_int8, x.to(torch.bfloat16)) == ep.EP_ERR_ARG
        assert code_of(ep.quantize_mxint8, torch.zeros((), dtype=torch.bfloat16)) == ep.EP_ERR_ARG
        assert code_of(ep.quantize_int8, torch.zeros((), dtype=torch.bfloat16)) == ep.EP_ERR_ARG
    assert code_of(ep.Router(64, 4, score="tanh").c) == ep.EP_ERR_ARG
    assert code_of(ep.Router(64 + (1 << 32), 4).c) == ep.EP_ERR_ARG
    assert code_of(ep.route, x.half(), ep.Router(64, 4)) == ep.EP_ERR_ARG
    assert code_of(ep.route, x[0], ep.Router(64, 4)) == ep.EP_ERR_ARG
