"""What the experts' binding and C ABI refuse before anything is launched, in
sizes and tensors that no GPU is needed for."""
import os
import re
import subprocess

import pytest
import torch

from combine_get_dispatch_amd import build as epbuild
from combine_get_dispatch_amd import ep

MIB = 1 << 20
FAR = (1 << 32) + 256  # as a 32-bit int: 256


@pytest.fixture(scope="module", autouse=True)
def library():
    if not os.path.exists(ep.LIB_PATH):
        epbuild.build()
    return ep.load()


def groups(**kw):
    g = dict(offsets=MIB, counts=MIB, num_experts=8, num_ranks=2, cap_rows=64, region_rows=0, rows_hint=0)
    g.update(kw)
    return ep.EpGroups(*[g[n] for n, _ in ep.EpGroups._fields_])


def code_of(f, *args, **kw):
    with pytest.raises(ep.EpError) as e:
        f(*args, **kw)
    return e.value.code


@pytest.mark.parametrize("K,N", [(FAR, 256), (256, FAR), (FAR, FAR), (256 - (1 << 32), 256)])
def test_products_of_channels_past_32_bits(K, N):
    a, b, c, s = MIB << 4, MIB << 5, MIB << 6, MIB << 7
    assert code_of(ep.ep_expert_gemm, groups(), ep.EP_FORM_BF16, a, None, b, None, K, N, c, 0) == ep.EP_ERR_ARG
    assert code_of(ep.ep_expert_gemm, groups(), ep.EP_FORM_FP8, a, s, b, s, K, N, c, 0) == ep.EP_ERR_ARG
    assert code_of(ep.ep_expert_gemm_dgrad, groups(), a, b, K, N, c, 0) == ep.EP_ERR_ARG
    assert code_of(ep.ep_expert_gemm_wgrad, groups(), a, b, K, N, c, True, False, 0) == ep.EP_ERR_ARG


def test_rows_of_channels_past_32_bits():
    a, b, c = MIB << 4, MIB << 5, MIB << 6
    assert code_of(ep.ep_swiglu, None, a, 1, FAR, ep.EP_FORM_BF16, b, None, 0) == ep.EP_ERR_ARG
    assert code_of(ep.ep_swiglu, groups(), a, 128, FAR, ep.EP_FORM_FP8, b, c, 0) == ep.EP_ERR_ARG
    assert code_of(ep.ep_swiglu_backward, None, a, b, 1, FAR, c, 0) == ep.EP_ERR_ARG
    assert code_of(ep.ep_quantize_mxfp4, None, a, 1, FAR, b, c, 0) == ep.EP_ERR_ARG
    assert code_of(ep.ep_dequantize_mxfp4, None, a, b, 1, FAR, c, 0) == ep.EP_ERR_ARG


@pytest.fixture
def as_if_on_gpu(monkeypatch):
    """CPU tensors pass for the current GPU's; the calls of the C ABI are recorded in its place."""
    calls, lib = [], ep.load()

    class Library:
        ep_strerror = lib.ep_strerror

        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or ep.EP_OK

    monkeypatch.setattr(ep, "_torch", torch)
    monkeypatch.setattr(ep, "_device", lambda: 0)
    monkeypatch.setattr(ep, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(ep, "load", Library)
    return calls


@pytest.mark.parametrize("field", ["num_experts", "num_ranks"])
def test_groups_past_32_bits(as_if_on_gpu, field):
    """Sizes that the C struct's 32-bit fields cannot hold (views of one number stand for the large arrays)."""
    one = torch.zeros(1, dtype=torch.int32)
    sizes = dict(num_experts=8, num_ranks=2, cap_rows=64)
    sizes[field] += 1 << 32
    g = ep.Groups(one.expand(sizes["num_experts"]), one.expand(sizes["num_experts"]), **sizes)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(torch.Tensor, "is_contiguous", lambda t: True)
        assert code_of(g.c) == ep.EP_ERR_ARG


# Every output on an input's first and last 16 bytes, and on another output's. (Sizes: 128 rows, 8 experts, K = 256 and N = 64
# channels.) The arrays' places are never touched: every call is refused.
ROWS, E, K, N = 128, 8, 256, 64
BASE = 1 << 40


def overlapping(arrays, outputs):
    """Places {name: address} 1 GiB apart but for one output, which overlaps another array by 16 bytes on either side."""
    for o in outputs:
        for other in arrays:
            if other != o:
                for side in (0, 1):
                    at = {n: BASE + (i << 30) for i, n in enumerate(arrays)}
                    at[o] = at[other] - arrays[o] + 16 if side else at[other] + arrays[other] - 16
                    yield f"{o} on {other}", at


@pytest.mark.parametrize("form", [ep.EP_FORM_BF16, ep.EP_FORM_FP8, ep.EP_FORM_MXFP4])
def test_products_on_their_operands(form):
    width = {ep.EP_FORM_BF16: 2 * K, ep.EP_FORM_FP8: K, ep.EP_FORM_MXFP4: K // 2}[form]
    arrays = dict(rows=ROWS * width, weights=E * N * width, out=ROWS * N * 2)
    if form == ep.EP_FORM_FP8:
        arrays.update(row_scales=ROWS * K // 128 * 4, weight_scales=E * K // 128 * 4)
    elif form == ep.EP_FORM_MXFP4:
        arrays.update(row_scales=ROWS * K // 32, weight_scales=E * N * K // 32)
    for what, p in overlapping(arrays, ["out"]):
        assert code_of(ep.ep_expert_gemm, groups(), form, p["rows"], p.get("row_scales"), p["weights"],
                       p.get("weight_scales"), K, N, p["out"], 0) == ep.EP_ERR_ARG, what


def test_gradients_on_their_operands():
    for what, p in overlapping(dict(d=ROWS * N * 2, w=E * N * K * 2, out=ROWS * K * 2), ["out"]):
        assert code_of(ep.ep_expert_gemm_dgrad, groups(), p["d"], p["w"], K, N, p["out"], 0) == ep.EP_ERR_ARG, what
    for f32 in (False, True):
        for what, p in overlapping(dict(d=ROWS * N * 2, x=ROWS * K * 2, out=E * N * K * (4 if f32 else 2)), ["out"]):
            assert code_of(ep.ep_expert_gemm_wgrad, groups(), p["d"], p["x"], K, N, p["out"], f32, False,
                           0) == ep.EP_ERR_ARG, what


@pytest.mark.parametrize("grouped", [False, True])
def test_row_operators_on_their_operands(grouped):
    g = groups() if grouped else None
    n = ROWS * K
    for form, size, scales in ((ep.EP_FORM_BF16, 2 * n, 0), (ep.EP_FORM_FP8, n, n // 32), (ep.EP_FORM_MXFP4, n // 2, n // 32)):
        arrays = dict(x=4 * n, out=size, **(dict(scales=scales) if scales else {}))
        for what, p in overlapping(arrays, [a for a in arrays if a != "x"]):
            assert code_of(ep.ep_swiglu, g, p["x"], ROWS, K, form, p["out"], p.get("scales"), 0) == ep.EP_ERR_ARG, what
    for what, p in overlapping(dict(d=2 * n, x=4 * n, out=4 * n), ["out"]):
        assert code_of(ep.ep_swiglu_backward, g, p["d"], p["x"], ROWS, K, p["out"], 0) == ep.EP_ERR_ARG, what
    for what, p in overlapping(dict(x=2 * n, q=n // 2, scales=n // 32), ["q", "scales"]):
        assert code_of(ep.ep_quantize_mxfp4, g, p["x"], ROWS, K, p["q"], p["scales"], 0) == ep.EP_ERR_ARG, what
    for what, p in overlapping(dict(x=2 * n, q=n // 2, scales=n // 32), ["x"]):
        assert code_of(ep.ep_dequantize_mxfp4, g, p["q"], p["scales"], ROWS, K, p["x"], 0) == ep.EP_ERR_ARG, what
    # in place over an input that is another array's too
    assert code_of(ep.ep_swiglu_backward, g, BASE, BASE, ROWS, K, BASE, 0) == ep.EP_ERR_ARG


# Tensors wrong in one respect. (The names of the arguments, in the order of the call; `out` last, a tuple of them where the
# call has two outputs.)
def binding_calls():
    i32, bf, u8, f32 = torch.int32, torch.bfloat16, torch.uint8, torch.float32
    t = lambda dtype, *shape: torch.zeros(shape, dtype=dtype)  # noqa: E731
    E, R, cap, K, N = 4, 2, 8, 256, 136
    n = R * cap
    g = dict(counts=t(i32, E), offsets=t(i32, E))
    gemm = {
        "bf16": dict(rows=t(bf, n, K), weights=t(bf, E, N, K)),
        "fp8": dict(rows=t(u8, n, K), weights=t(u8, E, N, K), row_scales=t(f32, n, 2), weight_scales=t(f32, E, 2, 2)),
        "mxfp4": dict(rows=t(u8, n, K // 2), weights=t(u8, E, N, K // 2), row_scales=t(u8, n, 8),
                      weight_scales=t(u8, E, N, 8)),
    }
    mk = lambda d: ep.Groups(d.pop("counts"), d.pop("offsets"), num_experts=E, num_ranks=R, cap_rows=cap)  # noqa: E731
    calls = {f"expert_gemm {f}": (lambda d: ep.expert_gemm(groups=mk(d), **d), dict(g, **a, out=t(bf, n, N)))
             for f, a in gemm.items()}
    calls["expert_gemm_dgrad"] = (lambda d: ep.expert_gemm_dgrad(groups=mk(d), **d),
                                  dict(g, grad_out=t(bf, n, N), weights=t(bf, E, N, K), out=t(bf, n, K)))
    calls["expert_gemm_wgrad"] = (lambda d: ep.expert_gemm_wgrad(groups=mk(d), dtype=f32, **d),
                                  dict(g, grad_out=t(bf, n, N), rows=t(bf, n, K), out=t(f32, E, N, K)))
    pair = lambda d: (d.pop("out"), d.pop("scales"))  # noqa: E731
    calls["swiglu bf16"] = lambda d: ep.swiglu(groups=mk(d), **d), dict(g, gate_up=t(bf, n, 2 * K), out=t(bf, n, K))
    calls["swiglu fp8"] = (lambda d: ep.swiglu(d.pop("gate_up"), mk(d), "fp8", out=pair(d)),
                           dict(g, gate_up=t(bf, n, 2 * K), out=t(u8, n, K), scales=t(f32, n, 2)))
    calls["swiglu mxfp4"] = (lambda d: ep.swiglu(d.pop("gate_up"), mk(d), "mxfp4", out=pair(d)),
                             dict(g, gate_up=t(bf, n, 2 * K), out=t(u8, n, K // 2), scales=t(u8, n, 8)))
    calls["swiglu_backward"] = (lambda d: ep.swiglu_backward(groups=mk(d), **d),
                                dict(g, grad_out=t(bf, n, K), gate_up=t(bf, n, 2 * K), out=t(bf, n, 2 * K)))
    calls["quantize_mxfp4"] = (lambda d: ep.quantize_mxfp4(d.pop("x"), mk(d), out=pair(d)),
                               dict(g, x=t(bf, n, K), out=t(u8, n, K // 2), scales=t(u8, n, 8)))
    calls["dequantize_mxfp4"] = (lambda d: ep.dequantize_mxfp4(d.pop("q"), d.pop("scales"), mk(d), **d),
                                 dict(g, q=t(u8, n, K // 2), scales=t(u8, n, 8), out=t(bf, n, K)))
    return calls


def wrong(t):
    """The tensor with another type of the same size, another size, and other strides."""
    same_size = {torch.int32: torch.float32, torch.float32: torch.int32, torch.bfloat16: torch.float16,
                 torch.uint8: torch.int8}
    yield "type", t.view(same_size[t.dtype])
    yield "dimensions", t[None]
    for d in range(t.dim()):
        yield f"size {d}", torch.zeros([s + 32 if i == d else s for i, s in enumerate(t.shape)], dtype=t.dtype)
    if t.dim() > 1:
        yield "order", t.mT.contiguous().mT
    yield "stride", torch.zeros([2 * s if i == 0 else s for i, s in enumerate(t.shape)], dtype=t.dtype)[::2]


@pytest.mark.parametrize("name", list(binding_calls()))
def test_binding_refuses_each_tensor(as_if_on_gpu, name):
    call, tensors = binding_calls()[name]
    call(dict(tensors))
    assert [c for c, _ in as_if_on_gpu] == ["ep_" + name.split()[0]]  # as it should be: it reaches the C call, once
    as_if_on_gpu.clear()
    for arg, t in tensors.items():
        for what, bad in wrong(t):
            try:
                call(dict(tensors, **{arg: bad}))
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


# ---------------------------------------------------------------------------
# the compiled kernels
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    """(assembly, the compiler's messages) of the experts' kernels, device and host passes."""
    out = str(tmp_path_factory.mktemp("experts") / "experts.s")
    cmd = [epbuild.hipcc()] + epbuild.flags() + ["-S", "-o", out, os.path.join(epbuild.CSRC, "ep_experts.hip")]
    done = subprocess.run(cmd + ["--offload-device-only"], check=True, capture_output=True, text=True)
    host = subprocess.run([epbuild.hipcc()] + epbuild.flags() + ["--offload-host-only", "-fsyntax-only", cmd[-1]],
                          check=True, capture_output=True, text=True)
    return open(out).read(), done.stderr + host.stderr


@pytest.mark.slow
def test_no_warnings(compiled):
    """But for the driver's own about flags that one of its passes does not use."""
    found = [l for l in compiled[1].splitlines()
             if "warning:" in l and "argument unused" not in l and "packed-fp32-ops" not in l]
    assert not found, "\n".join(found[:5])


@pytest.mark.slow
def test_only_the_copies_touch_m0(compiled):
    """The copies to LDS write M0 in asm, which cannot be named as a clobber (the compiler reserves it): no instruction of
    the compiler's own may write it, nor read it but as the copies do."""
    in_asm, copies, others = False, 0, []
    for line in compiled[0].splitlines():
        t = line.strip()
        if t.startswith(";;#ASM"):
            in_asm = "START" in t
        t = t.split(";")[0].strip()
        if re.search(r"\bm0\b", t):
            copies += in_asm
            others += [] if in_asm else [t]
        elif not in_asm:
            # instructions that read it without naming it
            others += [t] if re.match(r"(global|buffer)_load_lds|ds_gws|s_sendmsg\b|s_movrel|v_movrel|ds_\w+_addtid", t) else []
    assert copies > 1000 and not others, others[:5]
