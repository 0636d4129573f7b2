"""The experts' operators without a GPU: refusals of the C ABI and of the
binding, and the assembly of the products' kernels."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from combine_get_dispatch_amd import build as epbuild
from combine_get_dispatch_amd import ep

P16, P8, P4, P2 = (ctypes.c_void_p(v) for v in (1 << 20, (1 << 20) + 8, (1 << 20) + 4, (1 << 20) + 2))
CALLS = ("ep_expert_gemm", "ep_expert_gemm_dgrad", "ep_expert_gemm_wgrad", "ep_swiglu", "ep_swiglu_backward",
         "ep_quantize_mxfp4", "ep_dequantize_mxfp4")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ep.LIB_PATH):
        epbuild.build()
    return ep.load()


def groups(**kw):
    g = dict(offsets=P16, counts=P16, num_experts=8, num_ranks=2, cap_rows=64, region_rows=0, rows_hint=0)
    g.update(kw)
    return ep.EpGroups(*[g[n] for n, _ in ep.EpGroups._fields_])


def arguments(call, g, **kw):
    """The call's arguments, valid but for the pointers' memory, with changes by name."""
    v = dict(g=None if g is None else ctypes.byref(g), form=ep.EP_FORM_BF16, rows=P16, row_scales=None, weights=P16,
             weight_scales=None, K=256, N=64, out=P16, out_f32=1, accumulate=0, n=128, scales=None)
    v.update(kw)
    order = {"ep_expert_gemm": "g form rows row_scales weights weight_scales K N out",
             "ep_expert_gemm_dgrad": "g rows weights K N out",
             "ep_expert_gemm_wgrad": "g rows weights K N out out_f32 accumulate",
             "ep_swiglu": "g rows n K form out scales",
             "ep_swiglu_backward": "g rows weights n K out",
             "ep_quantize_mxfp4": "g rows n K out scales",
             "ep_dequantize_mxfp4": "g rows scales n K out"}[call]
    return [v[name] for name in order.split()] + [None]


def needed(call):
    return dict(scales=P16) if "mxfp4" in call else {}


@pytest.mark.parametrize("bad", [
    dict(num_experts=0), dict(num_experts=1025, num_ranks=1), dict(num_ranks=0), dict(num_ranks=65), dict(num_ranks=3),
    dict(cap_rows=-1), dict(cap_rows=1 << 30), dict(cap_rows=1 << 62), dict(region_rows=-1), dict(rows_hint=-1),
    dict(counts=None), dict(offsets=None), dict(region_rows=8), dict(region_rows=9, offsets=None),
    dict(region_rows=1 << 61, offsets=None),
])
@pytest.mark.parametrize("call", CALLS)
def test_bad_groups(lib, call, bad):
    g = groups(**bad)
    n = max(0, min(g.num_ranks * g.cap_rows, 1 << 40))
    assert getattr(lib, call)(*arguments(call, g, n=n, **needed(call))) == ep.EP_ERR_ARG


@pytest.mark.parametrize("call", CALLS)
def test_misaligned(lib, call):
    ok = needed(call)
    for name in ("rows", "out") + (("weights",) if "gemm" in call or "backward" in call else ()):
        assert getattr(lib, call)(*arguments(call, groups(), **dict(ok, **{name: P8}))) == ep.EP_ERR_ALIGN, name
    assert getattr(lib, call)(*arguments(call, groups(counts=P2), **ok)) == ep.EP_ERR_ALIGN
    assert getattr(lib, call)(*arguments(call, groups(offsets=P2), **ok)) == ep.EP_ERR_ALIGN


@pytest.mark.parametrize("call", CALLS)
def test_null_and_empty(lib, call):
    ok = needed(call)
    for name in ("rows", "out") + (("weights",) if "gemm" in call or "backward" in call else ()):
        assert getattr(lib, call)(*arguments(call, groups(), **dict(ok, **{name: None}))) == ep.EP_ERR_ARG, name
    if call != "ep_expert_gemm_wgrad":  # (whose result is zeros then)
        empty = arguments(call, groups(cap_rows=0), n=0, rows=None, weights=None, out=None)
        assert getattr(lib, call)(*empty) == ep.EP_OK
    if "gemm" in call:
        assert getattr(lib, call)(*arguments(call, None)) == ep.EP_ERR_ARG


@pytest.mark.parametrize("K,N", [(0, 64), (4, 64), (12, 64), (65544, 64), (64, 0), (64, 12), (64, 65544), (-8, 64)])
def test_bad_channels(lib, K, N):
    for call in CALLS[:3]:
        assert getattr(lib, call)(*arguments(call, groups(), K=K, N=N)) == ep.EP_ERR_ARG


def test_forms(lib):
    f = lib.ep_expert_gemm
    s = dict(row_scales=P16, weight_scales=P16)
    assert f(*arguments("ep_expert_gemm", groups(), form=3)) == ep.EP_ERR_ARG
    assert f(*arguments("ep_expert_gemm", groups(), form=-1)) == ep.EP_ERR_ARG
    assert f(*arguments("ep_expert_gemm", groups(), **s)) == ep.EP_ERR_ARG             # bf16 has no scales
    for form in (ep.EP_FORM_FP8, ep.EP_FORM_MXFP4):
        assert f(*arguments("ep_expert_gemm", groups(), form=form)) == ep.EP_ERR_ARG   # these need them
        assert f(*arguments("ep_expert_gemm", groups(), form=form, row_scales=P16)) == ep.EP_ERR_ARG
        assert f(*arguments("ep_expert_gemm", groups(), form=form, K=200, **s)) == ep.EP_ERR_ARG
        assert f(*arguments("ep_expert_gemm", groups(), form=form, **dict(s, row_scales=P2))) == ep.EP_ERR_ALIGN
    assert f(*arguments("ep_expert_gemm", groups(), form=ep.EP_FORM_MXFP4, **dict(s, row_scales=P4))) == ep.EP_ERR_ALIGN
    # an expert's regions over 4 GiB of rows: 2 * 2^14 rows of 128 KiB
    far = groups(offsets=None, region_rows=1 << 14, cap_rows=8 << 14)
    assert f(*arguments("ep_expert_gemm", far, K=65536)) == ep.EP_ERR_ARG
    assert lib.ep_expert_gemm_dgrad(*arguments("ep_expert_gemm_dgrad", far, N=65536)) == ep.EP_ERR_ARG
    w = lib.ep_expert_gemm_wgrad
    assert w(*arguments("ep_expert_gemm_wgrad", groups(), out_f32=0, accumulate=1)) == ep.EP_ERR_ARG


@pytest.mark.parametrize("form,I", [(0, 12), (0, 0), (0, 65544), (1, 64), (1, 192), (2, 48), (2, 8), (3, 128), (-1, 128)])
def test_swiglu_sizes(lib, form, I):
    s = None if form == 0 else P16
    assert lib.ep_swiglu(*arguments("ep_swiglu", groups(), form=form, K=I, scales=s)) == ep.EP_ERR_ARG


def test_row_counts(lib):
    for call in CALLS[3:]:
        f = getattr(lib, call)
        ok = needed(call)
        assert f(*arguments(call, groups(), n=127, **ok)) == ep.EP_ERR_ARG       # not the groups' rows
        assert f(*arguments(call, None, n=-1, **ok)) == ep.EP_ERR_ARG
        assert f(*arguments(call, None, n=1 << 31, **ok)) == ep.EP_ERR_ARG
    assert lib.ep_swiglu(*arguments("ep_swiglu", groups(), form=1)) == ep.EP_ERR_ARG              # no scales
    assert lib.ep_swiglu(*arguments("ep_swiglu", groups(), scales=P16)) == ep.EP_ERR_ARG          # bf16 has none
    for call in CALLS[5:]:
        assert getattr(lib, call)(*arguments(call, groups(), K=48, scales=P16)) == ep.EP_ERR_ARG  # cols % 32
        assert getattr(lib, call)(*arguments(call, groups())) == ep.EP_ERR_ARG                    # no scales


def refused(f, *a, **kw):
    with pytest.raises(ep.EpError) as e:
        f(*a, **kw)
    assert e.value.code == ep.EP_ERR_ARG


def test_binding_refuses(lib):
    """Types, shapes, strides and devices that the C ABI cannot see (here all
    tensors are on the CPU, which alone is refused)."""
    i32 = torch.zeros(8, dtype=torch.int32)
    g = ep.Groups(i32, i32, num_experts=8, num_ranks=2, cap_rows=64)
    x, w = torch.zeros(128, 64, dtype=torch.bfloat16), torch.zeros(8, 32, 64, dtype=torch.bfloat16)
    refused(ep.expert_gemm, x, w, g)
    refused(ep.swiglu, x)
    refused(ep.swiglu, x, kind="fp4")
    refused(ep.swiglu_backward, x, x)
    refused(ep.quantize_mxfp4, x)
    refused(ep.quantize_mxfp4, torch.zeros((), dtype=torch.bfloat16))
    refused(ep.dequantize_mxfp4, torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    for bad in (torch.zeros(8), torch.zeros(9, dtype=torch.int32), torch.zeros(16, dtype=torch.int32)[::2]):
        with pytest.raises(ep.EpError):
            ep.Groups(bad, i32, num_experts=8, num_ranks=2, cap_rows=64).c()


# ---------------------------------------------------------------------------
# the assembly
# ---------------------------------------------------------------------------

def registers(text):
    found = set()
    for kind, lo, hi, k, one in re.findall(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", text):
        found.update(f"{kind}{i}" for i in range(int(lo), int(hi) + 1)) if kind else found.add(k + one)
    return found


@pytest.mark.slow
def test_matrix_instructions_written_as_asm(tmp_path):
    """The compiler keeps the distances that matrix instructions need between
    each other and other instructions, except for those written as asm: no
    vector instruction may write one of their operands in the two wait states
    before, and nothing else may touch their results in the 18 after. The same
    for the copies to LDS: a vector instruction writes the scalar registers of
    their base no later than five wait states before."""
    out = str(tmp_path / "experts.s")
    subprocess.run([epbuild.hipcc()] + epbuild.flags() + ["-S", "--offload-device-only", "-o", out,
                   os.path.join(epbuild.CSRC, "ep_experts.hip")], check=True, capture_output=True)
    seen, copies, window, in_asm = 0, 0, [], False
    for line in open(out):
        t = line.strip()
        if t.startswith(";;#ASM"):
            in_asm = "START" in t
        t = t.split(";")[0].strip()
        if not t or t.endswith(":") or t.startswith("."):
            continue
        op, _, rest = t.partition(" ") if " " in t else t.partition("\t")
        operands = re.split(r",(?![^\[]*\])", rest)
        states = int(rest) + 1 if op == "s_nop" else 1
        if op in ("s_branch", "s_endpgm"):
            window = []
            continue
        entry = None
        if "mfma" in op:
            seen += in_asm
            if in_asm:
                read = registers(",".join(operands[1:]))
                late = [w for kind, w, ago in window if kind == "valu" and ago < 2 and w & read]
                assert not late, f"operand written right before: {t}"
                entry = ("asm", registers(operands[0]), 0)
        elif op.startswith("global_load_lds"):
            copies += 1
            base = {f"s{i}" for lo, hi in re.findall(r"\bs\[(\d+):(\d+)\]", rest) for i in range(int(lo), int(hi) + 1)}
            late = [w for kind, w, ago in window if kind == "scalar" and ago < 5 and w & base]
            assert not late, f"base written right before: {t}"
        elif op.startswith(("v_", "global_", "ds_", "scratch_", "buffer_")):
            touched = registers(rest)
            early = [w for kind, w, ago in window if kind == "asm" and ago < 18 and w & touched]
            assert not early, f"result touched too early: {t}"
            scalar = {f"s{i}" for i in re.findall(r"\bs(\d+)\b", operands[0])}
            scalar |= {f"s{i}" for lo, hi in re.findall(r"\bs\[(\d+):(\d+)\]", operands[0])
                       for i in range(int(lo), int(hi) + 1)}
            if op.startswith("v_"):
                entry = ("scalar", scalar, 0) if scalar else ("valu", registers(operands[0]), 0)
        window = [(k, w, ago + states) for k, w, ago in window if ago + states < 18] + ([entry] if entry else [])
    assert seen > 1000 and copies > 1000  # (there are some)
