"""What the experts' binding and C ABI refuse before anything is launched, in
sizes and tensors that no GPU is needed for."""
import os

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
