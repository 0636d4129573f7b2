"""The experts' products on the values their formats end with: NaN codes and
scales, infinities, the smallest and largest scales, subnormal numbers, every
FP8 and MXFP4 code. In tiles of both widths."""
import numpy as np
import pytest
import torch

import experts_helpers as xh
from combine_get_dispatch_amd import ep

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8  # a rounding's largest relative error
SIZES = {"narrow": [5, 0, 40, 130], "wide": [5, 3000, 4400, 130]}
E = 4


def groups_for(size):
    counts = SIZES[size]
    off, cap, rows = xh.packed_groups(counts, 1, slack=3)
    g = ep.Groups(torch.tensor(counts, dtype=torch.int32).cuda(), torch.from_numpy(off).cuda(), num_experts=E, num_ranks=1,
                  cap_rows=cap, rows_hint=sum(counts))
    return g, cap, rows, 2056 if size == "wide" else 136


def product(g, x, xs, w, ws):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    out = torch.zeros((g.num_rows, w.shape[1]), dtype=torch.bfloat16, device="cuda")
    return ep.expert_gemm(dev(x), dev(w), g, row_scales=dev(xs), weight_scales=dev(ws), out=out).cpu()


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("form,K", [("fp8", 256), ("fp8", 512), ("mxfp4", 256), ("mxfp4", 384), ("mxfp4", 512)])
def test_nan_stays_where_it_is(form, K, size):
    """A NaN code or scale of a row: that row; of a weight (FP8 scale: of its 128 channels): those channels of its expert."""
    g, cap, rows, N = groups_for(size)
    rng = np.random.default_rng([K, 61])
    x, xs = xh.make_operand(rng, (cap, K), form)
    w, ws = xh.make_operand(rng, (E, N, K), form, weights=True)
    clean = product(g, x, xs, w, ws)
    assert not torch.isnan(clean).any()
    bad_rows, bad = [rows[0][1], rows[2][7], rows[3][129]], torch.zeros_like(clean, dtype=torch.bool)
    bad[bad_rows] = True
    if form == "fp8":
        x[bad_rows[0], K - 1], x[bad_rows[1], 0], xs[bad_rows[2], 1] = 0x7F, 0xFF, float("nan")
        w[2, 70, 100], ws[3, 1, 0] = 0x7F, float("nan")
        bad[rows[2], 70] = True
        bad[rows[3][0]:rows[3][-1] + 1, 128:256] = True
    else:
        xs[bad_rows[0], 0], xs[bad_rows[1], K // 32 - 1], xs[bad_rows[2], 3] = 255, 255, 255
        x[bad_rows[0], :16] = 0  # zero codes, as quantization leaves them
        ws[2, 70, 1], ws[3, N - 1, K // 32 - 1] = 255, 255
        bad[rows[2], 70] = True
        bad[rows[3], N - 1] = True
    got = product(g, x, xs, w, ws)
    assert torch.equal(torch.isnan(got), bad)
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("sx,sw", [(0, 254), (254, 0), (1, 253), (100, 27), (60, 60), (200, 60), (190, 190), (0, 0)])
@pytest.mark.parametrize("K", [384, 512])
def test_mxfp4_scales_from_end_to_end(K, sx, sw, size):
    """Scale bytes whose product is moderate, next to the fp32 range's ends, and past them."""
    g, cap, rows, N = groups_for(size)
    rng = np.random.default_rng([K, sx, sw])
    x, xs = xh.make_operand(rng, (cap, K), "mxfp4")
    w, ws = xh.make_operand(rng, (E, N, K), "mxfp4", weights=True)
    xs[:], ws[:] = sx, sw
    got = product(g, x, xs, w, ws).double()
    for e, r in enumerate(rows):
        if r:
            # the codes' product is a multiple of 1/4 below 2^15: exact in fp32, and so is its product with a power of two
            # from 2^-126 to the fp32 range's end
            exact = xh.e2m1_values(x[r]) @ xh.e2m1_values(w[e]).t() * 2.0 ** (sx + sw - 254)
            want = exact.float().to(torch.bfloat16).double()
            size_sum = xh.e2m1_values(x[r]).abs() @ xh.e2m1_values(w[e]).abs().t() * 2.0 ** (sx + sw - 254)
            # where the products' magnitudes together pass the fp32 range, so may a part of the sum, of either sign, whatever
            # the whole sum is: fp32 sums of inf and finite numbers stay inf, of both infinities are NaN
            may_pass = size_sum > torch.finfo(torch.float32).max
            inside = torch.isfinite(got[r]) & torch.isfinite(want)
            assert bool((inside | may_pass).all())
            diff = (got[r] - want).abs()[inside]
            assert bool((diff <= 2.0 ** -126).all()), float(diff.max())  # results below may be taken as 0


@pytest.mark.parametrize("size", list(SIZES))
def test_every_fp8_code(size):
    """Rows that hold one code in one channel, against weights of one: each code's value, subnormal ones too."""
    g, cap, rows, N = groups_for(size)
    K = 256
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    x = torch.zeros((cap, K), dtype=torch.uint8)
    at = torch.arange(cap)
    x[at, at * 37 % K] = codes[at % len(codes)]
    w = torch.full((E, N, K), 0x38, dtype=torch.uint8)  # 1.0
    got = product(g, x, torch.ones(cap, 2), w, torch.ones(E, (N + 127) // 128, 2)).double()
    want = x.view(torch.float8_e4m3fn).double().sum(1)  # exact in bf16
    for r in rows:
        assert torch.equal(got[r], want[r][:, None].expand(len(r), N))


@pytest.mark.parametrize("size", list(SIZES))
def test_bf16_subnormal_and_infinite_operands(size):
    g, cap, rows, N = groups_for(size)
    K = 72
    rng = np.random.default_rng(62)
    w = xh.bf16(rng, (E, N, K))
    x = torch.zeros((cap, K), dtype=torch.bfloat16)
    x[:, 3] = 2.0 ** -130   # a subnormal bf16
    w[:, :, 3] = 2.0 ** 120
    first, last = rows[0][0], rows[3][-1]
    x[first, 5], x[last, 71] = float("inf"), -float("inf")
    got = product(g, x, None, w, None).float()
    plain = torch.tensor([r for e in rows for r in e if r not in (first, last)])
    assert bool((got[plain] == 2.0 ** -10).all())
    assert torch.equal(got[first], torch.sign(w[0, :, 5].float()) * float("inf"))
    assert torch.equal(got[last], -torch.sign(w[3, :, 71].float()) * float("inf"))
