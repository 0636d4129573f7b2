"""Inputs and plain 64-bit forms for the tests of the experts' operators
(grouped products, SwiGLU, MXFP4). CPU only; no code of the library."""
from __future__ import annotations

import numpy as np
import torch


def bf16(rng, shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(scale)).to(torch.bfloat16)


def e4m3(rng, shape, scale=100.0):
    v = torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(scale)).clamp(-448, 448)
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def e2m1_values(q: torch.Tensor) -> torch.Tensor:
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    return table[torch.stack((q & 15, q >> 4), -1).flatten(-2).long()]


def mx_values(q, scales):
    """float64 values of packed e2m1 codes and e8m0 scale bytes (255: NaN)."""
    s = torch.ldexp(torch.ones(scales.shape, dtype=torch.float64), scales.to(torch.int32) - 127)
    s[scales == 255] = float("nan")
    v = e2m1_values(q)
    return (v.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def mx_quantized(x):
    """(q, scales) of float64 values [.., 32 n] by the rule: exact in 64 bits, one element at a time."""
    b = x.double().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    exponent = torch.frexp(torch.where(bad, 1.0, amax)).exponent - 1
    e = torch.where(amax > 0, exponent - 2, torch.full_like(exponent, -127)).clamp(min=-127)
    v = torch.ldexp(torch.where(bad.unsqueeze(-1), 0.0, b), -e.unsqueeze(-1))
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    dist = (v.abs().unsqueeze(-1) - values).abs()
    # nearest, ties to the even code: an odd code at the same distance loses
    code = (dist + torch.tensor([0, 1, 0, 1, 0, 1, 0, 1]) * 1e-12).argmin(-1)
    code = torch.where(torch.signbit(b) & ~bad.unsqueeze(-1), code + 8, code).flatten(-2).to(torch.uint8)
    scales = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def packed_groups(counts, R, slack=5):
    """Offsets, cap_rows and each expert's rows for counts [E] on R ranks."""
    E = len(counts)
    per = np.asarray(counts).reshape(R, E // R)
    off = (np.cumsum(per, 1) - per).reshape(-1).astype(np.int32)
    cap = int(per.sum(1).max()) + slack
    rows = [list(range((e // (E // R)) * cap + off[e], (e // (E // R)) * cap + off[e] + counts[e])) for e in range(E)]
    return off, cap, rows


def region_groups(counts, region):
    """cap_rows and each expert's rows for counts [E, R] of regions of `region` rows."""
    E, R = counts.shape
    rows = [[(e * R + s) * region + i for s in range(R) for i in range(counts[e, s])] for e in range(E)]
    return E * region, rows


def operand(q, scales, form, weights=False):
    """float64 values of a product's operand."""
    if form == "bf16":
        return q.double()
    if form == "mxfp4":
        return mx_values(q, scales)
    v = q.view(torch.float8_e4m3fn).double()
    s = scales.double().repeat_interleave(128, -1)
    if weights:
        s = s.repeat_interleave(128, -2)[..., :v.shape[-2], :]
    return v * s


def make_operand(rng, shape, form, weights=False):
    """Random (q, scales) [.., K] of a form; weights [E, N, K] get 128 x 128 scales."""
    K = shape[-1]
    if form == "bf16":
        return bf16(rng, shape), None
    if form == "fp8":
        sshape = (shape[0], (shape[1] + 127) // 128, K // 128) if weights else shape[:-1] + (K // 128,)
        s = torch.from_numpy(np.exp2(rng.uniform(-9, -5, sshape)).astype(np.float32))
        return e4m3(rng, shape), s
    q = torch.from_numpy(rng.integers(0, 256, shape[:-1] + (K // 2,), dtype=np.uint8))
    s = torch.from_numpy(rng.integers(120, 130, shape[:-1] + (K // 32,), dtype=np.uint8))
    return q, s
