"""Plain 64-bit forms of the 8-bit operators, for the tests (see include/s2frame.h), on the CPU."""
import numpy as np
import torch

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
STEP = 2.0 ** -24          # half a step of fp32, relative


def pitch(cols):
    return -(-cols // 16) * 16


def coded(v, factor=1.0):
    """Rows v * factor (fp64) -> (codes int64, scales fp64, distance of each quotient to a border between codes).
    factor [rows, 1] is common to a row."""
    peak = v.abs().amax(-1, keepdim=True)
    step = (peak * factor / 127).clamp(min=2.0 ** -126)
    small = peak * factor < 127 * 2.0 ** -126
    q = torch.where(small, v * factor / step, 127 * v / peak.clamp(min=2.0 ** -1000))
    code = torch.round(q)
    bad = ~torch.isfinite(v).all(-1, keepdim=True) | ~torch.isfinite((step.float()))
    code = torch.where(bad, torch.zeros_like(code), code)
    most = np.nextafter(np.finfo(np.float32).max / np.float32(127), np.float32(0))       # what 127 times is finite
    scale = torch.where(bad, torch.full_like(step, float("nan")), step.clamp(max=float(most)))[:, 0]
    return code.long(), scale, 0.5 - (q - torch.round(q)).abs()


def norm(x, weight, eps, residual=None):
    """(products h w, the rows' factor, total)"""
    total = x if residual is None else (residual.double() + x.double()).to(x.dtype)
    h = total.double()
    r = 1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    return h * weight.double(), r, total


def gate(x):
    f = x.shape[1] // 2
    g, u = x[:, :f].double(), x[:, f:].double()
    return g / (1 + torch.exp(-g)) * u


def product(x_codes, x_scales, codes, scales, dtype):
    """The operator's own roundings on the exact sums: equal to the last bit."""
    total = x_codes.numpy().astype(np.float64) @ codes.numpy().astype(np.float64).T     # whole numbers below 2^53
    assert np.abs(total).max() < 2.0 ** 31
    y = total.astype(np.float32) * x_scales.numpy()[:, None] * scales.numpy()
    return torch.from_numpy(y).to(dtype)


def check_codes(got, want, distance, sure=0.0):
    """Codes are equal, but where a quotient is within `sure` of a border (the 64-bit form's own roundings)."""
    cols = want.shape[1]
    assert got.shape[1] == pitch(cols) and (got[:, cols:] == 0).all()
    off = got[:, :cols].long() != want
    assert not (off & (distance > sure)).any(), int((off & (distance > sure)).sum())
