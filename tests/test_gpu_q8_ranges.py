"""Rows as 8-bit integers at the ends of their types' ranges: values that fp32 holds, made of factors or through products that it does
not, against the 64-bit forms.  Tolerances are those of tests/test_gpu_q8_rows.py."""
import math

import pytest
import torch

from tests import eight_bit as eb

pytestmark = pytest.mark.gpu

SURE = 127 * 2.0 ** -41
# a warp's row, a block's, one that a block's threads do not hold whole (quantiser and gate of fp32, norms)
COLS = [200, 1500, 9728, 20001]


def _uniform(shape, seed, low=-1.0, high=1.0):
    return low + (high - low) * torch.rand(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _check_gate(x, dt):
    """x [rows][2 f] fp64, rounded to dt first."""
    import dual_ar_tts_gb300 as pkg
    x = x.to(dt)
    assert torch.isfinite(x).all()
    codes, scales = pkg.swiglu_q8(x.cuda())
    v = eb.gate(x)
    assert (v.abs() <= torch.finfo(torch.float32).max).all()
    want, scale, distance = eb.coded(v)
    assert ((scales.cpu().double() - scale).abs() <= 16 * eb.STEP * scale).all(), (scales.cpu(), scale)
    eb.check_codes(codes.cpu(), want, distance, SURE)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("cols", COLS)
def test_gate_products_past_the_range(cols, dtype):
    """gate * up passes fp32's range where silu(gate) * up does not."""
    most = torch.finfo(eb.TYPES[dtype]).max
    g, u = _rand((6, cols), 1), _uniform((6, cols), 2) * most
    g[0] = torch.where(g[0] > 0, -10.0, -80.0)
    g[1] = _uniform(cols, 3, 0.5, 1.2)                                # values up to 3.1e38
    g[2], u[2] = g[2].clamp(-3, 3), _rand(cols, 4)
    g[2, 17], u[2, 17] = -10.0, 5e37                                  # -2.3e34, alone at the top
    g[3], u[3] = g[3].clamp(-2, 1), u[3] / 100
    g[3, 5], u[3, 5] = 2.0, 1.8e38                                    # 3.17e38
    g[4] = 1.2
    g[5], u[5] = -_uniform(cols, 5, 1.0, 80.0), u[5].sign() * most
    _check_gate(torch.cat([g, u], 1), eb.TYPES[dtype])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("cols", [255, 1500])
@pytest.mark.parametrize("gate,power", [(2.03125, 120), (1.296875, -113), (-10.0625, -100), (3.015625, -122)])
def test_gate_halves_at_the_ends(gate, power, cols, dtype):
    """Elements that share their row's largest one's gate: exact halves go to the even code where the product of gate and up passes
    the range, or its last places fall below it."""
    import dual_ar_tts_gb300 as pkg
    dt = eb.TYPES[dtype]
    half = torch.arange(0.5, 64.0, 1.0, dtype=torch.float64)          # 7 bits
    up = torch.cat([half, torch.tensor([127.0]), -half]).repeat(cols // 127 + 1)[:cols]
    x = torch.cat([torch.full((cols,), gate, dtype=torch.float64), up * 2.0 ** power])[None].to(dt)
    assert torch.equal(x[0, cols:].double(), up * 2.0 ** power) and x[0, 0] == gate
    codes, scales = pkg.swiglu_q8(x.cuda())
    assert scales.item() > 2.0 ** -126 and torch.equal(codes.cpu()[0, :cols].double(), torch.round(up) * math.copysign(1, gate))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("cols", COLS)
def test_gates_as_large_as_their_type(cols, dtype):
    """A finite gate of any size is one: past 87.3 its exponential counts as nothing."""
    import dual_ar_tts_gb300 as pkg
    dt = eb.TYPES[dtype]
    most = torch.finfo(dt).max
    g, u = _rand((6, cols), 12), _rand((6, cols), 13).clamp(-4, 4)
    g[0, 3], u[0, 3] = 3e38, 0.5
    g[1, cols - 1], u[1, cols - 1] = -3e38, 2.0
    g[2], u[2] = g[2].sign() * most, u[2] / 5
    g[3], u[3] = -most, u[3] * 1e30
    g[4, 7], u[4, 7] = 2.4e38, 1e-38
    g[5] *= 1e37
    x = torch.cat([g, u], 1)
    _check_gate(x, dt)
    x = x.to(dt)
    for at, v in ((3, math.inf), (3, -math.inf), (3, math.nan), (cols + 3, math.inf), (cols + 3, math.nan)):
        y = x.clone()
        y[:, at] = v
        codes, scales = pkg.swiglu_q8(y.cuda())
        assert torch.isnan(scales).all() and (codes == 0).all(), (at, v)
