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
def test_gate_of_small_rows(cols, dtype):
    """Values about the least step and below, ordinary gates: codes are still the exact quotients'."""
    rows = max(4, 1_000_000 // cols)
    g, u = _rand((rows, cols), 6), _uniform((rows, cols), 7)
    u *= 2.0 ** _uniform((rows, 1), 8, -122, -117)
    _check_gate(torch.cat([g, u], 1), eb.TYPES[dtype])


@pytest.mark.parametrize("cols", COLS)
def test_gate_borders_at_the_least_step(cols):
    """Values as near as fp32 operands bring them to borders between multiples of the least step: fp32's own roundings would put many of
    them on the wrong side."""
    g = _rand((20, cols), 18).float().double()
    g = torch.where(g.abs() < 0.1, torch.full_like(g, 0.7), g)
    v = (torch.floor(_uniform((20, cols), 19, -126, 126)) + 0.5) * 2.0 ** -126
    _check_gate(torch.cat([g, v * (1 + torch.exp(-g)) / g], 1), torch.float32)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("cols", COLS)
def test_gate_below_the_range(cols, dtype):
    """Gates (and their silu) below fp32's normal range times numbers that bring the values back into it."""
    rows = max(4, 300_000 // cols)
    g, u = _rand((rows, cols), 9), _uniform((rows, cols), 10)
    g, u = g * 2.0 ** _uniform((rows, 1), 8, -140, -126), u * 2.0 ** _uniform((rows, 1), 11, 20, 127)
    _check_gate(torch.cat([g, u], 1), eb.TYPES[dtype])


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


def _check_norm(x, w, eps, dt, residual=False):
    import dual_ar_tts_gb300 as pkg
    x, w = x.to(dt), w.float()
    assert torch.isfinite(x).all() and torch.isfinite(w).all()
    res = (x.double() / 2).to(dt) if residual else None
    out = pkg.rms_norm_q8(x.cuda(), w.cuda(), eps, residual=None if res is None else res.cuda())
    eps = float(torch.tensor(eps, dtype=torch.float32))
    v, r, total = eb.norm(x, w, eps, res)
    assert ((v * r).abs() <= torch.finfo(torch.float32).max).all()
    want, scale, distance = eb.coded(v, r)
    if residual:
        assert torch.equal(out[2].cpu(), total)
    # as many additions as a thread's elements (32 of up to 1024 columns; 16, or eight of every 3328 at least), then as there
    cols = x.shape[1]
    adds = 32 if cols <= 1024 else max(16, 8 * math.ceil(cols / 3328))
    got = out[1].cpu().double()
    assert ((got - scale).abs() <= ((adds + 12) / 2 + 7) * eb.STEP * scale).all(), (got / scale)
    least = scale <= 2.0 ** -126
    eb.check_codes(out[0].cpu()[~least], want[~least], distance[~least], SURE)
    # at the least step a code is the value's, as fp32 has it: off by the factor's roundings
    tol = ((adds + 12) / 2 + 7) * eb.STEP * 127
    eb.check_codes(out[0].cpu()[least], want[least], distance[least], tol)


# (of x, of the weight, eps): all below are what a finite norm is made of
SMALL = [(1e-12, 1e-25, 1e-6), (1e-13, 1e-25, 1e-6), (1e-21, 1.0, 0.0), (1e-30, 1e-5, 0.0), (1e-37, 1.0, 0.0), (3e-39, 1e20, 1e-38),
         (1e-19, 1e-12, 1e-40),
         (1e-20, 1e-15, 1e-6), (1e-30, 1e20, 1e-20), (1.0, 1e-36, 1e-6), (1e30, 1e-30, 1e-6), (1e36, 1e-37, 0.0), (1e37, 1e3, 1e-6),
         (1e20, 1e-38, 1e-6), (1e-25, 1e-25, 1e-6),
         (1e-33, 1.0, 1e-6), (1e-36, 1.0, 1e-9), (1e-42, 1e3, 1e-12), (1e-24, 1e-24, 1e-14)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("cols", [300, 1300, 5000, 20001])
@pytest.mark.parametrize("size,weight,eps", SMALL)
def test_norm_of_factors_out_of_range(size, weight, eps, cols, dtype):
    """Squares or products with the weight that leave fp32's range while the norm does not."""
    x, w = _rand((9, cols), 14) * size, torch.exp(0.3 * _rand(cols, 15)) * weight
    _check_norm(x, w, eps, eb.TYPES[dtype], residual=cols in (300, 5000))


@pytest.mark.parametrize("cols", [300, 5000])
def test_norm_of_small_fp16_rows(cols):
    for weight, eps in ((1e-25, 1e-6), (1e-30, 0.0), (1e30, 0.0)):
        _check_norm(_rand((5, cols), 16) * 3e-7, torch.exp(0.3 * _rand(cols, 15)) * weight, eps, torch.float16, residual=True)


@pytest.mark.parametrize("cols", [300, 5000])
def test_norm_of_uneven_factors(cols):
    """Large weights meet elements that are small or nothing."""
    w = torch.full((cols,), 1e-30, dtype=torch.float64)
    x = _rand((4, cols), 17) * 1e-12
    w[0], w[1], w[2] = 3e38, 1e38, 1e20
    x[:, 0], x[1, 1], x[2, 1] = 0.0, 1e-44, 0.0
    x[[0, 3], 1] = 0.0
    x[:3, 2] = 0.0
    _check_norm(x, w, 1e-6, torch.float32)
    _check_norm(x * 2.0 ** -90, w, 0.0, torch.float32)
    for at, v in ((0, math.inf), (cols - 1, math.nan)):
        import dual_ar_tts_gb300 as pkg
        y = x.clone().float()
        y[1, at] = v
        codes, scales = pkg.rms_norm_q8(y.cuda(), w.float().cuda(), 1e-6)
        assert torch.equal(torch.isnan(scales).cpu(), torch.tensor([False, True, False, False])) and (codes[1] == 0).all()


@pytest.mark.parametrize("cols", [255, 1500, 5000])
@pytest.mark.parametrize("weight,power", [(1.1, -113), (1.1e-20, -60), (1.1e-30, -30), (1.1e-37, 20), (1.1e37, 20), (1.1, 100)])
def test_norm_halves_at_the_ends(weight, power, cols):
    """Elements under one weight: exact halves go to the even code, whatever range the products are in."""
    import dual_ar_tts_gb300 as pkg
    half = torch.arange(0.5, 127.0, 1.0, dtype=torch.float64)
    x = torch.cat([half, torch.tensor([127.0]), -half]).repeat(cols // 255 + 1)[:cols]
    codes, scales = pkg.rms_norm_q8((x * 2.0 ** power)[None].float().cuda(), torch.full((cols,), weight, device="cuda"), 0.0)
    if 1.7 * weight >= 127 * 2.0 ** -126:         # the largest of the norm: 127 / rms
        assert torch.equal(codes.cpu()[0, :cols].double(), torch.round(x))
    rms = x.square().mean().sqrt().item()
    want = float(torch.tensor(weight)) / rms
    assert abs(scales.item() / max(want, 2.0 ** -126) - 1) <= ((32 + 12) / 2 + 7) * eb.STEP


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("cols", [300, 2560, 17000])
def test_norm_rows_out_of_range_in_place(cols, which):
    """Rows past the range, whose sum lies over an operand, beside ordinary ones, whose bits are those of any other batch."""
    import dual_ar_tts_gb300 as pkg
    scale = torch.tensor([1.0, 1e30, 1e-36, 1.0, 0.0, 1e36, 1e-40, 1.0], dtype=torch.float64)[:, None]
    x, res = [(_rand((8, cols), s) * scale).float().cuda() for s in (20, 21)]
    w = torch.exp(0.3 * _rand(cols, 22)).float().cuda()
    for eps in (0.0, 1e-6):
        want = pkg.rms_norm_q8(x, w, eps, residual=res)
        v, r, total = eb.norm(x.cpu(), w.cpu(), eps, res.cpu())
        live = (total != 0).any(1) if eps == 0.0 else torch.ones(8, dtype=torch.bool)
        codes, step, distance = eb.coded(v[live], r[live])
        usual = step > 2.0 ** -126
        eb.check_codes(want[0].cpu()[live][usual], codes[usual], distance[usual], SURE)
        assert torch.equal(torch.isnan(want[1]).cpu(), ~live) and torch.equal(want[2].cpu(), total)
        a, b = x.clone(), res.clone()
        got = pkg.rms_norm_q8(a, w, eps, residual=b, total=a if which == "x" else b)
        for p, q in zip(got, want):
            assert torch.equal(p.nan_to_num(7.0) if p.is_floating_point() else p, q.nan_to_num(7.0) if q.is_floating_point() else q)
        rest = torch.tensor([0, 3, 7], device="cuda")
        alone = pkg.rms_norm_q8(x[rest], w, eps, residual=res[rest])
        for p, q in zip(alone, want):
            assert torch.equal(p, q[rest])
