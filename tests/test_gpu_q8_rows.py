"""Rows as 8-bit integers: the quantiser, the norm and the gate with such outputs, and reading back, against their 64-bit
forms.  Codes have to be equal: the kernels decide what lies next to a border exactly."""
import math

import pytest
import torch

from tests import eight_bit as eb

pytestmark = pytest.mark.gpu

# one column, odd ones, a warp's most, a block's least, the model's, more than a block's threads hold
SHAPES = [(1, 1), (3, 7), (9, 16), (5, 250), (33, 1001), (2, 1024), (3, 1025), (4, 2560), (2, 9728), (2, 20001)]
# a quotient of the 64-bit form is off by a few 2^-53 of up to 127, the two-term sums by 2^-42 of it
SURE = 127 * 2.0 ** -41


def _rand(shape, seed, std=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std


def _rows_per_thread(cols):
    """Elements that one thread adds up, at most."""
    return 32 if cols <= 1024 else 16 + 8 * math.ceil(max(0, cols - 16384) / 8192)


@pytest.mark.parametrize("dtype", list(eb.TYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantise(rows, cols, dtype):
    import dual_ar_tts_gb300 as pkg
    x = (_rand((rows, cols), 1) * torch.exp(_rand(cols, 2))).to(eb.TYPES[dtype])
    if rows > 2:
        x[1] = 0
    codes, scales = pkg.quantize_q8(x.cuda())
    want, scale, distance = eb.coded(x.double())
    # 127 v / peak of 64 bits is within 2^-52 of 127; exact halves of 16-bit rows come out exactly
    eb.check_codes(codes.cpu(), want, distance, 127 * 2.0 ** -51 if dtype == "fp32" else 0.0)
    assert torch.equal(scales.cpu(), scale.float())
    for dt in eb.TYPES.values():
        y = pkg.dequantize_q8(codes, scales, cols, dtype=dt)
        assert torch.equal(y.cpu(), (codes.cpu()[:, :cols].float() * scales.cpu()[:, None]).to(dt))


@pytest.mark.parametrize("dtype", list(eb.TYPES))
def test_quantise_halves(dtype):
    """Quotients that are exact halves go to the even code, and their neighbours to their own sides."""
    import dual_ar_tts_gb300 as pkg
    dt = eb.TYPES[dtype]
    half = torch.arange(-126.5, 127.0, 1.0, dtype=torch.float64)
    for power in (-20, 0, 7):
        x = torch.cat([half, torch.tensor([127.0])]) * 2.0 ** power
        x = torch.stack([x, -x, x.flip(0)]).to(dt)
        exact = x.double() / 2.0 ** power
        codes, scales = pkg.quantize_q8(x.cuda())
        assert (scales == 2.0 ** power).all()
        assert torch.equal(codes.cpu()[:, :255].long(), torch.round(exact).long())     # bf16 rounds the larger halves
    if dtype == "fp32":
        up = torch.nextafter(half.float(), torch.tensor(1e9))
        down = torch.nextafter(half.float(), torch.tensor(-1e9))
        for x, want in ((up, torch.floor(half) + 1), (down, torch.ceil(half) - 1)):
            row = torch.cat([x, torch.tensor([127.0])])[None]
            assert torch.equal(pkg.quantize_q8(row.cuda())[0].cpu()[0, :254].long(), want.long())


@pytest.mark.parametrize("dtype", list(eb.TYPES))
def test_halves_of_norm_and_gate(dtype):
    """Elements that share their row's largest one's weight or gate: quotients that are exact halves go to the even code."""
    import dual_ar_tts_gb300 as pkg
    dt = eb.TYPES[dtype]
    half = torch.arange(-126.5, 127.0, 1.0, dtype=torch.float64)
    x = (torch.cat([half, torch.tensor([127.0])]) / 16).to(dt)
    x = torch.stack([x, -x, x.flip(0)])                  # bf16 rounds the larger halves
    want = torch.round(x.double() * 16).long()
    for weight in (1.0, 1.1, 0.3, 7e-3):
        w = torch.full((255,), weight, device="cuda")
        assert torch.equal(pkg.rms_norm_q8(x.cuda(), w)[0].cpu()[:, :255].long(), want)
    for gate in (2.296875, -1.3, 0.1, 11.0, -20.5, 61.0):
        g = torch.full((3, 255), gate).to(dt)
        codes = pkg.swiglu_q8(torch.cat([g, x], 1).cuda())[0]
        assert torch.equal(codes.cpu()[:, :255].long(), want * (1 if gate > 0 else -1)), gate


@pytest.mark.parametrize("dtype", list(eb.TYPES))
@pytest.mark.parametrize("cols", [40, 1300])
def test_quantise_extremes(cols, dtype):
    """The type's largest and smallest numbers; rows with an infinity or a NaN stand for NaN and leave others alone."""
    import dual_ar_tts_gb300 as pkg
    dt = eb.TYPES[dtype]
    f = torch.finfo(dt)
    x = _rand((9, cols), 3).to(dt)
    x[0] = x[0].sign() * f.max
    x[1] = (x[1].float().clamp(-3, 3) * (f.max / 4)).to(dt)
    x[2] = (x[2].float() * f.tiny).to(dt)
    x[3] = 0
    x[3, -1] = f.smallest_normal * f.eps        # the least number there is
    x[4, 17] = math.inf
    x[5, cols - 1] = -math.inf
    x[6, 3] = math.nan
    x[7] = -0.0
    codes, scales = pkg.quantize_q8(x.cuda())
    want, scale, distance = eb.coded(x.double())
    eb.check_codes(codes.cpu(), want, distance, 127 * 2.0 ** -51 if dtype == "fp32" else 0.0)
    assert torch.equal(torch.isnan(scales).cpu(), torch.tensor([False] * 4 + [True] * 3 + [False] * 2))
    live = ~torch.isnan(scale)
    assert torch.equal(scales.cpu()[live], scale[live].float())
    y = pkg.dequantize_q8(codes, scales, cols)
    assert torch.isnan(y[4:7]).all() and torch.isfinite(y[[0, 1, 2, 3, 7, 8]]).all()


@pytest.mark.parametrize("dtype", list(eb.TYPES))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm(rows, cols, residual, dtype):
    import dual_ar_tts_gb300 as pkg
    dt = eb.TYPES[dtype]
    x = (_rand((rows, cols), 4) * torch.exp(0.5 * _rand(cols, 5))).to(dt)
    res = _rand((rows, cols), 6, 2.0).to(dt) if residual else None
    w = torch.exp(0.3 * _rand(cols, 7))
    out = pkg.rms_norm_q8(x.cuda(), w.cuda(), 1e-6, residual=None if res is None else res.cuda())
    v, r, total = eb.norm(x, w, 1e-6, res)
    want, scale, distance = eb.coded(v, r)
    eb.check_codes(out[0].cpu(), want, distance, SURE)
    # the squares' sum: as many additions as a thread's elements, ten across threads; its root halves that; then the mean,
    # eps, root, reciprocal, product with the largest (itself rounded) and quotient
    tol = ((_rows_per_thread(cols) + 12) / 2 + 7) * eb.STEP
    assert ((out[1].cpu().double() - scale).abs() <= tol * scale).all()
    if residual:
        assert len(out) == 3 and torch.equal(out[2].cpu(), total)


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("cols", [136, 2560, 17000])
def test_norm_in_place(cols, which):
    import dual_ar_tts_gb300 as pkg
    x, res, w = [_rand((5, cols), s).bfloat16().cuda() for s in (8, 9, 10)]
    w = w[0].float().contiguous()
    want = pkg.rms_norm_q8(x, w, residual=res)
    target = x if which == "x" else res
    got = pkg.rms_norm_q8(x, w, residual=res, total=target)
    assert got[2] is target and all(torch.equal(a, b) for a, b in zip(got, want))


def test_norm_extremes():
    """Rows whose squares or products pass fp32's range while the norm does not; rows that are not finite; eps alone."""
    import dual_ar_tts_gb300 as pkg
    cols = 300
    x = _rand((8, cols), 11)
    x[0] *= 1e30                     # squares past the range
    x[1] *= 1e-30                    # squares below it: eps is what is left
    x[2] = 0
    x[3, 5] = math.inf
    x[4, 6] = math.nan
    x[5] *= 1e37
    w = 1 + 0.1 * _rand(cols, 12)
    for weight, eps in ((w, 1e-6), (w * 1e25, 1e-6), (w * 1e-25, 1e-5)):
        codes, scales = pkg.rms_norm_q8(x.cuda(), weight.cuda(), eps)
        v, r, _ = eb.norm(x, weight, eps)
        want, scale, distance = eb.coded(v, r)
        bad = torch.tensor([i in (3, 4) for i in range(8)])
        assert torch.equal(torch.isnan(scales).cpu(), bad) and torch.equal(torch.isnan(scale), bad)
        usual = ~bad & (scale > 2.0 ** -126)
        eb.check_codes(codes.cpu()[usual], want[usual], distance[usual], SURE)
        tol = ((32 + 12) / 2 + 7) * eb.STEP
        assert ((scales.cpu().double() - scale).abs()[~bad] <= tol * scale[~bad]).all()
        assert (codes[3:5] == 0).all() and (codes[2] == 0).all()
        # where the scale is at its least, a code is off by the value's own roundings at most
        rest = ~bad & ~usual
        assert ((codes.cpu()[rest][:, :cols].long() - want[rest]).abs() <= 1).all()
    # a norm past fp32's range
    codes, scales = pkg.rms_norm_q8(x[:1].cuda(), (w * 3e38).clamp(max=3.4e38).cuda(), 0.0)
    assert torch.isnan(scales).all() and (codes == 0).all()
    codes, scales = pkg.rms_norm_q8(torch.zeros((2, 40), device="cuda"), torch.ones(40, device="cuda"), 0.0)
    assert torch.isnan(scales).all() and (codes == 0).all()      # 0 / 0


@pytest.mark.parametrize("dtype", list(eb.TYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_gate(rows, cols, dtype):
    import dual_ar_tts_gb300 as pkg
    x = _rand((rows, 2 * cols), 13, 1.5).to(eb.TYPES[dtype])
    codes, scales = pkg.swiglu_q8(x.cuda())
    want, scale, distance = eb.coded(eb.gate(x))
    eb.check_codes(codes.cpu(), want, distance, SURE)
    assert ((scales.cpu().double() - scale).abs() <= 16 * eb.STEP * scale).all()


def test_gate_many():
    """Ten million elements whose quotients come as near to a border as chance has it."""
    import dual_ar_tts_gb300 as pkg
    x = _rand((512, 2 * 9728), 14, 2.0)
    codes, scales = pkg.swiglu_q8(x.cuda())
    want, _, distance = eb.coded(eb.gate(x))
    assert (distance < 1e-6).any()
    eb.check_codes(codes.cpu(), want, distance, SURE)


def test_gate_extremes():
    import dual_ar_tts_gb300 as pkg
    cols = 200
    x = _rand((10, 2 * cols), 15)
    x[0, :cols] *= 40                       # from nothing to the identity
    x[1, :cols] = -90 - x[1, :cols].abs()   # silu below 2^-126
    x[2, :cols] = torch.linspace(-87, -60, cols)
    x[3, :cols] = torch.linspace(55, 65, cols)
    x[4] *= 1e30                            # products past fp32's range
    x[5, 3] = math.inf
    x[6, cols + 3] = -math.inf
    x[7, 3] = math.nan
    x[8] = 0
    x[9, :cols] *= 1e-20
    codes, scales = pkg.swiglu_q8(x.cuda())
    v = eb.gate(x)
    want, scale, distance = eb.coded(v)
    bad = torch.tensor([i in (4, 5, 6, 7) for i in range(10)])
    assert torch.equal(torch.isnan(scales).cpu(), bad) and (codes[4:8] == 0).all()
    usual = torch.tensor([0, 2, 3, 8, 9])
    eb.check_codes(codes.cpu()[usual], want[usual], distance[usual], SURE)
    assert ((scales.cpu().double() - scale).abs()[usual] <= 16 * eb.STEP * scale[usual]).all()
    # exp(-|g|) below 2^-126 has few bits
    assert ((codes.cpu()[1, :cols].float() * scales.cpu()[1]).double() - v[1]).abs().max() <= 2.0 ** -120


@pytest.mark.parametrize("dtype", list(eb.TYPES))
@pytest.mark.parametrize("cols", [48, 250, 2560])
def test_rows_of_other_tensors(cols, dtype):
    """Rows anywhere in a wider tensor, of any alignment, columns apart, and a single row of any stride."""
    import dual_ar_tts_gb300 as pkg
    dt = eb.TYPES[dtype]
    wide = _rand((7, 2 * cols + 24), 16).to(dt).cuda()
    res = _rand((7, 2 * cols + 9), 17).to(dt).cuda()
    w = (1 + 0.1 * _rand(cols + 3, 18)).cuda()
    for x in (wide, wide[:, 1:], wide[:, 8:], wide[::2], wide.t().contiguous().t(), wide[:1], wide[2:3, 3:]):
        part, gates, n = x[:, :cols], x[:, :2 * cols], x.shape[0]
        same = lambda t: torch.empty(t.shape, dtype=t.dtype, device="cuda").copy_(t)   # noqa: E731
        for a, b in zip(pkg.quantize_q8(part), pkg.quantize_q8(same(part))):
            assert torch.equal(a, b)
        for a, b in zip(pkg.swiglu_q8(gates), pkg.swiglu_q8(same(gates))):
            assert torch.equal(a, b)
        for o in (0, 1, 3):
            weight, r = w[o:o + cols], res[:n, o:o + cols]
            for a, b in zip(pkg.rms_norm_q8(part, weight, residual=r),
                            pkg.rms_norm_q8(same(part), same(weight), residual=same(r))):
                assert torch.equal(a, b)
            for a, b in zip(pkg.rms_norm_q8(part, weight), pkg.rms_norm_q8(same(part), same(weight))):
                assert torch.equal(a, b)


def test_outputs_given():
    """Given outputs are the ones written, whole, and nothing around them."""
    import dual_ar_tts_gb300 as pkg
    x = _rand((3, 100), 19).cuda()
    room = torch.full((5, 112), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((5,), -1.0, device="cuda")
    got = pkg.quantize_q8(x, codes=room[1:4], scales=scales[1:4])
    want = pkg.quantize_q8(x)
    assert torch.equal(room[1:4], want[0]) and torch.equal(scales[1:4], want[1])
    assert (room[0] == 77).all() and (room[4] == 77).all() and scales[0] == -1 and scales[4] == -1
    assert got[0].data_ptr() == room[1:4].data_ptr()
    y = torch.full((5, 100), -1.0, device="cuda")
    pkg.dequantize_q8(*want, 100, out=y[1:4])
    assert (y[0] == -1).all() and (y[4] == -1).all() and torch.equal(y[1:4], pkg.dequantize_q8(*want, 100))


@pytest.mark.parametrize("dtype", list(eb.TYPES))
def test_no_rows(dtype):
    import dual_ar_tts_gb300 as pkg
    x = torch.empty((0, 100), dtype=eb.TYPES[dtype], device="cuda")
    w = torch.ones(100, device="cuda")
    codes, scales = pkg.quantize_q8(x)
    assert codes.shape == (0, 112) and scales.shape == (0,)
    assert pkg.dequantize_q8(codes, scales, 100).shape == (0, 100)
    assert [t.shape for t in pkg.rms_norm_q8(x, w, residual=x)] == [(0, 112), (0,), (0, 100)]
    assert pkg.swiglu_q8(x)[0].shape == (0, 64)
    weights = pkg.quantize_q8(torch.randn((5, 100), device="cuda"))
    assert pkg.q8_matmul(codes, scales, *weights).shape == (0, 5)
    assert pkg.q8_matmul(*weights, codes, scales).shape == (5, 0)


def test_many_short_rows():
    """More rows than a launch's other dimensions could count."""
    import dual_ar_tts_gb300 as pkg
    x = torch.randn((600_001, 3), device="cuda")
    codes, scales = pkg.quantize_q8(x)
    want, scale, distance = eb.coded(x.cpu().double())
    eb.check_codes(codes.cpu(), want, distance, 127 * 2.0 ** -51)
    assert torch.equal(scales.cpu(), scale.float())
    assert torch.equal(pkg.dequantize_q8(codes, scales, 3), codes[:, :3].float() * scales[:, None])


def test_norm_sum_between_rows():
    """A sum that lies between the operand's rows, and in the operand of a single row, is taken."""
    import dual_ar_tts_gb300 as pkg
    x, r, w = _rand((3, 700), 1), _rand((3, 100), 2).cuda(), torch.ones(100, device="cuda")
    want = pkg.rms_norm_q8(x[:, :100].cuda(), w, residual=r)
    held = x.cuda()
    total = held.view(-1)[100:400].view(3, 100)       # behind the first row, before the second
    got = pkg.rms_norm_q8(held[:, :100], w, residual=r, total=total)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(held.cpu()[:, :100], x[:, :100]) and torch.equal(total, want[2])
    one = x.cuda()[:1, :100]
    got = pkg.rms_norm_q8(one, w, residual=r[:1], total=one)
    assert torch.equal(one, want[2][:1]) and torch.equal(got[0], want[0][:1])
    with pytest.raises(pkg.S2Error):
        pkg.rms_norm_q8(held[:, :100], w, residual=r, total=held.view(-1)[600:900].view(3, 100))


@pytest.mark.parametrize("dtype", list(eb.TYPES))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("cols", [4097, 5000, 9985, 17003])
def test_wide_norms(cols, residual, dtype):
    """More rows than SMs, wider than a block holds, or than it is by one; a row has the same bits in any batch."""
    import dual_ar_tts_gb300 as pkg
    rows, dt = 160, eb.TYPES[dtype]
    x, w = _rand((rows, cols), cols).to(dt), torch.exp(0.3 * _rand(cols, 7))
    res = _rand((rows, cols), 6, 2.0).to(dt) if residual else None
    call = lambda a, b: pkg.rms_norm_q8(a.cuda(), w.cuda(), 1e-6, residual=None if b is None else b.cuda())    # noqa: E731
    out = call(x, res)
    v, r, total = eb.norm(x, w, 1e-6, res)
    want, scale, distance = eb.coded(v, r)
    eb.check_codes(out[0].cpu(), want, distance, SURE)
    # a thread adds eight elements of every 3328 at least, the others as above
    tol = ((8 * math.ceil(cols / 3328) + 12) / 2 + 7) * eb.STEP
    assert ((out[1].cpu().double() - scale).abs() <= tol * scale).all()
    if residual:
        assert torch.equal(out[2].cpu(), total)
    for at in (slice(0, 1), slice(3, 10)):
        for a, b in zip(call(x[at], None if res is None else res[at]), out):
            assert torch.equal(a, b[at])
