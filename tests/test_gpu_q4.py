"""4-bit weights (s2_quantize_q4, s2_q4_matmul) against their definitions.

Quantisation is compared bit for bit: the scale is one fp32 division (by 8, exact but for subnormal
results) rounded to bf16, a code one fp32 division and a rounding to nearest even, the same on both
sides.  A product is held to half a step of its type plus (k/16 + 32) roundings of 2^-23 of
sum |x w|: no path of its sum, in lanes, warps or matrix instructions of 16 terms, is longer."""
import math

import pytest
import torch

from tests import four_bit as fb

pytestmark = pytest.mark.gpu


def _weights(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, cols), generator=g) * 0.02 * torch.exp(torch.randn((rows, 1), generator=g))).to(dtype)


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("rows,cols,group", [(1, 32, 32), (3, 128, 32), (5, 160, 32), (17, 320, 64), (33, 384, 128),
                                             (64, 1088, 64)])
def test_quantise_is_the_definition(dtype, rows, cols, group):
    import dual_ar_tts_gb300 as pkg
    w = _weights(rows, cols, fb.TYPES[dtype], rows + cols)
    w[0, :32] = 0
    w[rows - 1, cols - 5] = w[rows - 1].float().abs().max() * -3      # a negative extreme
    w[rows // 2, 1], w[rows // 2, 9] = 0.5, -0.5                      # a tie of the largest: the first one counts
    codes, scales = pkg.quantize_q4(w.cuda(), group)
    want_c, want_s = fb.q4_quantise(w, group)
    assert torch.equal(scales.cpu().view(torch.int16), want_s.view(torch.int16))
    assert torch.equal(codes.cpu(), want_c)
    # half a step from every weight; a whole one where the far end of the range is clipped (the scale is bf16)
    v = fb.q4_values(codes, scales, cols, group)
    s = scales.cpu().double().abs().repeat_interleave(group, 1)[:, :cols]
    assert ((v - w.double()).abs() <= s * 1.04 + 1e-300).all()


def test_quantise_edge_groups():
    import dual_ar_tts_gb300 as pkg
    w = torch.zeros((8, 128))
    w[1, 3], w[2, 40], w[3, 70] = math.nan, math.inf, -math.inf
    w[4] = 3e38
    w[5, :32] = 1e-45                                                  # the scale rounds to 0
    w[6] = torch.linspace(-1, 1, 128)
    w[7, 127] = -1e-30
    codes, scales = pkg.quantize_q4(w.cuda(), 32)
    want_c, want_s = fb.q4_quantise(w, 32)
    got = scales.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want_s))
    ok = ~torch.isnan(want_s)
    assert torch.equal(got[ok], want_s[ok]) and torch.equal(codes.cpu(), want_c)
    y = pkg.q4_matmul(torch.ones((1, 128), device="cuda"), codes, scales, 32).cpu()[0]
    assert torch.isnan(y[1:4]).all() and y[0] == 0 and torch.isfinite(y[[0, 5, 6, 7]]).all()
    assert y[4] == math.inf                                            # 128 * 3e38 is beyond fp32


SHAPES = [  # n, m, k, group
    (1, 1, 32, 32), (1, 16, 128, 128), (2, 17, 64, 64), (3, 97, 160, 32), (5, 130, 320, 64), (8, 64, 256, 32),
    (9, 33, 1088, 64), (13, 200, 96, 32), (16, 48, 640, 128), (17, 49, 416, 32), (31, 65, 384, 128), (32, 40, 2560, 32),
    (64, 100, 704, 64), (65, 19, 256, 128), (130, 36, 128, 32), (1, 2560, 9728, 128), (4, 5000, 512, 32)]


def _check(y, x, codes, scales, k, group):
    w = fb.q4_values(codes, scales, k, group)
    xd = x.cpu().double()
    want, size = xd @ w.t(), xd.abs() @ w.abs().t()
    tol = (k / 16 + 32) * 2.0 ** -23 * size + fb.rounding(want, x.dtype)
    err = (y.cpu().double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("n,m,k,group", SHAPES)
def test_matmul(dtype, n, m, k, group):
    import dual_ar_tts_gb300 as pkg
    g = torch.Generator().manual_seed(n * 7 + m)
    codes, scales = pkg.quantize_q4(_weights(m, k, torch.bfloat16, n + k).cuda(), group)
    x = torch.randn((n, k), generator=g).to(fb.TYPES[dtype])
    out = torch.full((n + 1, m), 7.0, dtype=x.dtype, device="cuda")
    y = pkg.q4_matmul(x.cuda(), codes, scales, group, out=out[:n])
    _check(y, x, codes, scales, k, group)
    assert (out[n] == 7).all()                                         # nothing behind the last row
    assert torch.equal(y, pkg.q4_matmul(x.cuda(), codes, scales, group))   # the same bits again


@pytest.mark.parametrize("dtype", list(fb.TYPES))
def test_matmul_strided_and_magnitudes(dtype):
    """Rows of a wider tensor, rows that start off a 16-byte boundary, large, tiny and cancelling activations."""
    import dual_ar_tts_gb300 as pkg
    k, m = 416, 75
    codes, scales = pkg.quantize_q4(_weights(m, k, torch.float32, 3).cuda(), 32)
    g = torch.Generator().manual_seed(5)
    wide = torch.randn((6, 2 * k + 3), generator=g).to(fb.TYPES[dtype]).cuda()
    big = 3e4 if dtype == "fp16" else 1e30
    wide[1] *= big
    wide[2] *= 1e-3 if dtype == "fp16" else 1e-30
    wide[3, 1::2] = -wide[3, 0:-1:2]
    for x in (wide[:, :k], wide[:, 8:8 + k], wide[:, 3:3 + k], wide[::2, 1:1 + k]):
        y = pkg.q4_matmul(x, codes, scales, 32)
        w = fb.q4_values(codes, scales, k, 32)
        want = x.cpu().double() @ w.t()
        fits = want.abs().amax(1) < torch.finfo(x.dtype).max
        _check(y[fits.cuda()], x[fits.cuda()], codes, scales, k, 32)


def test_matmul_non_finite_rows_stay_their_own():
    import dual_ar_tts_gb300 as pkg
    codes, scales = pkg.quantize_q4(_weights(40, 256, torch.bfloat16, 1).cuda(), 64)
    for dtype in fb.TYPES.values():
        x = torch.randn((7, 256), generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
        clean = pkg.q4_matmul(x, codes, scales, 64)
        x[2, 5], x[4, 100] = math.nan, math.inf
        y = pkg.q4_matmul(x, codes, scales, 64)
        assert torch.isnan(y[2]).all() and not torch.isfinite(y[4]).all()
        for r in (0, 1, 3, 5, 6):
            assert torch.equal(y[r], clean[r])


def test_matmul_on_another_stream_and_in_a_graph():
    import dual_ar_tts_gb300 as pkg
    codes, scales = pkg.quantize_q4(_weights(300, 512, torch.bfloat16, 1).cuda(), 32)
    x = torch.randn((3, 512), device="cuda")
    want = pkg.q4_matmul(x, codes, scales, 32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = pkg.q4_matmul(x, codes, scales, 32)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        pkg.q4_matmul(x, codes, scales, 32, out=out)
    x.copy_(torch.randn((3, 512), device="cuda"))
    graph.replay()
    assert torch.equal(out, pkg.q4_matmul(x, codes, scales, 32))
