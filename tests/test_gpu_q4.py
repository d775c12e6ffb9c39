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


MANY = [  # n, m, k, group: tiles of 32, 64 and 128 columns, their ends, split and whole sums, one code block and many
    (33, 129, 32, 32), (47, 1, 128, 128), (63, 257, 1920, 64), (127, 300, 1056, 32), (128, 128, 640, 128),
    (129, 40, 9728, 64), (200, 1000, 2688, 128), (257, 2500, 224, 32), (600, 640, 512, 64)]


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("n,m,k,group", MANY)
def test_matmul_of_many_rows(dtype, n, m, k, group):
    test_matmul(dtype, n, m, k, group)


def test_matmul_of_many_rows_takes_rows_as_they_are():
    """Every row's result does not depend on the rows beside it: not on their magnitudes, nor on what is no number."""
    import dual_ar_tts_gb300 as pkg
    codes, scales = pkg.quantize_q4(_weights(300, 1600, torch.bfloat16, 9).cuda(), 32)
    for dtype in fb.TYPES.values():
        x = torch.randn((150, 1600), generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
        clean = pkg.q4_matmul(x, codes, scales, 32)
        x[7] *= 1000
        x[20, 5], x[140, 1000], x[149] = math.nan, -math.inf, 0
        y = pkg.q4_matmul(x, codes, scales, 32)
        assert torch.isnan(y[20]).all() and not torch.isfinite(y[140]).all() and (y[149] == 0).all()
        keep = [r for r in range(149) if r not in (7, 20, 140)]
        assert torch.equal(y[keep], clean[keep])
        _check(y[7:8], x[7:8], codes, scales, 1600, 32)


def test_matmul_of_many_rows_of_weights_of_many_sizes():
    """Weight rows of magnitudes from 1e-30 to 1e30, groups a millionfold apart in a row, groups of zeros, a row of
    zeros, and a group that is no number: only its row is none."""
    import dual_ar_tts_gb300 as pkg
    m, k = 140, 1280
    w = _weights(m, k, torch.float32, 12)
    for r in range(m):
        w[r] *= 10.0 ** (r % 61 - 30)
    w[3, 32:64], w[5, :640], w[9] = 0, w[5, :640] * 1e-6, 0
    w[11, 70] = math.inf
    codes, scales = pkg.quantize_q4(w.cuda(), 32)
    x = torch.randn((70, k), generator=torch.Generator().manual_seed(8)).cuda()
    y = pkg.q4_matmul(x, codes, scales, 32)
    assert torch.isnan(y[:, 11]).all() and (y[:, 9] == 0).all()
    keep = torch.tensor([r for r in range(m) if r != 11])
    _check(y[:, keep.cuda()], x, codes[keep.cuda()], scales[keep.cuda()], k, 32)
    tail = x.clone()
    tail[:, 640:] = 0                                                   # only the small groups of row 5 count
    y = pkg.q4_matmul(tail, codes, scales, 32)
    _check(y[:, 5:6], tail, codes[5:6], scales[5:6], k, 32)


def test_matmul_of_many_rows_in_a_graph_beside_another():
    """Two captured calls on two streams, replayed at once with new inputs; a workspace of the caller's."""
    import dual_ar_tts_gb300 as pkg
    codes, scales = pkg.quantize_q4(_weights(700, 1024, torch.bfloat16, 1).cuda(), 64)
    runs = []
    for n in (100, 260):
        x, out = torch.randn((n, 1024), device="cuda"), torch.empty((n, 700), device="cuda")
        ws = torch.empty(pkg.load().s2_q4_matmul_workspace(n, 1024, pkg.S2_F32), dtype=torch.uint8, device="cuda")
        pkg.q4_matmul(x, codes, scales, 64, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkg.q4_matmul(x, codes, scales, 64, out=out, workspace=ws)
        x.copy_(torch.randn((n, 1024), device="cuda"))
        runs.append((graph, x, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, _, _, stream in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, x, out, _ in runs:
        assert torch.equal(out, pkg.q4_matmul(x, codes, scales, 64))


@pytest.mark.parametrize("dtype,n", [("bf16", 17), ("fp16", 32), ("fp32", 9), ("fp32", 16)])
@pytest.mark.parametrize("m,k,group", [(1300, 9728, 128), (5000, 2560, 64), (4930, 2560, 32)])
def test_matmul_of_large_matrices(dtype, n, m, k, group):
    """17 to 32 columns (an fp32 row is two) of matrices on both sides of 12 Mi weights."""
    test_matmul(dtype, n, m, k, group)
    test_matmul(dtype, n, (12 << 20) // k - 1, k, group)


@pytest.mark.parametrize("n,m,k,group", [(1, 3000, 128, 32), (1, 5000, 1536, 32), (3, 2000, 1536, 32), (13, 700, 1536, 32),
                                         (1, 2000, 64, 64), (2, 2000, 2560, 32), (14, 1000, 160, 32)])
def test_matmul_keeps_fp32(n, m, k, group):
    """The error of fp32 products of few rows, 2-norm over 2-norm.  A tensor core cuts a sum off at its last bit, half of
    it on average: a group of 32 (64) columns is 2 (4) such additions of 2^-24 of a partial sum.  Splitting an
    activation into two fp16 terms leaves 2^-23 / sqrt(3) of it.  At most 2560 / 32 / 2 group sums are added one by
    one, each rounding 2^-25 and independent.  4 * 2^-24 + 0.7e-7 + sqrt(40) * 2^-25 = 5e-7; 6e-7 asked."""
    import dual_ar_tts_gb300 as pkg
    for seed in range(4):
        codes, scales = pkg.quantize_q4(_weights(m, k, torch.float32, seed).cuda(), group)
        w = fb.q4_values(codes, scales, k, group)
        x = torch.randn((n, k), generator=torch.Generator().manual_seed(100 + seed))
        want = x.double() @ w.t()
        off = (pkg.q4_matmul(x.cuda(), codes, scales, group).cpu().double() - want).norm(dim=1) / want.norm(dim=1)
        assert off.max() <= 6e-7, (seed, off.max())


@pytest.mark.parametrize("n,m,k,group", [(9, 2560, 9728, 128), (40, 1300, 9728, 32), (200, 640, 9728, 32), (150, 500, 2560, 64),
                                         (17, 300, 384, 32), (70, 257, 128, 128)])
def test_matmul_of_many_rows_keeps_fp32(n, m, k, group):
    """As above for more rows.  Sums of two code blocks are 16 additions on the tensor core, each of which cuts off half of
    the last bit (2^-24 to 2^-23 of a partial sum, 0.72 * 2^-23 on average; the partial sums' sizes average 0.7 of
    the whole): 16 * 0.5 * 0.72 * 0.7 * 2^-23 = 4.8e-7, in one direction.  These are added one by one, 38 of them at
    most, and over up to eight blocks: sqrt(38 + 8) * 2^-25 = 2e-7, independent; 0.7e-7 for the split: 7.5e-7 in all, 8e-7 asked."""
    import dual_ar_tts_gb300 as pkg
    for seed in range(2):
        codes, scales = pkg.quantize_q4(_weights(m, k, torch.float32, seed).cuda(), group)
        w = fb.q4_values(codes, scales, k, group)
        x = torch.randn((n, k), generator=torch.Generator().manual_seed(100 + seed))
        want = x.double() @ w.t()
        off = (pkg.q4_matmul(x.cuda(), codes, scales, group).cpu().double() - want).norm(dim=1) / want.norm(dim=1)
        assert off.max() <= 8e-7, (seed, off.max())


@pytest.mark.parametrize("dtype,n", [("bf16", 40), ("fp16", 64), ("bf16", 300), ("fp32", 17), ("fp32", 100)])
@pytest.mark.parametrize("m,k", [(300, 2560), (300, 256), (20000, 640)])
def test_matmul_of_many_rows_whose_waits_give_up(dtype, n, m, k):
    """No tries: every wait gives up at once.  No number comes out, and the next call is as ever."""
    import dual_ar_tts_gb300 as pkg
    codes, scales = pkg.quantize_q4(_weights(m, k, torch.bfloat16, 1).cuda(), 32)
    x = torch.randn((n, k), generator=torch.Generator().manual_seed(2)).to(fb.TYPES[dtype]).cuda()
    want = pkg.q4_matmul(x, codes, scales, 32)
    out = torch.full((n + 1, m), 7.0, dtype=x.dtype, device="cuda")
    pkg.s2_set_wait_limit(0)
    try:
        pkg.q4_matmul(x, codes, scales, 32, out=out[:n])
        torch.cuda.synchronize()
    finally:
        pkg.s2_set_wait_limit(-1)
    assert torch.isnan(out[:n]).all() and (out[n] == 7).all()
    assert torch.equal(pkg.q4_matmul(x, codes, scales, 32), want) and torch.isfinite(want).all()


@pytest.mark.parametrize("dtype", list(fb.TYPES))
def test_matmul_of_one_row_of_any_stride(dtype):
    import dual_ar_tts_gb300 as pkg
    k, m = 256, 75
    codes, scales = pkg.quantize_q4(_weights(m, k, torch.float32, 3).cuda(), 32)
    wide = torch.randn((4, 260), generator=torch.Generator().manual_seed(1)).to(fb.TYPES[dtype]).cuda()
    column = wide[:2].flatten()[:2 * k].view(k, 2)
    for x in (wide[:1, :k], wide[1:2, 1:1 + k], wide[3:, 4:], column[:, :1].t(), column[:, 1:].t(), column[:, :1].clone().t()):
        _check(pkg.q4_matmul(x, codes, scales, 32), x, codes, scales, k, 32)


@pytest.mark.parametrize("dtype,n", [("bf16", 17), ("fp16", 32), ("fp32", 9)])
def test_matmul_of_larger_matrices(dtype, n):
    """The same on both sides of 32 Mi weights."""
    k = 2560
    for m in ((32 << 20) // k + 1, (32 << 20) // k - 1):
        test_matmul(dtype, n, m, k, 64)


@pytest.mark.parametrize("dtype,n", [("fp32", 1), ("bf16", 3), ("fp16", 14), ("bf16", 50), ("fp32", 70)])
@pytest.mark.parametrize("k,group", [(128, 128), (1408, 128), (2560, 128), (640, 64), (160, 32)])
def test_matmul_of_a_part_of_the_rows(k, group, dtype, n):
    """Rows of a quantised matrix, from the second, the third and the last on: their scales start on 2, 4 or 8 bytes."""
    import dual_ar_tts_gb300 as pkg
    codes, scales = pkg.quantize_q4(_weights(90, k, torch.bfloat16, 1).cuda(), group)
    x = torch.randn((n, k), generator=torch.Generator().manual_seed(2)).to(fb.TYPES[dtype]).cuda()
    for a, b in ((1, 90), (2, 33), (7, 8), (89, 90)):
        _check(pkg.q4_matmul(x, codes[a:b], scales[a:b], group), x, codes[a:b], scales[a:b], k, group)
    held = torch.empty(codes.numel() + 4, dtype=torch.uint8, device="cuda")[4:].view(codes.shape).copy_(codes)
    _check(pkg.q4_matmul(x, held, scales, group), x, codes, scales, k, group)
