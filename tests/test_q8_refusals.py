"""What the 8-bit calls refuse before anything is launched (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from dual_ar_tts_gb300 import build
    build.build()
    import dual_ar_tts_gb300 as pkg
    return pkg.load()


P = 0x10000                      # an aligned address that no refused call touches
EINVAL = 1


def _bad(fn, good, **changes):
    for name, values in changes.items():
        for v in values if isinstance(values, (list, tuple)) else [values]:
            args = dict(good)
            args[name] = v
            assert fn(*args.values()) == EINVAL, (name, v)


OUT = dict(codes=[None, P + 8], scales=[None, P + 2])


def test_rows(lib):
    quantise = dict(x=P, dtype=0, stride=100, rows=3, cols=100, codes=P, scales=P, stream=None)
    rows = dict(x=[None, P + 2], dtype=[3, -1], stride=[99, 0, -100], rows=[0, -1, 1 << 31], cols=[0, -1, (1 << 24) + 1])
    _bad(lib.s2_quantize_q8, quantise, **rows, **OUT)
    _bad(lib.s2_swiglu_q8, dict(quantise, stride=200), **dict(rows, stride=[199, 100, 0]), **OUT)
    _bad(lib.s2_dequantize_q8, dict(codes=P, scales=P, rows=3, cols=100, out=P, dtype=0, stream=None), rows=[0, 1 << 31],
         cols=[0, (1 << 24) + 1], out=[None, P + 2], dtype=[3], **OUT)


def test_norm(lib):
    nan, inf = float("nan"), float("inf")
    good = dict(x=P, dtype=0, stride=100, res=None, rstride=0, weight=P, eps=1e-6, rows=3, cols=100, total=None, codes=P,
                scales=P, stream=None)
    _bad(lib.s2_rms_norm_q8, good, x=[None, P + 2], dtype=[3, -1], stride=[99, 0], weight=[None, P + 2],
         eps=[-1.0, nan, inf], rows=[0, 1 << 31], cols=[0, (1 << 24) + 1], total=[P], res=[P], **OUT)
    _bad(lib.s2_rms_norm_q8, dict(good, res=P, rstride=100, total=P), res=[None, P + 1], rstride=[99, 0], total=[None, P + 2])


def test_norm_sum_in_place(lib):
    """The residual's sum may be one of the operands, not part of one, or of its rows."""
    fn, size = lib.s2_rms_norm_q8, 3 * 100 * 4
    good = dict(x=P, dtype=0, stride=100, res=4 * P, rstride=100, weight=P, eps=1e-6, rows=3, cols=100, total=8 * P, codes=P,
                scales=P, stream=None)
    assert 4 * P - P > size
    _bad(fn, good, total=[P + 4, P + 400, P + size - 4, P - size + 4, 4 * P - 4, 4 * P + size - 4])
    # rows apart: a sum over them, and over the last one's end
    apart = dict(good, stride=1000)
    _bad(fn, apart, total=[P, P + 396, P + 4000, P + 8396, P + 4000 - size + 4, P - 4])
    _bad(fn, dict(good, rstride=101), total=[4 * P])


def test_matmul(lib):
    good = dict(n=2, x=P, xs=P, w=P, ws=P, m=3, k=32, y=P, dtype=1, stream=None)
    _bad(lib.s2_q8_matmul, good, n=[0, -1, (1 << 21) - 31], x=[None, P + 8], xs=[None, P + 2], w=[None, P + 4], ws=[None, P + 1],
         m=[0, -1, (1 << 28) + 1], k=[0, -16, 8, 24, 1 << 17], y=[None, P + 1], dtype=[3, -1])


def test_python_checks():
    torch = pytest.importorskip("torch")
    import dual_ar_tts_gb300 as pkg
    x, w = torch.zeros((2, 64)), torch.zeros(64)
    c = torch.zeros((2, 64), dtype=torch.int8)
    for call in (lambda: pkg.quantize_q8(x), lambda: pkg.swiglu_q8(x), lambda: pkg.rms_norm_q8(x, w),
                 lambda: pkg.dequantize_q8(c, w[:2]), lambda: pkg.q8_matmul(c, w[:2], c, w[:2])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_python_refusals():
    import torch
    import dual_ar_tts_gb300 as pkg
    x = torch.zeros((3, 100), device="cuda")
    w = torch.ones(100, device="cuda")
    c, s = pkg.quantize_q8(x)
    i8 = dict(dtype=torch.int8, device="cuda")
    bad = [
        lambda: pkg.quantize_q8(x.double()), lambda: pkg.quantize_q8(x[0]), lambda: pkg.quantize_q8(x[:, :0]),
        lambda: pkg.quantize_q8(x, codes=torch.empty((3, 100), **i8)), lambda: pkg.quantize_q8(x, codes=c.t()),
        lambda: pkg.quantize_q8(x, codes=torch.empty(3 * 112 + 1, **i8)[1:].view(3, 112)),
        lambda: pkg.quantize_q8(x, scales=s.double()), lambda: pkg.quantize_q8(x, scales=s[:2]),
        lambda: pkg.swiglu_q8(x[:, :99]), lambda: pkg.swiglu_q8(x.int()),
        lambda: pkg.rms_norm_q8(x, w[:50]), lambda: pkg.rms_norm_q8(x, w.half()), lambda: pkg.rms_norm_q8(x, w.cpu()),
        lambda: pkg.rms_norm_q8(x, w, residual=x.half()), lambda: pkg.rms_norm_q8(x, w, residual=x[:2]),
        lambda: pkg.rms_norm_q8(x, w, total=x), lambda: pkg.rms_norm_q8(x, w, residual=x, total=x[:, ::2]),
        lambda: pkg.rms_norm_q8(x, w, residual=x, total=x.t().contiguous().t()),
        lambda: pkg.dequantize_q8(c, s, 96), lambda: pkg.dequantize_q8(c, s, 113), lambda: pkg.dequantize_q8(c, s, 0),
        lambda: pkg.dequantize_q8(c, s, dtype=torch.int8), lambda: pkg.dequantize_q8(c, s[:2]),
        lambda: pkg.dequantize_q8(c, s, 100, out=torch.empty((3, 112), device="cuda")),
        lambda: pkg.q8_matmul(c, s, c[:, :96], s), lambda: pkg.q8_matmul(c, s, c, s[:2]),
        lambda: pkg.q8_matmul(c[:, :100], s, c[:, :100], s), lambda: pkg.q8_matmul(c, s, c, s, dtype=torch.float64),
        lambda: pkg.q8_matmul(c, s.double(), c, s), lambda: pkg.q8_matmul(c.view(torch.uint8), s, c, s),
        lambda: pkg.q8_matmul(c, s, c, s, out=torch.empty((3, 3), device="cuda")),
        lambda: pkg.q8_matmul(c, s, c.cpu(), s),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(pkg.S2Error):
        pkg.rms_norm_q8(x, w, -1.0)
    # more columns than exact sums can be of
    wide = torch.zeros((1, 1 << 17), dtype=torch.int8, device="cuda")
    with pytest.raises(pkg.S2Error):
        pkg.q8_matmul(wide, s[:1], wide, s[:1])
