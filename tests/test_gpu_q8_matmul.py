"""Products of 8-bit integers: bits equal to those of the exact sums, rounded as the operator says."""
import math

import pytest
import torch

from tests import eight_bit as eb

pytestmark = pytest.mark.gpu


def _operands(n, m, k, seed):
    g = torch.Generator().manual_seed(seed)
    code = lambda r: torch.randint(-128, 128, (r, k), generator=g).to(torch.int8)    # noqa: E731
    scale = lambda r: torch.exp(torch.randn(r, generator=g)) * 1e-2                  # noqa: E731
    return code(n), scale(n), code(m), scale(m)


def _check(ops, dtype):
    import dual_ar_tts_gb300 as pkg
    y = pkg.q8_matmul(*[t.cuda() for t in ops], dtype=dtype)
    want = eb.product(*ops, dtype)
    assert torch.equal(torch.isnan(y).cpu(), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y.cpu()), torch.nan_to_num(want))


@pytest.mark.parametrize("dtype", list(eb.TYPES))
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 255, 256, 257, 300, 513])
def test_rows(n, dtype):
    _check(_operands(n, 301, 400, n), eb.TYPES[dtype])


@pytest.mark.parametrize("n", [1, 12, 32, 60, 200, 300])
@pytest.mark.parametrize("k", [16, 32, 112, 128, 144, 256, 1008, 1024, 1040, 2560, 9728])
def test_columns(n, k):
    _check(_operands(n, 150, k, k), torch.float32)


@pytest.mark.parametrize("n", [1, 12, 32, 60, 200, 300])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 127, 128, 129, 255, 256, 257, 2049])
def test_weights(n, m):
    _check(_operands(n, m, 272, m), torch.bfloat16)


@pytest.mark.parametrize("n", [3, 20, 40, 270])
@pytest.mark.parametrize("k", [1024, 1040, 4096, (1 << 17) - 16])
def test_largest_sums(n, k):
    """All codes at an end of their range: sums up to 2^31, which no rounding may touch."""
    one = torch.ones
    for a, b in ((-128, -128), (127, 127), (-128, 127)):
        x = torch.full((n, k), a, dtype=torch.int8)
        w = torch.full((130, k), b, dtype=torch.int8)
        x[1, ::7], w[5, ::3] = 1, -1
        _check((x, one(n), w, one(130)), torch.float32)


@pytest.mark.parametrize("n", [5, 100])
def test_scales(n):
    """Scales that are NaN, infinite, zero or at the ends of fp32."""
    ops = list(_operands(n, 140, 96, 5))
    ops[1][0], ops[1][1], ops[1][2], ops[1][3] = math.nan, math.inf, 0.0, 1e38
    ops[3][:6] = torch.tensor([math.nan, -math.inf, 0.0, 1e38, 1e-38, 2.0 ** -126])
    ops[2][10] = 0                       # sums of zero
    for dt in eb.TYPES.values():
        _check(ops, dt)


@pytest.mark.parametrize("n", [1, 40, 300])
def test_rows_of_matrices(n):
    """Rows of larger operands, and operands that do not start on 16 bytes."""
    import dual_ar_tts_gb300 as pkg
    x, xs, w, ws = [t.cuda() for t in _operands(n + 2, 500, 256, 8)]
    want = pkg.q8_matmul(x, xs, w, ws, dtype=torch.float32)
    got = pkg.q8_matmul(x[2:], xs[2:], w[101:400], ws[101:400], dtype=torch.float32)
    assert torch.equal(got, want[2:, 101:400])
    odd = torch.empty(w.numel() + 1, dtype=torch.int8, device="cuda")[1:].view(w.shape).copy_(w)
    assert torch.equal(pkg.q8_matmul(x, xs, odd, ws, dtype=torch.float32), want)
    out = torch.full((n + 4, 500), -7.0, device="cuda")
    pkg.q8_matmul(x, xs, w, ws, dtype=torch.float32, out=out[1:n + 3])
    assert torch.equal(out[1:n + 3], want) and (out[0] == -7).all() and (out[-1] == -7).all()


@pytest.mark.parametrize("n,m,k", [(1, 19456, 2560), (7, 6144, 2560), (32, 2560, 9728), (77, 19456, 2560), (600, 9728, 2560)])
def test_model_sizes(n, m, k):
    """Projections of the model, against the exact sums of the same codes taken on the GPU in 64 bits."""
    import dual_ar_tts_gb300 as pkg
    g = torch.Generator(device="cuda").manual_seed(n)
    x, w = [torch.randint(-128, 128, (r, k), generator=g, device="cuda").to(torch.int8) for r in (n, m)]
    xs, ws = [torch.rand(r, generator=g, device="cuda") + 0.5 for r in (n, m)]
    y = pkg.q8_matmul(x, xs, w, ws, dtype=torch.float32)
    total = x.double() @ w.double().t()
    assert torch.equal(y, total.float() * xs[:, None] * ws)
