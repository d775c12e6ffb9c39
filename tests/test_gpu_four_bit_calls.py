"""Calls of the 4-bit operators that nothing is to be done for, and what they leave alone."""
import pytest
import torch

from tests import four_bit as fb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(fb.TYPES))
def test_no_rows(dtype):
    """An empty batch: empty results of the right shapes, checked as others are, and pages as they were."""
    import dual_ar_tts_gb300 as pkg
    dt = fb.TYPES[dtype]
    none = lambda *shape: torch.empty(shape, dtype=dt, device="cuda")   # noqa: E731
    codes, scales = pkg.quantize_q4(none(0, 256), 64)
    assert codes.shape == (0, 128) and scales.shape == (0, 4)
    assert pkg.q4_matmul(none(3, 256), codes, scales, 64).shape == (3, 0)
    codes, scales = pkg.quantize_q4(torch.randn((5, 256), device="cuda").to(dt), 64)
    y = pkg.q4_matmul(none(0, 256), codes, scales, 64)
    assert y.shape == (0, 5) and y.dtype == dt
    pages = pkg.kv4_pages(2, 2, 64)
    pages.fill_(7)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for place in ((ints(0, 1).view(2, 1), ints(0, 0, 0), ints(5, 0)),
                  (torch.empty((0, 1), dtype=torch.int32, device="cuda"), ints(0), ints())):
        q = pkg.kv4_append(none(0, 6 * 64), pages, *place, pkg.rope_table(8, 64), 2)
        assert q.shape == (0, 2, 64) and q.dtype == dt and (pages == 7).all()
        k, v = pkg.kv4_read(pages, *place, 0)
        assert k.shape == v.shape == (2, 0, 64)
        assert pkg.kv4_attention(q, pages, *place).shape == (0, 2, 64)
    assert pkg.adjust_logits(none(0, 9)).shape == (0, 9) and pkg.adjust_logits(none(4, 0)).shape == (4, 0)
    with pytest.raises(ValueError):
        pkg.q4_matmul(none(0, 128), codes, scales, 64)
    with pytest.raises(ValueError):
        pkg.kv4_append(none(0, 5 * 64), pages, *place, pkg.rope_table(8, 64), 2)
