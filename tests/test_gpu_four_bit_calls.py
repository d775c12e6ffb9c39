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


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("rows", [3, 600])
def test_append_of_rows_of_a_wider_tensor(rows, dtype):
    """Rows that start on 16 bytes are read where they lie, others are copied: the same bytes and queries."""
    import dual_ar_tts_gb300 as pkg
    hq, hkv, hd = 3, 2, 64
    width, dt = (hq + 2 * hkv) * hd, fb.TYPES[dtype]
    wide = torch.randn((rows, width + 24), generator=torch.Generator().manual_seed(1)).to(dt).cuda()
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    place = (torch.randperm(10, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()[None].contiguous(),
             ints(0, rows), ints(rows + 5))
    rope = pkg.rope_table(rows + 5, hd)
    for x in (wide[:, :width], wide[:, 16:16 + width], wide[:, 3:3 + width], wide[:, :width].t().contiguous().t()):
        got, want = pkg.kv4_pages(10, hkv, hd), pkg.kv4_pages(10, hkv, hd)
        q = pkg.kv4_append(x, got, *place, rope, hq)
        same = torch.empty((rows, width), dtype=dt, device="cuda").copy_(x)
        assert torch.equal(q, pkg.kv4_append(same, want, *place, rope, hq)) and torch.equal(got, want)
