"""Logits adjusted before a draw (s2_adjust_logits) against the definition in 64 bits: at most five fp32
roundings of terms no larger than |l| * rep + freq * c + pres + |bias|."""
import math

import numpy as np
import pytest
import torch

from tests import four_bit as fb

pytestmark = pytest.mark.gpu


def _want(x, hist, hist_len, pen, bias, mask, entry):
    x = x.double().numpy().copy()
    size = np.abs(x)
    rows, n = x.shape
    for r in range(rows):
        if hist is not None:
            rep, freq, pres = [float(v) for v in pen[r]]
            ln = hist.shape[1] if hist_len is None else min(max(int(hist_len[r]), 0), hist.shape[1])
            count = np.zeros(n)
            for t in hist[r, :ln].tolist():
                e = entry(t)
                if e is not None:
                    count[e] += 1
            hit = count > 0
            with np.errstate(invalid="ignore"):
                y = np.where(x[r] > 0, x[r] / rep, x[r] * rep) - freq * count - pres
            size[r] = np.where(hit, size[r] * max(rep, 1 / rep) + abs(freq) * count + abs(pres), size[r])
            x[r] = np.where(hit, y, x[r])
    if bias is not None:
        size = size + bias.double().abs().numpy()
        x = x + bias.double().numpy()
    if mask is not None:
        i = np.arange(n)
        bits = (mask.numpy().view(np.uint32)[:, i // 32] >> (i % 32).astype(np.uint32)) & 1
        x = np.where(np.broadcast_to(bits, x.shape) != 0, x, -math.inf)
    return x, size


def _compare(y, x, size):
    y = y.cpu().double().numpy()
    assert np.array_equal(np.isnan(y), np.isnan(x))
    fin = np.isfinite(x)
    assert np.array_equal(y[~fin & ~np.isnan(x)], x[~fin & ~np.isnan(x)])
    assert (np.abs(y[fin] - x[fin]) <= 5 * 2.0 ** -24 * size[fin] * 1.01).all()


CASES = [  # rows, n, hist columns, shared bias, shared mask, (sem_begin, im_end)
    (1, 1, 1, True, True, (-1, 0)), (1, 33, 5, False, False, (-1, 0)), (3, 65, 64, True, False, (4096, 4160)),
    (2, 4097, 10, False, True, (151678, 151645)), (5, 4096, 300, True, True, (-1, 0)),
    (4, 2049, 2048, False, False, (-1, 0)), (7, 20011, 513, True, False, (-1, 0)), (2, 155776, 4096, False, False, (-1, 0))]


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("rows,n,cols,one_bias,one_mask,ids", CASES)
def test_adjust(dtype, rows, n, cols, one_bias, one_mask, ids):
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(rows * n + cols)
    sem, end = ids
    x = torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32) * 4).to(fb.TYPES[dtype])
    x[0, 0] = -math.inf
    x[rows - 1, n - 1] = math.nan
    x[rows // 2, n // 2] = math.inf
    base = 0 if sem < 0 else sem
    hist = base + rng.integers(0, max(1, n // 3), (rows, cols)).astype(np.int32)
    hist[:, 0] = base + n - 1 if sem < 0 else end
    if cols > 3:
        hist[:, 1], hist[:, 2], hist[:, 3] = -5, base + n + 7, 2 ** 31 - 1     # ids that no entry has
    hist_len = rng.integers(0, cols + 1, rows).astype(np.int32)
    hist_len[0] = cols
    if rows > 2:
        hist_len[1], hist_len[2] = 0, cols + 100                               # empty; longer than its row
    pen = np.stack([rng.uniform(0.8, 1.5, rows), rng.uniform(-0.2, 0.6, rows), rng.uniform(-0.2, 0.6, rows)], 1).astype(np.float32)
    bias = torch.from_numpy(rng.standard_normal((1 if one_bias else rows, n)).astype(np.float32))
    bias[0, n // 3] = -math.inf
    mask = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (1 if one_mask else rows, -(-n // 32))).astype(np.int32))

    def entry(t):
        if sem < 0:
            return t if 0 <= t < n else None
        if t == end:
            return n - 1
        return t - sem if 0 <= t - sem < n - 1 else None

    th, tl, tp = torch.from_numpy(hist), torch.from_numpy(hist_len), torch.from_numpy(pen)
    for use_h, use_l, use_b, use_m in ((1, 1, 1, 1), (1, 0, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (0, 0, 0, 0)):
        kw = dict(sem_begin=sem, im_end=end)
        if use_h:
            kw.update(history=th.cuda(), penalties=tp.cuda(), hist_len=tl.cuda() if use_l else None)
        if use_b:
            kw["bias"] = bias.cuda()
        if use_m:
            kw["mask"] = mask.cuda()
        want, size = _want(x, th if use_h else None, tl if use_l else None, tp, bias if use_b else None,
                           mask if use_m else None, entry)
        _compare(pkg.adjust_logits(x.cuda(), **kw), want, size)


def test_adjust_in_place_rows_without_entries_and_the_draw():
    """In place on fp32; a mask that leaves a row nothing; the draw takes the result (one entry allowed wins)."""
    import dual_ar_tts_gb300 as pkg
    n = 4097
    x = torch.randn((3, n), device="cuda")
    mask = torch.zeros((3, -(-n // 32)), dtype=torch.int32, device="cuda")
    mask[1, 2049 // 32] = 1 << (2049 % 32)
    mask[2, (n - 1) // 32] = 1 << ((n - 1) % 32)
    want = pkg.adjust_logits(x, mask=mask)
    got = pkg.adjust_logits(x, mask=mask, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)
    ids = pkg.draw(got, torch.ones((3, 30), device="cuda"), 0.7, 0.9, 151678, 151645).tolist()
    assert ids == [-1, 151678 + 2049, 151645]


def test_adjust_strided_rows_and_empty_history():
    import dual_ar_tts_gb300 as pkg
    wide = torch.randn((4, 300), device="cuda").bfloat16()
    x = wide[::2, 5:260]
    hist = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    y = pkg.adjust_logits(x, history=hist, penalties=torch.ones((2, 3), device="cuda"))
    assert torch.equal(y, x.float())
