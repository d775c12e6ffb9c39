"""More of the paged 4-bit cache: attention where sequences bring many rows (its own kernel) over bad pages, lengths past
the page table, hints, pools past 32 bits and many splits; one position against thousands in both kernels; appending
hundreds of rows.  Bounds: tests/four_bit.py."""
import math

import numpy as np
import pytest
import torch

from tests import four_bit as fb
from tests import test_gpu_kv4 as kv

pytestmark = pytest.mark.gpu


def _made(spans, hq, hkv, hd, dtype, seed, extra=3, cols=0):
    rng = np.random.default_rng(seed)
    table, q_start, lengths, pool = kv._layout(spans, rng, extra, cols)
    pages = torch.zeros((pool, hkv, 80 * hd), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    q = torch.from_numpy(rng.standard_normal((int(q_start[-1]), hq, hd)).astype(np.float32) * 1.5).to(fb.TYPES[dtype])
    return q, pages, table, q_start, lengths


def _check_present(got, q, pages, table, q_start, lengths, scale, dt, most=None):
    """As kv._check_attention, over the positions whose page is in the pool and in the first `most` of a sequence."""
    hq, hkv, pool = q.shape[1], pages.shape[1], pages.shape[0]
    for s, length in enumerate(int(v) for v in lengths):
        a, b = int(q_start[s]), int(q_start[s + 1])
        upto = min(length, most or length)
        there = [0 <= int(table[s, t // 64]) < pool for t in range(upto)]
        before = np.cumsum([0] + there)                              # positions present below t
        seen = [int(before[min(max(length - (b - a) + i + 1, 0), upto)]) for i in range(b - a)]
        ids = [int(p) if 0 <= int(p) < pool else 0 for p in table[s, :-(-upto // 64)]]
        if not any(there):
            assert (got[a:b] == 0).all()
            continue
        for h in range(hq):
            k, v = [fb.get(pages[:, h // (hq // hkv)][:, None], part, ids)[0, :upto][there] for part in range(2)]
            o, rel, wv, tiny = fb.attention(q[a:b, h], k, v, seen, scale)
            err = (got[a:b, h].cpu().double() - o).abs()
            assert (err <= fb.attention_tol(o, rel, wv, tiny, dt)).all(), (s, h)


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("hd", [64, 128])
def test_bad_pages_are_not_attended(hd, dtype):
    import dual_ar_tts_gb300 as pkg
    q, pages, table, q_start, lengths = _made([(70, 500), (130, 130), (40, 2000), (64, 64)], 8, 2, hd, dtype, 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = table.copy()
    bad[0, 2], bad[0, 7], bad[1, 0], bad[2, 5:9], bad[2, 30] = len(pages), -1, -1, 2 ** 31 - 1, -2 ** 31
    bad[3, 0] = -5                                                   # nothing is left to see
    got = kv._attend(pkg, q, pages, bad, q_start, lengths, status=status)
    assert int(status) == pkg.S2_EINVAL
    assert (got[200 + 40:] == 0).all()
    _check_present(got, q, pages, bad, q_start, lengths, hd ** -0.5, fb.TYPES[dtype])


@pytest.mark.parametrize("dtype", list(fb.TYPES))
def test_lengths_past_the_page_table(dtype):
    """Positions behind the table's pages are not attended; the others are, at the rows' own positions."""
    import dual_ar_tts_gb300 as pkg
    q, pages, table, q_start, _ = _made([(100, 640), (30, 640), (50, 600)], 4, 2, 64, dtype, 2)
    lengths = np.asarray([690, 5000, 600], np.int32)                 # rows from 591, 4971 and 551 on; the table ends at 640
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kv._attend(pkg, q, pages, table, q_start, lengths, status=status)
    assert int(status) == pkg.S2_EINVAL
    _check_present(got, q, pages, table, q_start, lengths, 0.125, fb.TYPES[dtype], most=640)


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("hd,hq,hkv", [(64, 8, 2), (128, 8, 1), (128, 12, 4)])
def test_many_splits_and_hints(hd, hq, hkv, dtype):
    """16 rows over thousands of positions: more splits than one warp joins; hints below, at and above the length."""
    import dual_ar_tts_gb300 as pkg
    q, pages, table, q_start, lengths = _made([(16, 7000), (20, 3), (18, 1500)], hq, hkv, hd, dtype, 3, cols=120)
    for hint in (0, 64, 700, 7000, 100000):
        got = kv._attend(pkg, q, pages, table, q_start, lengths, max_len=hint)
        _check_present(got, q, pages, table, q_start, lengths, hd ** -0.5, fb.TYPES[dtype])
        assert torch.equal(got, kv._attend(pkg, q, pages, table, q_start, lengths, max_len=hint))


def test_shared_pages_and_a_pool_past_32_bits():
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(21)
    n_pages, hd = (1 << 32) // (80 * 128) + 50, 128
    small = torch.zeros((6, 1, 80 * hd), dtype=torch.uint8)
    fb.fill_random(small, rng)
    pages = torch.empty((n_pages, 1, 80 * hd), dtype=torch.uint8, device="cuda")
    first = n_pages - 6
    pages[first:] = small.cuda()
    local = np.asarray([[0, 1, 2], [0, 1, 3], [4, 5, -1]], np.int32)
    table = np.where(local >= 0, local + first, -1).astype(np.int32)
    q_start, lengths = np.asarray([0, 70, 110, 200], np.int32), np.asarray([170, 190, 90], np.int32)
    for dtype, dt in fb.TYPES.items():
        q = torch.from_numpy(rng.standard_normal((200, 4, hd)).astype(np.float32)).to(dt)
        got = pkg.kv4_attention(q.cuda(), pages, *kv._gpu(table, q_start, lengths))
        kv._check_attention(got, q, small, local, q_start, lengths, hd ** -0.5, dt)
    del pages
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", list(fb.TYPES))
def test_captured_and_replayed_with_other_lengths(dtype):
    import dual_ar_tts_gb300 as pkg
    q, pages, table, q_start, lengths = _made([(60, 1500), (33, 700)], 8, 2, 64, dtype, 5)
    gp, gq = pages.cuda(), q.cuda()
    gt, gs, gl = kv._gpu(table, q_start, lengths)
    pkg.kv4_attention(gq, gp, gt, gs, gl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pkg.kv4_attention(gq, gp, gt, gs, gl, max_len=300)
    for new in ((1500, 700), (60, 33), (20, 640), (0, 65)):
        gl.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        kv._check_attention(out, q, pages, table, q_start, np.asarray(new), 0.125, fb.TYPES[dtype])


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("spans", [[(1, 4000), (1, 4000)], [(40, 4000), (3, 3)]])
@pytest.mark.parametrize("where", [0, 1777, 3950])
def test_one_position_against_thousands(where, spans, dtype):
    """A query that singles one key out (along its offset from the mean key, by the inverse of their covariance), whose
    score is 10 nats over all others together: thousands of weights of which each is
    some 2^-26 of the largest, early, in the middle and last of what is seen."""
    import dual_ar_tts_gb300 as pkg
    q, pages, table, q_start, lengths = _made(spans, 4, 1, 64, dtype, 7)
    dt = fb.TYPES[dtype]
    ids = [int(p) for p in table[0, :-(-4000 // 64)]]
    k, v = [fb.get(pages, part, ids)[0, :4000].double() for part in range(2)]
    others = torch.arange(4000) != where

    def margin(x):
        s = k @ x * 0.125
        return float(s[where] - torch.logsumexp(s[others], 0))

    lo, hi = 0.0, 1000.0                                             # |q| by bisection
    along = torch.linalg.solve(k.t().cov(), k[where] - k.mean(0))
    along /= along.norm()
    for _ in range(60):
        lo, hi = ((lo + hi) / 2, hi) if margin(along * (lo + hi) / 2) < 10 else (lo, (lo + hi) / 2)
    last = int(q_start[1]) - 1                                       # sees all 4000 (row 0 of the many at least 3961)
    for row in {0, last}:
        q[row, 0] = (along * hi).to(dt)
    assert 9 < margin(q[last, 0].double()) < 11
    got = kv._attend(pkg, q, pages, table, q_start, lengths)
    kv._check_attention(got, q, pages, table, q_start, lengths, 0.125, dt)
    # the one value all but alone, and the others' share of e^-10 in it
    for row in {0, last}:
        seen = 4000 - (last - row)
        p = torch.softmax(k[:seen] @ q[row, 0].double() * 0.125, 0)
        assert 0.9999 < float(p[where]) < 1 - 1e-5
        rest = (p[:, None] * v[:seen])[others[:seen]].sum(0)
        if dtype == "fp32":
            off = got[row, 0].cpu().double() - p[where] * v[where] - rest
            assert off.abs().max() <= 0.05 * rest.abs().max()


kv.SPANS["hundreds"] = [(400, 460), (1, 70), (131, 131)]             # 532 rows: appended a block a row


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("hq,hkv,hd", [(4, 2, 64), (9, 3, 64), (14, 2, 64), (5, 2, 128), (16, 1, 128), (6, 1, 128), (32, 8, 128)])
@pytest.mark.parametrize("norm", [False, True])
def test_append_and_read_of_hundreds_of_rows(hq, hkv, hd, dtype, norm):
    """Heads that end inside, at and one behind a turn of a block's four warps (16 heads of 64, 8 of 128)."""
    kv.test_append_and_read("hundreds", hq, hkv, hd, dtype, norm)


@pytest.mark.parametrize("rows", [511, 512, 513])
def test_append_alike_on_both_sides_of_512_rows(rows):
    """The rows of one call appended in two: the same bytes."""
    import dual_ar_tts_gb300 as pkg
    hq, hkv, hd = 9, 3, 64
    qkv = torch.randn((rows, (hq + 2 * hkv) * hd), generator=torch.Generator().manual_seed(rows)).bfloat16().cuda()
    w = [(1 + 0.1 * torch.randn(hd, generator=torch.Generator().manual_seed(i))).cuda() for i in range(2)]
    table = np.random.default_rng(rows).permutation(9)[None].astype(np.int32)
    rope = pkg.rope_table(rows, hd)
    one, two = [pkg.kv4_pages(9, hkv, hd) for _ in range(2)]
    q = pkg.kv4_append(qkv, one, *kv._gpu(table, np.asarray([0, rows], np.int32), np.asarray([rows], np.int32)), rope, hq, *w)
    got = []
    for a, b in ((0, 200), (200, rows)):
        at = kv._gpu(table, np.asarray([0, b - a], np.int32), np.asarray([b], np.int32))
        got.append(pkg.kv4_append(qkv[a:b], two, *at, rope, hq, *w))
    assert torch.equal(one, two) and torch.equal(q, torch.cat(got))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("spans,hq,hkv,hd", [([(1, 2500), (1, 700)], 32, 8, 128), ([(1, 2500), (2, 900)], 16, 2, 64),
                                             ([(3, 2000)], 12, 3, 128), ([(40, 2500), (100, 300)], 8, 2, 128),
                                             ([(130, 1500)], 8, 2, 64)])
def test_16_bit_results_are_the_rounded_ones(spans, hq, hkv, hd, dtype):
    """Of 16-bit queries too a weight has two terms, so that a result before its rounding is some 3e-6 off at most (fp32 sums
    on the tensor core, cut off at their last bit at each of up to 160 additions).  A result then takes the neighbour of the
    rounded 64-bit one where that lies as near to a border between two: 0.8 * 3e-6 over steps of 2^-10.5 (fp16, in the
    mean) or 2^-7.5, three times that since some results are small beside what they are sums of: 1 % and 0.13 %; 3 % and
    0.5 % asked.  Weights rounded to fp16, 1.2e-4 off, gave 14 to 27 % and 4 to 6 %, and 2.4e-4 for the error of fp16 results, whose
    rounding alone is 2^-11 / sqrt(3) * 0.735 (its mean over a binade) = 2.07e-4; 2.15e-4 asked."""
    import dual_ar_tts_gb300 as pkg
    q, pages, table, q_start, lengths = _made(spans, hq, hkv, hd, dtype, 31)
    got = kv._attend(pkg, q, pages, table, q_start, lengths).cpu()
    want = torch.empty(q.shape, dtype=torch.float64)
    for s, (n, length) in enumerate(spans):
        ids, rows = [int(p) for p in table[s, :-(-length // 64)]], slice(int(q_start[s]), int(q_start[s + 1]))
        for h in range(hq):
            k, v = [fb.get(pages[:, h // (hq // hkv)][:, None], part, ids)[0, :length] for part in range(2)]
            want[rows, h] = fb.attention(q[rows, h], k, v, range(length - n + 1, length + 1), hd ** -0.5)[0]
    differ = float((got != want.to(got.dtype)).float().mean())
    assert differ <= (0.03 if dtype == "fp16" else 0.005), differ
    if dtype == "fp16":
        off = float((got.double() - want).norm() / want.norm())
        assert off <= 2.15e-4, off
