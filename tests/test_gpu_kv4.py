"""The paged 4-bit cache (s2_kv4_append, s2_kv4_read, s2_kv4_attention) against its definition.

Appended codes and parameters are compared with a plain form that rounds every fp32 operation by
itself (as the kernel does); with the norm, the plain form's mean square comes from 64 bits and the
kernel's from pairs of fp32, both rounded to fp32 once, so that bits can differ only where a sum lies
on a rounding border of the last place: a few elements in a million may then take the neighbouring
code.  Rotated queries: six fp32 roundings and the type's own.  Attention: tests/four_bit.py."""
import math

import numpy as np
import pytest
import torch

from tests import four_bit as fb

pytestmark = pytest.mark.gpu


def _layout(spans, rng, extra=3, cols=0):
    """table, q_start, lengths, pages in the pool for spans of (new rows, length)."""
    need = [-(-length // fb.PAGE) for _, length in spans]
    pool = sum(need) + extra
    order = rng.permutation(pool).astype(np.int32)
    table = np.full((len(spans), max(need + [1, cols])), -7, np.int32)     # entries past a length are never read
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    q_start = np.cumsum([0] + [n for n, _ in spans]).astype(np.int32)
    lengths = np.asarray([length for _, length in spans], np.int32)
    return table, q_start, lengths, pool


def _gpu(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


SPANS = {
    "one": [(1, 1)],
    "page_end": [(1, 64), (1, 65), (2, 128)],
    "ragged": [(3, 17), (0, 9), (70, 70), (1, 200), (0, 0), (5, 133)],
    "decode": [(1, n) for n in (1, 63, 64, 65, 700, 2, 33, 129)],
    "prompt": [(150, 150), (64, 640)],
}
HEADS = [(4, 2, 64), (32, 8, 128), (3, 3, 64), (16, 1, 128), (6, 2, 128)]


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("hq,hkv,hd", HEADS)
@pytest.mark.parametrize("spans", ["one", "page_end", "ragged", "prompt"])
@pytest.mark.parametrize("norm", [False, True])
def test_append_and_read(spans, hq, hkv, hd, dtype, norm):
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(hq * hd + len(spans))
    table, q_start, lengths, pool = _layout(SPANS[spans], rng)
    rows = int(q_start[-1])
    dt = fb.TYPES[dtype]
    heads = hq + 2 * hkv
    x = rng.standard_normal((rows, heads, hd)) * np.exp(rng.standard_normal((heads, hd)))
    x[..., 3] += 5.0                                                    # a biased channel
    qkv = torch.from_numpy(x.astype(np.float32)).to(dt)
    qkv[0, hq, :32] = 0                                                 # a group of zeros
    qkv[0, hq + hkv, :32] = 0.75                                        # a constant group
    n_pos = int(lengths.max()) + 2
    rope = pkg.rope_table(n_pos, hd)
    qw, kw = [torch.from_numpy((1 + 0.1 * rng.standard_normal(hd)).astype(np.float32)) if norm else None for _ in "qk"]
    pages = torch.full((pool, hkv, 80 * hd), 0xA5, dtype=torch.uint8)
    want = pages.clone()
    gp = pages.cuda()
    gt, gs, gl = _gpu(table, q_start, lengths)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((rows + 2, hq, hd), 9.0, dtype=dt, device="cuda")
    more = torch.cat([qkv.flatten(1), torch.full((2, heads * hd), math.nan, dtype=dt)]).cuda()  # rows behind the last
    got = pkg.kv4_append(more, gp, gt, gs, gl, rope, hq, q_norm=None if qw is None else qw.cuda(),
                         k_norm=None if kw is None else kw.cuda(), eps=1e-6, q_out=q_out, status=status)
    seq = np.repeat(np.arange(len(lengths)), np.diff(q_start))
    pos = lengths[seq] - (q_start[seq + 1] - np.arange(rows))
    cs = rope.cpu()[torch.from_numpy(pos).long()][:, None]
    f = qkv.float()
    q64 = f[:, :hq].double()
    if norm:
        q64 = q64 * (q64.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * qw.double()
    a, b, c, s = q64[..., 0::2], q64[..., 1::2], cs[..., 0].double(), cs[..., 1].double()
    q64, mag = [torch.stack(t, -1).flatten(-2) for t in
                ((a * c - b * s, b * c + a * s), ((a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()))]
    err = (got[:rows].cpu().double() - q64).abs()
    assert (err <= 10 * 2.0 ** -24 * mag + fb.rounding(q64, dt)).all()
    assert (got[rows:] == 9).all() and int(status) == 0
    k = fb.norm_rotate(f[:, hq:hq + hkv], kw, 1e-6, cs)
    for i in range(rows):
        fb.put(want, int(table[seq[i], pos[i] // 64]), int(pos[i] % 64), k[i], f[i, hq + hkv:])
    if norm:
        off = (gp.cpu() != want).float().mean().item()
        assert off <= max(1e-5, 2.0 / want.numel()), off
    else:
        assert torch.equal(gp.cpu(), want)                              # every other byte as it was
    rk, rv = pkg.kv4_read(gp, gt, gs, gl, rows + 2, k_out=torch.full((hkv, rows + 2, hd), 9, dtype=torch.float16, device="cuda"))
    kept = gp.cpu()
    for part, r in enumerate((rk, rv)):
        for i in range(rows):
            full = fb.get(kept, part, [int(table[seq[i], pos[i] // 64])])[:, pos[i] % 64]
            assert torch.equal(r[:, i].cpu(), full)
    assert (rk[:, rows:] == 9).all()
    # half a step of the group's scale from what went in (one step where the range was clipped by the zero point)
    vs = fb.kv_quantise(f[:, hq + hkv:])[1].float().repeat_interleave(32, -1)
    assert ((rv[:, :rows].transpose(0, 1).cpu().float() - f[:, hq + hkv:]).abs() <= vs * 1.02 + 1e-6).all()


def test_append_non_finite_and_large_values():
    import dual_ar_tts_gb300 as pkg
    hkv, hd = 2, 128
    qkv = torch.randn((1, 2 * hkv, hd), generator=torch.Generator().manual_seed(0))
    qkv[0, 0, 5] = math.nan
    qkv[0, 1, 40] = math.inf
    qkv[0, 2, 70] = -3e38
    qkv[0, 3, :32] = 1e-9                                               # the scale rounds to zero
    qkv[0, 3, 32:64] = torch.linspace(100.0, 100.5, 32)                 # narrow and far from zero
    rope = torch.zeros((1, hd // 2, 2))
    rope[..., 0] = 1
    pages = pkg.kv4_pages(1, hkv, hd)
    one = _gpu(np.zeros((1, 1), np.int32), np.asarray([0, 1], np.int32), np.asarray([1], np.int32))
    pkg.kv4_append(qkv.flatten(1).cuda(), pages, *one, rope.cuda(), 0)
    k, v = [t[:, 0].cpu() for t in pkg.kv4_read(pages, *one, 1)]
    assert torch.isnan(k[0, :32]).all() and torch.isfinite(k[0, 32:]).all()
    # a key is rotated before it is quantised: inf * sin(0) is NaN in the pair, so the group's scale is
    assert torch.isnan(k[1, 32:64]).all() and torch.isfinite(k[1, :32]).all() and torch.isfinite(k[1, 64:]).all()
    assert torch.isfinite(v).all() and v[0, 70] < -5e4 and (v[1, :32] == 0).all()
    assert ((v[1, 32:64].float() - qkv[0, 3, 32:64]).abs() <= 100.5 / 127 * 1.01).all()


def test_append_leaves_out_bad_rows():
    """A page out of range, a position below zero, behind the rotation table or behind the page table."""
    import dual_ar_tts_gb300 as pkg
    hq, hkv, hd = 4, 2, 64
    spans = [(2, 70), (1, 1), (3, 2), (1, 65), (1, 130)]
    table = np.asarray([[0, 9], [1, -1], [2, -1], [3, -1], [4, 5]], np.int32)   # 9 and -1 do not exist
    q_start = np.cumsum([0] + [n for n, _ in spans]).astype(np.int32)
    lengths = np.asarray([n for _, n in spans], np.int32)
    rows = int(q_start[-1])
    qkv = torch.randn((rows, (hq + 2 * hkv) * hd), generator=torch.Generator().manual_seed(1)).cuda()
    pages = pkg.kv4_pages(6, hkv, hd)
    before = pages.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((rows, hq, hd), 9.0, device="cuda")
    gt, gs, gl = _gpu(table, q_start, lengths)
    pkg.kv4_append(qkv, pages, gt, gs, gl, pkg.rope_table(100, hd), hq, q_out=q_out, status=status)
    assert int(status) == pkg.S2_EINVAL
    skipped = torch.tensor([True, True, False, True, False, False, True, True])
    assert torch.equal((q_out.cpu() == 9).flatten(1).all(1), skipped)
    changed = (pages != before).flatten(1).any(1).cpu()
    assert changed.tolist() == [False, True, True, False, False, False]
    status.zero_()
    k, v = pkg.kv4_read(pages, gt, gs, gl, rows, status=status)
    assert int(status) == pkg.S2_EINVAL
    for i in range(rows):
        bad = i in (0, 1, 3, 6)
        assert bool((k[:, i] == 0).all()) == (bad or i == 7)            # row 7: its (empty) page can be read


def _attend(pkg, q, pages, table, q_start, lengths, **kw):
    gt, gs, gl = _gpu(table, q_start, lengths)
    return pkg.kv4_attention(q.cuda(), pages.cuda(), gt, gs, gl, **kw)


def _check_attention(got, q, pages, table, q_start, lengths, scale, dt, live=None):
    hq, hkv = q.shape[1], pages.shape[1]
    worst = 0.0
    for s in range(len(lengths)):
        a, b = int(q_start[s]), int(q_start[s + 1])
        if a == b:
            continue
        n = b - a
        L = int(lengths[s])
        ids = [int(p) for p in table[s, :-(-L // 64)]] if L > 0 else []
        seen = [max(0, L - n + i + 1) for i in range(n)]
        for h in range(hq):
            kv = [(fb.get(pages[:, h // (hq // hkv)][:, None], part, ids)[0, :L] if ids else torch.zeros((0, q.shape[2])))
                  for part in range(2)]
            o, rel, wv, tiny = fb.attention(q[a:b, h], kv[0], kv[1], seen, scale) if L > 0 else \
                (torch.zeros((n, q.shape[2])), 0, torch.zeros((n, q.shape[2])), 0)
            tol = fb.attention_tol(o, rel, wv, tiny, dt) if L > 0 else torch.zeros_like(o)
            err = (got[a:b, h].cpu().double() - o).abs()
            assert (err <= tol).all(), (s, h, float((err - tol).max()))
            worst = max(worst, float((err / tol.clamp(min=1e-30)).max()))
    return worst


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("hq,hkv,hd", HEADS + [(40, 2, 64), (7, 1, 128)])
@pytest.mark.parametrize("spans", ["one", "page_end", "ragged", "decode", "prompt"])
def test_attention(spans, hq, hkv, hd, dtype):
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(hq + hd + len(spans))
    table, q_start, lengths, pool = _layout(SPANS[spans], rng, cols=6)
    rows = int(q_start[-1])
    dt = fb.TYPES[dtype]
    pages = torch.zeros((pool, hkv, 80 * hd), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    q = torch.from_numpy(rng.standard_normal((rows + 1, hq, hd)).astype(np.float32) * 1.5).to(dt)
    out = torch.full((rows + 1, hq, hd), 9.0, dtype=dt, device="cuda")
    got = _attend(pkg, q, pages, table, q_start, lengths, out=out)
    assert (got[rows:] == 9).all()
    _check_attention(got, q, pages, table, q_start, lengths, hd ** -0.5, dt)
    again = _attend(pkg, q, pages, table, q_start, lengths, max_len=int(lengths.max()))
    _check_attention(again, q, pages, table, q_start, lengths, hd ** -0.5, dt)


@pytest.mark.parametrize("dtype", list(fb.TYPES))
def test_attention_long_and_split(dtype):
    """Lengths that are split over blocks; the hint below, at and above the length; the same bits again."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(11)
    spans = [(1, 5003), (2, 3000), (1, 1), (1, 64)]
    table, q_start, lengths, pool = _layout(spans, rng, cols=200)
    dt = fb.TYPES[dtype]
    pages = torch.zeros((pool, 2, 80 * 128), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    q = torch.from_numpy(rng.standard_normal((5, 8, 128)).astype(np.float32) * 3).to(dt)
    for hint in (0, 64, 2000, 5003, 12800):
        got = _attend(pkg, q, pages, table, q_start, lengths, max_len=hint)
        _check_attention(got, q, pages, table, q_start, lengths, 128 ** -0.5, dt)
        assert torch.equal(got, _attend(pkg, q, pages, table, q_start, lengths, max_len=hint))


@pytest.mark.parametrize("dtype", list(fb.TYPES))
def test_attention_ignores_what_is_masked(dtype):
    """Slots past a length and in the future of a row hold NaN and infinities; a row that sees nothing gets zeros."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(3)
    spans = [(4, 70), (5, 3), (2, 128), (3, 0), (2, 1)]
    table, q_start, lengths, pool = _layout(spans, rng)
    dt = fb.TYPES[dtype]
    hq, hkv, hd = 8, 2, 128
    pages = torch.zeros((pool, hkv, 80 * hd), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    for s, (_, L) in enumerate(spans):
        if L % 64:
            for part in range(2):
                codes, par = fb._parts(pages, part)
                par[int(table[s, L // 64]), :, L % 64:] = torch.tensor([math.nan, math.inf]).half()
                codes[int(table[s, L // 64]), :, L % 64:] = 255
    q = torch.from_numpy(rng.standard_normal((16, hq, hd)).astype(np.float32)).to(dt)
    got = _attend(pkg, q, pages, table, q_start, lengths)
    assert torch.isfinite(got).all()
    assert (got[4:6] == 0).all() and (got[11:14] == 0).all() and (got[14] == 0).all()
    _check_attention(got, q, pages, table, q_start, lengths, hd ** -0.5, dt)
    # a key in a row's future: NaN there, rows before it are as they were
    codes, par = fb._parts(pages, 0)
    par[int(table[2, 1]), :, 63] = math.nan
    later = _attend(pkg, q, pages, table, q_start, lengths)
    assert torch.equal(later[9], got[9]) and torch.isnan(later[10]).all()


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_of_many_rows_ignores_what_is_masked(dtype, hd):
    """As above for sequences of many rows: NaN behind a length and in the future of some rows, in keys or values."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(4)
    spans = [(70, 100), (130, 130), (40, 20), (64, 0)]
    table, q_start, lengths, pool = _layout(spans, rng)
    dt = fb.TYPES[dtype]
    hq, hkv = 8, 2
    pages = torch.zeros((pool, hkv, 80 * hd), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    for s, (_, L) in enumerate(spans):
        if L % 64:
            for part in range(2):
                codes, par = fb._parts(pages, part)
                par[int(table[s, L // 64]), :, L % 64:] = torch.tensor([math.nan, -math.inf]).half()
    q = torch.from_numpy(rng.standard_normal((int(q_start[-1]), hq, hd)).astype(np.float32)).to(dt)
    got = _attend(pkg, q, pages, table, q_start, lengths)
    assert torch.isfinite(got).all()
    assert (got[200:220] == 0).all() and (got[240:] == 0).all()     # rows before their sequence, and of an empty one
    _check_attention(got, q, pages, table, q_start, lengths, hd ** -0.5, dt)
    # sequence 0: position 80 is seen by its rows 50 on; sequence 1: position 70 by its rows 70 on
    codes, par = fb._parts(pages, 1)
    par[int(table[0, 1]), :, 16, 1] = math.nan                       # one group of the values
    codes, par = fb._parts(pages, 0)
    par[int(table[1, 1]), 0, 6] = math.nan                           # a key of KV head 0
    later = _attend(pkg, q, pages, table, q_start, lengths)
    assert torch.equal(later[:50], got[:50]) and torch.equal(later[70:140], got[70:140])
    assert torch.isnan(later[50:70, :, 32:64]).all()
    assert torch.equal(later[50:70, :, :32], got[50:70, :, :32])
    assert torch.isnan(later[140:200, :4]).all() and torch.equal(later[140:200, 4:], got[140:200, 4:])


@pytest.mark.parametrize("dtype", list(fb.TYPES))
def test_many_sequences(dtype):
    """More sequences than a warp has lanes, empty ones among them, appended, read and attended."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(8)
    spans = [(int(rng.integers(0, 3)), int(rng.integers(3, 90))) for _ in range(75)] + [(1, 200)]
    table, q_start, lengths, pool = _layout(spans, rng)
    rows, dt, hq, hkv, hd = int(q_start[-1]), fb.TYPES[dtype], 6, 2, 64
    pages = torch.zeros((pool, hkv, 80 * hd), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    qkv = torch.from_numpy(rng.standard_normal((rows, (hq + 2 * hkv) * hd)).astype(np.float32)).to(dt)
    gp = pages.cuda()
    gt, gs, gl = _gpu(table, q_start, lengths)
    rope = pkg.rope_table(256, hd)
    q = pkg.kv4_append(qkv.cuda(), gp, gt, gs, gl, rope, hq)
    want = pages.clone()
    f = qkv.float().view(rows, -1, hd)
    seq = np.repeat(np.arange(len(lengths)), np.diff(q_start))
    pos = lengths[seq] - (q_start[seq + 1] - np.arange(rows))
    k = fb.norm_rotate(f[:, hq:hq + hkv], None, 0, rope.cpu()[torch.from_numpy(pos).long()][:, None])
    for i in range(rows):
        fb.put(want, int(table[seq[i], pos[i] // 64]), int(pos[i] % 64), k[i], f[i, hq + hkv:])
    assert torch.equal(gp.cpu(), want)
    got = pkg.kv4_attention(q, gp, gt, gs, gl)
    _check_attention(got, q.cpu(), want, table, q_start, lengths, hd ** -0.5, dt)


@pytest.mark.parametrize("dtype", list(fb.TYPES))
def test_attention_magnitudes(dtype):
    """Scores far apart (one position takes all; 10 nats below it thousands share the rest), queries of 1e-6 and
    1e4, tiny value scales."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(5)
    dt = fb.TYPES[dtype]
    spans = [(1, 4000), (1, 4000), (1, 333), (3, 3)]
    table, q_start, lengths, pool = _layout(spans, rng)
    pages = torch.zeros((pool, 1, 80 * 64), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    codes, par = fb._parts(pages, 1)
    par[..., 0] *= 1e-3
    par[..., 1] = 7
    q = torch.from_numpy(rng.standard_normal((6, 4, 64)).astype(np.float32))
    q[0] *= 8
    q[1] *= 1e-6 if dtype != "fp16" else 1e-4
    q[2] *= 1e4 if dtype != "fp16" else 50
    # one key that matches q[0] head 0, about 10 nats over the others' mass
    k = fb.get(pages, 0, [int(table[0, 0])])
    q = q.to(dt)
    got = _attend(pkg, q, pages, table, q_start, lengths)
    assert k.shape[1] == 64
    _check_attention(got, q, pages, table, q_start, lengths, 0.125, dt)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 1.0])
def test_attention_scales(scale):
    """A scale of zero (all seen positions alike), a negative one, one that underflows, and none."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(17)
    for spans in ([(1, 70), (2, 33)], [(50, 100), (3, 3)]):
        table, q_start, lengths, pool = _layout(spans, rng)
        pages = torch.zeros((pool, 1, 80 * 64), dtype=torch.uint8)
        fb.fill_random(pages, rng)
        for dt in fb.TYPES.values():
            q = torch.from_numpy(rng.standard_normal((int(q_start[-1]), 4, 64)).astype(np.float32)).to(dt)
            got = _attend(pkg, q, pages, table, q_start, lengths, scale=scale)
            _check_attention(got, q, pages, table, q_start, lengths, scale, dt)


def test_attention_bad_pages_are_not_attended():
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(9)
    table, q_start, lengths, pool = _layout([(1, 200), (2, 64), (1, 300)], rng)
    pages = torch.zeros((pool, 2, 80 * 64), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    q = torch.from_numpy(rng.standard_normal((4, 4, 64)).astype(np.float32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _attend(pkg, q, pages, table, q_start, lengths, status=status)
    assert int(status) == 0
    bad = table.copy()
    bad[0, 1], bad[1, 0], bad[2, 0] = pool, -1, 2 ** 31 - 1
    got = _attend(pkg, q, pages, bad, q_start, lengths, status=status)
    assert int(status) == pkg.S2_EINVAL
    assert (got[1:3] == 0).all()
    # sequence 0 without its second page: the same as its other pages alone, where no causal limit cuts in
    cut = np.asarray([[table[0, 0], table[0, 2], table[0, 3]]], np.int32)
    want = _attend(pkg, q[:1], pages, cut, np.asarray([0, 1], np.int32), np.asarray([136], np.int32))
    assert (got[0] - want[0]).abs().max() <= 1e-5 * want[0].abs().max()
    # a length past the page table
    status.zero_()
    got = _attend(pkg, q[:1], pages, table[:1, :2], np.asarray([0, 1], np.int32), np.asarray([1000], np.int32), status=status)
    assert int(status) == pkg.S2_EINVAL
    want = _attend(pkg, q[:1], pages, table[:1, :2], np.asarray([0, 1], np.int32), np.asarray([128], np.int32))
    assert (got - want).abs().max() <= 1e-5 * want.abs().max()


def test_shared_pages_and_a_pool_past_32_bits():
    """Two sequences read the same prefix pages; the pool is larger than 4 GiB and its last pages are in use."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(21)
    n_pages = (1 << 32) // (80 * 128) + 50
    small = torch.zeros((5, 1, 80 * 128), dtype=torch.uint8)
    fb.fill_random(small, rng)
    pages = torch.empty((n_pages, 1, 80 * 128), dtype=torch.uint8, device="cuda")
    first = n_pages - 5
    pages[first:] = small.cuda()
    local = np.asarray([[0, 1, 2], [0, 1, 3], [4, -1, -1]], np.int32)
    table = np.where(local >= 0, local + first, -1).astype(np.int32)
    q_start, lengths = np.asarray([0, 1, 3, 4], np.int32), np.asarray([170, 190, 20], np.int32)
    q = torch.from_numpy(rng.standard_normal((4, 4, 128)).astype(np.float32)).bfloat16()
    gt, gs, gl = _gpu(table, q_start, lengths)
    got = pkg.kv4_attention(q.cuda(), pages, gt, gs, gl)
    _check_attention(got, q, small, local, q_start, lengths, 128 ** -0.5, torch.bfloat16)
    qkv = torch.randn((4, 3 * 128), device="cuda")
    own = _gpu(np.asarray([[first + 4]], np.int32), np.asarray([0, 4], np.int32), np.asarray([64], np.int32))
    pkg.kv4_append(qkv, pages, *own, pkg.rope_table(64, 128), 1)
    k, v = pkg.kv4_read(pages, *own, 4)
    assert torch.equal(v.cpu(), fb.get(pages[first:].cpu(), 1, [4])[:, 60:])
    del pages
    torch.cuda.empty_cache()


def test_attention_captured_and_replayed_with_other_lengths():
    """One graph; lengths, tables and queries change between replays.  A second graph has its own workspace, and
    the two run on two streams at the same time."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(2)
    table, q_start, lengths, pool = _layout([(1, 3000), (1, 1500)], rng)
    pages = torch.zeros((pool, 2, 80 * 128), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    gp = pages.cuda()
    gt, gs, gl = _gpu(table, q_start, lengths)
    q = torch.randn((2, 8, 128), device="cuda").half()
    nbytes = pkg.load().s2_kv4_attention_workspace(2, 2, 8, 2, 128, 3000)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    torch.cuda.synchronize()
    for s in side:
        ws = torch.empty(max(16, nbytes), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pkg.kv4_attention(q, gp, gt, gs, gl, max_len=3000, workspace=ws, out=out)
        graphs.append((g, ws, out))
    for new in ((3000, 1500), (1, 1472), (2900, 64)):
        gl.copy_(torch.tensor(new, dtype=torch.int32))
        q.copy_(torch.randn((2, 8, 128)).half())
        torch.cuda.synchronize()
        for (g, _, _), s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][2], graphs[1][2])
        _check_attention(graphs[0][2], q.cpu(), pages, table, q_start, np.asarray(new), 128 ** -0.5, torch.float16)


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("fp32", 128)])
def test_attention_of_many_rows_beside_products_on_other_streams(dtype, hd):
    """Calls of both operators that use tensor memory, on three streams at once: each gives its own bits."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(17)
    spans = [(60, 700), (200, 1300), (33, 64)]
    table, q_start, lengths, pool = _layout(spans, rng, cols=24)
    dt = fb.TYPES[dtype]
    pages = torch.zeros((pool, 8, 80 * hd), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    q = torch.from_numpy(rng.standard_normal((293, 32, hd)).astype(np.float32)).to(dt).cuda()
    args = (q, pages.cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(q_start).cuda(),
            torch.from_numpy(lengths).cuda())
    w = torch.randn((2500, 1280), generator=torch.Generator().manual_seed(2)).cuda()
    codes, scales = pkg.quantize_q4(w, 64)
    xs = [torch.randn((n, 1280), generator=torch.Generator().manual_seed(n)).to(dt).cuda() for n in (40, 300)]
    calls = [lambda: pkg.kv4_attention(*args)] + [lambda x=x: pkg.q4_matmul(x, codes, scales, 64) for x in xs]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(20):
        for f, s, g in zip(calls, streams, got):
            with torch.cuda.stream(s):
                g.append(f())
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, y) for y in g)


@pytest.mark.parametrize("hd,hq,hkv", [(64, 4, 1), (128, 8, 2)])
@pytest.mark.parametrize("spans,hint", [([(1, 20000)], 64), ([(1, 3000), (2, 700)], 0), ([(200, 3000), (60, 60)], 0),
                                        ([(40, 20000)], 64), ([(130, 1000)], 0)])
def test_attention_keeps_fp32(spans, hint, hd, hq, hkv):
    """The error of fp32 attention, 2-norm over 2-norm of a sequence, for queries and keys of unit size.  A score: the split
    of the query leaves 2^-23 / sqrt(3) of its terms (1e-7 of their size), hd / 16 = 8 additions on the tensor core cut
    off half of the last bit each, 0.72 * 2^-23 on average, of sums 0.7 as large: 2.4e-7 of the score, whose size is
    about 1.5: 3.6e-7 of a weight.  ex2 and its argument: 2^-22.  Output: a page's (a step's) 4 additions: 1.2e-7; its sums,
    added one by one: 2^-25 sqrt(470) / 2 = 3e-7 at 20000 positions (of a size that grows as its root).  Independent but for
    the two cuts: sqrt(1^2 + 2.4^2 + 3^2) + 3.6 + 1.2 = 8.8e-7; 1e-6 asked."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(hd + len(spans))
    table, q_start, lengths, pool = _layout(spans, rng)
    pages = torch.zeros((pool, hkv, 80 * hd), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    q = torch.from_numpy(rng.standard_normal((int(q_start[-1]), hq, hd)).astype(np.float32))
    got = _attend(pkg, q, pages, table, q_start, lengths, max_len=hint).cpu().double()
    for s, (n, length) in enumerate(spans):
        ids, rows = [int(p) for p in table[s, :-(-length // 64)]], slice(int(q_start[s]), int(q_start[s + 1]))
        want = torch.empty((n, hq, hd), dtype=torch.float64)
        for h in range(hq):
            k, v = [fb.get(pages[:, h // (hq // hkv)][:, None], part, ids)[0, :length] for part in range(2)]
            want[:, h] = fb.attention(q[rows, h], k, v, range(length - n + 1, length + 1), hd ** -0.5)[0]
        off = float((got[rows] - want).norm() / want.norm())
        assert off <= 1e-6, off


@pytest.mark.parametrize("dtype", list(fb.TYPES))
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("spans", [[(70, 100), (130, 130)], [(300, 4000), (20, 64)]])
def test_attention_of_many_rows_whose_waits_give_up(spans, hd, dtype):
    """No tries: every wait gives up at once.  No number comes out, the status says so, and the next call is as ever."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(4)
    table, q_start, lengths, pool = _layout(spans, rng)
    rows = int(q_start[-1])
    pages = torch.zeros((pool, 2, 80 * hd), dtype=torch.uint8)
    fb.fill_random(pages, rng)
    q = torch.from_numpy(rng.standard_normal((rows + 1, 8, hd)).astype(np.float32)).to(fb.TYPES[dtype])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((rows + 1, 8, hd), 9.0, dtype=q.dtype, device="cuda")
    want = _attend(pkg, q, pages, table, q_start, lengths, out=out.clone(), status=status)
    assert int(status) == 0 and torch.isfinite(want).all()
    pkg.s2_set_wait_limit(0)
    try:
        got = _attend(pkg, q, pages, table, q_start, lengths, out=out, status=status)
        torch.cuda.synchronize()
    finally:
        pkg.s2_set_wait_limit(-1)
    assert int(status) == pkg.S2_ETIMEOUT
    assert torch.isnan(got[:rows]).all() and (got[rows:] == 9).all()
    status.zero_()
    assert torch.equal(_attend(pkg, q, pages, table, q_start, lengths, out=out, status=status), want) and int(status) == 0


@pytest.mark.parametrize("dtype", list(fb.TYPES))
def test_append_of_one_row_of_any_stride(dtype):
    import dual_ar_tts_gb300 as pkg
    hq, hkv, hd = 2, 1, 64
    width = (hq + 2 * hkv) * hd
    wide = torch.randn((3, width + 3), generator=torch.Generator().manual_seed(1)).to(fb.TYPES[dtype]).cuda()
    one = _gpu(np.zeros((1, 1), np.int32), np.asarray([0, 1], np.int32), np.asarray([9], np.int32))
    rope = pkg.rope_table(16, hd)
    for x in (wide[1:2, :width], wide[2:, 3:], wide[:1, 1:1 + width], wide[:1, :width].t().contiguous().t()):
        pages, want = [pkg.kv4_pages(1, hkv, hd) for _ in range(2)]
        q = pkg.kv4_append(x, pages, *one, rope, hq)
        same = torch.empty((1, width), dtype=x.dtype, device="cuda").copy_(x)
        assert torch.equal(q, pkg.kv4_append(same, want, *one, rope, hq)) and torch.equal(pages, want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hq,hkv,hd", [(9, 3, 64), (32, 8, 128), (3, 2, 128)])
def test_append_norm_of_large_rows(hq, hkv, hd, dtype):
    """Rows whose sum of squares, or mean square too, is past fp32's range: the definition gives numbers where the
    mean fits (rounded from 64 bits), and zeros where it does not (1 / sqrt(inf)).  A query: 12 roundings of 2^-24 in its
    mean, half of that after the root, 6 more of the norm and 3 of the rotation: 15; and 9 of the plain form's."""
    import dual_ar_tts_gb300 as pkg
    rng = np.random.default_rng(3)
    dt, heads, sizes = fb.TYPES[dtype], hq + 2 * hkv, (1.0, 2e17, 1.5e18, 1e19, 1.7e19, 3e19, 1e25, 1e37)
    rows = len(sizes)
    x = rng.standard_normal((rows, heads, hd)).clip(-3, 3) * np.asarray(sizes)[:, None, None]
    x[4, :, 1:] *= 1e-8                                                # one element has it all
    f = torch.from_numpy(x.astype(np.float32)).to(dt)
    qw, kw = [torch.from_numpy((1 + 0.1 * rng.standard_normal(hd)).astype(np.float32)) for _ in "qk"]
    one = _gpu(np.zeros((1, 1), np.int32), np.asarray([0, rows], np.int32), np.asarray([rows], np.int32))
    rope = pkg.rope_table(rows, hd)
    pages = pkg.kv4_pages(1, hkv, hd)
    q = pkg.kv4_append(f.flatten(1).cuda(), pages, *one, rope, hq, q_norm=qw.cuda(), k_norm=kw.cuda()).cpu().double()
    cs = rope.cpu()[:, None]
    f = f.float()
    want = fb.norm_rotate(f[:, :hq], qw, 1e-6, cs).double()
    a, b = want[..., 0::2].abs(), want[..., 1::2].abs()
    mag = (a + b).repeat_interleave(2, -1) * 1.5                       # of what was rotated: at most sqrt(2) of this
    assert ((q - want).abs() <= 24 * 2.0 ** -24 * mag + fb.rounding(want, dt)).all()
    assert (q[6:] == 0).all() and (q[:5].abs().amax((1, 2)) > 0.5).all()
    want = torch.zeros((1, hkv, 80 * hd), dtype=torch.uint8)
    k = fb.norm_rotate(f[:, hq:hq + hkv], kw, 1e-6, cs)
    assert torch.isfinite(k).all()
    for i in range(rows):
        fb.put(want, 0, i, k[i], f[i, hq + hkv:])
    assert (pages.cpu() != want).sum() <= 2                            # a mean on a rounding border may move a code


@pytest.mark.parametrize("dtype", list(fb.TYPES))
def test_append_query_bits_do_not_depend_on_the_heads_beside_it(dtype):
    import dual_ar_tts_gb300 as pkg
    rows, hd = 300, 64
    x = torch.randn((rows, 6, hd), generator=torch.Generator().manual_seed(1)).to(fb.TYPES[dtype]).cuda()
    w = torch.ones(hd, device="cuda")
    place = _gpu(np.arange(5, dtype=np.int32)[None], np.asarray([0, rows], np.int32), np.asarray([rows], np.int32))
    rope = pkg.rope_table(rows, hd)
    got = []
    for heads, hq in (([0, 1, 2, 3, 4, 5], 4), ([0, 4, 5], 1), ([1, 0, 4, 5], 2)):
        qkv = x[:, heads].flatten(1).contiguous()
        got.append(pkg.kv4_append(qkv, pkg.kv4_pages(5, 1, hd), *place, rope, hq, q_norm=w, k_norm=w)[:, heads.index(0)])
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
