"""What the stateless 4-bit calls refuse before anything is launched (no GPU needed: a refusal is
decided from the arguments alone)."""
import ctypes

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


def test_quantize_q4(lib):
    good = dict(w=P, dtype=1, rows=4, cols=128, group=32, codes=P, scales=P, stream=None)
    _bad(lib.s2_quantize_q4, good, w=[None, P + 1], dtype=[3, -1], rows=[0, -1, 1 << 40], cols=[0, -32, 100],
         group=[0, 16, 48, 256], codes=[None, P + 8], scales=[None, P + 1])
    _bad(lib.s2_quantize_q4, dict(good, group=128), cols=[64, 160])


def test_q4_matmul(lib):
    good = dict(n=2, x=P, dtype=1, x_stride=128, codes=P, scales=P, m=4, k=128, group=32, y=P, ws=None, nb=0,
                stream=None)
    _bad(lib.s2_q4_matmul, good, ws=[P + 8], n=[0, -1], x=[None, P + 2], dtype=[3, 9], x_stride=[127, 132, 0], codes=[None, P + 4],
         scales=[None, P + 2], m=[0, -3], k=[0, 100, -32], group=[0, 31, 256], y=[None, P + 1])
    for dtype in (0, 1, 2):
        need = lib.s2_q4_matmul_workspace(40, 2560, dtype)
        assert need > 0 and lib.s2_q4_matmul_workspace(1, 2560, dtype) == 0
        _bad(lib.s2_q4_matmul, dict(good, n=40, k=2560, x_stride=2560, dtype=dtype, ws=P, nb=need), nb=[0, need - 1],
             ws=[None])
    for bad in ((0, 128, 1), (1, 0, 1), (1, 128, 3), (-1, 128, 0), (1 << 30, 128, 0)):
        assert lib.s2_q4_matmul_workspace(*bad) == 0


def _cache(pkg, **over):
    f = dict(pages=P, n_pages=4, n_kv_head=2, head_dim=64, table=P, table_cols=3, n_seq=2, q_start=P, lengths=P,
             n_rows=2, status=None)
    f.update(over)
    return pkg.s2_kv4(*f.values())


BAD_CACHE = [dict(pages=None), dict(pages=P + 8), dict(n_pages=0), dict(n_kv_head=0), dict(head_dim=96),
             dict(head_dim=256), dict(table=None), dict(table=P + 2), dict(table_cols=0), dict(table_cols=1 << 30),
             dict(n_seq=0), dict(q_start=None), dict(q_start=P + 1), dict(lengths=None), dict(lengths=P + 3),
             dict(n_rows=0), dict(n_rows=-1), dict(status=P + 2), dict(n_kv_head=1 << 20)]


def test_kv4(lib):
    import dual_ar_tts_gb300 as pkg
    c = ctypes.byref(_cache(pkg))
    append = dict(c=c, qkv=P, dtype=1, stride=512, n_head=4, rope=P, n_pos=64, qn=None, kn=None, eps=1e-6, q_out=P,
                  stream=None)
    read = dict(c=c, k=P, v=P, stream=None)
    attend = dict(c=c, q=P, dtype=1, n_head=4, scale=0.1, max_len=0, out=P, ws=None, n=0, stream=None)
    for over in BAD_CACHE:
        bad = ctypes.byref(_cache(pkg, **over))
        for fn, good in ((lib.s2_kv4_append, append), (lib.s2_kv4_read, read), (lib.s2_kv4_attention, attend)):
            _bad(fn, good, c=[bad])
    nan, inf = float("nan"), float("inf")
    _bad(lib.s2_kv4_append, append, c=[None], qkv=[None, P + 2], dtype=[3], stride=[511, 516, 0], n_head=[-1, 1 << 20],
         rope=[None, P + 4], n_pos=[0], qn=[P + 4], kn=[P + 8], eps=[-1.0, nan, inf], q_out=[None, P + 2])
    _bad(lib.s2_kv4_read, read, c=[None], k=[None, P + 2], v=[None, P + 8])
    _bad(lib.s2_kv4_attention, attend, c=[None], q=[None, P + 2], dtype=[-1, 3], n_head=[0, 3, -2], scale=[nan, inf],
         max_len=[-1], out=[None, P + 4], ws=[P + 8])
    big = _cache(pkg, n_rows=2, table_cols=600)
    need = lib.s2_kv4_attention_workspace(2, 2, 4, 2, 64, 600 * 64)
    if need:
        _bad(lib.s2_kv4_attention, dict(attend, c=ctypes.byref(big), ws=P, n=need - 1), ws=[P, None])


def test_kv4_sizes(lib):
    assert lib.s2_kv4_page_bytes(8, 128) == 8 * 80 * 128 and lib.s2_kv4_page_bytes(2, 64) == 2 * 80 * 64
    for bad in ((0, 64), (2, 96), (-1, 128), (2, 0)):
        assert lib.s2_kv4_page_bytes(*bad) == -1
    for bad in ((0, 1, 4, 2, 64, 0), (1, 0, 4, 2, 64, 0), (1, 1, 3, 2, 64, 0), (1, 1, 4, 2, 96, 9), (1, 1, 4, 2, 64, -1)):
        assert lib.s2_kv4_attention_workspace(*bad) == 0


def test_adjust_logits(lib):
    good = dict(rows=2, n=100, sem=-1, end=0, logits=P, dtype=0, hist=P, hlen=P, cols=5, pen=P, bias=P, bs=100, mask=P,
                ms=4, out=P, stream=None)
    _bad(lib.s2_adjust_logits, good, rows=[0, 65536], n=[0, -1], logits=[None, P + 2], dtype=[3], hist=[None, P + 1],
         hlen=[P + 2], cols=[0, -1], pen=[None, P + 2], bias=[P + 2], bs=[99, -1], mask=[P + 1], ms=[3, -1],
         out=[None, P + 2])
    _bad(lib.s2_adjust_logits, dict(good, sem=5), n=[1])


def test_python_checks():
    torch = pytest.importorskip("torch")
    import dual_ar_tts_gb300 as pkg
    x = torch.zeros((2, 64))
    for call in (lambda: pkg.quantize_q4(x), lambda: pkg.q4_matmul(x, x, x), lambda: pkg.adjust_logits(x),
                 lambda: pkg.adjust_logits(x.double()), lambda: pkg.kv4_read(x, x, x, x, 1),
                 lambda: pkg.kv4_attention(x[None], x, x, x, x), lambda: pkg.kv4_append(x, x, x, x, x, x, 1),
                 lambda: pkg.kv4_pages(1, 1, 96)):
        with pytest.raises(ValueError):
            call()


def test_q4_matmul_sizes(lib):
    """The largest counts are taken, one more is not; a workspace serves whatever matrix follows."""
    import dual_ar_tts_gb300 as pkg
    assert lib.s2_q4_matmul_workspace(1 << 21, 128, pkg.S2_F32) > 0
    assert lib.s2_q4_matmul_workspace((1 << 21) + 1, 128, pkg.S2_F32) == 0
    assert lib.s2_q4_matmul_workspace(40, (1 << 28) + 1, pkg.S2_BF16) == 0
    sizes = [lib.s2_q4_matmul_workspace(n, 2560, pkg.S2_BF16) for n in (1, 8, 9, 16, 17, 32, 33, 64, 65, 500)]
    assert sizes[0] == 0 and all(a <= b for a, b in zip(sizes[2:], sizes[3:]))


def test_rows_of_any_stride_are_taken():
    """What q4_matmul and kv4_append do with their rows: a start and a stride that the library takes, the values as
    they were.  torch lets a single row have any stride."""
    torch = pytest.importorskip("torch")
    import dual_ar_tts_gb300 as pkg
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        wide, k = torch.randn((4, 260)).to(dt), 256
        rows = [wide[:, :k], wide[0:1, :k], wide[1:2, 1:1 + k], wide[:1, 2:2 + k], wide[3:, 4:], wide[::2, :k],
                torch.randn((k, 1)).to(dt).t(), torch.randn((k, 3)).to(dt).t(), torch.randn((k, 3)).to(dt).t()[1:2],
                wide[:1, :k].expand(3, k), torch.randn(k).to(dt).as_strided((1, k), (0, 1)),
                torch.randn(2 * k).to(dt)[::2][None], torch.randn(k + 1).to(dt)[1:][None]]
        for x in rows:
            y, stride = pkg._rows16(x)
            assert y.shape == x.shape and torch.equal(y, x)
            assert y.data_ptr() % 16 == 0 and stride >= k and stride * y.element_size() % 16 == 0
            assert y.stride(1) == 1 and (y.shape[0] == 1 or y.stride(0) == stride)


def test_q4_matmul_alignment_of_scales(lib):
    good = dict(n=2, x=P, dtype=1, x_stride=128, codes=P, scales=P, m=4, k=128, group=32, y=P, ws=None, nb=0,
                stream=None)
    _bad(lib.s2_q4_matmul, good, scales=[P + 1, P + 2, P + 4, P + 12])
    for group in (64, 128):
        _bad(lib.s2_q4_matmul, dict(good, group=group), scales=[P + 1, P + 2, P + 6])
