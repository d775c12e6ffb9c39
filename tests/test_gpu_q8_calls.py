"""Calls of the 8-bit operators as programs make them: more blocks than a launch's other dimensions count, behind a join of two streams,
eager and captured, and what 8 bits cost."""
import threading

import pytest
import torch

from tests import eight_bit as eb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(1_100_000, 3), (131_100, 1025), (140_000, 2064)])
def test_more_than_65535_blocks(rows, cols):
    """A block holds 16 rows of 3 columns, one of more than 1024; reading back takes 2048 elements a block, 4096 of whole sixteens."""
    import dual_ar_tts_gb300 as pkg
    x = torch.randn((rows, cols), device="cuda", dtype=torch.bfloat16)
    w = torch.rand(cols, device="cuda") + 0.5
    codes, scales = pkg.quantize_q8(x)
    for at in (slice(0, 100), slice(65535 - 50, 65536 + 50), slice(rows - 100, rows)):
        for a, b in zip(pkg.quantize_q8(x[at]), (codes, scales)):
            assert torch.equal(a, b[at])
        want, scale, distance = eb.coded(x[at].cpu().double())
        eb.check_codes(codes[at].cpu(), want, distance)
        assert torch.equal(scales[at].cpu(), scale.float())
    back = pkg.dequantize_q8(codes, scales, cols, dtype=torch.bfloat16)
    # (in parts: the codes in fp32 would be four times as much)
    for part in torch.arange(rows, device="cuda").split(20_000):
        at = slice(int(part[0]), int(part[-1]) + 1)
        assert torch.equal(back[at], (codes[at, :cols].float() * scales[at, None]).bfloat16())
    codes, scales, total = pkg.rms_norm_q8(x, w, residual=back)
    for at in (slice(65536, 65636), slice(rows - 100, rows)):
        for a, b in zip(pkg.rms_norm_q8(x[at], w, residual=back[at]), (codes, scales, total)):
            assert torch.equal(a, b[at])
    if cols < 2000:
        gates = pkg.swiglu_q8(x[:, :cols - 1])
        for a, b in zip(pkg.swiglu_q8(x[rows - 100:, :cols - 1]), gates):
            assert torch.equal(a, b[rows - 100:])


def _join(pkg, st, other):
    """Activations on this stream, weights on the other, their product behind both."""
    main = torch.cuda.current_stream()
    other.wait_stream(main)
    pkg.rms_norm_q8(st["x"], st["norm"], codes=st["c"], scales=st["s"])
    with torch.cuda.stream(other):
        pkg.quantize_q8(st["w"], codes=st["wc"], scales=st["ws"])
    main.wait_stream(other)
    pkg.q8_matmul(st["c"], st["s"], st["wc"], st["ws"], out=st["y"], dtype=torch.float32)
    # and out again: the weights change on the other stream when the product has read them
    other.wait_stream(main)
    with torch.cuda.stream(other):
        pkg.dequantize_q8(st["wc"], st["ws"], out=st["w"])
    pkg.swiglu_q8(st["y"], codes=st["ac"], scales=st["as"])
    main.wait_stream(other)


def _state(n, m, k):
    i8 = dict(dtype=torch.int8, device="cuda")
    f32 = dict(device="cuda")
    return dict(x=torch.randn((n, k), **f32), norm=torch.rand(k, **f32) + 0.5, w=torch.randn((m, k), **f32), c=torch.empty((n, k), **i8),
                s=torch.empty(n, **f32), wc=torch.empty((m, k), **i8), ws=torch.empty(m, **f32), y=torch.empty((n, m), **f32),
                ac=torch.empty((n, m // 2), **i8), **{"as": torch.empty(n, **f32)})


@pytest.mark.parametrize("n,m,k", [(3, 6144, 2560), (60, 6144, 2560), (300, 4864, 2560)])
def test_joined_streams(n, m, k):
    """A call behind two streams' work, eager and as a captured fork and join, reads what both wrote."""
    import dual_ar_tts_gb300 as pkg
    st = _state(n, m, k)
    other = torch.cuda.Stream()
    _join(pkg, st, other)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _join(pkg, st, other)
    for step in range(12):
        st["x"].copy_(torch.randn_like(st["x"]))
        st["w"].copy_(torch.randn_like(st["w"]))
        for key in ("c", "wc", "ac"):
            st[key].zero_()
        x, w = st["x"].clone(), st["w"].clone()
        torch.cuda.synchronize()
        if step % 2:
            _join(pkg, st, other)
        else:
            graph.replay()
        torch.cuda.synchronize()
        c, wc = pkg.rms_norm_q8(x, st["norm"]), pkg.quantize_q8(w)
        torch.cuda.synchronize()
        y = pkg.q8_matmul(*c, *wc, dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(st["y"], y), step
        assert torch.equal(st["w"], pkg.dequantize_q8(*wc)) and torch.equal(st["ac"], pkg.swiglu_q8(y)[0]), step


def test_threads():
    """Calls from several threads at once, each on its own stream."""
    import dual_ar_tts_gb300 as pkg
    states = [_state(n, 2560, 1024) for n in (2, 40, 130, 300)]
    failed = []

    def work(st):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                pkg.rms_norm_q8(st["x"], st["norm"], codes=st["c"], scales=st["s"])
                pkg.quantize_q8(st["w"], codes=st["wc"], scales=st["ws"])
                pkg.q8_matmul(st["c"], st["s"], st["wc"], st["ws"], out=st["y"], dtype=torch.float32)
            torch.cuda.current_stream().synchronize()
            want = (st["c"].double() @ st["wc"].double().t()).float() * st["s"][:, None] * st["ws"]
            if not torch.equal(st["y"], want):
                failed.append(st["x"].shape)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(st,)) for st in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_cost_of_eight_bits():
    """A row of 2560 normal numbers has a largest one of 3.47 deviations (root mean square), its step is that / 127 and the rounding's
    deviation step / sqrt(12), 0.79 % of a value's; a product has two of them, 1.12 %.  A bit less on one side makes 1.8 %."""
    import dual_ar_tts_gb300 as pkg
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = [torch.randn(s, generator=g, device="cuda") for s in ((64, 2560), (2560, 2560))]
    y = pkg.q8_matmul(*pkg.quantize_q8(x), *pkg.quantize_q8(w), dtype=torch.float32)
    want = x.double() @ w.double().t()
    assert 0.010 < ((y.double() - want).norm() / want.norm()) < 0.0125
