"""Products of 8-bit integers on tcgen05: every form of the kernel (single blocks, split ones, pairs; results by TMA and by plain
stores), many tiles a block, weights that come late, waits that give up, streams and graphs."""
import pytest
import torch

from tests import eight_bit as eb

pytestmark = pytest.mark.gpu


def _operands(n, m, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, w = [torch.randint(-128, 128, (r, k), generator=g, device="cuda").to(torch.int8) for r in (n, m)]
    xs, ws = [torch.rand(r, generator=g, device="cuda") * 0.01 + 0.005 for r in (n, m)]
    return x, xs, w, ws


def _want(ops, dtype):
    x, xs, w, ws = ops
    return ((x.double() @ w.double().t()).float() * xs[:, None] * ws).to(dtype)


# one tile, split K, whole rounds, several tiles a block, pairs; rows of results on 16 bytes and not; a last step and a last tile
# that are not whole
FORMS = [(65, 1024, 4096), (130, 1030, 4112), (512, 2560, 272), (520, 2555, 1040), (3000, 1000, 1024), (3000, 1001, 1040),
         (40, 19456, 256), (300, 19457, 1040), (256, 19456, 1024), (1030, 9728, 1152), (2100, 9721, 144), (700, 10000, 16)]


@pytest.mark.parametrize("dtype", list(eb.TYPES))
@pytest.mark.parametrize("n,m,k", FORMS)
def test_forms(n, m, k, dtype):
    import dual_ar_tts_gb300 as pkg
    ops, dt = _operands(n, m, k, n + k), eb.TYPES[dtype]
    # rows behind and before the result stay as they were
    room = torch.full((n + 2, m), 7.0, dtype=dt, device="cuda")
    out = room[1:n + 1]
    pkg.q8_matmul(*ops, dtype=dt, out=out)
    assert torch.equal(out, _want(ops, dt))
    assert (room[0] == 7).all() and (room[-1] == 7).all()


@pytest.mark.parametrize("n,m,k", [(40, 2560, 9728), (128, 2560, 9728), (33, 19456, 2560), (600, 6144, 2560)])
def test_many_calls_on_cold_weights(n, m, k):
    """Copies that arrive late and out of order: calls in a row, each on weights that are not in L2."""
    import dual_ar_tts_gb300 as pkg
    sets = [_operands(n, m, k, i) for i in range(8)]
    want = [_want(ops, torch.float32) for ops in sets]
    out = [torch.empty((n, m), device="cuda") for _ in sets]
    for _ in range(25):
        for ops, y in zip(sets, out):
            pkg.q8_matmul(*ops, dtype=torch.float32, out=y)
    for y, w in zip(out, want):
        assert torch.equal(y, w)


@pytest.mark.parametrize("n,m,k", [(100, 6144, 512), (64, 2560, 4096), (128, 2560, 4096), (300, 19456, 512), (2100, 9721, 144)])
def test_waits_that_give_up(n, m, k):
    """A wait on the device that gives up leaves NaN, whatever was in the output, and the next call is right."""
    import dual_ar_tts_gb300 as pkg
    ops = _operands(n, m, k, 3)
    out = torch.zeros((n, m), device="cuda")
    pkg.s2_set_wait_limit(0)
    try:
        pkg.q8_matmul(*ops, dtype=torch.float32, out=out)
        torch.cuda.synchronize()
    finally:
        pkg.s2_set_wait_limit(-1)
    assert torch.isnan(out).all()
    pkg.q8_matmul(*ops, dtype=torch.float32, out=out)
    assert torch.equal(out, _want(ops, torch.float32))


def test_streams():
    """Calls of every form at once, on streams of their own."""
    import dual_ar_tts_gb300 as pkg
    shapes = [(3, 6144, 2560), (64, 2560, 9728), (300, 19456, 512), (100, 6144, 512)]
    sets = [_operands(*s, i) for i, s in enumerate(shapes)]
    want = [_want(ops, torch.bfloat16) for ops in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    out = [torch.empty(w.shape, dtype=torch.bfloat16, device="cuda") for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for ops, y, st in zip(sets, out, streams):
            with torch.cuda.stream(st):
                pkg.q8_matmul(*ops, out=y)
    torch.cuda.synchronize()
    for y, w in zip(out, want):
        assert torch.equal(y, w)


@pytest.mark.parametrize("n,m,k", [(3, 2560, 2560), (60, 2560, 4096), (300, 19456, 512)])
def test_captured(n, m, k):
    """Two graphs of the same call replayed on inputs that change under them."""
    import dual_ar_tts_gb300 as pkg
    ops = _operands(n, m, k, 1)
    outs = [torch.empty((n, m), device="cuda") for _ in range(2)]
    pkg.q8_matmul(*ops, dtype=torch.float32, out=outs[0])
    torch.cuda.synchronize()
    graphs = []
    for y in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkg.q8_matmul(*ops, dtype=torch.float32, out=y)
        graphs.append(g)
    for seed in (2, 3):
        for t, s in zip(ops, _operands(n, m, k, seed)):
            t.copy_(s)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = _want(ops, torch.float32)
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_first_call_captured():
    """The first call of a form may be a captured one."""
    import subprocess
    import sys
    code = ("import torch, dual_ar_tts_gb300 as pkg\n"
            "x = torch.randint(-9, 9, (70, 512), device='cuda', dtype=torch.int8)\n"
            "w = torch.randint(-9, 9, (2560, 512), device='cuda', dtype=torch.int8)\n"
            "a, b = torch.rand(70, device='cuda'), torch.rand(2560, device='cuda')\n"
            "y = torch.empty((70, 2560), device='cuda')\n"
            "torch.cuda.synchronize()\n"
            "g = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(g):\n"
            "    pkg.q8_matmul(x, a, w, b, dtype=torch.float32, out=y)\n"
            "g.replay()\n"
            "torch.cuda.synchronize()\n"
            "assert torch.equal(y, (x.double() @ w.double().t()).float() * a[:, None] * b)\n")
    assert subprocess.run([sys.executable, "-c", code], timeout=240).returncode == 0
