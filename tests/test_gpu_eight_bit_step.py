"""The 8-bit operators run together: a layer of a small model over a batch of streams, its projections in 8-bit integers, its cache
in 4 bits.  Each stage is compared with its 64-bit form on what the stage before it left on the GPU, and a captured layer,
replayed while its inputs change, gives the eager bits."""
import pytest
import torch

import synth
from tests import eight_bit as eb

pytestmark = pytest.mark.gpu

D = synth.CONFIGS["tiny"]["dims"]
SURE = 127 * 2.0 ** -41


class Layer:
    def __init__(self, pkg, dtype, lengths):
        g = torch.Generator().manual_seed(4)
        self.pkg, self.dt, self.n = pkg, eb.TYPES[dtype], len(lengths)
        hq, hkv, hd, dim, f = D["n_head"], D["n_kv_head"], D["head_dim"], D["dim"], D["ffn"]
        shapes = dict(qkv=((hq + 2 * hkv) * hd, dim), wo=(dim, hq * hd), w13=(2 * f, dim), w2=(dim, f))
        self.w = {k: pkg.quantize_q8((torch.randn(s, generator=g) * 0.08).bfloat16().cuda()) for k, s in shapes.items()}
        self.norms = [(1 + 0.1 * torch.randn(dim, generator=g)).cuda() for _ in range(2)]
        self.rope = pkg.rope_table(512, hd, D["rope_base"])
        self.pages = pkg.kv4_pages(self.n * 4, hkv, hd)
        self.table = torch.randperm(self.n * 4, generator=g).to(torch.int32).view(self.n, 4).cuda().contiguous()
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.q_start = torch.arange(self.n + 1, dtype=torch.int32, device="cuda")
        self.x = torch.randn((self.n, dim), generator=g).to(self.dt).cuda()
        self.out = {}

    def run(self):
        p, o, dt, eps = self.pkg, self.out, self.dt, D["norm_eps"]
        place = (self.pages, self.table, self.q_start, self.lengths)
        o["h"] = p.rms_norm_q8(self.x, self.norms[0], eps)
        o["qkv"] = p.q8_matmul(*o["h"], *self.w["qkv"], dtype=dt)
        q = p.kv4_append(o["qkv"], *place, self.rope, D["n_head"])
        o["att"] = p.kv4_attention(q, *place).flatten(1)
        o["att8"] = p.quantize_q8(o["att"])
        o["proj"] = p.q8_matmul(*o["att8"], *self.w["wo"], dtype=dt)
        *o["h2"], o["mid"] = p.rms_norm_q8(o["proj"], self.norms[1], eps, residual=self.x)
        o["gate_up"] = p.q8_matmul(*o["h2"], *self.w["w13"], dtype=dt)
        o["act"] = p.swiglu_q8(o["gate_up"])
        o["down"] = p.q8_matmul(*o["act"], *self.w["w2"], dtype=dt)
        return o


def _product(codes, weights, dt):
    cpu = lambda t: t.cpu()    # noqa: E731
    return eb.product(cpu(codes[0]), cpu(codes[1]), cpu(weights[0]), cpu(weights[1]), dt)


def _codes(got, v, factor=1.0):
    want, scale, distance = eb.coded(v, factor)
    eb.check_codes(got[0].cpu(), want, distance, SURE)
    # 256 to 768 columns: 32 additions a thread, 12 across, as the operators' own tests count
    assert ((got[1].cpu().double() - scale).abs() <= ((32 + 12) / 2 + 16) * eb.STEP * scale).all()


@pytest.mark.parametrize("dtype", list(eb.TYPES))
@pytest.mark.parametrize("streams", [1, 4, 40])
def test_layer_stage_by_stage(streams, dtype):
    import dual_ar_tts_gb300 as pkg
    st = Layer(pkg, dtype, [1 + 5 * i for i in range(streams)])
    o, dt = st.run(), st.dt
    x, norms = st.x.cpu(), [t.cpu() for t in st.norms]
    v, r, _ = eb.norm(x, norms[0], D["norm_eps"])
    _codes(o["h"], v, r)
    assert torch.equal(o["qkv"].cpu(), _product(o["h"], st.w["qkv"], dt))
    _codes(o["att8"], o["att"].cpu().double())
    assert torch.equal(o["proj"].cpu(), _product(o["att8"], st.w["wo"], dt))
    v, r, total = eb.norm(o["proj"].cpu(), norms[1], D["norm_eps"], x)
    assert torch.equal(o["mid"].cpu(), total)
    _codes(o["h2"], v, r)
    assert torch.equal(o["gate_up"].cpu(), _product(o["h2"], st.w["w13"], dt))
    _codes(o["act"], eb.gate(o["gate_up"].cpu()))
    assert torch.equal(o["down"].cpu(), _product(o["act"], st.w["w2"], dt))


@pytest.mark.parametrize("streams", [2, 40])
def test_captured_layer(streams):
    import dual_ar_tts_gb300 as pkg
    eager, graph = [Layer(pkg, "bf16", [3 + i for i in range(streams)]) for _ in range(2)]
    graph.run()
    torch.cuda.synchronize()
    graph.pages.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.run()
    for step in range(3):
        want = eager.run()
        g.replay()
        for key in ("qkv", "att", "proj", "mid", "gate_up", "down"):
            assert torch.equal(graph.out[key], want[key]), (step, key)
        for st in (eager, graph):
            st.x.copy_((st.out["mid"] + st.out["down"]) / 1.5)
            st.lengths += 1


def test_quality_of_a_layer():
    """What 8 bits cost: a projection of normal activations and weights is within a few thousandths of the unquantised one (a step is
    max / 127, some 3.5 deviations; its rounding's deviation, step / sqrt(12), is 0.8 % of a value's on either side)."""
    import dual_ar_tts_gb300 as pkg
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = [torch.randn(s, generator=g, device="cuda") for s in ((64, 2560), (2560, 2560))]
    y = pkg.q8_matmul(*pkg.quantize_q8(x), *pkg.quantize_q8(w), dtype=torch.float32)
    want = x.double() @ w.double().t()
    assert ((y.double() - want).norm() / want.norm()) < 0.02


@pytest.mark.parametrize("n,m,k", [(1, 512, 2560), (12, 2560, 512), (40, 2560, 1024), (300, 4864, 512)])
def test_run_on_the_same_buffers(n, m, k):
    """Calls may begin before the one in front of them has ended: a run of them in which each writes what the one in front reads,
    and reads what it writes, eager and captured, gives what calls with buffers of their own give."""
    import dual_ar_tts_gb300 as pkg
    g = torch.Generator(device="cuda").manual_seed(n)
    ws = [pkg.quantize_q8(torch.randn((m, k), generator=g, device="cuda") * 0.05) for _ in range(3)]
    raw = [pkg.dequantize_q8(*w) for w in ws]
    xs = [torch.randn((n, k), generator=g, device="cuda") for _ in range(3)]
    norm = 1 + 0.1 * torch.randn(k, generator=g, device="cuda")
    want = []
    for i in range(12):
        c, s, total = pkg.rms_norm_q8(xs[i % 3], norm, residual=xs[(i + 1) % 3])
        torch.cuda.synchronize()
        y = pkg.q8_matmul(c, s, *ws[i % 3], dtype=torch.float32)
        torch.cuda.synchronize()
        want.append((c, s, total, y, *pkg.swiglu_q8(y)))
        torch.cuda.synchronize()
    i8 = dict(dtype=torch.int8, device="cuda")
    f32 = dict(device="cuda")
    codes, scales, total = torch.empty((n, k), **i8), torch.empty(n, **f32), torch.empty((n, k), **f32)
    wc, wsc, y = torch.empty((m, k), **i8), torch.empty(m, **f32), torch.empty((n, m), **f32)
    act = torch.empty((n, (m // 2 + 15) // 16 * 16), **i8), torch.empty(n, **f32)
    got = [[torch.empty_like(t) for t in w] for w in want]

    def run():
        for i in range(12):
            pkg.quantize_q8(raw[i % 3], wc, wsc)                        # the weights that the product before this reads
            pkg.rms_norm_q8(xs[i % 3], norm, 1e-6, xs[(i + 1) % 3], total, codes, scales)
            pkg.q8_matmul(codes, scales, wc, wsc, out=y, dtype=torch.float32)
            pkg.swiglu_q8(y, *act)
            if i % 4 == 3:                                              # (a kernel of another kind now and then)
                for a, b in zip(got[i], (codes, scales, total, y, *act)):
                    a.copy_(b)

    def check():
        for i in range(3, 12, 4):
            for j, (a, b) in enumerate(zip(got[i], want[i])):
                assert torch.equal(a, b), (i, j)

    for _ in range(20):
        run()
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(20):
        for o in got:
            for t in o:
                t.zero_()
        graph.replay()
        check()
