"""The 4-bit operators run together, as a decode step and as a stream's store.

A step of a small model over a batch of streams: q/k/v projection with 4-bit weights, append (norm,
rotation, 4-bit cache), attention, output projection, logits, adjustment, draw.  Each stage is
compared with its plain 64-bit form on the inputs that the stage before it produced on the GPU (a
rounding of a cached code is a step, not an error that a tolerance could follow through), and a
captured step, replayed while lengths and histories advance on the device, gives the eager bits.

A stream's keys and values kept in the 4-bit cache are read back into s2_stream_import, and the
decoder continues from them exactly as from the same fp16 values."""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests import four_bit as fb

pytestmark = pytest.mark.gpu

D = synth.CONFIGS["tiny"]["dims"]


class Step:
    """One layer and the logits of a small model, on caller buffers."""

    def __init__(self, pkg, dtype, lengths, group):
        g = torch.Generator().manual_seed(4)
        self.pkg, self.group, self.dt = pkg, group, fb.TYPES[dtype]
        hq, hkv, hd = D["n_head"], D["n_kv_head"], D["head_dim"]
        self.n = len(lengths)
        shapes = dict(qkv=((hq + 2 * hkv) * hd, D["dim"]), wo=(D["dim"], hq * hd), head=(D["codebook_size"] + 1, D["dim"]))
        self.w = {k: pkg.quantize_q4((torch.randn(s, generator=g) * 0.08).bfloat16().cuda(), group) for k, s in shapes.items()}
        self.qn, self.kn = [(1 + 0.1 * torch.randn(hd, generator=g)).cuda() for _ in range(2)]
        self.rope = pkg.rope_table(512, hd, D["rope_base"])
        cols = 4
        self.pages = pkg.kv4_pages(self.n * cols, hkv, hd)
        host = torch.zeros(self.pages.shape, dtype=torch.uint8)
        fb.fill_random(host, np.random.default_rng(1))
        self.pages.copy_(host)
        perm = torch.randperm(self.n * cols, generator=g).to(torch.int32)
        self.table = perm.view(self.n, cols).cuda().contiguous()
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.q_start = torch.arange(self.n + 1, dtype=torch.int32, device="cuda")
        self.pen = torch.tensor([[1.2, 0.1, 0.2]] * self.n, device="cuda")
        self.hist = torch.zeros((self.n, 64), dtype=torch.int32, device="cuda")
        self.hist_len = torch.zeros(self.n, dtype=torch.int32, device="cuda")
        self.mask = torch.full((1, 3), -1, dtype=torch.int32, device="cuda")
        self.mask[0, 1] = 0x0F0F0F0F
        self.x = (torch.randn((self.n, D["dim"]), generator=g)).to(self.dt).cuda()
        self.expo = -torch.log(torch.rand((self.n, 30), generator=g)).cuda().clamp(min=1e-6)
        self.out = {}

    def run(self):
        p, o = self.pkg, self.out
        one = (self.pages, self.table, self.q_start, self.lengths)
        o["qkv"] = p.q4_matmul(self.x, *self.w["qkv"], self.group)
        o["q"] = p.kv4_append(o["qkv"], *one, self.rope, D["n_head"], self.qn, self.kn, D["norm_eps"])
        o["att"] = p.kv4_attention(o["q"], *one)
        o["proj"] = p.q4_matmul(o["att"].flatten(1), *self.w["wo"], self.group)
        o["logits"] = p.q4_matmul(self.x + o["proj"], *self.w["head"], self.group)
        o["adjusted"] = p.adjust_logits(o["logits"], history=self.hist, hist_len=self.hist_len, penalties=self.pen,
                                        mask=self.mask, sem_begin=D["sem_begin"], im_end=D["im_end"])
        o["ids"] = p.draw(o["adjusted"], self.expo, 0.8, 0.8, D["sem_begin"], D["im_end"])
        return o

    def advance(self):
        """What a serving loop does between steps, on the device."""
        self.hist.scatter_(1, self.hist_len[:, None].long(), self.out["ids"][:, None])
        self.hist_len += 1
        self.lengths += 1
        self.x.copy_((self.x + self.out["proj"]) / 1.5)


@pytest.mark.parametrize("dtype,group", [("fp32", 32), ("bf16", 64), ("fp16", 128)])
def test_step_stage_by_stage(dtype, group):
    import dual_ar_tts_gb300 as pkg
    st = Step(pkg, dtype, [1, 64, 65, 130], group)
    ids = oracle.admissible_ids(D)
    for _ in range(3):
        o = {k: v.cpu() for k, v in st.run().items()}
        x = st.x.cpu()
        res = (st.x + st.out["proj"]).cpu()
        for name, a, k in (("qkv", x, D["dim"]), ("proj", o["att"].flatten(1), D["n_head"] * D["head_dim"]),
                           ("logits", res, D["dim"])):
            w = fb.q4_values(*st.w[{"qkv": "qkv", "proj": "wo", "logits": "head"}[name]], k, group)
            want, size = a.double() @ w.t(), a.double().abs() @ w.abs().t()
            tol = (k / 16 + 32) * 2.0 ** -23 * size + fb.rounding(want, st.dt)
            assert ((o[name].double() - want).abs() <= tol).all(), name
        pages, table, lengths = st.pages.cpu(), st.table.cpu(), st.lengths.tolist()
        hq, hkv, hd = D["n_head"], D["n_kv_head"], D["head_dim"]
        cs = st.rope.cpu()[torch.tensor(lengths) - 1][:, None]
        f = o["qkv"].float().view(st.n, -1, hd)
        k32 = fb.norm_rotate(f[:, hq:hq + hkv], st.kn.cpu(), D["norm_eps"], cs)
        q32 = fb.norm_rotate(f[:, :hq], st.qn.cpu(), D["norm_eps"], cs)
        # both sides round fp32 six times at most, from a mean square equal to one rounding, then to the type
        assert ((o["q"].float() - q32).abs() <= 16 * 2.0 ** -24 * q32.abs().amax(-1, keepdim=True)
                + 2 * fb.rounding(q32, st.dt)).all()
        for i, L in enumerate(lengths):
            page, slot = [int(p) for p in table[i, :-(-L // 64)]], (L - 1) % 64
            for part, row in ((0, k32[i]), (1, f[i, hq + hkv:])):
                c, s, z = fb.kv_quantise(row)
                got = fb.get(pages, part, page[-1:])[:, slot]
                off = (got.float() - fb.kv_value(c, s, z).float()).abs()
                assert (off <= s.float().repeat_interleave(32, -1) * 1.01).all() and (off > 0).float().mean() < 0.01
            for h in range(hq):
                kv = [fb.get(pages[:, h // (hq // hkv)][:, None], part, page)[0, :L] for part in range(2)]
                want, rel, wv, tiny = fb.attention(o["q"][i, h][None], *kv, [L], hd ** -0.5)
                assert ((o["att"][i, h][None].double() - want).abs() <= fb.attention_tol(want, rel, wv, tiny, st.dt)).all()
        for i in range(st.n):
            l = o["logits"][i].double().numpy().copy()
            seen = st.hist[i, :int(st.hist_len[i])].cpu().numpy()
            for e, t in enumerate(ids):
                c = int((seen == t).sum())
                if c:
                    l[e] = (l[e] / 1.2 if l[e] > 0 else l[e] * 1.2) - 0.1 * c - 0.2
            bits = (st.mask.cpu().numpy().view(np.uint32)[0, np.arange(len(l)) // 32] >> (np.arange(len(l)) % 32)) & 1
            l[bits == 0] = -np.inf
            got = o["adjusted"][i].numpy()
            assert np.array_equal(np.isinf(got), np.isinf(l)) and np.abs(got[bits == 1] - l[bits == 1]).max() <= 1e-5
            tok, diag = oracle.draw(got.copy(), 0.8, 0.8, 30, st.expo[i].cpu().numpy(), ids)
            if float(diag[1]) > 1e-5 and float(diag[2]) - float(diag[3]) > 1e-5:
                assert int(o["ids"][i]) == int(tok)
        st.advance()


def test_step_captured_and_replayed():
    import dual_ar_tts_gb300 as pkg
    eager, graphed = [Step(pkg, "bf16", [60, 63, 100], 32) for _ in range(2)]
    want = []
    for _ in range(6):
        want.append({k: v.clone() for k, v in eager.run().items()})
        eager.advance()
    state = ("pages", "lengths", "hist", "hist_len", "x")
    first = {k: getattr(graphed, k).clone() for k in state}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.run()
        graphed.advance()
    torch.cuda.synchronize()
    for k, v in first.items():
        getattr(graphed, k).copy_(v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed.run()
        graphed.advance()
    for i in range(6):
        g.replay()
        for k, v in want[i].items():
            assert torch.equal(graphed.out[k], v), (i, k)
    assert torch.equal(graphed.pages, eager.pages)


def test_stream_kept_in_four_bits_continues():
    """Keys and values of every layer in one pool of pages; read back, imported, decoded: the same frames as from
    the fp16 values that the definition gives."""
    import dual_ar_tts_gb300 as pkg
    d = synth.MINI
    n_pos, n_frames = 150, 4
    L, H, hd = d["n_layer"], d["n_kv_head"], d["head_dim"]
    k16, v16, x_last = synth.kv_state(5, 0, d, n_pos)
    kd, vd = [torch.from_numpy(a.view(np.int16)).cuda().view(torch.float16) for a in (k16, v16)]
    rope = torch.zeros((n_pos, hd // 2, 2), device="cuda")             # the keys are rotated already
    rope[..., 0] = 1
    cols = -(-n_pos // 64)
    pages = pkg.kv4_pages(L * cols, H, hd)
    q_start = torch.tensor([0, n_pos], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([n_pos], dtype=torch.int32, device="cuda")
    ks, vs = [], []
    for l in range(L):
        table = torch.arange(l * cols, (l + 1) * cols, dtype=torch.int32, device="cuda")[None].contiguous()
        rows = torch.cat([kd[l].transpose(0, 1), vd[l].transpose(0, 1)], 1).flatten(1).contiguous()
        pkg.kv4_append(rows, pages, table, q_start, lengths, rope, 0)
        k, v = pkg.kv4_read(pages, table, q_start, lengths, n_pos)
        ks.append(k)
        vs.append(v)
    k, v = torch.stack(ks), torch.stack(vs)
    for got, src in ((k, kd), (v, vd)):
        assert torch.equal(got.cpu(), fb.kv_value(*fb.kv_quantise(src.cpu())))
    w = pkg.upload_weights(synth.make_weights(d, 5, norm_jitter=0.1))
    expo = torch.from_numpy(synth.expo(5, 0, n_frames)).cuda()[None]
    s = synth.sampling("tiny", min_tokens_before_end=n_frames)
    outs = []
    for kk, vv in ((k, v), [fb.kv_value(*fb.kv_quantise(t.cpu())).cuda() for t in (kd, vd)]):
        dec = pkg.Decoder(d, w, max_streams=1, kv_slots=256)
        dec.import_stream(0, kk, vv, torch.from_numpy(x_last).cuda())
        outs.append(dec.decode(n_frames, s, expo)["codes"].cpu())
        assert dec.sync_status() == pkg.S2_OK
        dec.close()
    assert torch.equal(*outs)
