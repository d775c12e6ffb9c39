"""What is measured of the 4-bit serving operators: projections with 4-bit weights, the paged 4-bit
key/value cache (appending to it, reading it back, attention over it) and the adjustment of logits
before a draw.

``own`` chooses the side: False computes every operator in its plain form (elementary torch
operations in 32 bits, rounded once at the end), True calls ``dual_ar_tts_gb300``.  Both take the
same tensors in the layouts that ``include/s2frame.h`` describes.
"""
import math
import random

import torch

own = False

PAGE = 64            # positions in a cache page
GROUP = 32           # head elements that share a scale and a zero point in the cache
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one row through a small model's projection: the smallest call, all latency
        dict(name="matmul small", op="matmul", rows=3, m=97, k=256, group=32, dtype="fp16"),
        # one stream's gate and up projection, fp32 activations as the decode keeps them
        dict(name="matmul gate/up 1 row", op="matmul", rows=1, m=19456, k=2560, group=32, dtype="fp32"),
        # 32 streams decoded together: the down projection
        dict(name="matmul down 32 rows", op="matmul", rows=32, m=2560, k=9728, group=128, dtype="bf16"),
        # one token of a small model appended and read back
        dict(name="append 1 token", op="append", seqs=1, q_most=1, len_lo=33, len_hi=33, hq=4, hkv=2, hd=64,
             norm=False, dtype="fp32", mix=1),
        # 32 streams, one token each, with the per-head norms
        dict(name="append 32 streams", op="append", seqs=32, q_most=1, len_lo=512, len_hi=4096, hq=32, hkv=8, hd=128,
             norm=True, dtype="bf16", mix=2),
        # prompts of several streams, whole
        dict(name="append prompts", op="append", seqs=8, q_most=1000, len_lo=1000, len_hi=1500, hq=32, hkv=8, hd=128,
             norm=True, dtype="fp16", mix=3),
        # one token of one small stream: latency
        dict(name="attention short", op="attention", seqs=1, q_most=1, len_lo=17, len_hi=17, hq=4, hkv=2, hd=64,
             dtype="fp32", mix=4),
        # 32 streams of different lengths, one token each
        dict(name="attention 32 streams", op="attention", seqs=32, q_most=1, len_lo=512, len_hi=4096, hq=32, hkv=8,
             hd=128, dtype="fp16", mix=5),
        # 8 streams with 30000 positions each
        dict(name="attention long context", op="attention", seqs=8, q_most=1, len_lo=30000, len_hi=30000, hq=32, hkv=8,
             hd=128, dtype="bf16", mix=6),
        # pieces of prompts of several streams after what is cached of them
        dict(name="attention prompt pieces", op="attention", seqs=5, q_most=512, len_lo=700, len_hi=3000, hq=32, hkv=8,
             hd=128, dtype="bf16", mix=7),
        # one stream's main logits before its draw
        dict(name="logits 1 row", op="logits", rows=1, n=4097, hist=10, per_row_bias=False, dtype="fp32", mix=8),
        # 32 rows over the whole vocabulary, long histories, a grammar mask for each row
        dict(name="logits vocabulary", op="logits", rows=32, n=155776, hist=2048, per_row_bias=True, dtype="bf16", mix=9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["matmul", "append", "attention", "logits"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    mix = rng.randrange(1 << 20)
    if op == "matmul":
        group = rng.choice([32, 64, 128])
        k = group * max(1, _log(rng, 64, 9728) // group)
        return dict(op=op, rows=_log(rng, 1, 32), m=_log(rng, 40, 19456 * 2560 // max(k, 2560)), k=k, group=group,
                    dtype=dtype)
    if op == "logits":
        return dict(op=op, rows=_log(rng, 1, 32), n=_log(rng, 33, 155776), hist=_log(rng, 1, 2048),
                    per_row_bias=rng.random() < 0.5, dtype=dtype, mix=mix)
    hq, hkv = rng.choice([(32, 8), (8, 8), (4, 2), (16, 1), (12, 4), (9, 3)])
    hd = rng.choice([64, 128])
    if op == "append":
        seqs = _log(rng, 1, 32)
        q_most = 1 if rng.random() < 0.4 else _log(rng, 2, 4000 // seqs)
        lo = _log(rng, q_most, 4000)
        return dict(op=op, seqs=seqs, q_most=q_most, len_lo=lo, len_hi=_log(rng, lo, 4200), hq=hq, hkv=hkv, hd=hd,
                    norm=rng.random() < 0.5, dtype=dtype, mix=mix)
    if rng.random() < 0.6:
        seqs = _log(rng, 1, 32)
        hi = _log(rng, 1, min(30000, 240000 // seqs))
        return dict(op=op, seqs=seqs, q_most=1, len_lo=_log(rng, 1, hi), len_hi=hi, hq=hq, hkv=hkv, hd=hd, dtype=dtype,
                    mix=mix)
    seqs = _log(rng, 1, 5)
    q_most = _log(rng, 2, 512)
    lo = _log(rng, 1, 2500)
    return dict(op=op, seqs=seqs, q_most=q_most, len_lo=lo, len_hi=_log(rng, lo, 3000), hq=hq, hkv=hkv, hd=hd,
                dtype=dtype, mix=mix)


def _spans(case):
    """(new rows, cached length with them) of each sequence, from the case alone."""
    r = random.Random(case["mix"])
    out = []
    for i in range(case["seqs"]):
        n = case["q_most"] if i == 0 else r.randint(1, case["q_most"])
        out.append((n, max(n, _log(r, case["len_lo"], case["len_hi"]))))
    return out


# ---------------------------------------------------------------- the inputs

def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _triangle(g, shape):
    """Bytes of two 4-bit codes, each more likely near the middle of its range."""
    a = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    b = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    lo = ((a & 15) + (b & 15)) >> 1
    hi = ((a >> 4) + (b >> 4)) >> 1
    return lo | (hi << 4)


def _cache(case, g, spans, filled):
    """A pool of pages with the table of each sequence's pages (in no order), the rows' bounds and the lengths."""
    hkv, hd = case["hkv"], case["hd"]
    need = [-(-length // PAGE) for _, length in spans]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).tolist()
    table = torch.zeros((len(spans), max(need)), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    half, meta = PAGE * hd // 2, PAGE * hd // GROUP * 4
    pages = torch.zeros((n_pages, hkv, 2 * (half + meta)), dtype=torch.uint8, device="cuda")
    if filled:
        for part in range(2):
            o = part * (half + meta)
            pages[:, :, o:o + half] = _triangle(g, (n_pages, hkv, half))
            m = pages[:, :, o + half:o + half + meta].view(torch.float16)
            shape = (n_pages, hkv, PAGE * hd // GROUP)
            m[:, :, 0::2] = (0.27 * torch.exp(0.2 * torch.randn(shape, generator=g, device="cuda"))).half()
            m[:, :, 1::2] = torch.randint(5, 11, shape, generator=g, device="cuda").half()
    q_start = [0]
    for n, _ in spans:
        q_start.append(q_start[-1] + n)
    return dict(pages=pages, table=table.cuda(), q_start=torch.tensor(q_start, dtype=torch.int32, device="cuda"),
                lengths=torch.tensor([length for _, length in spans], dtype=torch.int32, device="cuda"),
                rows=q_start[-1], q_most=max(n for n, _ in spans), max_len=max(length for _, length in spans))


def _rope(n_pos, hd, base=1e6):
    """cos and sin of position * base^(-2i/hd), angles in 64 bits, held in bf16 precision as the decode's table."""
    theta = base ** (-2.0 * torch.arange(hd // 2, device="cuda", dtype=torch.float64) / hd)
    a = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * theta
    return torch.stack([a.cos(), a.sin()], -1).float().bfloat16().float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "matmul":
        m, k, group = case["m"], case["k"], case["group"]
        kp = -(-k // 128) * 128
        codes = _triangle(g, (m, kp // 2))
        scales = (0.01 * torch.exp(0.3 * torch.randn((m, kp // group), generator=g, device="cuda"))).bfloat16()
        if kp > k:  # what pads a row to whole blocks of 128
            c = codes.view(m, kp // 128, 4, 4, 4)
            c[:, -1, :, (k % 128) // 32:] = 0x88
            scales[:, k // group:] = 0
        return dict(case=case, x=_normal(g, (case["rows"], k), dt), codes=codes, scales=scales)
    if op == "logits":
        rows, n = case["rows"], case["n"]
        hist = torch.randint(0, n, (rows, case["hist"]), generator=g, device="cuda", dtype=torch.int32)
        again = torch.rand(hist.shape, generator=g, device="cuda") < 0.4  # repeated tokens
        hist = torch.where(again, hist[:, :1] % max(1, n // 2) + hist % 7 % n, hist).clamp_(max=n - 1)
        r = random.Random(case["mix"])
        hist_len = [case["hist"] if i == 0 else r.randint(0, case["hist"]) for i in range(rows)]
        pen = torch.rand((rows, 3), generator=g, device="cuda")
        pen = torch.stack([1.0 + 0.4 * pen[:, 0], 0.5 * pen[:, 1], 0.5 * pen[:, 2]], -1).contiguous()
        bias = _normal(g, (rows if case["per_row_bias"] else 1, n), torch.float32, 0.5)
        mask = torch.randint(-2 ** 31, 2 ** 31, (rows, -(-n // 32)), generator=g, device="cuda").to(torch.int32)
        return dict(case=case, logits=_normal(g, (rows, n), dt, 3.0), hist=hist.contiguous(),
                    hist_len=torch.tensor(hist_len, dtype=torch.int32, device="cuda"), pen=pen, bias=bias, mask=mask)
    spans = _spans(case)
    s = _cache(case, g, spans, op == "attention")
    s["case"] = case
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    if op == "append":
        std = torch.exp(0.5 * torch.randn((hq + 2 * hkv) * hd, generator=g, device="cuda"))
        s["qkv"] = (torch.randn((s["rows"], (hq + 2 * hkv) * hd), generator=g, device="cuda") * std).to(dt)
        s["rope"] = _rope(s["max_len"], hd)
        s["q_norm"] = (1.0 + _normal(g, (hd,), torch.float32, 0.1)) if case["norm"] else None
        s["k_norm"] = (1.0 + _normal(g, (hd,), torch.float32, 0.1)) if case["norm"] else None
    else:
        s["q"] = _normal(g, (s["rows"], hq, hd), dt)
    return s


# ------------------------------------------------------------- the plain forms

def _nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _weights(codes, scales, k, group, dtype):
    """The matrix that codes and scales stand for.  In a block of 128 columns, word 4c + j (8 codes) holds columns
    32j + 8c .. 32j + 8c + 7."""
    m = codes.shape[0]
    c = _nibbles(codes.view(m, -1, 4, 4, 4).transpose(2, 3).reshape(m, -1)).to(dtype) - 8.0
    return (c.view(m, -1, group) * scales.to(dtype)[:, :, None]).view(m, -1)[:, :k]


def _plain_matmul(s):
    c = s["case"]
    w = _weights(s["codes"], s["scales"], c["k"], c["group"], torch.float32)
    return (s["x"].float() @ w.t()).to(s["x"].dtype)


def _plain_logits(s):
    n = s["case"]["n"]
    hist, rows = s["hist"].long(), s["hist"].shape[0]
    live = torch.arange(hist.shape[1], device="cuda")[None] < s["hist_len"][:, None]
    count = torch.zeros((rows, n), device="cuda").scatter_add_(1, hist, live.float())
    x = s["logits"].float()
    rep, freq, pres = s["pen"][:, 0:1], s["pen"][:, 1:2], s["pen"][:, 2:3]
    x = torch.where(count > 0, torch.where(x > 0, x / rep, x * rep) - freq * count - pres, x) + s["bias"]
    bit = (s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    return torch.where(bit.reshape(rows, -1)[:, :n] != 0, x, -math.inf)


def _places(s):
    """Sequence and position of each row."""
    row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["q_start"][1:], row, right=True)
    return seq, s["lengths"][seq] - (s["q_start"][seq + 1] - row)


def _norm_rotate(x, w, eps, cs):
    if w is not None:
        mean = x.double().square().mean(-1, keepdim=True).float()
        x = x * (1.0 / torch.sqrt(mean + eps)) * w
    a, b = x[..., 0::2], x[..., 1::2]
    c, t = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.stack([a * c - b * t, b * c + a * t], -1).flatten(-2)


def _quantised(x):
    """Codes, scale and zero point of groups of 32, and the values they stand for."""
    g = x.clamp(-57344.0, 57344.0).unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = torch.maximum((hi - lo) / 15.0, torch.maximum(-lo, hi) / 127.0).half().float()
    some = scale > 0
    div = torch.where(some, scale, 1.0)
    zero = torch.where(some, torch.round(-lo / div).clamp(-127.0, 127.0), 0.0)
    code = torch.where(some, (torch.round(g / div) + zero).clamp(0.0, 15.0), 0.0)
    return code.flatten(-2).to(torch.uint8), scale, zero, (scale * (code - zero)).half().flatten(-2)


def _plain_append(s):
    c = s["case"]
    hq, hkv, hd, dt = c["hq"], c["hkv"], c["hd"], s["qkv"].dtype
    q, k, v = s["qkv"].float().unflatten(-1, (-1, hd)).split([hq, hkv, hkv], 1)
    seq, pos = _places(s)
    cs = s["rope"][pos]
    q = _norm_rotate(q, s["q_norm"], 1e-6, cs).to(dt)
    k = _norm_rotate(k, s["k_norm"], 1e-6, cs)
    page, slot = s["table"][seq, pos // PAGE], pos % PAGE
    half, meta = PAGE * hd // 2, PAGE * hd // GROUP * 4
    values = []
    for part, x in enumerate((k, v)):
        code, scale, zero, value = _quantised(x)
        o = part * (half + meta)
        to = s["pages"][:, :, o:o + half].unflatten(-1, (PAGE, hd // 2))
        to[page, :, slot] = code[..., 0::2] | (code[..., 1::2] << 4)
        to = s["pages"][:, :, o + half:o + half + meta].view(torch.float16).unflatten(-1, (PAGE, hd // GROUP, 2))
        to[page, :, slot] = torch.cat([scale, zero], -1).half()
        values.append(value.transpose(0, 1).contiguous())
    return q, values[0], values[1]


def _cached(s, part, dtype):
    """The keys (part 0) or values (1) of every sequence, [seq][head][position][head_dim], as held in fp16."""
    hd, table = s["case"]["hd"], s["table"].long()
    half, meta = PAGE * hd // 2, PAGE * hd // GROUP * 4
    o = part * (half + meta)
    code = s["pages"][:, :, o:o + half][table].unflatten(-1, (PAGE, hd // 2))
    m = s["pages"][:, :, o + half:o + half + meta].view(torch.float16)[table].unflatten(-1, (PAGE, hd // GROUP, 2))
    x = _nibbles(code).unflatten(-1, (-1, GROUP)).float()
    x = ((x - m[..., 1:].float()) * m[..., :1].float()).half().flatten(-2).transpose(1, 2)
    return x.flatten(2, 3).to(dtype)


def _plain_attention(s):
    c = s["case"]
    hq, hkv, hd = c["hq"], c["hkv"], c["hd"]
    seqs, most, n = s["lengths"].shape[0], s["q_most"], s["table"].shape[1] * PAGE
    at = torch.arange(most, device="cuda")
    count = (s["q_start"][1:] - s["q_start"][:-1])[:, None]
    live = at[None] < count
    row = torch.where(live, s["q_start"][:-1, None] + at, 0)
    q = s["q"][row].float().unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = q @ _cached(s, 0, torch.float32).transpose(2, 3) * (1.0 / math.sqrt(hd))
    last = s["lengths"][:, None] - count + at[None]  # the last position that a row sees
    seen = torch.arange(n, device="cuda")[None, None] <= last[:, :, None]
    score = score.view(seqs, hkv, -1, most, n).masked_fill_(~seen[:, None, None], -math.inf)
    score = score - score.amax(-1, keepdim=True)
    p = score.exp_()
    o = p.view(seqs, hkv, -1, n) @ _cached(s, 1, torch.float32)
    o = o / p.view(seqs, hkv, -1, n).sum(-1, keepdim=True)
    o = o.view(seqs, hkv, -1, most, hd).permute(0, 3, 1, 2, 4).reshape(seqs, most, hq, hd)
    return o[live].to(s["q"].dtype)


PLAIN = {"matmul": _plain_matmul, "append": _plain_append, "attention": _plain_attention, "logits": _plain_logits}


# --------------------------------------------------------- the framework's calls

def _own(s):
    import dual_ar_tts_gb300 as pkg
    c = s["case"]
    if c["op"] == "matmul":
        return pkg.q4_matmul(s["x"], s["codes"], s["scales"], c["group"])
    if c["op"] == "logits":
        return pkg.adjust_logits(s["logits"], history=s["hist"], hist_len=s["hist_len"], penalties=s["pen"],
                                 bias=s["bias"], mask=s["mask"])
    if c["op"] == "append":
        q = pkg.kv4_append(s["qkv"], s["pages"], s["table"], s["q_start"], s["lengths"], s["rope"], c["hq"],
                           q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6)
        k, v = pkg.kv4_read(s["pages"], s["table"], s["q_start"], s["lengths"], s["rows"])
        return q, k, v
    return pkg.kv4_attention(s["q"], s["pages"], s["table"], s["q_start"], s["lengths"], max_len=s["max_len"])


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------------------- work

def work(case):
    op, size = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op == "matmul":
        n, m, k = case["rows"], case["m"], case["k"]
        return {"bytes": m * k / 2 + 2 * m * (k // case["group"]) + size * n * (m + k), "flops": 2.0 * n * m * k}
    if op == "logits":
        n, rows = case["n"], case["rows"]
        bias = n * 4 * (rows if case["per_row_bias"] else 1)
        return {"bytes": rows * n * (size + 4) + bias + rows * (n / 8 + 4 * case["hist"]), "flops": 6.0 * rows * n}
    spans, hq, hkv, hd = _spans(case), case["hq"], case["hkv"], case["hd"]
    rows = sum(n for n, _ in spans)
    cached = 2 * hkv * (hd / 2 + hd / GROUP * 4)  # bytes of a position
    if op == "append":  # rows in, rotated queries and codes out, codes read back, values out
        moved = size * (2 * hq + 2 * hkv) * hd + 2 * cached + 2 * hkv * hd * 2 + hd * 4
        return {"bytes": rows * moved, "flops": rows * (10.0 * hq + 40.0 * hkv) * hd}
    seen = sum((length - n) * n + n * (n + 1) / 2 for n, length in spans)
    return {"bytes": sum(length for _, length in spans) * cached + 2 * size * rows * hq * hd,
            "flops": 4.0 * hq * hd * seen}


# ---------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, f8 = case["op"], torch.float64
    if op == "matmul":
        m, k, group = case["m"], case["k"], case["group"]
        col = torch.arange(k, device="cuda")
        byte = col // 128 * 64 + (col % 32 // 8) * 16 + (col % 128 // 32) * 4 + col % 8 // 2
        out = torch.empty((case["rows"], m), dtype=f8, device="cuda")
        for a in range(0, m, 4096):
            c = (s["codes"][a:a + 4096][:, byte] >> (col % 2 * 4).to(torch.uint8)) & 15
            w = (c.to(f8) - 8) * s["scales"][a:a + 4096].to(f8)[:, col // group]
            out[:, a:a + 4096] = s["x"].to(f8) @ w.t()
        return out
    if op == "logits":
        out = s["logits"].to(f8)
        for r in range(case["rows"]):
            rep, freq, pres = s["pen"][r].to(f8)
            tok, cnt = torch.unique(s["hist"][r, :int(s["hist_len"][r])].long(), return_counts=True)
            x = out[r, tok]
            out[r, tok] = torch.where(x > 0, x / rep, x * rep) - freq * cnt.to(f8) - pres
        out = out + s["bias"].to(f8)
        i = torch.arange(case["n"], device="cuda")
        out[((s["mask"].long()[:, i // 32] >> (i % 32)) & 1) == 0] = -math.inf
        return out
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    spans, table = _spans(case), s["table"].tolist()
    if op == "append":
        x = s["qkv"].to(f8).view(s["rows"], -1, hd)
        pos = torch.cat([torch.arange(length - n, length, device="cuda") for n, length in spans])
        turn = torch.view_as_complex(s["rope"].to(f8))[pos][:, None]
        if case["norm"]:
            r = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
            x = torch.cat([x[:, :hq] * r[:, :hq] * s["q_norm"].to(f8),
                           x[:, hq:hq + hkv] * r[:, hq:hq + hkv] * s["k_norm"].to(f8), x[:, hq + hkv:]], 1)
        qk = torch.view_as_complex(x[:, :hq + hkv].reshape(s["rows"], -1, hd // 2, 2).contiguous()) * turn
        qk = torch.view_as_real(qk).flatten(-2)
        out = [qk[:, :hq]]
        for y in (qk[:, hq:], x[:, hq + hkv:]):
            y = y.reshape(s["rows"], hkv, -1, GROUP).clamp(-57344, 57344)
            lo, hi = y.min(-1, True).values, y.max(-1, True).values
            step = torch.maximum((hi - lo) / 15, y.abs().amax(-1, keepdim=True) / 127).half().to(f8)
            zero = torch.round(-lo / step).clamp(-127, 127)
            value = step * ((torch.round(y / step) + zero).clamp(0, 15) - zero)
            value = torch.where(step > 0, value, torch.zeros_like(value))
            out.append(value.reshape(s["rows"], hkv, hd).transpose(0, 1).contiguous())
        return tuple(out)
    out = torch.empty((s["rows"], hq, hd), dtype=f8, device="cuda")
    half, meta = PAGE * hd // 2, PAGE * hd // GROUP * 4
    first = 0
    for i, (n, length) in enumerate(spans):
        kv = []
        for part in range(2):
            o = part * (half + meta)
            block = s["pages"][torch.tensor(table[i][:-(-length // PAGE)], device="cuda")]
            b = block[:, :, o:o + half].reshape(-1, hkv, PAGE, hd // 2)
            code = torch.empty(b.shape[:-1] + (hd,), dtype=f8, device="cuda")
            code[..., 0::2], code[..., 1::2] = (b & 15).to(f8), (b >> 4).to(f8)
            m = block[:, :, o + half:o + half + meta].contiguous().view(torch.float16).reshape(-1, hkv, PAGE, hd // 32, 2)
            x = (code - m[..., 1].to(f8).repeat_interleave(32, -1)) * m[..., 0].to(f8).repeat_interleave(32, -1)
            kv.append(x.half().to(f8).transpose(0, 1).reshape(hkv, -1, hd)[:, :length])
        late = torch.arange(length, device="cuda")[None] > torch.arange(length - n, length, device="cuda")[:, None]
        for h in range(hq):
            x = s["q"][first:first + n, h].to(f8) @ kv[0][h // (hq // hkv)].t() / math.sqrt(hd)
            out[first:first + n, h] = torch.softmax(x.masked_fill(late, -math.inf), -1) @ kv[1][h // (hq // hkv)]
        first += n
    return out
