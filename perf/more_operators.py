"""What is measured of the 8-bit serving operators: rows quantised to 8-bit integers with a scale each,
RMSNorm with the residual's sum and the feed-forward's gate with such an output, and the product of
8-bit activations with 8-bit weights.

``own`` chooses the side: False computes every operator in its plain form (elementary torch
operations, in 64 bits where values next to a rounding border of a code matter, else in 32), True
calls ``dual_ar_tts_gb300``.  What a row's codes stand for is returned, not the codes.

A row of codes is padded with zeros to a multiple of 16 columns; it has the scale
max|v| / 127 (2^-126 at least), and the code of v is the nearest whole number to v / scale.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
TINY = 2.0 ** -126


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # attention's output of 32 streams, before the output projection
        dict(name="quantise 32 streams", op="quantise", rows=32, cols=4096, dtype="bf16"),
        # the gate and up matrix, quantised when it is loaded
        dict(name="quantise gate/up weights", op="quantise", rows=19456, cols=2560, dtype="bf16"),
        # one stream's hidden state before a projection: latency
        dict(name="norm 1 stream", op="norm", rows=1, cols=2560, residual=True, dtype="fp32"),
        # an odd width without a residual, as a model's first norm
        dict(name="norm odd", op="norm", rows=45, cols=1001, residual=False, dtype="fp16"),
        # prompts of eight streams, whole
        dict(name="norm prompts", op="norm", rows=5916, cols=2560, residual=True, dtype="bf16"),
        # one stream's feed-forward
        dict(name="gate 1 stream", op="gate", rows=1, cols=9728, dtype="fp32"),
        # a prompt's feed-forward
        dict(name="gate prompt", op="gate", rows=2048, cols=9728, dtype="bf16"),
        # a small model's projection, few rows of odd sizes: the smallest call
        dict(name="matmul small", op="matmul", rows=3, m=97, k=250, dtype="fp16"),
        # one stream's gate and up projection
        dict(name="matmul gate/up 1 row", op="matmul", rows=1, m=19456, k=2560, dtype="fp32"),
        # seven streams: the projection to queries, keys and values
        dict(name="matmul qkv 7 rows", op="matmul", rows=7, m=6144, k=2560, dtype="bf16"),
        # 32 streams decoded together: the down projection
        dict(name="matmul down 32 rows", op="matmul", rows=32, m=2560, k=9728, dtype="bf16"),
        # prompts: the gate and up projection
        dict(name="matmul gate/up 2048 rows", op="matmul", rows=2048, m=19456, k=2560, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["quantise", "norm", "gate", "matmul"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op == "matmul":
        rows, k = _log(rng, 1, 2048), _log(rng, 64, 9728)
        return dict(op=op, rows=rows, m=_log(rng, 40, 19456 * 2560 // max(k, 2560)), k=k, dtype=dtype)
    cols = _log(rng, 64, 9728)
    if op == "quantise":
        return dict(op=op, rows=_log(rng, 1, 2048 * 9728 // cols), cols=cols, dtype=dtype)
    if op == "gate":
        return dict(op=op, rows=_log(rng, 1, 1024 * 9728 // cols), cols=cols, dtype=dtype)
    return dict(op=op, rows=_log(rng, 1, 5916 * 2560 // max(cols, 2560)), cols=cols, residual=rng.random() < 0.7,
                dtype=dtype)


# ---------------------------------------------------------------- the inputs

def _pad(k):
    return -(-k // 16) * 16


def _activations(g, rows, cols):
    """Normal values whose channels differ in size, as hidden states' do."""
    size = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    return torch.randn((rows, cols), generator=g, device="cuda") * size


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt, rows = case["op"], DTYPES[case["dtype"]], case["rows"]
    s = dict(case=case)
    if op == "quantise":
        s["x"] = _activations(g, rows, case["cols"]).to(dt)
    elif op == "norm":
        s["x"] = (0.3 * _activations(g, rows, case["cols"])).to(dt)
        s["residual"] = _activations(g, rows, case["cols"]).to(dt) if case["residual"] else None
        s["weight"] = torch.exp(0.3 * torch.randn(case["cols"], generator=g, device="cuda"))
    elif op == "gate":
        s["x"] = (1.5 * torch.randn((rows, 2 * case["cols"]), generator=g, device="cuda")).to(dt)
    else:
        m, k = case["m"], case["k"]
        x = _activations(g, rows, k)
        step = x.abs().amax(-1) / 127
        s["x_codes"] = torch.zeros((rows, _pad(k)), dtype=torch.int8, device="cuda")
        s["x_codes"][:, :k] = (x / step[:, None]).round().clamp(-127, 127).to(torch.int8)
        s["x_scales"] = step
        s["codes"] = torch.zeros((m, _pad(k)), dtype=torch.int8, device="cuda")
        s["codes"][:, :k] = (torch.randn((m, k), generator=g, device="cuda") * 34).round().clamp(-127, 127).to(torch.int8)
        s["scales"] = 6e-4 * torch.exp(0.3 * torch.randn(m, generator=g, device="cuda"))
    return s


# ------------------------------------------------------------- the plain forms

def _steps(v, factor=1.0):
    """What the codes of rows v * factor (64 bits) stand for, in 32 bits, and the scales.  A code is a
    ratio within its row, so a factor of the whole row only meets the scale."""
    most = v.abs().amax(-1, keepdim=True)
    step = (most * factor / 127).clamp(min=TINY).float()
    code = torch.round(v * 127 / most.clamp(min=1e-300)).float()
    return code * step, step[:, 0]


def _plain_quantise(s):
    x = s["x"]
    values, scales = _steps(x.double())
    return values.to(x.dtype), scales


def _plain_norm(s):
    x, res = s["x"], s["residual"]
    total = x if res is None else (res.float() + x.float()).to(x.dtype)
    h = total.double()
    values, scales = _steps(h * s["weight"].double(), 1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS))
    out = (values.to(x.dtype), scales)
    return out if res is None else out + (total,)


def _plain_gate(s):
    x, f = s["x"], s["case"]["cols"]
    a, b = x[:, :f].double(), x[:, f:].double()
    values, scales = _steps(a / (1.0 + torch.exp(-a)) * b)
    return values.to(x.dtype), scales


def _plain_matmul(s):
    y = s["x_codes"].float() @ s["codes"].float().t()
    return (y * s["x_scales"][:, None] * s["scales"]).to(DTYPES[s["case"]["dtype"]])


PLAIN = {"quantise": _plain_quantise, "norm": _plain_norm, "gate": _plain_gate, "matmul": _plain_matmul}


# --------------------------------------------------------- the framework's calls

def _own(s):
    import dual_ar_tts_gb300 as pkg
    c = s["case"]
    if c["op"] == "matmul":
        return pkg.q8_matmul(s["x_codes"], s["x_scales"], s["codes"], s["scales"], dtype=DTYPES[c["dtype"]])
    more = ()
    if c["op"] == "quantise":
        codes, scales = pkg.quantize_q8(s["x"])
    elif c["op"] == "gate":
        codes, scales = pkg.swiglu_q8(s["x"])
    elif c["residual"]:
        codes, scales, total = pkg.rms_norm_q8(s["x"], s["weight"], EPS, residual=s["residual"])
        more = (total,)
    else:
        codes, scales = pkg.rms_norm_q8(s["x"], s["weight"], EPS)
    return (pkg.dequantize_q8(codes, scales, c["cols"], dtype=s["x"].dtype), scales) + more


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------------------- work

def work(case):
    op, size, rows = case["op"], 4 if case["dtype"] == "fp32" else 2, case["rows"]
    if op == "matmul":
        m, k = case["m"], case["k"]
        return {"bytes": (m + rows) * (k + 4) + size * rows * m, "flops": 2.0 * rows * m * k}
    cols = case["cols"]
    coded = rows * (2 * cols + size * cols + 8)  # codes and scales written and read back, values written
    if op == "quantise":
        return {"bytes": size * rows * cols + coded, "flops": 4.0 * rows * cols}
    if op == "gate":
        return {"bytes": 2 * size * rows * cols + coded, "flops": 9.0 * rows * cols}
    moved = (3 if case["residual"] else 1) * size * rows * cols + 4 * cols
    return {"bytes": moved + coded, "flops": 9.0 * rows * cols}


# ---------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, f8 = case["op"], torch.float64
    if op == "matmul":
        out = torch.empty((case["rows"], case["m"]), dtype=f8, device="cuda")
        x = s["x_codes"].to(f8)
        for a in range(0, case["m"], 4096):
            out[:, a:a + 4096] = x @ s["codes"][a:a + 4096].to(f8).t()
        return out.mul_(s["x_scales"].to(f8)[:, None]).mul_(s["scales"].to(f8))

    def held(v):
        """(values, scales) of rows v: halves go to the even code, as in torch.round."""
        peak = v.abs().max(-1, keepdim=True).values
        code = torch.round(127 * v / peak)
        scale = torch.clamp(peak / 127, min=TINY)
        return scale * code, scale.squeeze(-1)

    if op == "quantise":
        return held(s["x"].to(f8))
    if op == "gate":
        up = s["x"][:, case["cols"]:].to(f8)
        gate = s["x"][:, :case["cols"]].to(f8)
        return held(torch.sigmoid(gate) * gate * up)
    h = s["x"].to(f8)
    if case["residual"]:
        h = (h + s["residual"].to(f8)).to(s["x"].dtype).to(f8)
    # codes before the row's common factor, which would move products that lie on a border
    value, scale = held(h * s["weight"].to(f8))
    r = (h.pow(2).sum(-1) / case["cols"] + EPS) ** -0.5
    out = (value * r[:, None], scale * r)
    return out + (h,) if case["residual"] else out
