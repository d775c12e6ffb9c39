"""Plain 64-bit forms of the 4-bit operators, for the tests: the layouts of include/s2frame.h read and
written element by element with numpy/torch, on the CPU."""
import math

import numpy as np
import torch

PAGE, GROUP = 64, 32
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def rounding(value, dtype):
    """How far rounding values near `value` to dtype may be off: half a step, relative or of a subnormal."""
    f = torch.finfo(dtype)
    return f.eps / 2 * value.abs() * 1.01 + f.smallest_normal * f.eps / 2


# ------------------------------------------------------------- 4-bit weights

def q4_columns(cols):
    """(byte in the row, shift) of each column's code."""
    k = np.arange(cols)
    return k // 128 * 64 + k % 32 // 8 * 16 + k % 128 // 32 * 4 + k % 8 // 2, k % 2 * 4


def q4_quantise(w, group):
    """w [rows][cols] torch CPU -> (codes uint8, scales bf16) from the definition (fp32 divisions)."""
    rows, cols = w.shape
    f = w.float()
    g = f.view(rows, -1, group)
    finite = torch.isfinite(g).all(-1, keepdim=True)
    big = torch.where(torch.isfinite(g), g, 0).abs().argmax(-1, keepdim=True)      # the first of equals
    scale = (g.gather(-1, big) / -8.0).bfloat16() + 0.0          # no -0
    scale = torch.where(finite, scale, torch.tensor(math.nan, dtype=torch.bfloat16))
    s = scale.float()
    live = finite & (s != 0)
    code = torch.where(live, (torch.round(g / torch.where(live, s, 1.0)) + 8).clamp(0, 15), 8.0)
    code = code.view(rows, cols).to(torch.uint8).numpy()
    blocks = -(-cols // 128)
    codes = np.full((rows, blocks * 64), 0x88, np.uint8)
    byte, shift = q4_columns(cols)
    for sh in (0, 4):
        m = shift == sh
        codes[:, byte[m]] = (codes[:, byte[m]] & (0xf0 if sh == 0 else 0x0f)) | (code[:, m] << sh)
    scales = torch.zeros((rows, blocks * (128 // group)), dtype=torch.bfloat16)
    scales[:, :cols // group] = scale[..., 0]
    return torch.from_numpy(codes), scales


def q4_values(codes, scales, cols, group):
    byte, shift = q4_columns(cols)
    c = (codes.cpu().numpy()[:, byte] >> shift) & 15
    return (torch.from_numpy(c.astype(np.float64)) - 8) * \
        scales.cpu().double()[:, torch.arange(cols) // group]


# -------------------------------------------------------------- 4-bit cache

def kv_quantise(x):
    """Values [..., hd] fp32 -> (codes, scale, zero) per the definition (each fp32 operation rounded by itself)."""
    g = x.float().clamp(-57344.0, 57344.0).unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = torch.maximum((hi - lo) / 15.0, torch.maximum(-lo, hi) / 127.0).half()
    s = scale.float()
    live = s > 0
    d = torch.where(live, s, 1.0)
    zero = torch.where(live, torch.round(-lo / d).clamp(-127, 127), 0.0)
    code = torch.where(live, (torch.round(g / d) + zero).clamp(0, 15), 0.0)
    return code.flatten(-2).to(torch.uint8), scale[..., 0], zero[..., 0].half()


def kv_value(code, scale, zero):
    c = code.float().unflatten(-1, (-1, GROUP))
    return (scale.float()[..., None] * (c - zero.float()[..., None])).half().flatten(-2)


def _parts(pages, part):
    hd = pages.shape[2] // 80
    half = PAGE * (hd // 2 + hd // 8)
    p = pages[:, :, part * half:(part + 1) * half]
    codes = p[:, :, :PAGE * hd // 2].unflatten(-1, (PAGE, hd // 2))
    par = p[:, :, PAGE * hd // 2:].view(torch.float16).unflatten(-1, (PAGE, hd // GROUP, 2))
    return codes, par


def put(pages, page, slot, k, v):
    """Quantise k, v [n_kv_head][hd] into one slot of CPU pages."""
    for part, x in enumerate((k, v)):
        codes, par = _parts(pages, part)
        c, s, z = kv_quantise(x)
        codes[page, :, slot] = c[..., 0::2] | (c[..., 1::2] << 4)
        par[page, :, slot, :, 0], par[page, :, slot, :, 1] = s, z


def get(pages, part, ids):
    """Values of the pages `ids` in order: [n_kv_head][64 * len(ids)][hd] fp16 (CPU pages)."""
    codes, par = _parts(pages, part)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[ids]
    x = kv_value(c, par[ids][..., 0], par[ids][..., 1])
    return x.transpose(0, 1).flatten(1, 2)


def fill_random(pages, rng):
    """Every slot of CPU pages: bell-shaped codes, scales near a unit normal's, zero points around the middle."""
    for part in range(2):
        codes, par = _parts(pages, part)
        a = rng.integers(0, 16, codes.shape + (4,), dtype=np.uint8)
        codes[:] = torch.from_numpy((a[..., 0] + a[..., 1]) // 2 | ((a[..., 2] + a[..., 3]) // 2) << 4)
        par[..., 0] = torch.from_numpy((0.27 * np.exp(0.3 * rng.standard_normal(par.shape[:-1]))).astype(np.float16))
        par[..., 1] = torch.from_numpy(rng.integers(-4, 20, par.shape[:-1]).astype(np.float16))


def norm_rotate(x, w, eps, cs):
    """fp32 [..., hd] by the definition: 64-bit mean square rounded to fp32, every further operation in fp32."""
    if w is not None:
        mean = x.double().square().mean(-1, keepdim=True).float()
        x = x * (1.0 / torch.sqrt(mean + eps)) * w
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1]], -1).flatten(-2)


def attention(q, k, v, seen, scale):
    """One head in 64 bits: q [n][hd], k/v [L][hd], row i sees the first seen[i] positions.  Returns
    (out, the bound of the error of a kernel with fp32 sums, without the rounding of its result): see below."""
    q, k, v = q.double(), k.double(), v.double()
    n, hd, L = q.shape[0], q.shape[1], k.shape[0]
    s = q @ k.t() * scale
    dead = torch.arange(L)[None] >= torch.as_tensor(seen)[:, None]
    s = s.masked_fill(dead, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.where(dead, torch.zeros((), dtype=torch.float64), (s - torch.where(m == -math.inf, 0.0, m)).exp())
    l = p.sum(-1, keepdim=True)
    w = torch.where(l > 0, p / l, 0.0)
    # A score: at most hd/16 + 32 roundings of 2^-23 along any path of its sum, of terms that add up to
    # sum |q k|, and the same again for the split of q into two fp16 parts (22 bits).  It shifts the row's
    # weights by twice its error; exp and its argument's product with log2(e) add 2^-21 + |s - m| 2^-23;
    # sums over positions L/16 + 64 roundings of 2^-23.
    ab = (q.abs() @ k.abs().t() * abs(scale)).masked_fill(dead, 0)
    ds = 2 * (hd / 16 + 32) * 2.0 ** -23 * ab.amax(-1, keepdim=True)
    spread = torch.where(dead, torch.zeros((), dtype=torch.float64), (m - s).clamp(max=60)).amax(-1, keepdim=True)
    rel = 2 * ds + 2 * (2.0 ** -21 + spread * 2.0 ** -23) + (L / 16 + 64) * 2.0 ** -23
    top = v.abs().amax() if v.numel() else torch.zeros((), dtype=torch.float64)
    return w @ v, rel, w @ v.abs(), 2.0 ** -24 * top


def attention_tol(o, rel, wv, tiny, dtype):
    """Weights of 16-bit types are rounded to fp16 (2^-11 each) before their product with the values."""
    return rounding(o, dtype) + (rel + (2.0 ** -11 * 1.01 if dtype != torch.float32 else 0)) * wv + tiny
