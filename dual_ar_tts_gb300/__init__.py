"""GB300 (sm_103a) Dual-AR frame decoder for S2-Pro — thin Python binding of ``libs2frame.so``.

The functions named ``s2_*`` mirror the C ABI in ``include/s2frame.h`` one to one and only
marshal arguments; every step of the decode runs in the library's CUDA kernels.  PyTorch is
used for device memory and streams.  There is no CPU fallback: if the CUDA library is missing
or no GPU is present, calls raise.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libs2frame.so")

S2_F32, S2_BF16, S2_F16 = 0, 1, 2
S2_OK, S2_EINVAL, S2_ENOMEM, S2_ECAPACITY, S2_ECUDA, S2_ETIMEOUT, S2_ESTATE = range(7)
STATUS_NAMES = {0: "S2_OK", 1: "S2_EINVAL", 2: "S2_ENOMEM", 3: "S2_ECAPACITY", 4: "S2_ECUDA", 5: "S2_ETIMEOUT",
                6: "S2_ESTATE"}

EXPORTS = ("s2_weight_count", "s2_weight_info", "s2_frame_workspace_bytes", "s2_frame_init", "s2_prefill",
           "s2_decode_frames", "s2_fast_logits", "s2_sync_status", "s2_set_spin_limit", "s2_set_trace",
           "s2_phase_count", "s2_frame_free", "s2_last_error", "s2_fast_logits_static", "s2_stream_import",
           "s2_stop_stream", "s2_stream_progress", "s2_codec_latent", "s2_quantize_e4m3", "s2_set_barrier_base",
           "s2_draw", "s2_quantize_q4", "s2_q4_matmul_workspace", "s2_q4_matmul",
           "s2_kv4_page_bytes", "s2_kv4_append", "s2_kv4_read",
           "s2_kv4_attention_workspace", "s2_kv4_attention", "s2_adjust_logits", "s2_set_wait_limit",
           "s2_quantize_q8", "s2_dequantize_q8", "s2_rms_norm_q8", "s2_swiglu_q8", "s2_q8_matmul")

S2_KV4_PAGE = 64


class s2_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dim", "n_layer", "n_head", "n_kv_head", "head_dim", "ffn", "vocab",
                                            "sem_begin", "sem_end", "im_end", "n_codebooks", "codebook_size")] + \
               [(n, ctypes.c_float) for n in ("sem_scale", "norm_eps", "rope_base")] + \
               [(n, ctypes.c_int) for n in ("qk_norm", "rope_table_bf16", "fast_dim", "fast_n_layer", "fast_n_head",
                                            "fast_n_kv_head", "fast_head_dim", "fast_ffn", "fast_window",
                                            "has_fast_project_in", "weight_dtype", "kv_dtype", "weight_fp8")]


class s2_sampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_p", ctypes.c_float), ("ras_temperature", ctypes.c_float),
                ("ras_top_p", ctypes.c_float), ("top_k", ctypes.c_int), ("ras_window", ctypes.c_int),
                ("min_tokens_before_end", ctypes.c_int), ("max_frames", ctypes.c_int)]


class s2_debug_taps(ctypes.Structure):
    _fields_ = [("main_logits", ctypes.c_void_p), ("fast_logits", ctypes.c_void_p), ("hidden", ctypes.c_void_p),
                ("draws", ctypes.c_void_p)]


class s2_kv4(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("n_kv_head", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("table", ctypes.c_void_p), ("table_cols", ctypes.c_int),
                ("n_seq", ctypes.c_int), ("q_start", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("n_rows", ctypes.c_int), ("status", ctypes.c_void_p)]


class S2Error(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn} -> {STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


_lib = None


def load(path: str = LIB_PATH):
    """Load the CUDA library (build it first with ``dual_ar_tts_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
    P = ctypes.POINTER
    sig = {
        "s2_weight_count": (i32, [P(s2_dims)]),
        "s2_weight_info": (i64, [P(s2_dims), i32, ctypes.c_char_p, i32]),
        "s2_frame_workspace_bytes": (sz, [P(s2_dims), i32, i32]),
        "s2_frame_init": (i32, [P(s2_dims), P(vp), i32, vp, sz, i32, i32, P(vp)]),
        "s2_prefill": (i32, [vp, i32, P(i32), vp, P(i32), vp]),
        "s2_decode_frames": (i32, [vp, i32, P(i32), i32, P(s2_sampling), vp, vp, vp, vp, P(s2_debug_taps), vp]),
        "s2_fast_logits": (i32, [vp, i32, vp, vp, vp, vp]),
        "s2_sync_status": (i32, [vp, vp]),
        "s2_set_spin_limit": (i32, [vp, i64]),
        "s2_set_trace": (i32, [vp, vp, i32]),
        "s2_set_barrier_base": (i32, [vp, ctypes.c_uint]),
        "s2_phase_count": (i32, [vp, i32]),
        "s2_frame_free": (i32, [vp]),
        "s2_last_error": (ctypes.c_char_p, [vp]),
        "s2_fast_logits_static": (i32, [P(s2_dims), P(vp), i32, i32, vp, vp, vp, vp, vp]),
        "s2_stream_import": (i32, [vp, i32, i32, vp, vp, vp, vp]),
        "s2_stop_stream": (i32, [vp, i32, vp]),
        "s2_codec_latent": (i32, [i32, i32, i32, P(vp), i32, vp, vp, vp, vp]),
        "s2_quantize_e4m3": (i32, [vp, ctypes.c_longlong, i32, vp, vp, vp]),
        "s2_stream_progress": (i32, [vp, i32, P(i32), vp, vp]),
        "s2_draw": (i32, [i32, vp, i32, i32, i32, i32, ctypes.c_float, ctypes.c_float, vp, vp, vp]),
        "s2_quantize_q4": (i32, [vp, i32, i64, i32, i32, vp, vp, vp]),
        "s2_q4_matmul_workspace": (sz, [i32, i32, i32]),
        "s2_q4_matmul": (i32, [i32, vp, i32, i64, vp, vp, i32, i32, i32, vp, vp, sz, vp]),
        "s2_kv4_page_bytes": (i64, [i32, i32]),
        "s2_kv4_append": (i32, [P(s2_kv4), vp, i32, i64, i32, vp, i32, vp, vp, ctypes.c_float, vp, vp]),
        "s2_kv4_read": (i32, [P(s2_kv4), vp, vp, vp]),
        "s2_kv4_attention_workspace": (sz, [i32, i32, i32, i32, i32, i32]),
        "s2_kv4_attention": (i32, [P(s2_kv4), vp, i32, i32, ctypes.c_float, i32, vp, vp, sz, vp]),
        "s2_set_wait_limit": (i32, [i32]),
        "s2_quantize_q8": (i32, [vp, i32, i64, i64, i32, vp, vp, vp]),
        "s2_dequantize_q8": (i32, [vp, vp, i64, i32, vp, i32, vp]),
        "s2_rms_norm_q8": (i32, [vp, i32, i64, vp, i64, vp, ctypes.c_float, i64, i32, vp, vp, vp, vp]),
        "s2_swiglu_q8": (i32, [vp, i32, i64, i64, i32, vp, vp, vp]),
        "s2_q8_matmul": (i32, [i32, vp, vp, vp, vp, i32, i32, vp, i32, vp]),
        "s2_adjust_logits": (i32, [i32, i32, i32, i32, vp, i32, vp, vp, i32, vp, vp, i64, vp, i64, vp, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(fn, rc, ctx=None):
    if rc != S2_OK:
        raise S2Error(fn, rc, load().s2_last_error(ctx).decode())
    return rc


def _ints(seq):
    arr = (ctypes.c_int * len(seq))(*[int(v) for v in seq])
    return arr


# ------------------------------------------------------------------ the C ABI

def make_dims(d: dict) -> s2_dims:
    s = s2_dims()
    for name, _ in s2_dims._fields_:
        setattr(s, name, d.get(name, 0) if name == "weight_fp8" else d[name])
    return s


def s2_weight_count(dims: s2_dims) -> int:
    return load().s2_weight_count(ctypes.byref(dims))


def s2_weight_info(dims: s2_dims, i: int):
    buf = ctypes.create_string_buffer(128)
    n = load().s2_weight_info(ctypes.byref(dims), i, buf, 128)
    return buf.value.decode(), n


def s2_frame_workspace_bytes(dims: s2_dims, max_streams: int, kv_slots: int) -> int:
    return load().s2_frame_workspace_bytes(ctypes.byref(dims), max_streams, kv_slots)


def s2_frame_init(dims: s2_dims, weight_ptrs, workspace_ptr: int, ws_bytes: int, max_streams: int, kv_slots: int):
    n = len(weight_ptrs)
    arr = (ctypes.c_void_p * n)(*[p if p else None for p in weight_ptrs])
    out = ctypes.c_void_p()
    rc = load().s2_frame_init(ctypes.byref(dims), arr, n, workspace_ptr, ws_bytes, max_streams, kv_slots,
                              ctypes.byref(out))
    _check("s2_frame_init", rc, None)
    return out.value


def s2_prefill(ctx, stream_ids, tokens_ptr: int, lengths, stream: int = 0):
    rc = load().s2_prefill(ctx, len(stream_ids), _ints(stream_ids), tokens_ptr, _ints(lengths), stream)
    return _check("s2_prefill", rc, ctx)


def s2_stream_import(ctx, stream_id: int, n_pos: int, k_ptr: int, v_ptr: int, x_last_ptr: int, stream: int = 0):
    rc = load().s2_stream_import(ctx, stream_id, n_pos, k_ptr, v_ptr, x_last_ptr, stream)
    return _check("s2_stream_import", rc, ctx)


def s2_stop_stream(ctx, stream_id: int, side_stream: int = 0):
    return _check("s2_stop_stream", load().s2_stop_stream(ctx, stream_id, side_stream), ctx)


def s2_stream_progress(ctx, stream_ids, out_ptr: int, side_stream: int = 0):
    rc = load().s2_stream_progress(ctx, len(stream_ids), _ints(stream_ids), out_ptr, side_stream)
    return _check("s2_stream_progress", rc, ctx)


def s2_codec_latent(n_codebooks: int, codebook_size: int, dim: int, quantizer_ptrs, n_frames: int, codes_ptr: int,
                    latent_ptr: int, status_ptr: int | None = None, stream: int = 0):
    """Codec latent = Σ_cb quantizer_cb[code] per frame (device pointers; see s2frame.h)."""
    arr = (ctypes.c_void_p * len(quantizer_ptrs))(*quantizer_ptrs)
    rc = load().s2_codec_latent(n_codebooks, codebook_size, dim, arr, n_frames, codes_ptr, latent_ptr, status_ptr,
                                stream)
    return _check("s2_codec_latent", rc)


def s2_quantize_e4m3(w_ptr: int, rows: int, cols: int, codes_ptr: int, scales_ptr: int, stream: int = 0):
    """e4m3 codes + fp32 row scales of bf16 rows (device pointers; see s2frame.h)."""
    return _check("s2_quantize_e4m3", load().s2_quantize_e4m3(w_ptr, rows, cols, codes_ptr, scales_ptr, stream))


def s2_draw(rows: int, logits_ptr: int, n: int, sem_begin: int, im_end: int, block_end: bool, temperature: float,
            top_p: float, expo_ptr: int, out_ptr: int, stream: int = 0):
    """The S2 draw on device logits rows (see s2frame.h)."""
    rc = load().s2_draw(rows, logits_ptr, n, sem_begin, im_end, 1 if block_end else 0, temperature, top_p, expo_ptr,
                        out_ptr, stream)
    return _check("s2_draw", rc)


def draw(logits, expo, temperature: float, top_p: float, sem_begin: int = -1, im_end: int = 0,
         block_end: bool = False):
    """Device fp32 logits [rows][n] and variates [rows][30] (torch) -> drawn ids, int32 [rows]."""
    import torch
    if logits.dtype != torch.float32 or logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("draw takes 2-D fp32 CUDA logits")
    if expo.dtype != torch.float32 or tuple(expo.shape) != (logits.shape[0], 30) or not expo.is_cuda:
        raise ValueError("draw takes fp32 CUDA variates of shape [rows][30]")
    logits, expo = logits.contiguous(), expo.contiguous()
    out = torch.empty(logits.shape[0], dtype=torch.int32, device=logits.device)
    s2_draw(logits.shape[0], logits.data_ptr(), logits.shape[1], sem_begin, im_end, block_end, temperature, top_p,
            expo.data_ptr(), out.data_ptr(), torch.cuda.current_stream().cuda_stream)
    return out


def quantize_e4m3(w):
    """Device bf16 matrix (torch, [rows][cols]) -> (uint8 codes [rows][cols], fp32 scales [rows])."""
    import torch
    if w.dtype != torch.bfloat16 or w.dim() != 2 or not w.is_cuda:
        raise ValueError("quantize_e4m3 takes a 2-D bf16 CUDA tensor")
    w = w.contiguous()
    codes = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    scales = torch.empty(w.shape[0], dtype=torch.float32, device=w.device)
    s2_quantize_e4m3(w.data_ptr(), w.shape[0], w.shape[1], codes.data_ptr(), scales.data_ptr(),
                     torch.cuda.current_stream().cuda_stream)
    return codes, scales


# ------------------------------------- 4-bit weights, 4-bit cache, adjusted logits

# A call of a few microseconds is soon outweighed by what Python does around it (torch's own x.add_(1) takes 7.5 us
# on a Grace core), so what these calls use of torch is looked up once, and their checks are few expressions that
# read each property of a tensor once: 13.3 us a call of a small matmul became 12.7, of which 3 are the launch and 3
# the output's allocation.

class _Hot:
    """What the calls below use of torch and of the library."""
    __slots__ = ("torch", "lib", "kinds", "stream", "device", "empty", "u8", "i32", "f16", "bf16", "f32")

    def __init__(self):
        import torch
        self.torch, self.lib, self.empty = torch, load(), torch.empty
        self.kinds = {torch.float32: S2_F32, torch.bfloat16: S2_BF16, torch.float16: S2_F16}
        self.stream = torch._C._cuda_getCurrentRawStream     # of a device number, as an integer
        self.device = torch._C._cuda_getDevice               # the current one's number
        self.u8, self.i32 = torch.uint8, torch.int32
        self.f16, self.bf16, self.f32 = torch.float16, torch.bfloat16, torch.float32


_hot = None


def _bind():
    global _hot
    _hot = _Hot()
    return _hot


def _bad(msg):
    raise ValueError(msg)


def _launch(h, fn, dev, *args):
    """Call an entry point on the current stream of device number `dev`, with that device current meanwhile."""
    if dev == h.device():
        rc = fn(*args, h.stream(dev))
    else:
        with h.torch.cuda.device(dev):
            rc = fn(*args, h.stream(dev))
    if rc != S2_OK:
        raise S2Error(fn.__name__, rc, "see include/s2frame.h for what the call takes")


def _off(dev, *tensors):
    """Whether one of the given tensors is not on CUDA device number `dev`."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            return True
    return False


_DEVICE = "tensors must be on one CUDA device, the operand fp32, bf16 or fp16"


def _rows16(x):
    """x [n][k], k elements a multiple of 16 bytes, as rows that start on 16 bytes (a copy where they do not), and
    their stride."""
    k = x.shape[1]
    s0, s1 = x.stride()
    if x.shape[0] == 1:  # one row: its stride may be anything, for torch too
        s0 = k
    if s1 == 1 and s0 >= k and s0 * x.element_size() % 16 == 0 and x.data_ptr() % 16 == 0:
        return x, s0
    x = x.contiguous()
    return x.clone() if x.data_ptr() % 16 else x, k


def quantize_q4(w, group: int = 32):
    """Device matrix [rows][cols] (fp32, bf16 or fp16) -> (uint8 codes [rows][ceil(cols/128)*64], bf16 scales
    [rows][ceil(cols/128)*(128/group)]): 4-bit codes with a scale per `group` (32, 64 or 128) columns; layout in
    s2frame.h."""
    h = _hot or _bind()
    dt, dev = h.kinds.get(w.dtype), w.get_device()
    if dt is None or dev < 0:
        _bad(_DEVICE)
    if w.dim() != 2 or group not in (32, 64, 128) or w.shape[1] % group or not w.shape[1]:
        _bad("quantize_q4 takes a 2-D tensor, its columns a multiple of group: 32, 64 or 128")
    w = w.contiguous()
    rows, cols = w.shape
    blocks = -(-cols // 128)
    codes = h.empty((rows, blocks * 64), dtype=h.u8, device=w.device)
    scales = h.empty((rows, blocks * (128 // group)), dtype=h.bf16, device=w.device)
    if rows:
        _launch(h, h.lib.s2_quantize_q4, dev, w.data_ptr(), dt, rows, cols, group, codes.data_ptr(),
                scales.data_ptr())
    return codes, scales


def q4_matmul(x, codes, scales, group: int = 32, out=None, workspace=None):
    """x [n][k] (fp32, bf16 or fp16) times the transposed 4-bit matrix of quantize_q4, or consecutive rows of it
    (codes[a:b], scales[a:b]) -> [n][rows] in x's type.
    workspace, a uint8 tensor of s2_q4_matmul_workspace bytes, is allocated where none is given."""
    h = _hot or _bind()
    dt, dev = h.kinds.get(x.dtype), x.get_device()
    if dt is None or dev < 0 or codes.get_device() != dev or scales.get_device() != dev:
        _bad(_DEVICE)
    if x.dim() != 2 or codes.dim() != 2 or group not in (32, 64, 128):
        _bad("q4_matmul takes x [n][k], codes and scales of quantize_q4 and its group: 32, 64 or 128")
    n, k = x.shape
    m, width = codes.shape
    if k % group or width != -(-k // 128) * 64 or scales.shape != (m, width * 2 // group) or \
            codes.dtype is not h.u8 or scales.dtype is not h.bf16 or not codes.is_contiguous() or \
            not scales.is_contiguous():
        _bad("codes must be contiguous uint8 [rows][ceil(k/128)*64] and scales contiguous bf16 "
             "[rows][ceil(k/128)*(128/group)], k a multiple of group")
    if codes.data_ptr() % 16:
        codes = codes.clone()
    if scales.data_ptr() % (8 if group == 32 else 4):  # rows of a quantised matrix, from an odd number of scales on
        scales = scales.clone()
    x, stride = _rows16(x)
    if out is None:
        out = h.empty((n, m), dtype=x.dtype, device=x.device)
    elif out.dtype is not x.dtype or out.shape != (n, m) or out.get_device() != dev or not out.is_contiguous():
        _bad("out must be contiguous [n][rows] of x's type, on its device")
    if not n or not m:
        return out
    if workspace is None:
        nbytes = h.lib.s2_q4_matmul_workspace(n, k, dt)
        workspace = h.empty(nbytes, dtype=h.u8, device=x.device) if nbytes else None
    else:
        nbytes = _workspace(workspace, dev)
    ws = None if workspace is None else workspace.data_ptr()
    _launch(h, h.lib.s2_q4_matmul, dev, n, x.data_ptr(), dt, stride, codes.data_ptr(), scales.data_ptr(), m, k,
            group, out.data_ptr(), ws, nbytes)
    return out


def _workspace(workspace, dev):
    """Bytes of a caller's workspace."""
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _bad("workspace must be contiguous, on the operand's device")
    return workspace.nbytes


def rope_table(n_pos: int, head_dim: int, base: float = 1e6, bf16: bool = True, device="cuda"):
    """fp32 [n_pos][head_dim/2][2] of (cos, sin) of position * base^(-2i/head_dim), angles in fp64, the values
    rounded to bf16 precision as the decode's own table (bf16=False: to fp32)."""
    import torch
    theta = base ** (-2.0 * torch.arange(head_dim // 2, dtype=torch.float64, device=device) / head_dim)
    a = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * theta
    t = torch.stack([a.cos(), a.sin()], -1).float()
    return (t.bfloat16().float() if bf16 else t).contiguous()


def kv4_pages(n_pages: int, n_kv_head: int, head_dim: int, device="cuda"):
    """The pages of one layer's 4-bit cache: uint8 [n_pages][n_kv_head][80*head_dim], zeroed."""
    import torch
    nbytes = load().s2_kv4_page_bytes(n_kv_head, head_dim)
    if nbytes < 0 or n_pages < 1:
        _bad("kv4_pages takes head_dim 64 or 128 and positive counts")
    return torch.zeros((n_pages, n_kv_head, nbytes // n_kv_head), dtype=torch.uint8, device=device)


def _kv4(h, dev, pages, table, q_start, lengths, n_rows, status):
    if dev < 0 or pages.get_device() != dev or table.get_device() != dev or q_start.get_device() != dev or \
            lengths.get_device() != dev or (status is not None and status.get_device() != dev):
        _bad(_DEVICE)
    i32 = h.i32
    if pages.dim() != 3 or table.dim() != 2 or pages.dtype is not h.u8 or table.dtype is not i32 or \
            not pages.is_contiguous() or not table.is_contiguous():
        _bad("pages must be contiguous uint8 [n_pages][n_kv_head][80*head_dim], table contiguous int32 [n_seq][cols]")
    n_pages, n_kv_head, block = pages.shape
    n_seq, cols = table.shape
    if block not in (80 * 64, 80 * 128):
        _bad("pages must be uint8 [n_pages][n_kv_head][80*head_dim], head_dim 64 or 128")
    if q_start.dtype is not i32 or lengths.dtype is not i32 or q_start.shape != (n_seq + 1,) or \
            lengths.shape != (n_seq,) or not q_start.is_contiguous() or not lengths.is_contiguous() or \
            (status is not None and (status.dtype is not i32 or status.numel() != 1)):
        _bad("q_start must be int32 [n_seq+1], lengths int32 [n_seq], status one int32")
    return s2_kv4(pages.data_ptr(), n_pages, n_kv_head, block // 80, table.data_ptr(), cols, n_seq, q_start.data_ptr(),
                  lengths.data_ptr(), n_rows, None if status is None else status.data_ptr())


def kv4_append(qkv, pages, table, q_start, lengths, rope, n_head: int, q_norm=None, k_norm=None, eps: float = 1e-6,
               q_out=None, status=None):
    """Append rows to a paged 4-bit cache (kv4_pages): qkv [n_rows][(n_head + 2 n_kv_head)*head_dim] (fp32, bf16 or
    fp16; q | k | v, head-major).  Queries and keys are normed per head where q_norm / k_norm (fp32 [head_dim]) are
    given and rotated by rope's (rope_table) row of their position; keys and values are quantised.  table int32
    [n_seq][cols], q_start int32 [n_seq + 1] and lengths int32 [n_seq] place the rows (see s2_kv4 in s2frame.h).
    Returns the rotated queries [n_rows][n_head][head_dim].  Rows behind the last sequence are left as they were, and so
    are rows whose position or page is out of range, of which status (one int32, zeroed by the caller) tells; in a q_out
    that the call allocates they hold nothing in particular."""
    h = _hot or _bind()
    dt, dev = h.kinds.get(qkv.dtype), qkv.get_device()
    if dt is None or qkv.dim() != 2:
        _bad("qkv must be fp32, bf16 or fp16 [n_rows][(n_head + 2 n_kv_head)*head_dim]")
    n_rows, width = qkv.shape
    c = _kv4(h, dev, pages, table, q_start, lengths, n_rows, status)
    hd, f32 = c.head_dim, h.f32
    if n_head < 0 or width != (n_head + 2 * c.n_kv_head) * hd:
        _bad("qkv must be [n_rows][(n_head + 2 n_kv_head)*head_dim]")
    if rope.dtype is not f32 or rope.dim() != 3 or rope.shape[1:] != (hd // 2, 2) or not rope.is_contiguous() or \
            rope.get_device() != dev:
        _bad("rope must be contiguous fp32 [n_pos][head_dim/2][2] on qkv's device")
    for w in (q_norm, k_norm):
        if w is not None and (w.dtype is not f32 or w.shape != (hd,) or not w.is_contiguous() or
                              w.get_device() != dev):
            _bad("norm weights must be fp32 [head_dim] on qkv's device")
    qkv, stride = _rows16(qkv)
    if q_out is None:
        q_out = h.empty((n_rows, n_head, hd), dtype=qkv.dtype, device=qkv.device)
    elif q_out.dtype is not qkv.dtype or q_out.shape != (n_rows, n_head, hd) or q_out.get_device() != dev or \
            not q_out.is_contiguous():
        _bad("q_out must be contiguous [n_rows][n_head][head_dim] of qkv's type, on its device")
    if not n_rows:
        return q_out
    _launch(h, h.lib.s2_kv4_append, dev, ctypes.byref(c), qkv.data_ptr(), dt, stride, n_head, rope.data_ptr(),
            rope.shape[0], None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(),
            eps, q_out.data_ptr())
    return q_out


def kv4_read(pages, table, q_start, lengths, n_rows: int, k_out=None, v_out=None, status=None):
    """What the rows' positions of a paged 4-bit cache stand for: (k, v) fp16 [n_kv_head][n_rows][head_dim]; zeros where a
    position or page is out of range (status, as kv4_append's, then tells).  Rows behind the last sequence are left as
    they were."""
    h = _hot or _bind()
    dev = pages.get_device()
    c = _kv4(h, dev, pages, table, q_start, lengths, n_rows, status)
    shape, f16 = (c.n_kv_head, n_rows, c.head_dim), h.f16
    if k_out is None:
        k_out = h.empty(shape, dtype=f16, device=pages.device)
    elif k_out.dtype is not f16 or k_out.shape != shape or k_out.get_device() != dev or not k_out.is_contiguous():
        _bad("outputs must be contiguous fp16 [n_kv_head][n_rows][head_dim] on the pages' device")
    if v_out is None:
        v_out = h.empty(shape, dtype=f16, device=pages.device)
    elif v_out.dtype is not f16 or v_out.shape != shape or v_out.get_device() != dev or not v_out.is_contiguous():
        _bad("outputs must be contiguous fp16 [n_kv_head][n_rows][head_dim] on the pages' device")
    if n_rows:
        _launch(h, h.lib.s2_kv4_read, dev, ctypes.byref(c), k_out.data_ptr(), v_out.data_ptr())
    return k_out, v_out


def kv4_attention(q, pages, table, q_start, lengths, scale: float | None = None, max_len: int = 0, workspace=None,
                  out=None, status=None):
    """Causal attention of q [n_rows][n_head][head_dim] (fp32, bf16 or fp16) over a paged 4-bit cache that holds
    the rows' own keys and values already (kv4_append).  scale defaults to 1/sqrt(head_dim); max_len (the largest
    length expected, 0: what the table can hold) only sets how the work is split; workspace, a uint8 tensor of
    s2_kv4_attention_workspace bytes, is allocated where none is given.  Pages out of range are not attended; status, as
    kv4_append's, tells of them.  Rows behind the last sequence are left as they were."""
    h = _hot or _bind()
    dt, dev = h.kinds.get(q.dtype), q.get_device()
    if dt is None or q.dim() != 3:
        _bad("q must be fp32, bf16 or fp16 [n_rows][n_head][head_dim]")
    n_rows, n_head, hd = q.shape
    c = _kv4(h, dev, pages, table, q_start, lengths, n_rows, status)
    n_kv = c.n_kv_head
    if hd != c.head_dim or n_kv < 1 or n_head % n_kv or max_len < 0:
        _bad("q's heads must be a multiple of the cache's, of the same head_dim")
    if not q.is_contiguous() or q.data_ptr() % 16:
        q = q.clone(memory_format=h.torch.contiguous_format)
    if out is None:
        out = h.empty((n_rows, n_head, hd), dtype=q.dtype, device=q.device)
    elif out.dtype is not q.dtype or out.shape != q.shape or out.get_device() != dev or not out.is_contiguous():
        _bad("out must be contiguous, of q's shape and type, on its device")
    if not n_rows or not n_head:
        return out
    if workspace is None:
        held = c.table_cols * S2_KV4_PAGE
        nbytes = h.lib.s2_kv4_attention_workspace(c.n_seq, n_rows, n_head, n_kv, hd, min(max_len or held, held))
        workspace = h.empty(nbytes, dtype=h.u8, device=q.device) if nbytes else None
    else:
        nbytes = _workspace(workspace, dev)
    _launch(h, h.lib.s2_kv4_attention, dev, ctypes.byref(c), q.data_ptr(), dt, n_head,
            hd ** -0.5 if scale is None else scale, max_len, out.data_ptr(),
            None if workspace is None else workspace.data_ptr(), nbytes)
    return out


def adjust_logits(logits, history=None, hist_len=None, penalties=None, bias=None, mask=None, sem_begin: int = -1,
                  im_end: int = 0, out=None):
    """Logits [rows][n] (fp32, bf16 or fp16) adjusted for a draw -> fp32 [rows][n] (see s2_adjust_logits).
    history int32 [rows][cols] with hist_len int32 [rows] and penalties fp32 [rows][3] of (repetition, frequency,
    presence); bias fp32 [rows or 1][n]; mask int32 or uint32 bits [rows or 1][ceil(n/32)].  Entry ids as in draw."""
    h = _hot or _bind()
    dt, dev = h.kinds.get(logits.dtype), logits.get_device()
    if dt is None or dev < 0 or _off(dev, history, hist_len, penalties, bias, mask, out):
        _bad(_DEVICE)
    if logits.dim() != 2:
        _bad("logits must be [rows][n]")
    rows, n = logits.shape
    i32, f32 = h.i32, h.f32
    cols = bias_stride = mask_stride = 0
    hp = lp = pp = bp = mp = None       # device pointers of what is given
    if history is not None:
        if history.dtype is not i32 or history.dim() != 2 or history.shape[0] != rows or \
                not history.is_contiguous() or penalties is None or penalties.dtype is not f32 or \
                penalties.shape != (rows, 3) or not penalties.is_contiguous():
            _bad("history must be contiguous int32 [rows][cols], with contiguous fp32 penalties [rows][3]")
        if hist_len is not None and (hist_len.dtype is not i32 or hist_len.shape != (rows,) or
                                     not hist_len.is_contiguous()):
            _bad("hist_len must be int32 [rows]")
        cols = history.shape[1]
        if cols:
            hp, pp = history.data_ptr(), penalties.data_ptr()
            lp = None if hist_len is None else hist_len.data_ptr()
    elif penalties is not None or hist_len is not None:
        _bad("penalties and hist_len go with a history")
    if bias is not None:
        if bias.dtype is not f32 or bias.shape not in ((1, n), (rows, n)) or not bias.is_contiguous():
            _bad("bias must be contiguous fp32 [rows or 1][n]")
        bp, bias_stride = bias.data_ptr(), n if bias.shape[0] > 1 else 0
    if mask is not None:
        words = -(-n // 32)
        if mask.dtype not in (i32, h.torch.uint32) or mask.shape not in ((1, words), (rows, words)) or \
                not mask.is_contiguous():
            _bad("mask must be contiguous 32-bit [rows or 1][ceil(n/32)]")
        mp, mask_stride = mask.data_ptr(), words if mask.shape[0] > 1 else 0
    if not logits.is_contiguous():
        logits = logits.contiguous()
    if out is None:
        out = h.empty((rows, n), dtype=f32, device=logits.device)
    elif out.dtype is not f32 or out.shape != (rows, n) or not out.is_contiguous():
        _bad("out must be contiguous fp32 [rows][n]")
    if not rows or not n:
        return out
    _launch(h, h.lib.s2_adjust_logits, dev, rows, n, sem_begin, im_end, logits.data_ptr(), dt, hp, lp, cols, pp, bp,
            bias_stride, mp, mask_stride, out.data_ptr())
    return out


# ------------------------------------------- projections in 8-bit integers

# The checks, outputs and launches of these are in csrc/calls.cpp: on a Grace core a call of one row takes 4.6 us there, 2.1
# with outputs given, and 13 from Python.

_q8 = None


def _bind_q8():
    global _q8
    import torch  # noqa: F401  (its libraries, which the module is linked against)
    load()
    try:
        from . import _calls as module
    except ImportError as e:
        raise ImportError(f"{e}: run `python -c 'import __graft_entry__ as g; g.build()'` where torch and Python's headers "
                          "are installed") from e
    module.set_error(S2Error)
    _q8 = module
    return module


def quantize_q8(x, codes=None, scales=None):
    """Rows [rows][cols] (fp32, bf16 or fp16; weights, or activations) -> (int8 codes [rows][cols rounded up to 16], fp32
    scales [rows]): scale = max|x| / 127 of the row, code = x / scale rounded (see s2_quantize_q8 in s2frame.h).  Outputs
    may be given."""
    return (_q8 or _bind_q8()).quantize_q8(x, codes, scales)


def dequantize_q8(codes, scales, cols: int | None = None, dtype=None, out=None):
    """The values that rows of codes stand for, scale * code -> [rows][cols] of dtype (fp32 where none is given); cols
    defaults to all that the codes hold."""
    return (_q8 or _bind_q8()).dequantize_q8(codes, scales, cols, dtype, out)


def rms_norm_q8(x, weight, eps: float = 1e-6, residual=None, total=None, codes=None, scales=None):
    """RMSNorm of rows [rows][cols] (fp32, bf16 or fp16) with fp32 weight [cols], as codes and scales of quantize_q8.  With a
    residual (x's shape and type) the norm is of total = residual + x, rounded to their type, which is returned third;
    total may be given, and be x or residual itself, but lie over neither otherwise."""
    return (_q8 or _bind_q8()).rms_norm_q8(x, weight, eps, residual, total, codes, scales)


def swiglu_q8(x, codes=None, scales=None):
    """The feed-forward's gate: rows [rows][2 f] (fp32, bf16 or fp16; gate | up) -> silu(gate) * up as codes and scales of
    quantize_q8, codes [rows][f rounded up to 16]."""
    return (_q8 or _bind_q8()).swiglu_q8(x, codes, scales)


def q8_matmul(x_codes, x_scales, codes, scales, dtype=None, out=None):
    """Activation rows [n][k] times the transposed weight rows [m][k], both as codes and scales of quantize_q8 (or rows of
    them; k a multiple of 16) -> [n][m] of dtype (bf16 where none is given).  The sums are exact integers."""
    return (_q8 or _bind_q8()).q8_matmul(x_codes, x_scales, codes, scales, dtype, out)


def s2_decode_frames(ctx, stream_ids, n_frames: int, params, expo_ptr: int, forced_ptr: int | None, codes_ptr: int,
                     n_out_ptr: int, taps: s2_debug_taps | None = None, stream: int = 0):
    n = len(stream_ids)
    arr = (s2_sampling * n)(*params)
    rc = load().s2_decode_frames(ctx, n, _ints(stream_ids), n_frames, arr, expo_ptr, forced_ptr, codes_ptr, n_out_ptr,
                                 ctypes.byref(taps) if taps is not None else None, stream)
    return _check("s2_decode_frames", rc, ctx)


def s2_fast_logits(ctx, n_frames: int, hidden_ptr: int, prefix_ptr: int, logits_ptr: int, stream: int = 0):
    rc = load().s2_fast_logits(ctx, n_frames, hidden_ptr, prefix_ptr, logits_ptr, stream)
    return _check("s2_fast_logits", rc, ctx)


def s2_sync_status(ctx, stream: int = 0) -> int:
    return load().s2_sync_status(ctx, stream)


def s2_set_spin_limit(ctx, limit: int):
    return _check("s2_set_spin_limit", load().s2_set_spin_limit(ctx, limit), ctx)


def s2_set_wait_limit(tries: int):
    return _check("s2_set_wait_limit", load().s2_set_wait_limit(tries))


def s2_set_barrier_base(ctx, base: int):
    return _check("s2_set_barrier_base", load().s2_set_barrier_base(ctx, base), ctx)


def s2_set_trace(ctx, buf_ptr: int | None, capacity: int):
    return _check("s2_set_trace", load().s2_set_trace(ctx, buf_ptr, capacity), ctx)


def s2_phase_count(ctx, fast_only: bool = False) -> int:
    return load().s2_phase_count(ctx, int(bool(fast_only)))


def s2_frame_free(ctx):
    return load().s2_frame_free(ctx)


def s2_last_error(ctx=None) -> str:
    return load().s2_last_error(ctx).decode()


def s2_fast_logits_static(dims: s2_dims, weight_ptrs, n_frames: int, hidden_ptr: int, prefix_ptr: int,
                          logits_ptr: int, status_ptr: int | None = None, stream: int = 0):
    """Fast-AR alone on the library's static scratch: no context, no workspace, no allocation.
    The caller passes every input and output (device pointers)."""
    arr = (ctypes.c_void_p * len(weight_ptrs))(*[p if p else None for p in weight_ptrs])
    rc = load().s2_fast_logits_static(ctypes.byref(dims), arr, len(weight_ptrs), n_frames, hidden_ptr, prefix_ptr,
                                      logits_ptr, status_ptr, stream)
    return _check("s2_fast_logits_static", rc)


def make_sampling(s: dict) -> s2_sampling:
    return s2_sampling(s["temperature"], s["top_p"], s["ras_temperature"], s["ras_top_p"], s["top_k"],
                       s["ras_window"], s["min_tokens_before_end"], s.get("max_frames", 0))


# ------------------------------------------------------- memory-owning helper

class Decoder:
    """Owns the device workspace (a torch tensor) and the weight tensors for one context."""

    def __init__(self, d: dict, weights, max_streams: int = 1, kv_slots: int = 0, device: str = "cuda"):
        import torch
        if not torch.cuda.is_available():
            raise RuntimeError("the frame decoder needs a CUDA GPU")
        load()
        self.d = d
        self.dims = make_dims(d)
        self.weights = weights          # torch device tensors (or None), table order
        ptrs = [w.data_ptr() if w is not None else 0 for w in weights]
        nbytes = s2_frame_workspace_bytes(self.dims, max_streams, kv_slots)
        if nbytes == 0:
            raise S2Error("s2_frame_workspace_bytes", S2_EINVAL, s2_last_error(None))
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.ctx = s2_frame_init(self.dims, ptrs, self.workspace.data_ptr(), nbytes, max_streams, kv_slots)
        self.max_streams = max_streams
        self.kv_slots = kv_slots

    def close(self):
        if getattr(self, "ctx", None):
            s2_frame_free(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def stream(self):
        import torch
        return torch.cuda.current_stream().cuda_stream

    def prefill(self, prompts, stream_ids=None):
        """prompts: list of [T][NCB+1] int32 arrays/tensors (host or device)."""
        import torch
        ids = list(range(len(prompts))) if stream_ids is None else list(stream_ids)
        toks = torch.cat([torch.as_tensor(p, dtype=torch.int32).reshape(-1) for p in prompts]).cuda()
        lens = [int(torch.as_tensor(p).shape[0]) for p in prompts]
        s2_prefill(self.ctx, ids, toks.data_ptr(), lens, self.stream())
        self._keep = toks
        return toks

    def stop(self, stream_id, side_stream=None):
        """Ask a stream to stop at its next frame boundary (takes effect during a running decode
        when side_stream is a non-blocking stream other than the decode's)."""
        import torch
        side = side_stream if side_stream is not None else torch.cuda.Stream()
        s2_stop_stream(self.ctx, stream_id, side.cuda_stream)
        side.synchronize()

    def progress(self, stream_ids, side_stream=None):
        """Frames emitted so far by the running (or last) decode call, per stream id."""
        import numpy as np
        import torch
        side = side_stream if side_stream is not None else torch.cuda.Stream()
        out = np.zeros(len(stream_ids), np.int32)
        s2_stream_progress(self.ctx, list(stream_ids), out.ctypes.data, side.cuda_stream)
        side.synchronize()
        return out

    def import_stream(self, stream_id, k, v, x_last):
        """k, v: device tensors [n_layer][n_kv_head][n_pos][head_dim] of the KV dtype; x_last: [dim] fp32."""
        n_pos = int(k.shape[2])
        s2_stream_import(self.ctx, stream_id, n_pos, k.data_ptr(), v.data_ptr(), x_last.data_ptr(), self.stream())

    def decode(self, n_frames, sampling, expo, forced=None, stream_ids=None, taps=False):
        """expo: [n][n_frames][11][30] float32 (device tensor); forced: optional [n][n_frames][11] int32.
        Returns dict of device tensors (codes, n_out and, with taps, the debug outputs)."""
        import torch
        n = expo.shape[0]
        ids = list(range(n)) if stream_ids is None else list(stream_ids)
        d = self.d
        dev = expo.device
        codes = torch.zeros((n, d["n_codebooks"] * n_frames), dtype=torch.int32, device=dev)
        n_out = torch.zeros(n, dtype=torch.int32, device=dev)
        out = dict(codes=codes, n_out=n_out)
        t = None
        if taps:
            A = d["codebook_size"] + 1
            out["main_logits"] = torch.full((n, n_frames, A), float("nan"), device=dev)
            out["fast_logits"] = torch.full((n, n_frames, d["n_codebooks"] - 1, d["codebook_size"]), float("nan"),
                                            device=dev)
            out["hidden"] = torch.full((n, n_frames, d["dim"]), float("nan"), device=dev)
            out["draws"] = torch.full((n, n_frames, 11), -2, dtype=torch.int32, device=dev)
            t = s2_debug_taps(out["main_logits"].data_ptr(), out["fast_logits"].data_ptr(), out["hidden"].data_ptr(),
                              out["draws"].data_ptr())
        params = [make_sampling(sampling) for _ in range(n)] if isinstance(sampling, dict) else \
            [make_sampling(s) for s in sampling]
        s2_decode_frames(self.ctx, ids, n_frames, params, expo.data_ptr(),
                         forced.data_ptr() if forced is not None else None, codes.data_ptr(), n_out.data_ptr(), t,
                         self.stream())
        return out

    def fast_logits(self, hidden, prefix):
        import torch
        n = hidden.shape[0]
        d = self.d
        out = torch.empty((n, d["n_codebooks"] - 1, d["codebook_size"]), dtype=torch.float32, device=hidden.device)
        s2_fast_logits(self.ctx, n, hidden.data_ptr(), prefix.data_ptr(), out.data_ptr(), self.stream())
        return out

    def sync_status(self) -> int:
        return s2_sync_status(self.ctx, self.stream())


def upload_weights(host_weights, device="cuda"):
    """Host arrays (fp32, or uint16 bf16 patterns) -> torch device tensors (bf16 / fp32)."""
    import numpy as np
    import torch
    out = []
    for w in host_weights:
        if w is None:
            out.append(None)
            continue
        if w.dtype == np.uint16:
            t = torch.from_numpy(w.view(np.int16)).to(device).view(torch.bfloat16)
        else:
            t = torch.from_numpy(np.ascontiguousarray(w, dtype=np.float32)).to(device)
        out.append(t)
    return out


def serve(decoder, requests, slots, frames_per_call, sampling, expo_fn, forced_fn=None):
    """Continuous batching over the decoder's stream slots.

    requests: list of (prompt [T][NCB+1] int32, n_frames).  A request holds a slot from its prefill
    until it has produced n_frames frames or stopped (im_end); its slot then takes the next waiting
    request.  The active slots are decoded together (one weight read per step) in calls of at most
    frames_per_call frames, cut so that no request overshoots.  expo_fn(request, first_frame, n)
    returns that request's exponential variates [n][11][30] (float32), so a request sees the same
    variates whatever the batch around it.  forced_fn(request, first_frame, n), when given, returns
    that request's forced draws [n][11] (int32; teacher forcing, as in s2_decode_frames).  Returns,
    per request, its codes [NCB][frames] (int32).
    """
    import collections
    import numpy as np
    import torch
    ncb = decoder.d["n_codebooks"]
    waiting = collections.deque(range(len(requests)))
    active = {}
    results = [None] * len(requests)
    while waiting or active:
        for slot in range(slots):
            if slot not in active and waiting:
                r = waiting.popleft()
                decoder.prefill([requests[r][0]], stream_ids=[slot])
                active[slot] = [r, 0, []]
        ids = sorted(active)
        n = min(frames_per_call, min(requests[active[k][0]][1] - active[k][1] for k in ids))
        expo = torch.from_numpy(np.stack([expo_fn(active[k][0], active[k][1], n) for k in ids])).cuda()
        if forced_fn is not None:
            forced = torch.from_numpy(np.stack([forced_fn(active[k][0], active[k][1], n) for k in ids])).cuda()
            out = decoder.decode(n, sampling, expo, forced=forced, stream_ids=ids)
        else:
            out = decoder.decode(n, sampling, expo, stream_ids=ids)
        n_out = out["n_out"].cpu().numpy()
        codes = out["codes"].cpu().numpy()
        for j, k in enumerate(ids):
            r, done, chunks = active[k]
            no = int(n_out[j])
            chunks.append(codes[j, :ncb * no].reshape(ncb, no))
            done += no
            active[k][1] = done
            if no < n or done >= requests[r][1]:
                results[r] = np.concatenate(chunks, axis=1)
                del active[k]
    return results
