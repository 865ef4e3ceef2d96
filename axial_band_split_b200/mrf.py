"""Python binding of libmrf (include/mrf.h): argument marshalling only.

Every step of the forward runs in the library's CUDA kernels; PyTorch is used here for
device memory and streams.  The binding raises if libmrf.so is missing or a call fails:
there is no fallback path.

    from axial_band_split_b200 import mrf
    model = mrf.Model(cfg, weights, max_batch=1, max_frames=1100)   # weights: name -> ndarray
    masks = model.forward(stft_repr)            # torch CUDA float32 [B, F*2, T, 2]

The block operators (rms_norm, rope, attention_packed) take and return torch CUDA tensors and need
no model: they are the steps between the matrix products of a transformer block over sequences of
different lengths packed without padding.  With stream= a call's new tensors belong to that stream;
tensors of another stream are the caller's to order before it and to keep until its work has run.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple

import numpy as np

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmrf.so")

MRF_FP16 = 0
MRF_BF16 = 1
MRF_FP32_DEBUG = 2
STATUS = {0: "MRF_OK", -1: "MRF_EINVAL", -2: "MRF_ESHAPE", -3: "MRF_ENOMEM", -4: "MRF_ECUDA",
          -5: "MRF_EUNSUPPORTED", -6: "MRF_ETIMEOUT", -7: "MRF_EWEIGHTS"}

# every symbol include/mrf.h declares
EXPORTS = ["mrf_create", "mrf_forward", "mrf_forward_separate", "mrf_stft", "mrf_istft", "mrf_separate_audio",
           "mrf_forward_host", "mrf_forward_host_async", "mrf_host_join", "mrf_sync_status", "mrf_destroy",
           "mrf_last_error", "mrf_band_tables", "mrf_set_timing", "mrf_kernel_times",
           "mrf_set_graph", "mrf_launches_per_forward", "mrf_debug_buffer", "mrf_forward_static",
           "mrf_debug_stall_next", "mrf_chunk_plan", "mrf_separate_audio_chunked", "mrf_rms_norm",
           "mrf_rope_table", "mrf_rope", "mrf_attention_workspace", "mrf_attention", "mrf_ops_sync_status"]


class MrfError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class mrf_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "sample_rate", "n_fft", "audio_channels", "num_bands", "dim", "depth", "heads", "dim_head",
        "ff_mult", "mask_hidden", "mask_depth", "num_stems", "zero_dc", "max_batch", "max_frames")] + \
        [("rope_theta", ctypes.c_float), ("compute", ctypes.c_int), ("ff_act", ctypes.c_int),
         ("dim_head_v", ctypes.c_int)]


class mrf_tensor(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("dtype", ctypes.c_int), ("ndim", ctypes.c_int),
                ("shape", ctypes.c_int64 * 4), ("host_data", ctypes.c_void_p)]


class mrf_kernel_time(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int), ("ms", ctypes.c_double)]


class mrf_rms_norm_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "residual", "weight", "out", "residual_out", "scales")] + \
        [(n, ctypes.c_int64) for n in ("rows", "x_stride", "residual_stride", "out_stride", "residual_out_stride")] + \
        [(n, ctypes.c_int) for n in ("dim", "dtype", "weight_dtype", "out_dtype", "group", "clamp")] + \
        [("eps", ctypes.c_float)]


class mrf_rope_config(ctypes.Structure):
    _fields_ = [("part", ctypes.c_int), ("scaling", ctypes.c_int)] + \
        [(n, ctypes.c_double) for n in ("theta", "factor", "original", "beta_fast", "beta_slow")]


class mrf_rope_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "q_out", "k_out", "positions", "turns")] + \
        [(n, ctypes.c_int64) for n in (
            "tokens", "q_token_stride", "q_head_stride", "k_token_stride", "k_head_stride", "q_out_token_stride",
            "q_out_head_stride", "k_out_token_stride", "k_out_head_stride")] + \
        [(n, ctypes.c_int) for n in ("heads", "kv_heads", "width", "part", "dtype", "positions_wide", "interleaved")] + \
        [("scale", ctypes.c_float)]


class mrf_attention_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "out", "lse", "q_offsets", "k_start", "k_len",
                                               "workspace")] + \
        [("workspace_bytes", ctypes.c_size_t)] + \
        [(n, ctypes.c_int64) for n in (
            "q_rows", "k_rows", "max_k", "q_token_stride", "q_head_stride", "k_token_stride", "k_head_stride",
            "v_token_stride", "v_head_stride", "out_token_stride", "out_head_stride")] + \
        [(n, ctypes.c_int) for n in ("seqs", "heads", "kv_heads", "width", "v_width", "dtype", "causal")] + \
        [("scale", ctypes.c_float)]


_lib = None


def lib():
    """The loaded libmrf.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is missing: run `python -m axial_band_split_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        P, I, V = ctypes.c_void_p, ctypes.c_int, None
        L.mrf_create.argtypes = [ctypes.POINTER(mrf_config), ctypes.POINTER(mrf_tensor), I, ctypes.POINTER(P)]
        L.mrf_create.restype = I
        L.mrf_forward.argtypes = [P, P, P, I, I, P]
        L.mrf_forward.restype = I
        L.mrf_forward_separate.argtypes = [P, P, P, I, I, P]
        L.mrf_forward_separate.restype = I
        L.mrf_stft.argtypes = [P, P, P, I, I, I, P]
        L.mrf_stft.restype = I
        L.mrf_istft.argtypes = [P, P, P, I, I, I, I, P]
        L.mrf_istft.restype = I
        L.mrf_separate_audio.argtypes = [P, P, P, I, I, P]
        L.mrf_separate_audio.restype = I
        L.mrf_separate_audio_chunked.argtypes = [P, P, P, I, I, I, P]
        L.mrf_separate_audio_chunked.restype = I
        L.mrf_forward_static.argtypes = [P, P, P, I, I, P]
        L.mrf_forward_static.restype = I
        L.mrf_forward_host.argtypes = [P, P, P, I, I, P]
        L.mrf_forward_host.restype = I
        L.mrf_forward_host_async.argtypes = [P, P, P, I, I, P]
        L.mrf_forward_host_async.restype = I
        L.mrf_host_join.argtypes = [P, P]
        L.mrf_host_join.restype = I
        L.mrf_sync_status.argtypes = [P, P]
        L.mrf_sync_status.restype = I
        L.mrf_destroy.argtypes = [P]
        L.mrf_destroy.restype = V
        L.mrf_last_error.argtypes = [P]
        L.mrf_last_error.restype = ctypes.c_char_p
        L.mrf_band_tables.argtypes = [ctypes.POINTER(mrf_config)] + [P] * 6
        L.mrf_band_tables.restype = I
        L.mrf_set_timing.argtypes = [P, I]
        L.mrf_set_timing.restype = I
        L.mrf_set_graph.argtypes = [P, I]
        L.mrf_set_graph.restype = I
        L.mrf_kernel_times.argtypes = [P, ctypes.POINTER(mrf_kernel_time), I, ctypes.POINTER(I)]
        L.mrf_kernel_times.restype = I
        L.mrf_debug_buffer.argtypes = [P, ctypes.c_char_p, P, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)]
        L.mrf_debug_buffer.restype = I
        L.mrf_debug_stall_next.argtypes = [P]
        L.mrf_debug_stall_next.restype = I
        L.mrf_launches_per_forward.argtypes = [P, I, I]
        L.mrf_launches_per_forward.restype = I
        IP = ctypes.POINTER(I)
        L.mrf_chunk_plan.argtypes = [I, I, I, IP, IP, IP, IP, P, P, P, I]
        L.mrf_chunk_plan.restype = I
        L.mrf_rms_norm.argtypes = [P, P]
        L.mrf_rms_norm.restype = I
        L.mrf_rope_table.argtypes = [ctypes.POINTER(mrf_rope_config), P, ctypes.POINTER(ctypes.c_float)]
        L.mrf_rope_table.restype = I
        L.mrf_rope.argtypes = [P, P]
        L.mrf_rope.restype = I
        L.mrf_attention_workspace.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        L.mrf_attention_workspace.restype = I
        L.mrf_attention.argtypes = [P, P]
        L.mrf_attention.restype = I
        L.mrf_ops_sync_status.argtypes = [P]
        L.mrf_ops_sync_status.restype = I
        _lib = L
    return _lib


def _check(status, handle=None):
    if status != 0:
        raise MrfError(status, lib().mrf_last_error(handle).decode(errors="replace"))


def make_config(cfg, max_batch=1, max_frames=1100, compute=MRF_FP16):
    """mrf_config from any object with the model fields (sample_rate, n_fft, ...)."""
    c = mrf_config()
    c.sample_rate, c.n_fft, c.audio_channels = cfg.sample_rate, cfg.n_fft, cfg.audio_channels
    c.num_bands, c.dim, c.depth, c.heads, c.dim_head = cfg.num_bands, cfg.dim, cfg.depth, cfg.heads, cfg.dim_head
    c.ff_mult, c.mask_hidden, c.mask_depth = cfg.ff_mult, cfg.dim * cfg.mask_hidden_mult, cfg.mask_depth
    c.num_stems, c.zero_dc = cfg.num_stems, int(cfg.zero_dc)
    c.max_batch, c.max_frames = max_batch, max_frames
    c.rope_theta, c.compute = cfg.rope_theta, compute
    c.ff_act = getattr(cfg, "ff_act", 0)
    c.dim_head_v = getattr(cfg, "dim_head_v", 0)
    return c


def band_tables(cfg):
    """The library's band tables for cfg: dict of numpy arrays (first_bin, last_bin, width,
    feat_row, row_weight)."""
    c = make_config(cfg)
    n_feat = ctypes.c_int(0)
    _check(lib().mrf_band_tables(ctypes.byref(c), None, None, None, None, None, ctypes.byref(n_feat)))
    nb, rows = cfg.num_bands, (cfg.n_fft // 2 + 1) * cfg.audio_channels
    out = {"first_bin": np.zeros(nb, np.int32), "last_bin": np.zeros(nb, np.int32),
           "width": np.zeros(nb, np.int32), "feat_row": np.zeros(n_feat.value, np.int32),
           "row_weight": np.zeros(rows, np.float32)}
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    _check(lib().mrf_band_tables(ctypes.byref(c), ptr(out["first_bin"]), ptr(out["last_bin"]),
                                 ptr(out["width"]), ptr(out["feat_row"]), ptr(out["row_weight"]), None))
    return out


def chunk_plan(sample_rate, length, chunk_samples=0):
    """mrf_chunk_plan: the separation loop's geometry for a mix of `length` samples (chunks of
    chunk_samples, 0: 8 s): dict with chunk, border, padded_length and the per-chunk arrays off,
    valid, mode (0 full, 1 reflect tail, 2 zero tail)."""
    vals = [ctypes.c_int(0) for _ in range(4)]
    _check(lib().mrf_chunk_plan(sample_rate, chunk_samples, length, *[ctypes.byref(v) for v in vals], None, None,
                                None, 0))
    n = vals[3].value
    out = {k: np.zeros(n, np.int32) for k in ("off", "valid", "mode")}
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    _check(lib().mrf_chunk_plan(sample_rate, chunk_samples, length, *[ctypes.byref(v) for v in vals],
                                ptr(out["off"]), ptr(out["valid"]), ptr(out["mode"]), n))
    out.update(chunk=vals[0].value, border=vals[1].value, padded_length=vals[2].value)
    return out


def _stream_ptr(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


# ------------------------------------------------------------------ block operators
# A call of these takes microseconds on the device, so the binding keeps its own share small: checks
# build no message unless they fail, and the argument structures (the ctypes classes above, laid out
# the same) are packed in one go.
_NORM = struct.Struct("6P5q6if0P")
_ROPE = struct.Struct("6P9q7if0P")
_ATTENTION = struct.Struct("9PN11q7if0P")


class _Torch:
    """What the block operators use of torch, looked up once."""

    def __init__(self):
        import torch
        self.codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
        self.e4m3, self.f32, self.i32, self.i64, self.u8 = (torch.float8_e4m3fn, torch.float32, torch.int32, torch.int64,
                                                            torch.uint8)
        self.empty_like = torch.empty_like  # keeps the order of the strides, so that is where outputs' strides come from
        self.grad, self.device, self.Tensor = torch.is_grad_enabled, torch.cuda.current_device, torch.Tensor
        self.forward = torch.autograd.forward_ad
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.stream = raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_torch = None


def _t():
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _code(t, x, name, dev=None):
    """mrf_dtype of a CUDA tensor (on device `dev`) of one of the block operators' types; they compute no gradients."""
    if not isinstance(x, t.Tensor):
        raise MrfError(-1, f"{name} must be a tensor, got {type(x).__name__}")
    code = t.codes.get(x.dtype)
    if code is None:
        raise MrfError(-1, f"{name} must be float32, float16 or bfloat16, got {x.dtype}")
    at = x.get_device()
    if at < 0 or (dev is not None and at != dev):
        raise MrfError(-1, f"{name} must be on {'a CUDA device' if dev is None else f'cuda:{dev}'}, is on {x.device}")
    if (x.requires_grad and t.grad()) or getattr(t.forward, "_current_level", 0) >= 0:
        _no_gradient(t, x, name)
    return code


def _no_gradient(t, x, name):
    """Refuses what a gradient or, within a level of forward-mode derivatives, a tangent would be lost of."""
    if (x.requires_grad and t.grad()) or t.forward.unpack_dual(x).tangent is not None:
        raise MrfError(-1, f"{name} requires a gradient; the library is for inference")


def _like(t, x, dtype, dev, shape, name):
    """`x` is a tensor of the given type, device and shape, its last dimension contiguous; its strides."""
    if not isinstance(x, t.Tensor) or x.dtype != dtype or x.get_device() != dev:
        raise MrfError(-1, f"{name} must be {dtype} on cuda:{dev}, is {getattr(x, 'dtype', type(x))} on {getattr(x, 'device', None)}")
    if x.shape != shape:
        raise MrfError(-2, f"{name} must be {tuple(shape)}, got {tuple(x.shape)}")
    st = x.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise MrfError(-1, f"{name}: the last dimension must be contiguous")
    if (x.requires_grad and t.grad()) or getattr(t.forward, "_current_level", 0) >= 0:
        _no_gradient(t, x, name)
    return st


def _new_like(t, x):
    """A new tensor in the order of x's heads and tokens, and its strides."""
    y = t.empty_like(x)
    st = y.stride()
    if st[-1] != 1:  # x's rows overlap (windows over one signal): another dimension came out innermost
        y = x.new_empty(x.shape)
        st = y.stride()
    return y, st


def _vector(t, x, dev, count, name, wide=False):
    """`x` is a contiguous int32 (or int64 where `wide`) vector of `count` values on device `dev`."""
    if not isinstance(x, t.Tensor) or x.get_device() != dev or not (x.dtype == t.i32 or (wide and x.dtype == t.i64)):
        raise MrfError(-1, f"{name} must be an int32{' or int64' if wide else ''} tensor on cuda:{dev}")
    if x.dim() != 1 or x.shape[0] != count or (count > 1 and x.stride(0) != 1):
        raise MrfError(-2, f"{name} must be a contiguous vector of {count} values, got {tuple(x.shape)}")


def _row_stride(x, st, dim, name):
    """The row stride of a [rows, dim] tensor, or of one with other leading dimensions (contiguous)."""
    if len(st) == 2:
        return st[0]
    if not x.is_contiguous():
        raise MrfError(-1, f"{name} with other than two dimensions must be contiguous")
    return dim


class _scope:
    """Device `dev` and `stream` (a torch stream, a pointer, or None for dev's current one) made torch's
    current ones, so that what a call allocates belongs to the stream it runs on."""

    def __init__(self, dev, stream):
        import torch
        self.on = [torch.cuda.device(dev)]
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", dev))
            if stream.device.index != dev:
                raise MrfError(-1, f"the stream must be on cuda:{dev}, is on {stream.device}")
            self.on.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.on:
            c.__enter__()

    def __exit__(self, *e):
        for c in reversed(self.on):
            c.__exit__(*e)


class RmsNorm(NamedTuple):
    """What rms_norm returns: the normed rows; the scales of an 8-bit output, else None; h = x +
    residual, None without a residual."""
    out: object
    scales: object
    residual: object


def rms_norm(x, weight=None, eps=1e-6, residual=None, out_dtype=None, group=0, clamp=False, out=None,
             residual_out=None, stream=None):
    """mrf_rms_norm: h = x + residual, then h * weight / sqrt(mean h^2 + eps) over the last dimension
    (with clamp: h * weight / max(sqrt(mean h^2), eps)).

    x: CUDA float32, float16 or bfloat16 [rows, dim] (any row stride), or contiguous with other leading
    dimensions; residual the same; weight [dim] of any of the three types.  out_dtype
    torch.float8_e4m3fn gives 8-bit rows and float32 scales [..., ceil(dim / group)], one for each
    `group` columns (0: the row), out * scale standing for the value.  out=x norms in place,
    residual_out=residual updates the residual in place; without residual_out h gets a new tensor.
    Returns RmsNorm(out, scales, residual)."""
    t = _torch or _t()
    code = _code(t, x, "x")
    dev = x.get_device()
    if stream is not None or dev != t.device():
        with _scope(dev, stream):
            return rms_norm(x, weight, eps, residual, out_dtype, group, clamp, out, residual_out)
    shape, dtype = x.shape, x.dtype
    if len(shape) == 0 or shape[-1] < 1:
        raise MrfError(-2, "x must have a last dimension of at least 1")
    dim = shape[-1]
    quant = out_dtype is t.e4m3
    if not quant and out_dtype is not None and out_dtype != dtype:
        raise MrfError(-1, f"out_dtype must be {dtype} or torch.float8_e4m3fn, got {out_dtype}")
    whole = x.is_contiguous()
    x_row = dim if whole else _row_stride(x, _like(t, x, dtype, dev, shape, "x"), dim, "x")
    w = wcode = res = res_row = res_out = res_out_row = scale_ptr = 0
    if weight is not None:
        wcode = _code(t, weight, "weight", dev)
        if weight.shape != (dim,) or not weight.is_contiguous():
            raise MrfError(-2, f"weight must be a contiguous vector of {dim} values, got {tuple(weight.shape)}")
        w = weight.data_ptr()
    h, scales = residual_out, None
    if residual is not None:
        res_row = _row_stride(residual, _like(t, residual, dtype, dev, shape, "residual"), dim, "residual")
        res = residual.data_ptr()
        if h is None:
            h, res_out_row = t.empty_like(x) if whole else x.new_empty(shape), dim
        else:
            res_out_row = _row_stride(h, _like(t, h, dtype, dev, shape, "residual_out"), dim, "residual_out")
        res_out = h.data_ptr()
    elif h is not None:
        raise MrfError(-1, "residual_out without residual")
    if quant:
        if out is None:
            out, out_row = t.empty_like(x, dtype=t.e4m3) if whole else x.new_empty(shape, dtype=t.e4m3), dim
        else:
            out_row = _row_stride(out, _like(t, out, t.e4m3, dev, shape, "out"), dim, "out")
        scales = x.new_empty(shape[:-1] + (-(-dim // group) if group > 0 else 1,), dtype=t.f32)
        scale_ptr = scales.data_ptr()
    elif out is None:
        out, out_row = t.empty_like(x) if whole else x.new_empty(shape), dim
    else:
        out_row = _row_stride(out, _like(t, out, dtype, dev, shape, "out"), dim, "out")
    status = (_lib or lib()).mrf_rms_norm(_NORM.pack(
        x.data_ptr(), res, w, out.data_ptr(), res_out, scale_ptr, x.numel() // dim, x_row, res_row, out_row, res_out_row,
        dim, code, wcode, 3 if quant else code, group, bool(clamp), eps), t.stream(dev))
    if status:
        _check(status)
    return RmsNorm(out, scales, h)


class RopeTable(NamedTuple):
    """Rotary frequencies of `part` dimensions on one device: turns (int64 [part / 2], binary fractions
    of a turn a position) and the factor on cos and sin."""
    turns: object
    scale: float
    part: int


def rope_table(part, theta=10000.0, scaling="none", factor=1.0, original=0, beta_fast=0.0, beta_slow=0.0, device="cuda"):
    """mrf_rope_table: the frequencies theta^(-2i / part), scaled for contexts longer than the training's
    by "linear" (positions / factor), "ntk" (a larger theta) or "yarn" (by parts; `original` is the
    training's context length).  Made once and kept; rope takes it."""
    import torch
    kinds = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
    if scaling not in kinds:
        raise MrfError(-1, f"scaling must be one of {sorted(kinds)}, got {scaling!r}")
    c = mrf_rope_config(part, kinds[scaling], theta, factor, original, beta_fast, beta_slow)
    turns = np.zeros(max(1, min(part, 1024) // 2), np.uint64)
    scale = ctypes.c_float(0)
    _check(lib().mrf_rope_table(ctypes.byref(c), turns.ctypes.data_as(ctypes.c_void_p), ctypes.byref(scale)))
    # (waited for, so that any stream may use it)
    return RopeTable(torch.from_numpy(turns.view(np.int64)).to(device), scale.value, part)


def rope(q, k, positions, table, interleaved=True, q_out=None, k_out=None, stream=None):
    """mrf_rope: the first table.part dimensions of every head of q [tokens, heads, width] and of k
    [tokens, kv_heads, width] (or None) turned by each token's position (int32 or int64 [tokens]), in pairs
    (2i, 2i + 1), or (i, i + part / 2) with interleaved=False.  Heads and tokens may have any strides
    (column ranges of a projection's rows); q_out=q and k_out=k turn in place.  Returns (q_out, k_out)."""
    t = _torch or _t()
    code = _code(t, q, "q")
    dev = q.get_device()
    if stream is not None or dev != t.device():
        with _scope(dev, stream):
            return rope(q, k, positions, table, interleaved, q_out, k_out)
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3:
        raise MrfError(-2, f"q must be [tokens, heads, width], got {tuple(shape)}")
    tokens, heads, width = shape
    qs = _like(t, q, dtype, dev, shape, "q")
    ks = kos = (0, 0, 1)
    kv_heads = k_ptr = k_out_ptr = 0
    if k is not None:
        if not isinstance(k, t.Tensor) or k.dim() != 3:
            raise MrfError(-2, f"k must be a tensor [tokens, kv_heads, width], got {tuple(getattr(k, 'shape', ()))}")
        kv_heads = k.shape[1]
        k_shape = (tokens, kv_heads, width)
        ks = _like(t, k, dtype, dev, k_shape, "k")
        if k_out is None:
            k_out, kos = _new_like(t, k)
        else:
            kos = _like(t, k_out, dtype, dev, k_shape, "k_out")
        k_ptr, k_out_ptr = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise MrfError(-1, "k_out without k")
    _vector(t, positions, dev, tokens, "positions", wide=True)
    turns = table.turns if isinstance(table, RopeTable) else None
    if not isinstance(turns, t.Tensor) or turns.dtype != t.i64 or turns.get_device() != dev:
        raise MrfError(-1, f"table must come from rope_table on cuda:{dev}")
    if 2 * turns.numel() != table.part or not turns.is_contiguous():
        raise MrfError(-2, f"table must have a contiguous value for each of its {table.part} / 2 pairs, has {tuple(turns.shape)}")
    if q_out is None:
        q_out, qos = _new_like(t, q)
    else:
        qos = _like(t, q_out, dtype, dev, shape, "q_out")
    status = (_lib or lib()).mrf_rope(_ROPE.pack(
        q.data_ptr(), k_ptr, q_out.data_ptr(), k_out_ptr, positions.data_ptr(), turns.data_ptr(), tokens, qs[0], qs[1],
        ks[0], ks[1], qos[0], qos[1], kos[0], kos[1], heads, kv_heads, width, table.part, code, positions.dtype is t.i64,
        bool(interleaved), table.scale), t.stream(dev))
    if status:
        _check(status)
    return q_out, k_out


def attention_packed(q, k, v, q_offsets, k_start=None, k_len=None, max_k=0, causal=True, scale=None, out=None,
                     return_lse=False, stream=None):
    """mrf_attention: softmax attention with grouped heads over sequences packed one after another.

    q [q_rows, heads, width], k [k_rows, kv_heads, width], v [k_rows, kv_heads, v_width]: CUDA float16,
    bfloat16 or float32 with any token and head strides.  Sequence b owns the query rows q_offsets[b] ..
    q_offsets[b + 1] (int32 [seqs + 1]) and the key rows k_start[b] .. k_start[b] + k_len[b] (int32 [seqs];
    without them its query rows).  causal: the last query sees all keys of its sequence.  max_k: an upper
    bound of the key counts known on the host (0: k's rows), which only decides how the work is split: new
    tokens over long caches are the faster the closer it is.
    Rows of no sequence keep what `out` held (a new `out` is uninitialised there).  Returns out
    [q_rows, heads, v_width], or (out, lse float32 [q_rows, heads]) with return_lse."""
    t = _torch or _t()
    code = _code(t, q, "q")
    dev = q.get_device()
    if stream is not None or dev != t.device():
        with _scope(dev, stream):
            return attention_packed(q, k, v, q_offsets, k_start, k_len, max_k, causal, scale, out, return_lse)
    if not isinstance(v, t.Tensor):
        raise MrfError(-1, f"v must be a tensor, got {type(v).__name__}")
    dtype, shape, v_shape = q.dtype, q.shape, v.shape
    if len(shape) != 3 or len(v_shape) != 3:
        raise MrfError(-2, f"q and v must be [rows, heads, width], got {tuple(shape)} and {tuple(v_shape)}")
    q_rows, heads, width = shape
    k_rows, kv_heads, v_width = v_shape
    q_st, q_sh, _ = _like(t, q, dtype, dev, shape, "q")
    k_st, k_sh, _ = _like(t, k, dtype, dev, (k_rows, kv_heads, width), "k")
    v_st, v_sh, _ = _like(t, v, dtype, dev, v_shape, "v")
    if not isinstance(q_offsets, t.Tensor) or q_offsets.dim() != 1 or q_offsets.shape[0] < 1:
        raise MrfError(-2, "q_offsets must be a vector of seqs + 1 values")
    seqs = q_offsets.shape[0] - 1
    _vector(t, q_offsets, dev, seqs + 1, "q_offsets")
    start_ptr = len_ptr = lse_ptr = space_ptr = 0
    if k_len is not None and k_start is not None:
        _vector(t, k_start, dev, seqs, "k_start")
        _vector(t, k_len, dev, seqs, "k_len")
        # (a vector of no values has a null pointer; any other says that k_start and k_len are given)
        start_ptr, len_ptr = (k_start.data_ptr(), k_len.data_ptr()) if seqs else (8, 8)
    elif k_len is not None or k_start is not None:
        raise MrfError(-1, "k_start and k_len go together")
    if out is None and v_width == width:
        out, (o_st, o_sh, _) = _new_like(t, q)
    elif out is None:
        out = q.new_empty((q_rows, heads, v_width))
        o_st, o_sh, _ = out.stride()
    else:
        o_st, o_sh, _ = _like(t, out, dtype, dev, (q_rows, heads, v_width), "out")
    lse = None
    if return_lse:
        lse = q.new_empty((q_rows, heads), dtype=t.f32)
        lse_ptr = lse.data_ptr()
    L, need = _lib or lib(), ctypes.c_size_t()
    head = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr, q_offsets.data_ptr(), start_ptr, len_ptr)
    tail = (q_rows, k_rows, max_k, q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh, seqs, heads, kv_heads, width, v_width, code,
            bool(causal), width ** -0.5 if scale is None else scale)
    packed = _ATTENTION.pack(*head, 0, 0, *tail)
    status = L.mrf_attention_workspace(packed, ctypes.byref(need))
    if status:
        _check(status)
    if need.value:
        space = q.new_empty(need.value, dtype=t.u8)
        packed = _ATTENTION.pack(*head, space.data_ptr(), need.value, *tail)
    status = L.mrf_attention(packed, t.stream(dev))
    if status:
        _check(status)
    return (out, lse) if return_lse else out


def ops_sync_status(stream=None):
    """mrf_ops_sync_status: wait for `stream` and raise if a block operator's kernel on the current device gave up a wait
    since this thread last asked (nothing else reports it)."""
    _check(lib().mrf_ops_sync_status(_stream_ptr(stream)))


class Model:
    """A created libmrf handle: weights on the device, workspace for max_batch x max_frames."""

    def __init__(self, cfg, weights, max_batch=1, max_frames=1100, compute=MRF_FP16):
        self.cfg = cfg
        self.rows = (cfg.n_fft // 2 + 1) * cfg.audio_channels
        c = make_config(cfg, max_batch, max_frames, compute)
        keep, table = [], (mrf_tensor * len(weights))()
        for i, (name, a) in enumerate(weights.items()):
            a = np.ascontiguousarray(a)
            if a.dtype not in (np.float32, np.float16):
                a = a.astype(np.float32)
            keep.append(a)
            bname = name.encode()
            keep.append(bname)
            t = table[i]
            t.name = bname
            t.dtype = 0 if a.dtype == np.float32 else 1
            t.ndim = a.ndim
            for d in range(a.ndim):
                t.shape[d] = a.shape[d]
            t.host_data = a.ctypes.data
        h = ctypes.c_void_p()
        _check(lib().mrf_create(ctypes.byref(c), table, len(weights), ctypes.byref(h)))
        self._h = h
        self._host_pending = []  # (input, output) host tensors of forward_host_async calls not yet synced

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            lib().mrf_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check_input(self, x):
        """stft_repr must be a contiguous CUDA float32 [B, F*C, T, 2] of this model's rows."""
        import torch
        assert x.is_cuda and x.dtype == torch.float32 and x.is_contiguous(), "stft_repr: contiguous CUDA float32"
        assert x.dim() == 4 and x.shape[1] == self.rows and x.shape[3] == 2, \
            f"stft_repr must be [B, {self.rows}, T, 2], got {tuple(x.shape)}"

    def _check_host_input(self, x):
        """stft_repr for the host-buffer entry points: a contiguous host float32 [B, F*C, T, 2]."""
        import torch
        assert not x.is_cuda and x.dtype == torch.float32 and x.is_contiguous(), "stft_repr: contiguous host float32"
        assert x.dim() == 4 and x.shape[1] == self.rows and x.shape[3] == 2, \
            f"stft_repr must be [B, {self.rows}, T, 2], got {tuple(x.shape)}"

    def _check_out(self, x, out):
        """`out` must hold exactly B * num_stems * rows * T * 2 floats, on x's device."""
        import torch
        B, R, T, _ = x.shape
        need = B * self.cfg.num_stems * R * T * 2
        assert out.dtype == torch.float32 and out.is_contiguous(), "out: contiguous float32"
        assert out.device == x.device and out.is_cuda == x.is_cuda, "out must be on stft_repr's device"
        assert out.numel() == need, f"out holds {out.numel()} floats, the forward writes {need}"

    def _out_like(self, x, out):
        """[B, F*2, T, 2] for one stem, [B, stems, F*2, T, 2] for more."""
        import torch
        if out is not None:
            self._check_out(x, out)
            return out
        B, R, T, two = x.shape
        stems = self.cfg.num_stems
        shape = (B, R, T, two) if stems == 1 else (B, stems, R, T, two)
        return torch.empty(shape, dtype=x.dtype, device=x.device, pin_memory=not x.is_cuda and x.is_pinned())

    def forward(self, stft_repr, out=None, stream=None):
        """masks for a CUDA float32 tensor [B, F*2, T, 2] (queued on `stream`)."""
        self._check_input(stft_repr)
        B, R, T, two = stft_repr.shape
        out = self._out_like(stft_repr, out)
        _check(lib().mrf_forward(self._h, ctypes.c_void_p(stft_repr.data_ptr()),
                                 ctypes.c_void_p(out.data_ptr()), B, T, _stream_ptr(stream)), self._h)
        return out

    def separate(self, stft_repr, out=None, stream=None):
        """mrf_forward_separate: the separated spectra (masks times stft_repr, complex), same
        shape as forward's masks."""
        self._check_input(stft_repr)
        B, R, T, two = stft_repr.shape
        out = self._out_like(stft_repr, out)
        _check(lib().mrf_forward_separate(self._h, ctypes.c_void_p(stft_repr.data_ptr()),
                                          ctypes.c_void_p(out.data_ptr()), B, T, _stream_ptr(stream)), self._h)
        return out

    def stft(self, audio, hop, out=None, stream=None):
        """mrf_stft: CUDA float32 audio [B, C, L] -> stft_repr [B, (n_fft/2+1) C, 1 + L // hop, 2]."""
        import torch
        assert audio.is_cuda and audio.dtype == torch.float32 and audio.is_contiguous()
        B, C, L = audio.shape
        if out is None:
            out = torch.empty((B, (self.cfg.n_fft // 2 + 1) * C, 1 + L // hop, 2), dtype=audio.dtype,
                              device=audio.device)
        _check(lib().mrf_stft(self._h, ctypes.c_void_p(audio.data_ptr()), ctypes.c_void_p(out.data_ptr()), B, L,
                              hop, _stream_ptr(stream)), self._h)
        return out

    def istft(self, spec, hop, length, out=None, stream=None):
        """mrf_istft: CUDA float32 spectra [..., (n_fft/2+1) C, T, 2] -> audio [..., C, length]."""
        import torch
        assert spec.is_cuda and spec.dtype == torch.float32 and spec.is_contiguous()
        lead, FC, T = spec.shape[:-3], spec.shape[-3], spec.shape[-2]
        C = self.cfg.audio_channels
        S = int(np.prod(lead)) if lead else 1
        if out is None:
            out = torch.empty(tuple(lead) + (C, length), dtype=spec.dtype, device=spec.device)
        _check(lib().mrf_istft(self._h, ctypes.c_void_p(spec.data_ptr()), ctypes.c_void_p(out.data_ptr()), S, T,
                               hop, length, _stream_ptr(stream)), self._h)
        return out

    def separate_audio(self, mix, hop, out=None, stream=None, chunk_samples=0):
        """mrf_separate_audio(_chunked): CUDA float32 mix [C, L] -> stems [num_stems, C, L], in chunks
        of chunk_samples samples (0: 8 s)."""
        import torch
        assert mix.is_cuda and mix.dtype == torch.float32 and mix.is_contiguous()
        C, L = mix.shape
        if out is None:
            out = torch.empty((self.cfg.num_stems, C, L), dtype=mix.dtype, device=mix.device)
        assert out.is_cuda and out.dtype == torch.float32 and out.is_contiguous() and \
            out.numel() == self.cfg.num_stems * C * L
        _check(lib().mrf_separate_audio_chunked(self._h, ctypes.c_void_p(mix.data_ptr()),
                                                ctypes.c_void_p(out.data_ptr()), L, hop, chunk_samples,
                                                _stream_ptr(stream)), self._h)
        return out

    def forward_static(self, stft_repr, out, stream=None):
        """mrf_forward_static: the same forward with the library's fixed device scratch
        instead of the handle's workspace; allocates nothing (out must be given)."""
        self._check_input(stft_repr)
        self._check_out(stft_repr, out)
        B, R, T, _ = stft_repr.shape
        _check(lib().mrf_forward_static(self._h, ctypes.c_void_p(stft_repr.data_ptr()),
                                        ctypes.c_void_p(out.data_ptr()), B, T, _stream_ptr(stream)), self._h)
        return out

    def forward_host(self, stft_repr, out=None, stream=None):
        """masks for a host float32 array/tensor, copies inside the call; waits for the stream."""
        import torch
        x = stft_repr if isinstance(stft_repr, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(stft_repr))
        self._check_host_input(x)
        B, R, T, _ = x.shape
        out = self._out_like(x, out)
        _check(lib().mrf_forward_host(self._h, ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                                      B, T, _stream_ptr(stream)), self._h)
        return out

    def forward_host_async(self, stft_repr, out, stream=None):
        """enqueues H2D copy, forward and D2H copy of one host tensor and returns; `out` holds the
        masks once host_join and a stream synchronize (or sync_status) have followed.  Both
        tensors are kept referenced here until then; pin them for copies that overlap compute."""
        x = stft_repr
        self._check_host_input(x)
        self._check_out(x, out)
        B, R, T, _ = x.shape
        _check(lib().mrf_forward_host_async(self._h, ctypes.c_void_p(stft_repr.data_ptr()),
                                            ctypes.c_void_p(out.data_ptr()), B, T, _stream_ptr(stream)), self._h)
        self._host_pending.append((stft_repr, out))
        return out

    def host_join(self, stream=None):
        """makes `stream` wait for every copy forward_host_async enqueued (no host wait)."""
        _check(lib().mrf_host_join(self._h, _stream_ptr(stream)), self._h)

    def sync_status(self, stream=None):
        _check(lib().mrf_sync_status(self._h, _stream_ptr(stream)), self._h)
        self._host_pending = []

    def set_timing(self, on: bool):
        _check(lib().mrf_set_timing(self._h, int(on)), self._h)

    def set_graph(self, on: bool):
        _check(lib().mrf_set_graph(self._h, int(on)), self._h)

    def kernel_times(self):
        """{kernel name: (launches, total ms)} since the last call (timing mode)."""
        n = ctypes.c_int(0)
        buf = (mrf_kernel_time * 64)()
        _check(lib().mrf_kernel_times(self._h, buf, 64, ctypes.byref(n)), self._h)
        return {buf[i].name.decode(): (buf[i].launches, buf[i].ms) for i in range(n.value)}

    def debug_buffer(self, name, count):
        """First `count` float32 values of an internal buffer of the last forward ("X", "M")."""
        out = np.zeros(count, np.float32)
        n = ctypes.c_size_t(0)
        _check(lib().mrf_debug_buffer(self._h, name.encode(), out.ctypes.data_as(ctypes.c_void_p),
                                      out.nbytes, ctypes.byref(n)), self._h)
        return out[: n.value // 4]

    def debug_stall_next(self):
        """mrf_debug_stall_next: the next fp16 forward's first GEMM lets its bounded waits expire."""
        _check(lib().mrf_debug_stall_next(self._h), self._h)

    def launches_per_forward(self, B, T):
        return lib().mrf_launches_per_forward(self._h, B, T)
