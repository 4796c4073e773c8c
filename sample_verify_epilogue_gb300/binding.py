"""ctypes binding of libdspark.so: the C ABI of include/dspark.h with the same names.

Argument marshalling only.  Every step of the epilogue runs in the library's sm_103a
kernels; this module passes device pointers (``tensor.data_ptr()``) and the current torch
stream.  It raises if the library has not been built: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

from .build import LIB

DSPARK_OK = 0
DSPARK_BF16 = 0
DSPARK_FP32 = 1
DSPARK_MAX_TOP_LOGPROBS = 20
DSPARK_MAX_SPARSE_M = 256
DSPARK_MAX_TOP_LOGITS = 256
DSPARK_MAX_GRADS = 1 << 16
DSPARK_Q_DENSE, DSPARK_Q_SPARSE, DSPARK_Q_REDUCED = 0, 1, 2
DSPARK_LOGPROBS_RAW, DSPARK_LOGPROBS_PENALISED = 0, 1
Q_LAYOUTS = {"dense": DSPARK_Q_DENSE, "sparse": DSPARK_Q_SPARSE, "reduced": DSPARK_Q_REDUCED}
LOGPROB_MODES = {"raw": DSPARK_LOGPROBS_RAW, "penalised": DSPARK_LOGPROBS_PENALISED}

ROW_BAD_PARAMS = 1
ROW_BAD_DRAFT = 2
ROW_NONFINITE = 4
ROW_BAD_HISTORY = 8
ROW_INTERNAL = 16
ROW_BAD_BIAS = 32
ROW_BAD_MASK = 64
ROW_BAD_TEACHER = 128
ROW_BAD_TOKEN = 256
DSPARK_SAVED_FLOATS = 8

# dspark_row_params_t: float, int32, float, float, float, int32 (24 bytes)
ROW_PARAMS_DTYPE = np.dtype([
    ("temperature", np.float32), ("top_k", np.int32), ("top_p", np.float32),
    ("presence_penalty", np.float32), ("frequency_penalty", np.float32), ("num_drafts", np.int32),
])

# dspark_process_row_t: three floats and an int32 (16 bytes)
PROCESS_ROW_DTYPE = np.dtype([
    ("repetition_penalty", np.float32), ("presence_penalty", np.float32), ("frequency_penalty", np.float32),
    ("num_drafts", np.int32),
])


class dspark_counts_t(ctypes.Structure):
    _fields_ = [("row_offsets", ctypes.c_void_p), ("token_ids", ctypes.c_void_p), ("counts", ctypes.c_void_p)]


class dspark_extras_t(ctypes.Structure):
    _fields_ = [
        ("q_layout", ctypes.c_int32), ("q_row_len", ctypes.c_int32), ("q_ids", ctypes.c_void_p),
        ("d2t", ctypes.c_void_p), ("eos_ids", ctypes.c_void_p), ("out_stopped", ctypes.c_void_p),
        ("pos_counts", ctypes.c_void_p), ("logprob_mode", ctypes.c_int32),
    ]


class dspark_params_t(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("K_max", ctypes.c_int32), ("V", ctypes.c_int32), ("logits_dtype", ctypes.c_int32),
        ("rows", ctypes.c_void_p), ("want_logprobs", ctypes.c_int32), ("n_top_logprobs", ctypes.c_int32),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p),
        ("row_status", ctypes.c_void_p), ("stage_events", ctypes.c_void_p * 2),
        ("extras", ctypes.POINTER(dspark_extras_t)),
    ]


class dspark_bias_t(ctypes.Structure):
    _fields_ = [("row_offsets", ctypes.c_void_p), ("token_ids", ctypes.c_void_p), ("biases", ctypes.c_void_p)]


class dspark_mask_t(ctypes.Structure):
    _fields_ = [("words", ctypes.c_void_p), ("words_stride", ctypes.c_int64), ("n_rows", ctypes.c_int32),
                ("rows", ctypes.c_void_p)]


class dspark_process_params_t(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("K_max", ctypes.c_int32), ("V", ctypes.c_int32), ("logits_dtype", ctypes.c_int32),
        ("logits_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64), ("rows", ctypes.c_void_p),
        ("stream", ctypes.c_void_p), ("row_status", ctypes.c_void_p), ("history_nnz", ctypes.c_int32),
        ("bias_nnz", ctypes.c_int32),
    ]


class dspark_top_params_t(ctypes.Structure):
    _fields_ = [
        ("n_rows", ctypes.c_int32), ("V", ctypes.c_int32), ("logits_dtype", ctypes.c_int32),
        ("logits_stride", ctypes.c_int64), ("n", ctypes.c_int32), ("temperature", ctypes.c_float),
        ("stream", ctypes.c_void_p), ("row_status", ctypes.c_void_p),
    ]


class dspark_teacher_t(ctypes.Structure):
    _fields_ = [
        ("ids", ctypes.c_void_p), ("logits", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("n", ctypes.c_int32),
        ("t2d", ctypes.c_void_p), ("target_V", ctypes.c_int32),
    ]


class dspark_distill_params_t(ctypes.Structure):
    _fields_ = [
        ("n_rows", ctypes.c_int32), ("V", ctypes.c_int32), ("logits_dtype", ctypes.c_int32),
        ("student_stride", ctypes.c_int64), ("grad_stride", ctypes.c_int64), ("temperature", ctypes.c_float),
        ("weights", ctypes.c_void_p), ("stream", ctypes.c_void_p), ("row_status", ctypes.c_void_p),
    ]


class dspark_token_params_t(ctypes.Structure):
    _fields_ = [
        ("n_rows", ctypes.c_int32), ("V", ctypes.c_int32), ("logits_dtype", ctypes.c_int32),
        ("logits_stride", ctypes.c_int64), ("grad_stride", ctypes.c_int64), ("temperature", ctypes.c_float),
        ("tokens", ctypes.c_void_p), ("stream", ctypes.c_void_p), ("row_status", ctypes.c_void_p),
    ]


class dspark_policy_t(ctypes.Structure):
    _fields_ = [
        ("old_logprobs", ctypes.c_void_p), ("ref_logprobs", ctypes.c_void_p), ("advantages", ctypes.c_void_p),
        ("weights", ctypes.c_void_p), ("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float),
        ("kl_coef", ctypes.c_float), ("entropy_coef", ctypes.c_float),
    ]


class dspark_preference_t(ctypes.Structure):
    _fields_ = [
        ("n_pairs", ctypes.c_int32), ("row_offsets", ctypes.c_void_p), ("ref_logprobs", ctypes.c_void_p),
        ("weights", ctypes.c_void_p), ("beta", ctypes.c_float), ("margin", ctypes.c_float),
        ("label_smoothing", ctypes.c_float), ("mean", ctypes.c_int32),
    ]


class dspark_grad_t(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


def make_extras(q_layout="dense", q_row_len=0, q_ids=None, d2t=None, eos_ids=None, out_stopped=None,
                pos_counts=None, logprob_mode="raw"):
    """A dspark_extras_t; array arguments are raw addresses (int) or None."""
    x = dspark_extras_t()
    x.q_layout = Q_LAYOUTS[q_layout] if isinstance(q_layout, str) else int(q_layout)
    x.q_row_len = int(q_row_len)
    x.q_ids, x.d2t, x.eos_ids = q_ids, d2t, eos_ids
    x.out_stopped, x.pos_counts = out_stopped, pos_counts
    x.logprob_mode = LOGPROB_MODES[logprob_mode] if isinstance(logprob_mode, str) else int(logprob_mode)
    return x


_lib = None

EXPORTS = ("dspark_workspace_bytes", "dspark_verify_sample", "dspark_host_workspace_bytes",
           "dspark_verify_sample_host", "dspark_verify_sample_static", "dspark_status_string",
           "dspark_launches_per_call", "dspark_process_logits", "dspark_top_logits", "dspark_distill",
           "dspark_distill_backward", "dspark_token_logprobs", "dspark_token_logprobs_backward", "dspark_policy_loss",
           "dspark_policy_loss_backward", "dspark_preference_loss", "dspark_preference_loss_backward",
           "dspark_clip_workspace_bytes", "dspark_clip_grads")

DSPARK_STATIC_WORKSPACE_BYTES = 16 << 20


def load_library(path: str = LIB):
    """Load libdspark.so (built by ``sample_verify_epilogue_gb300.build.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    _lib = open_library(path)
    return _lib


def open_library(path: str):
    """A CDLL of a build of the library at ``path`` with the argument types set (not cached)."""
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} not found at {path}: build it first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(dspark_params_t)
    C = ctypes.POINTER(dspark_counts_t)
    vp = ctypes.c_void_p
    lib.dspark_workspace_bytes.argtypes = [P]
    lib.dspark_workspace_bytes.restype = ctypes.c_size_t
    lib.dspark_host_workspace_bytes.argtypes = [P, ctypes.c_int64]
    lib.dspark_host_workspace_bytes.restype = ctypes.c_size_t
    sig = [vp, vp, vp, C, P, vp, vp, vp, vp, vp, vp]
    lib.dspark_verify_sample.argtypes = sig
    lib.dspark_verify_sample.restype = ctypes.c_int
    lib.dspark_verify_sample_host.argtypes = sig
    lib.dspark_verify_sample_host.restype = ctypes.c_int
    lib.dspark_verify_sample_static.argtypes = sig
    lib.dspark_verify_sample_static.restype = ctypes.c_int
    lib.dspark_clip_workspace_bytes.argtypes = [ctypes.c_int32]
    lib.dspark_clip_workspace_bytes.restype = ctypes.c_size_t
    lib.dspark_status_string.argtypes = [ctypes.c_int]
    lib.dspark_status_string.restype = ctypes.c_char_p
    lib.dspark_launches_per_call.argtypes = []
    lib.dspark_launches_per_call.restype = ctypes.c_int32
    lib.dspark_process_logits.argtypes = [vp, vp, vp, C, ctypes.POINTER(dspark_bias_t), ctypes.POINTER(dspark_mask_t),
                                          ctypes.POINTER(dspark_process_params_t)]
    lib.dspark_process_logits.restype = ctypes.c_int
    lib.dspark_top_logits.argtypes = [vp, ctypes.POINTER(dspark_top_params_t), vp, vp, vp]
    lib.dspark_top_logits.restype = ctypes.c_int
    T, D = ctypes.POINTER(dspark_teacher_t), ctypes.POINTER(dspark_distill_params_t)
    lib.dspark_distill.argtypes = [vp, T, D, vp, vp, vp]
    lib.dspark_distill.restype = ctypes.c_int
    lib.dspark_distill_backward.argtypes = [vp, T, D, vp, vp, vp]
    lib.dspark_distill_backward.restype = ctypes.c_int
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def make_params(B, K_max, V, logits_dtype, *, rows=None, want_logprobs=False, n_top_logprobs=0,
                workspace=None, workspace_bytes=0, stream=None, row_status=None, stage_events=(None, None),
                extras=None):
    p = dspark_params_t()
    p.B, p.K_max, p.V = int(B), int(K_max), int(V)
    p.logits_dtype = DSPARK_BF16 if logits_dtype in ("bf16", DSPARK_BF16) else DSPARK_FP32
    p.rows = rows
    p.want_logprobs = int(bool(want_logprobs))
    p.n_top_logprobs = int(n_top_logprobs)
    p.workspace = workspace
    p.workspace_bytes = int(workspace_bytes)
    p.stream = stream
    p.row_status = row_status
    p.stage_events[0] = stage_events[0]
    p.stage_events[1] = stage_events[1]
    if extras is not None:
        p.extras = ctypes.pointer(extras)
    return p


def dspark_workspace_bytes(B, K_max, V, logits_dtype, n_top_logprobs=0, extras=None) -> int:
    lib = load_library()
    p = make_params(B, K_max, V, logits_dtype, n_top_logprobs=n_top_logprobs, extras=extras)
    return int(lib.dspark_workspace_bytes(ctypes.byref(p)))


def dspark_host_workspace_bytes(B, K_max, V, logits_dtype, n_top_logprobs=0, counts_nnz=0, extras=None) -> int:
    lib = load_library()
    p = make_params(B, K_max, V, logits_dtype, n_top_logprobs=n_top_logprobs, extras=extras)
    return int(lib.dspark_host_workspace_bytes(ctypes.byref(p), int(counts_nnz)))


def dspark_status_string(code: int) -> str:
    return load_library().dspark_status_string(int(code)).decode()


def dspark_launches_per_call() -> int:
    return int(load_library().dspark_launches_per_call())


def _check(code):
    if code != DSPARK_OK:
        raise RuntimeError(f"dspark: {dspark_status_string(code)} ({code})")


def _device_call(fn, logits, q, draft_ids, counts, rows, uniforms, out, row_status, workspace, want_logprobs,
                 n_top_logprobs, stream, stage_events, extras=None):
    import torch
    B, W, V = logits.shape
    if stream is None:
        stream = torch.cuda.current_stream(logits.device).cuda_stream
    dt = DSPARK_BF16 if logits.dtype == torch.bfloat16 else DSPARK_FP32
    p = make_params(B, W - 1, V, dt, rows=rows.data_ptr(), want_logprobs=want_logprobs,
                    n_top_logprobs=n_top_logprobs,
                    workspace=None if workspace is None else workspace.data_ptr(),
                    workspace_bytes=0 if workspace is None else workspace.numel() * workspace.element_size(),
                    stream=stream, row_status=row_status.data_ptr(),
                    stage_events=tuple(None if e is None else e for e in stage_events), extras=extras)
    c = None
    if counts is not None:
        c = dspark_counts_t(counts[0].data_ptr(), counts[1].data_ptr(), counts[2].data_ptr())
    code = fn(
        _ptr(logits), _ptr(q), _ptr(draft_ids), ctypes.byref(c) if c is not None else None, ctypes.byref(p),
        _ptr(uniforms), _ptr(out["accept_len"]), _ptr(out["tokens"]), _ptr(out.get("logprobs")),
        _ptr(out.get("top_ids")), _ptr(out.get("top_logprobs")))
    _check(code)


def dspark_verify_sample(logits, q, draft_ids, counts, rows, uniforms, *, out, row_status, workspace,
                         want_logprobs=False, n_top_logprobs=0, stream=None, stage_events=(None, None),
                         extras=None):
    """Enqueue the epilogue on ``stream`` (default: torch's current stream).

    logits [B, K_max+1, V] bf16/fp32, q [B, K_max, V] fp32 or None, draft_ids [B, K_max] int32,
    counts (offsets [B+1], ids, counts) int32 or None, rows: uint8 tensor of B packed
    dspark_row_params_t, uniforms [B, K_max+1, 2] fp32 -- all CUDA tensors.
    out: dict with "accept_len" [B], "tokens" [B, K_max+1] int32, and optionally
    "logprobs" [B, K_max+1], "top_ids" / "top_logprobs" [B, K_max+1, n] tensors.
    extras: a dspark_extras_t (``make_extras``, device addresses) or None.
    """
    _device_call(load_library().dspark_verify_sample, logits, q, draft_ids, counts, rows, uniforms, out,
                 row_status, workspace, want_logprobs, n_top_logprobs, stream, stage_events, extras)


def dspark_verify_sample_static(logits, q, draft_ids, counts, rows, uniforms, *, out, row_status,
                                want_logprobs=False, n_top_logprobs=0, stream=None, stage_events=(None, None),
                                extras=None):
    """The same call with the library's fixed device scratch (no workspace, no allocation);
    shapes needing more than DSPARK_STATIC_WORKSPACE_BYTES are refused.  Calls that overlap
    on the GPU race on that scratch."""
    _device_call(load_library().dspark_verify_sample_static, logits, q, draft_ids, counts, rows, uniforms, out,
                 row_status, None, want_logprobs, n_top_logprobs, stream, stage_events, extras)


def dspark_verify_sample_host(logits, q, draft_ids, counts, rows, uniforms, *, out, row_status, workspace,
                              logits_dtype, want_logprobs=False, n_top_logprobs=0, stream=None, extras=None):
    """The epilogue from host buffers (numpy or pinned torch CPU tensors); synchronous.

    ``workspace`` is a CUDA uint8 tensor of at least dspark_host_workspace_bytes bytes.
    Outputs are written into the host arrays of ``out`` and ``row_status``; ``extras`` holds
    host addresses."""
    lib = load_library()
    B, W, V = logits.shape

    def hp(a):
        if a is None:
            return None
        if isinstance(a, np.ndarray):
            assert a.flags.c_contiguous
            return ctypes.c_void_p(a.ctypes.data)
        return ctypes.c_void_p(a.data_ptr())

    p = make_params(B, W - 1, V, logits_dtype, rows=hp(rows).value, want_logprobs=want_logprobs,
                    n_top_logprobs=n_top_logprobs, workspace=workspace.data_ptr(),
                    workspace_bytes=workspace.numel() * workspace.element_size(), stream=stream,
                    row_status=hp(row_status).value, extras=extras)
    c = None
    if counts is not None:
        c = dspark_counts_t(hp(counts[0]).value, hp(counts[1]).value, hp(counts[2]).value)
    code = lib.dspark_verify_sample_host(
        hp(logits), hp(q), hp(draft_ids), ctypes.byref(c) if c is not None else None, ctypes.byref(p),
        hp(uniforms), hp(out["accept_len"]), hp(out["tokens"]), hp(out.get("logprobs")),
        hp(out.get("top_ids")), hp(out.get("top_logprobs")))
    _check(code)


# ---------------------------------------------------------------- around the epilogue
# These calls are a few microseconds of GPU work on small batches, so their checks are kept to
# one cheap comparison per property; device indices stand for devices.
class _Torch:
    """What the calls below use of torch, looked up once (this module is importable without it)."""

    def __init__(self):
        import torch
        self.i32, self.f32, self.u8 = torch.int32, torch.float32, torch.uint8
        self.dtypes = {torch.bfloat16: DSPARK_BF16, torch.float32: DSPARK_FP32}
        self.stream = torch._C._cuda_getCurrentRawStream
        self.device = torch._C._cuda_getDevice
        self.guard = torch.cuda.device


_torch = None


def _t():
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _dtype_of(logits):
    d = _t().dtypes.get(logits.dtype)
    if d is None:
        raise TypeError(f"logits are bfloat16 or float32, not {logits.dtype}")
    return d


def _packer(cls):
    """pack(*fields) -> the bytes of a structure: a quarter of the time that ctypes takes to make one (0 for a
    null pointer)."""
    kinds = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_void_p: "P"}
    layout = struct.Struct("@" + "".join(kinds[t] for _, t in cls._fields_) + "0P")
    assert layout.size == ctypes.sizeof(cls)
    return layout.pack


_counts, _bias, _mask, _process_params, _top_params, _teacher, _distill_params = map(_packer, (
    dspark_counts_t, dspark_bias_t, dspark_mask_t, dspark_process_params_t, dspark_top_params_t, dspark_teacher_t,
    dspark_distill_params_t))
_token_params, _policy, _preference, _grad = map(_packer, (dspark_token_params_t, dspark_policy_t, dspark_preference_t,
                                                           dspark_grad_t))


class _Calls:
    """The entry points around the epilogue, taking packed structures."""

    def __init__(self, lib):
        P, i32 = ctypes.c_void_p, ctypes.c_int32
        for name, args in (("dspark_process_logits", [P] * 7), ("dspark_top_logits", [P] * 5), ("dspark_distill", [P] * 6),
                           ("dspark_distill_backward", [P] * 6), ("dspark_token_logprobs", [P] * 5),
                           ("dspark_token_logprobs_backward", [P] * 6), ("dspark_policy_loss", [P] * 9),
                           ("dspark_policy_loss_backward", [P] * 6), ("dspark_preference_loss", [P] * 9),
                           ("dspark_preference_loss_backward", [P, P, i32, P, P, P]),
                           ("dspark_clip_grads", [P, i32, ctypes.c_float, P, P, P, ctypes.c_size_t, P])):
            fn = lib[name]
            fn.argtypes = args
            fn.restype = ctypes.c_int
            setattr(self, name, fn)


_calls_of = None


def _calls():
    global _calls_of
    if _calls_of is None:
        _calls_of = _Calls(load_library())
    return _calls_of


def _rows_of(name, t, like=None):
    """(rows, V, stride) of a tensor of logits [..., V]: each row contiguous, the rows evenly spaced."""
    shape = t.shape
    if like is not None and (shape != like.shape or t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must have the shape, dtype and device of the logits")
    if t.dim() < 1 or t.numel() == 0:
        raise ValueError(f"{name} is empty")
    V = shape[-1]
    if t.is_contiguous():
        return t.numel() // V, V, V
    if t.stride(-1) != 1 and V > 1:
        raise ValueError(f"{name}: the logits of a row must be contiguous")
    rows, stride = 1, V
    for d in range(t.dim() - 2, -1, -1):
        if shape[d] == 1:
            continue
        if rows == 1:
            stride = t.stride(d)
        elif t.stride(d) != rows * stride:
            raise ValueError(f"{name}: the rows must be evenly spaced")
        rows *= shape[d]
    if stride < V:
        raise ValueError(f"{name}: rows overlap")
    return rows, V, stride


def _flat(name, t, dtype, numel, dev):
    """The address of a contiguous tensor of ``numel`` elements on device ``dev``."""
    if t is None or t.dtype is not dtype or t.numel() != numel or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {numel} elements on the logits' device")
    return t.data_ptr()


def _device_of(name, t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _launch(fn, dev, *args):
    """Call ``fn`` with device ``dev`` current."""
    if _torch.device() == dev:
        code = fn(*args)
    else:
        with _torch.guard(dev):
            code = fn(*args)
    if code != DSPARK_OK:
        _check(code)


def dspark_process_logits(logits, rows, *, out, row_status, draft_ids=None, history=None, bias=None, mask=None,
                          mask_rows=None, stream=None):
    """Penalties, biases and grammar masks on the logits of every verify position, on ``stream``
    (default: torch's current stream).

    logits, out [B, K_max+1, V] bf16/fp32 (``out`` may be ``logits``), rows: uint8 tensor of B packed
    dspark_process_row_t (PROCESS_ROW_DTYPE), row_status [B] int32, draft_ids [B, K_max] int32,
    history (offsets [B+1], ids, counts) int32, bias (offsets [B+1] int32, ids int32, values fp32),
    mask [n, words >= ceil(V/32)] int32 bits of the allowed tokens (n may be 0 beside mask_rows), mask_rows
    [B, K_max+1] int32 rows of mask (-1: no grammar) or None (row b*(K_max+1) + j) -- all CUDA tensors.
    """
    T = _t()
    dev = _device_of("logits", logits)
    if logits.dim() != 3:
        raise ValueError("logits must be [B, K_max+1, V]")
    B, W, V = logits.shape
    stride = _rows_of("logits", logits)[2]
    out_stride = stride if out is logits else _rows_of("out", out, logits)[2]
    i32, f32 = T.i32, T.f32
    d = h = b = m = None
    n_history = n_bias = 0
    if draft_ids is not None and W > 1:
        d = _flat("draft_ids", draft_ids, i32, B * (W - 1), dev)
    if history is not None:
        off, ids, counts = history
        n_history = ids.numel()
        at = _flat("history offsets", off, i32, B + 1, dev)
        # (columns of no elements have no address, and none of them is read)
        h = _counts(at, _flat("history ids", ids, i32, n_history, dev) or at,
                    _flat("history counts", counts, i32, n_history, dev) or at)
    if bias is not None:
        off, ids, values = bias
        n_bias = ids.numel()
        at = _flat("bias offsets", off, i32, B + 1, dev)
        b = _bias(at, _flat("bias ids", ids, i32, n_bias, dev) or at, _flat("bias values", values, f32, n_bias, dev) or at)
    if mask is not None:
        if mask.dim() != 2 or mask.dtype is not i32 or mask.get_device() != dev or (mask.stride(1) != 1 and mask.shape[1] > 1):
            raise ValueError("mask must be [n, words] int32 rows on the logits' device")
        n, words = mask.shape
        if words < (V + 31) // 32:
            raise ValueError(f"mask rows have {words} words for {V} tokens")
        if n == 0 and mask_rows is None:
            raise ValueError("mask has no rows")
        m = _mask(mask.data_ptr(), mask.stride(0) if n > 1 else words, n,
                  0 if mask_rows is None else _flat("mask_rows", mask_rows, i32, B * W, dev))
    elif mask_rows is not None:
        raise ValueError("mask_rows without a mask")
    p = _process_params(B, W - 1, V, _dtype_of(logits), stride, out_stride, _flat("rows", rows, T.u8, B * 16, dev),
                        T.stream(dev) if stream is None else stream, _flat("row_status", row_status, i32, B, dev), n_history,
                        n_bias)
    _launch(_calls().dspark_process_logits, dev, logits.data_ptr(), out.data_ptr(), d, h, b, m, p)


def dspark_top_logits(logits, *, values, ids, row_status, lse=None, temperature=1.0, stream=None):
    """The n largest logits of every row and the row's log-sum-exp, on ``stream``.

    logits [..., V] bf16/fp32 of R rows, values fp32 and ids int32 [..., n], lse [...] fp32 or None,
    row_status [...] int32 -- all CUDA tensors; n is the last size of values.
    """
    T = _t()
    dev = _device_of("logits", logits)
    R, V, stride = _rows_of("logits", logits)
    n = values.shape[-1]
    i32, f32 = T.i32, T.f32
    p = _top_params(R, V, _dtype_of(logits), stride, n, temperature, T.stream(dev) if stream is None else stream,
                    _flat("row_status", row_status, i32, R, dev))
    _launch(_calls().dspark_top_logits, dev, logits.data_ptr(), p, _flat("values", values, f32, R * n, dev),
            _flat("ids", ids, i32, R * n, dev), None if lse is None else _flat("lse", lse, f32, R, dev))


def _distill_args(student, teacher_ids, teacher_logits, teacher_lse, t2d, weights, temperature, row_status, grad, stream):
    T = _t()
    dev = _device_of("student", student)
    R, V, stride = _rows_of("student", student)
    grad_stride = V if grad is None else stride if grad is student else _rows_of("grad", grad, student)[2]
    i32, f32 = T.i32, T.f32
    n = teacher_ids.shape[-1]
    t = _teacher(_flat("teacher_ids", teacher_ids, i32, R * n, dev), _flat("teacher_logits", teacher_logits, f32, R * n, dev),
                 0 if teacher_lse is None else _flat("teacher_lse", teacher_lse, f32, R, dev), n,
                 0 if t2d is None else _flat("t2d", t2d, i32, t2d.numel(), dev), 0 if t2d is None else t2d.numel())
    p = _distill_params(R, V, _dtype_of(student), stride, grad_stride, temperature,
                        0 if weights is None else _flat("weights", weights, f32, R, dev),
                        T.stream(dev) if stream is None else stream,
                        0 if row_status is None else _flat("row_status", row_status, i32, R, dev))
    return dev, R, t, p


def dspark_distill(student, teacher_ids, teacher_logits, *, loss, row_status, grad=None, saved=None, teacher_lse=None,
                   t2d=None, weights=None, temperature=1.0, stream=None):
    """Divergence of the student's softmax from a teacher's top logits, row by row, on ``stream``; with
    ``grad``, its gradient in the same launch.

    student [..., V] bf16/fp32 of R rows, teacher_ids int32 and teacher_logits fp32 [..., n] (id -1: no
    entry), teacher_lse [...] fp32 (the rest of the teacher's mass is one class) or None (the record
    is renormalised), t2d [target_V] int32 draft id of each target id or None, weights [...] fp32 or
    None; loss [...] fp32, row_status [...] int32, grad like student (may be student) or None, saved
    [..., 4] fp32 for dspark_distill_backward or None -- all CUDA tensors.
    """
    if row_status is None:
        raise ValueError("row_status is missing")
    dev, R, t, p = _distill_args(student, teacher_ids, teacher_logits, teacher_lse, t2d, weights, temperature,
                                 row_status, grad, stream)
    f32 = _torch.f32
    _launch(_calls().dspark_distill, dev, student.data_ptr(), t, p, _flat("loss", loss, f32, R, dev),
            None if saved is None else _flat("saved", saved, f32, 4 * R, dev), None if grad is None else grad.data_ptr())


def dspark_distill_backward(student, teacher_ids, teacher_logits, *, saved, grad, grad_loss=None, teacher_lse=None,
                            t2d=None, weights=None, temperature=1.0, row_status=None, stream=None):
    """The gradient of sum(grad_loss * loss) by the student's logits, from the inputs and the ``saved`` of
    a dspark_distill call; grad_loss [...] fp32 or None (all 1).  ``row_status``, if given, is written for rows
    alone that end with DSPARK_ROW_INTERNAL here."""
    if grad is None:
        raise ValueError("grad is missing")
    dev, R, t, p = _distill_args(student, teacher_ids, teacher_logits, teacher_lse, t2d, weights, temperature,
                                 row_status, grad, stream)
    f32 = _torch.f32
    _launch(_calls().dspark_distill_backward, dev, student.data_ptr(), t, p, _flat("saved", saved, f32, 4 * R, dev),
            None if grad_loss is None else _flat("grad_loss", grad_loss, f32, R, dev), grad.data_ptr())


# ---------------------------------------------------------------- training on decoded tokens
def _token_args(logits, tokens, temperature, row_status, grad, stream):
    T = _t()
    dev = _device_of("logits", logits)
    R, V, stride = _rows_of("logits", logits)
    grad_stride = V if grad is None else stride if grad is logits else _rows_of("grad", grad, logits)[2]
    p = _token_params(R, V, _dtype_of(logits), stride, grad_stride, temperature, _flat("tokens", tokens, T.i32, R, dev),
                      T.stream(dev) if stream is None else stream,
                      0 if row_status is None else _flat("row_status", row_status, T.i32, R, dev))
    return dev, R, p


def _saved(saved, R, dev):
    return _flat("saved", saved, _torch.f32, DSPARK_SAVED_FLOATS * R, dev)


def dspark_token_logprobs(logits, tokens, *, logprobs, row_status, entropy=None, saved=None, temperature=1.0, stream=None):
    """The log-probability of one token of every row, and the entropy of the row's distribution, on ``stream``
    (default: torch's current stream).

    logits [..., V] bf16/fp32 of R rows, tokens [...] int32 (-1: no token, the row is not read and gets 0),
    logprobs [...] fp32, row_status [...] int32, entropy [...] fp32 or None, saved [..., 8] fp32 for
    dspark_token_logprobs_backward or None -- all CUDA tensors.
    """
    dev, R, p = _token_args(logits, tokens, temperature, row_status, None, stream)
    f32 = _torch.f32
    _launch(_calls().dspark_token_logprobs, dev, logits.data_ptr(), p, _flat("logprobs", logprobs, f32, R, dev),
            None if entropy is None else _flat("entropy", entropy, f32, R, dev), None if saved is None else _saved(saved, R, dev))


def dspark_token_logprobs_backward(logits, tokens, *, saved, grad, grad_logprobs=None, grad_entropy=None, temperature=1.0,
                                   stream=None):
    """The gradient of sum(grad_logprobs * logprobs + grad_entropy * entropy) by the logits, from the inputs and the
    ``saved`` of a dspark_token_logprobs call; either of the two [...] fp32 may be None (all 0).  grad_entropy needs a call
    that asked for the entropy.  ``grad`` is like logits and may be logits."""
    if grad is None:
        raise ValueError("grad is missing")
    dev, R, p = _token_args(logits, tokens, temperature, None, grad, stream)
    f32 = _torch.f32
    _launch(_calls().dspark_token_logprobs_backward, dev, logits.data_ptr(), p, _saved(saved, R, dev),
            None if grad_logprobs is None else _flat("grad_logprobs", grad_logprobs, f32, R, dev),
            None if grad_entropy is None else _flat("grad_entropy", grad_entropy, f32, R, dev), grad.data_ptr())


def _policy_of(R, dev, old_logprobs, advantages, ref_logprobs, weights, clip_low, clip_high, kl_coef, entropy_coef):
    f32 = _torch.f32
    return _policy(_flat("old_logprobs", old_logprobs, f32, R, dev),
                   0 if ref_logprobs is None else _flat("ref_logprobs", ref_logprobs, f32, R, dev),
                   _flat("advantages", advantages, f32, R, dev),
                   0 if weights is None else _flat("weights", weights, f32, R, dev), clip_low, clip_high, kl_coef, entropy_coef)


def dspark_policy_loss(logits, tokens, old_logprobs, advantages, *, loss, row_status, ref_logprobs=None, weights=None,
                       logprobs=None, entropy=None, kl=None, saved=None, grad=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                       entropy_coef=0.0, temperature=1.0, stream=None):
    """The clipped policy loss of every row, with a KL term and an entropy bonus, on ``stream``; with ``grad``, its
    gradient as well.

    logits [..., V] bf16/fp32 of R rows, tokens [...] int32 (-1: no token), old_logprobs, advantages, ref_logprobs (or
    None), weights (or None) [...] fp32, the log-probabilities at this call's temperature (a verify call's raw ones are
    at 1); loss [...] fp32, row_status [...] int32, logprobs, entropy, kl [...] fp32 or None, saved [..., 8] fp32 (needed
    with grad and for dspark_policy_loss_backward) or None, grad like logits (may be
    logits) or None -- all CUDA tensors.
    """
    if row_status is None:
        raise ValueError("row_status is missing")
    if grad is not None and saved is None:
        raise ValueError("grad needs saved")
    dev, R, p = _token_args(logits, tokens, temperature, row_status, grad, stream)
    o = _policy_of(R, dev, old_logprobs, advantages, ref_logprobs, weights, clip_low, clip_high, kl_coef, entropy_coef)
    f32 = _torch.f32
    _launch(_calls().dspark_policy_loss, dev, logits.data_ptr(), o, p, _flat("loss", loss, f32, R, dev),
            None if logprobs is None else _flat("logprobs", logprobs, f32, R, dev),
            None if entropy is None else _flat("entropy", entropy, f32, R, dev),
            None if kl is None else _flat("kl", kl, f32, R, dev), None if saved is None else _saved(saved, R, dev),
            None if grad is None else grad.data_ptr())


def dspark_policy_loss_backward(logits, tokens, old_logprobs, advantages, *, saved, grad, grad_loss=None, ref_logprobs=None,
                                weights=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0, entropy_coef=0.0, temperature=1.0,
                                stream=None):
    """The gradient of sum(grad_loss * loss) by the logits, from the inputs and the ``saved`` of a dspark_policy_loss
    call; grad_loss [...] fp32 or None (all 1)."""
    if grad is None:
        raise ValueError("grad is missing")
    dev, R, p = _token_args(logits, tokens, temperature, None, grad, stream)
    o = _policy_of(R, dev, old_logprobs, advantages, ref_logprobs, weights, clip_low, clip_high, kl_coef, entropy_coef)
    _launch(_calls().dspark_policy_loss_backward, dev, logits.data_ptr(), o, p, _saved(saved, R, dev),
            None if grad_loss is None else _flat("grad_loss", grad_loss, _torch.f32, R, dev), grad.data_ptr())


def dspark_preference_loss(logits, tokens, row_offsets, *, loss, saved, row_status, pair_status, rewards=None,
                           logprobs=None, ref_logprobs=None, weights=None, grad=None, beta=0.1, margin=0.0, label_smoothing=0.0,
                           mean=False, temperature=1.0, stream=None):
    """The preference loss of P pairs of sequences, on ``stream``; with ``grad``, its gradient as well.

    logits [..., V] bf16/fp32 of R rows, tokens [...] int32 (-1: no token), row_offsets [2P + 1] int32: sequence 2i, rows
    row_offsets[2i] to row_offsets[2i + 1] - 1, is the chosen one of pair i, sequence 2i + 1 the rejected one;
    ref_logprobs [...] fp32 or None, weights [P] fp32 or None; loss [P] fp32, saved [..., 8] fp32 (for
    dspark_preference_loss_backward too), row_status [...] int32, pair_status [P] int32, rewards [P, 2] fp32 or None,
    logprobs [...] fp32 or None, grad like logits (may be logits) or None -- all CUDA tensors.  With ``mean`` the log ratios
    are averaged over a sequence's tokens instead of summed.
    """
    if row_status is None:
        raise ValueError("row_status is missing")
    dev, R, p = _token_args(logits, tokens, temperature, row_status, grad, stream)
    i32, f32 = _torch.i32, _torch.f32
    P = loss.numel()
    o = _preference(P, _flat("row_offsets", row_offsets, i32, 2 * P + 1, dev),
                    0 if ref_logprobs is None else _flat("ref_logprobs", ref_logprobs, f32, R, dev),
                    0 if weights is None else _flat("weights", weights, f32, P, dev), beta, margin, label_smoothing, bool(mean))
    _launch(_calls().dspark_preference_loss, dev, logits.data_ptr(), o, p, _flat("loss", loss, f32, P, dev),
            None if rewards is None else _flat("rewards", rewards, f32, 2 * P, dev),
            _flat("pair_status", pair_status, i32, P, dev), None if logprobs is None else _flat("logprobs", logprobs, f32, R, dev),
            _saved(saved, R, dev), None if grad is None else grad.data_ptr())


def dspark_preference_loss_backward(logits, tokens, *, saved, grad, grad_loss, temperature=1.0, stream=None):
    """The gradient of sum(grad_loss * loss) by the logits, from the inputs and the ``saved`` of a
    dspark_preference_loss call; grad_loss [P] fp32."""
    if grad is None:
        raise ValueError("grad is missing")
    dev, R, p = _token_args(logits, tokens, temperature, None, grad, stream)
    P = grad_loss.numel()
    _launch(_calls().dspark_preference_loss_backward, dev, logits.data_ptr(), p, P, _saved(saved, R, dev),
            _flat("grad_loss", grad_loss, _torch.f32, P, dev), grad.data_ptr())


def _dense(t):
    """Whether the elements of ``t`` fill its memory, each once, whatever the order of its dimensions."""
    n = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size != 1:
            if stride != n:
                return False
            n *= size
    return True


def _ordered_as(o, t):
    """Whether the dimensions of ``o`` lie in memory as those of ``t``."""
    return o is not None and all(n == 1 or a == b for n, a, b in zip(t.shape, o.stride(), t.stride()))


class GradTable:
    """A list of gradients as dspark_clip_grads takes it, made once for gradients that stay where they are.

    grads: bf16/fp32 CUDA tensors of one device whose elements fill their memory, in any order of dimensions (contiguous,
    transposed, channels-last), None entries left out; out: None (the gradients are clipped in place) or a tensor for each,
    of its shape and order and its dtype or fp32, that overlaps no gradient.  The table holds the tensors; it knows nothing
    of a ``.grad`` that is replaced later.
    """

    def __init__(self, grads, out=None):
        T = _t()
        grads = list(grads)
        out = grads if out is None else list(out)
        if len(out) != len(grads):
            raise ValueError(f"{len(grads)} gradients, {len(out)} outputs")
        pairs = [(g, o) for g, o in zip(grads, out) if g is not None]
        if not pairs:
            raise ValueError("no gradients")
        self.device = _device_of("a gradient", pairs[0][0])
        self.tensors, fields, held = pairs, [], []
        for g, o in pairs:
            if g.get_device() != self.device or not (g.is_contiguous() or _dense(g) and (o is g or _ordered_as(o, g))):
                raise ValueError("the gradients must be dense CUDA tensors of one device, their outputs of the same order")
            if o is not g and (o is None or o.shape != g.shape or o.get_device() != self.device or
                               (not o.is_contiguous() and not _ordered_as(o, g)) or
                               (o.dtype is not g.dtype and o.dtype is not T.f32)):
                raise ValueError("an output must be of its gradient's shape, order and device, and of its dtype or fp32")
            n = g.numel()
            if n:
                held.append((g.data_ptr(), n * g.element_size()))
                if o is not g:
                    held.append((o.data_ptr(), n * o.element_size()))
            fields.append(_grad(g.data_ptr(), o.data_ptr(), n, _dtype_of(g), _dtype_of(o)))
        held.sort()
        end = 0
        for at, size in held:
            if at < end:
                raise ValueError("gradients or outputs overlap, or one appears twice")
            end = at + size
        if len(fields) > DSPARK_MAX_GRADS:
            raise ValueError(f"more than {DSPARK_MAX_GRADS} gradients")
        self.packed = b"".join(fields)

    def __len__(self):
        return len(self.tensors)


def dspark_clip_workspace_bytes(table) -> int:
    return load_library().dspark_clip_workspace_bytes(len(table))


def dspark_clip_grads(table, max_norm, *, norm, status, workspace, stream=None):
    """The norm of the gradients of ``table`` (a GradTable, or a list to make one of) taken together, and the gradients
    scaled by max_norm / norm where the norm is larger than max_norm, on ``stream``.

    norm [1] fp32: before clipping; status [1] int32: 0, or ROW_NONFINITE when the norm is not finite (the gradients are
    then as they were); workspace: uint8 CUDA tensor of at least dspark_clip_workspace_bytes(table) bytes.
    """
    if not isinstance(table, GradTable):
        table = GradTable(table)
    T = _t()
    dev = table.device
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the gradients' device")
    _launch(_calls().dspark_clip_grads, dev, table.packed, len(table), max_norm, _flat("norm", norm, T.f32, 1, dev),
            _flat("status", status, T.i32, 1, dev), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            T.stream(dev) if stream is None else stream)
