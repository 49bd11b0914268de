"""Python binding of the expert-layer operators (include/csf_ops.h): what a
caller of csf.decode runs on either side of the decoded scales.

Argument marshalling only, as in csf.py: the kernels of libcsf.so do the work,
PyTorch supplies device memory and streams, and there is no CPU fallback.

Typical use (one layer of experts)::

    q, h = ops.rms_norm(x, norm_weight, ops.NVFP4, residual=h, tensor_scale=g)
    r = ops.route(logits, k=8)
    csf.decode(stack, ws, expert_start=r.expert_start, layout=csf.LAYOUT_BLOCKED)
    a = ops.expert_matmul(q, w_gate_up, ws, expert_start=r.expert_start, rows=r.rows, alpha=alpha,
                          activation="silu", gated=True, out=ops.NVFP4, out_tensor_scale=g2)
    y = ops.expert_matmul(a, w_down, down_ws, expert_start=r.expert_start, alpha=alpha2)

A call runs on the current stream, or on `stream`, where new results are then
that stream's.  Ordering the streams (wait_stream) is the caller's.
"""
from __future__ import annotations

import ctypes
import struct
import threading
from dataclasses import dataclass

import torch

from .csf import CsfError, _check, _es, lib

NVFP4 = 0     # rows of E2M1 codes, a UE4M3 scale per 16; goes with NVFP4 weights
MXFP8 = 1     # rows of E4M3 codes, a UE8M0 scale per 32; goes with MXFP4 weights
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ACTS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3}

_vp = ctypes.c_void_p


# The argument structs of csf_ops.h, packed as bytes: a fifth of the time that
# ctypes structures take to fill, which is what a one-token call waits for.
_ROWS = "iiqPqPqP"                                    # csf_rows
_RMS_NORM = struct.Struct("@PqPqPqPif" + _ROWS)       # csf_rms_norm_args
_ROUTE = struct.Struct("@PqiiiiiPPPPPPN")             # csf_route_args
_EXPERT_MATMUL = struct.Struct("@" + _ROWS + "PqiiPPPiPPiiiPPqiiPq" + _ROWS + "P")   # csf_expert_matmul_args
_NO_ROWS = (0, 0, 0, 0, 0, 0, 0, 0)

lib.csf_rms_norm.argtypes = [ctypes.c_char_p, _vp]
lib.csf_rms_norm.restype = ctypes.c_int
lib.csf_route.argtypes = [ctypes.c_char_p, _vp]
lib.csf_route.restype = ctypes.c_int
lib.csf_route_scratch_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32]
lib.csf_route_scratch_bytes.restype = ctypes.c_size_t
lib.csf_expert_matmul.argtypes = [ctypes.c_char_p, _vp]
lib.csf_expert_matmul.restype = ctypes.c_int

_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _launch(call, args: bytes, device: int, what: str):
    """The library call on the tensors' device (a stream's handle, 0 of the
    default one above all, means what it does on the current device) and that
    device's current stream."""
    if _current_device() == device:
        status = call(args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = call(args, _raw_stream(device))
    if status:
        _check(status, what)


_error_words: dict[int, torch.Tensor] = {}
_error_lock = threading.RLock()     # held from choosing a device's word to the launch, and while it is read and cleared


def _error_word(device: int) -> torch.Tensor:
    """The device's own error word, for calls that bring none."""
    word = _error_words.get(device)
    if word is None:
        with torch.cuda.device(device):
            capturing = torch.cuda.is_current_stream_capturing()
        if capturing:
            raise CsfError("no memory for the device's error word within a capture: call errors() before it, or give error_word")
        word = _error_words[device] = torch.zeros(1, dtype=torch.int32, device=torch.device("cuda", device))
        torch.cuda.synchronize(device)  # once: any stream may set it from here on
    return word


def errors(device: int | None = None) -> int:
    """CSF_DEV_ERR_* bits of the expert_matmul calls on a device that were given
    no error_word, and clears them.  Synchronises; calls of other threads wait
    meanwhile.  (Not so replays of captured calls: what one sets between the
    reading and the clearing is lost.)  Before a capture of such calls it makes
    the word that they report to."""
    device = torch.cuda.current_device() if device is None else device
    with _error_lock:
        word = _error_word(device)
        torch.cuda.synchronize(device)
        bits = int(word.item())
        if bits:
            word.zero_()
            torch.cuda.synchronize(device)      # before any stream's next call
    return bits


def _on(stream, call, *args):
    """The call with `stream` current, so that what it allocates is the
    stream's own; what it reads or writes of other streams' is kept until it
    has run, also where the caller lets go of it before."""
    device = (args[0].codes if isinstance(args[0], Quantized) else args[0]).get_device()
    if stream.device.index != device:
        raise CsfError(f"the stream is on cuda:{stream.device.index}, the tensors " +
                       (f"on cuda:{device}" if device >= 0 else "are not CUDA tensors"))
    with torch.cuda.stream(stream):
        result = call(*args)
    for a in args:
        for t in (a.codes, a.scales, a.tensor_scale) if isinstance(a, Quantized) else (a,):
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    return result


def _up(n: int, m: int) -> int:
    return (n + m - 1) // m * m


def _code_bytes(kind: int, cols: int) -> int:
    return _up(cols, 32) // (2 if kind == NVFP4 else 1)


def _scale_bytes(kind: int, cols: int) -> int:
    return _up(_up(cols, 32) // (16 if kind == NVFP4 else 32), 16)


@dataclass
class Quantized:
    """Quantised rows (csf_rows): uint8 codes [rows, code bytes] and scales
    [rows, scale bytes], rows 16-byte aligned.  `tensor_scale` is the NVFP4
    tensor scale they were made with (float32 [1]) or None; a product takes it
    through its alpha.  As an output they keep theirs where a call gives none."""
    kind: int
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int
    tensor_scale: torch.Tensor | None = None

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    def fields(self) -> tuple:
        """The fields of csf_rows."""
        c, s, t = self.codes, self.scales, self.tensor_scale
        return (self.kind, self.cols, c.shape[0], c.data_ptr(), c.stride(0), s.data_ptr(), s.stride(0),
                0 if t is None else t.data_ptr())


def empty_quantized(kind: int, rows: int, cols: int, device=None, tensor_scale: torch.Tensor | None = None) -> Quantized:
    """Quantised rows with undefined contents."""
    if kind not in (NVFP4, MXFP8):
        raise CsfError("quantised rows are NVFP4 or MXFP8")
    device = device if device is not None else "cuda"
    if cols < 1:
        raise CsfError("quantised rows have at least one column")
    return Quantized(kind, torch.empty((rows, _code_bytes(kind, cols)), dtype=torch.uint8, device=device),
                     torch.empty((rows, _scale_bytes(kind, cols)), dtype=torch.uint8, device=device), cols, tensor_scale)


def _where(device: int) -> str:
    return f" on cuda:{device}" if device >= 0 else ""


def _check_quantized(q: Quantized, what: str, device: int):
    c, s = q.codes, q.scales
    if q.kind not in (NVFP4, MXFP8):
        raise CsfError(f"{what}: quantised rows are NVFP4 or MXFP8")
    if c.dtype != torch.uint8 or s.dtype != torch.uint8 or device < 0 or c.get_device() != device or s.get_device() != device:
        raise CsfError(f"{what}: codes and scales must be uint8 CUDA tensors{_where(device)}")
    if c.dim() != 2 or s.dim() != 2 or c.shape[0] != s.shape[0] or c.stride(1) != 1 or s.stride(1) != 1:
        raise CsfError(f"{what}: codes and scales must be [rows, bytes] with contiguous rows")
    if q.cols < 1 or c.shape[1] < _code_bytes(q.kind, q.cols) or s.shape[1] < _scale_bytes(q.kind, q.cols):
        raise CsfError(f"{what}: codes or scales are too narrow for {q.cols} columns")


def _tensor_scale(out: Quantized, given: torch.Tensor | None, what: str, device: int) -> torch.Tensor | None:
    """The tensor scale of a quantised output: the argument, or the one it has."""
    scale = out.tensor_scale if given is None else given
    if scale is not None:
        if out.kind != NVFP4:
            raise CsfError(f"{what}: only NVFP4 rows have a tensor scale")
        _vector(scale, f"{what}: the tensor scale", 1, torch.float32, device)
    return scale


def _matrix(t, name: str, rows: int, cols: int, device: int, dtype=None):
    if device < 0 or t.get_device() != device or t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise CsfError(f"{name} must be a CUDA tensor of {dtype or 'bfloat16, float16 or float32'}{_where(device)}")
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols or (t.stride(1) != 1 and cols > 1):
        raise CsfError(f"{name} must be [{rows}, {cols}] with contiguous rows")
    return t.data_ptr(), (t.stride(0) if rows > 1 else max(t.stride(0), cols))


def _vector(t, name: str, n: int, dtype, device: int):
    if t is None:
        return 0
    if t.get_device() != device or t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise CsfError(f"{name} must be a contiguous CUDA tensor of {n} {dtype}{_where(device)}")
    return t.data_ptr()


def rms_norm(x: torch.Tensor, weight: torch.Tensor, kind: int, residual: torch.Tensor | None = None, eps: float = 1e-6,
             tensor_scale: torch.Tensor | None = None, out: Quantized | None = None,
             sum_out: torch.Tensor | None = None, stream=None):
    """Residual addition, root-mean-square norm and quantisation of the rows
    of `x` [rows, cols] in one launch (csf_rms_norm).  Returns the quantised
    rows and the sum x + residual (in `sum_out`, which may be `residual`
    itself, or a new tensor; None without a residual and a `sum_out`)."""
    if stream is not None:
        return _on(stream, rms_norm, x, weight, kind, residual, eps, tensor_scale, out, sum_out)
    if x.dim() != 2 or x.dtype not in _DTYPES:
        raise CsfError("rms_norm: x must be [rows, cols] of bfloat16, float16 or float32")
    rows, cols = x.shape
    device = x.get_device()
    xp, xs = _matrix(x, "rms_norm: x", rows, cols, device)
    rp, rs = (0, 0) if residual is None else _matrix(residual, "rms_norm: residual", rows, cols, device, x.dtype)
    if sum_out is None and residual is not None:
        sum_out = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
    sp, ss = (0, 0) if sum_out is None else _matrix(sum_out, "rms_norm: sum_out", rows, cols, device, x.dtype)
    wp = _vector(weight, "rms_norm: weight", cols, x.dtype, device)
    if out is None:
        out = empty_quantized(kind, rows, cols, x.device, tensor_scale)
    else:
        _check_quantized(out, "rms_norm: out", device)
        if out.kind != kind or out.rows != rows or out.cols != cols:
            raise CsfError("rms_norm: out does not match x and kind")
    out.tensor_scale = _tensor_scale(out, tensor_scale, "rms_norm", device)
    a = _RMS_NORM.pack(xp, xs, rp, rs, sp, ss, wp, _DTYPES[x.dtype], eps, *out.fields())
    _launch(lib.csf_rms_norm, a, device, "csf_rms_norm")
    return out, sum_out


@dataclass
class Routing:
    """The router's choice (csf_route).  Slots are numbered by expert, then by
    token; rows[slot] is a slot's token, slots[token, j] a choice's slot."""
    ids: torch.Tensor            # int32 [tokens, k], -1 where no expert was left
    weights: torch.Tensor        # float32 [tokens, k]
    expert_start: torch.Tensor   # int32 [experts + 1], as csf.decode takes it
    rows: torch.Tensor           # int32 [tokens * k]
    slots: torch.Tensor          # int32 [tokens, k]


def route(logits: torch.Tensor, k: int, renormalize: bool = True, stream=None) -> Routing:
    """Choose each token's k experts from `logits` [tokens, experts] and group
    the choices by expert (csf_route)."""
    if stream is not None:
        return _on(stream, route, logits, k, renormalize)
    if logits.dim() != 2:
        raise CsfError("route: logits must be [tokens, experts]")
    T, E = logits.shape
    if not 1 <= k <= min(32, E):
        raise CsfError(f"route: k must be 1 to {min(32, E)}")
    device = logits.get_device()
    lp, ls = _matrix(logits, "route: logits", T, E, device)
    dev = logits.device
    i32 = dict(dtype=torch.int32, device=dev)
    n = T * k
    r = Routing(torch.empty((T, k), **i32), torch.empty((T, k), dtype=torch.float32, device=dev),
                torch.empty(E + 1, **i32), torch.empty(n, **i32), torch.empty((T, k), **i32))
    need = lib.csf_route_scratch_bytes(T, E)
    scratch = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    a = _ROUTE.pack(lp, ls, _DTYPES[logits.dtype], T, E, k, renormalize, r.ids.data_ptr(), r.weights.data_ptr(),
                    r.expert_start.data_ptr(), r.rows.data_ptr(), r.slots.data_ptr(),
                    scratch.data_ptr() if need else 0, need)
    _launch(lib.csf_route, a, device, "csf_route")
    return r


def expert_matmul(x: Quantized, w: torch.Tensor, w_scales: torch.Tensor, expert_start: torch.Tensor | None = None,
                  rows: torch.Tensor | None = None, alpha: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                  activation: str | None = None, gated: bool = False, row_scale: torch.Tensor | None = None,
                  residual: torch.Tensor | None = None, out=torch.bfloat16, out_tensor_scale: torch.Tensor | None = None,
                  error_word: torch.Tensor | None = None, stream=None):
    """Block-scaled product of quantised rows with the experts' FP4 weights
    (csf_expert_matmul).

    `w` is uint8 [E, N, K/2] (NVFP4 weights for NVFP4 rows, MXFP4 for MXFP8),
    `w_scales` their scales as csf.decode(..., layout=LAYOUT_BLOCKED) writes
    them.  Slots [expert_start[e], expert_start[e+1]) belong to expert e; slot s
    reads row rows[s] of x (row s without `rows`).  Without `expert_start` the
    one expert owns every slot.  p = alpha[e] * (x . w) + bias[e]; y = act(p),
    or act(p[:N/2]) * p[N/2:] when `gated`; out = y * row_scale[s] + residual.
    `out` is a dtype, a tensor, NVFP4 or MXFP8 (a new Quantized), or a
    Quantized.  Activations: None, "relu", "silu", "gelu" (tanh form).
    Data errors reach `error_word` (int32 [1]) or, without one, errors()."""
    if stream is not None:
        return _on(stream, expert_matmul, x, w, w_scales, expert_start, rows, alpha, bias, activation, gated, row_scale,
                   residual, out, out_tensor_scale, error_word)
    device = x.codes.get_device()
    _check_quantized(x, "expert_matmul: x", device)
    if w.dtype != torch.uint8 or w.get_device() != device or w.dim() != 3 or not w.is_contiguous() or w.shape[2] * 2 != x.cols:
        raise CsfError(f"expert_matmul: w must be a contiguous uint8 CUDA tensor [E, N, {x.cols // 2}]{_where(device)}")
    E, N = w.shape[0], w.shape[1]
    C = x.cols // (16 if x.kind == NVFP4 else 32)
    if w_scales.dtype != torch.uint8 or w_scales.get_device() != device or not w_scales.is_contiguous() or \
            w_scales.numel() < E * _up(N, 128) * _up(C, 4):
        raise CsfError(f"expert_matmul: w_scales must be a contiguous uint8 CUDA tensor in the blocked layout{_where(device)}")
    if activation not in _ACTS:
        raise CsfError(f"expert_matmul: unknown activation {activation!r}")
    if rows is not None and (rows.get_device() != device or rows.dtype != torch.int32 or not rows.is_contiguous() or rows.dim() != 1):
        raise CsfError(f"expert_matmul: rows must be a contiguous int32 CUDA vector{_where(device)}")
    es, es64 = _es(expert_start)
    if expert_start is not None:
        if expert_start.get_device() != device:
            raise CsfError(f"expert_start must be a CUDA tensor{_where(device)}")
        if expert_start.numel() != E + 1:
            raise CsfError("expert_start must have E+1 entries")
    S = x.rows if rows is None else rows.shape[0]
    F = N // 2 if gated else N
    bias_dtype = 0
    if bias is not None:
        if bias.dtype not in _DTYPES:
            raise CsfError("expert_matmul: bias must be bfloat16, float16 or float32")
        bias_dtype = _DTYPES[bias.dtype]
    rp, rs = (0, 0) if residual is None else _matrix(residual, "expert_matmul: residual", S, F, device)
    if isinstance(out, torch.dtype):
        if out not in _DTYPES:
            raise CsfError("expert_matmul: out must be bfloat16, float16 or float32")
        out = torch.empty((S, F), dtype=out, device=x.codes.device)
    elif isinstance(out, int):
        out = empty_quantized(out, S, F, x.codes.device, out_tensor_scale)
    if isinstance(out, Quantized):
        _check_quantized(out, "expert_matmul: out", device)
        if out.rows != S or out.cols != F:
            raise CsfError("expert_matmul: out does not match the product")
        out.tensor_scale = _tensor_scale(out, out_tensor_scale, "expert_matmul", device)
        op, os_, odt, orows = 0, 0, 0, out.fields()
    else:
        op, os_ = _matrix(out, "expert_matmul: out", S, F, device)
        odt, orows = _DTYPES[out.dtype], _NO_ROWS
    own_word = error_word is None
    if own_word:
        _error_lock.acquire()
    try:
        a = _EXPERT_MATMUL.pack(
            *x.fields(), 0 if rows is None else rows.data_ptr(), S, E, N, w.data_ptr(), w_scales.data_ptr(), es or 0, es64,
            _vector(alpha, "expert_matmul: alpha", E, torch.float32, device),
            0 if bias is None else _vector(bias, "expert_matmul: bias", E * N, bias.dtype, device), bias_dtype, _ACTS[activation],
            gated, _vector(row_scale, "expert_matmul: row_scale", S, torch.float32, device), rp, rs,
            0 if residual is None else _DTYPES[residual.dtype], odt, op, os_, *orows,
            _error_word(device).data_ptr() if own_word else _vector(error_word, "expert_matmul: error_word", 1, torch.int32, device))
        _launch(lib.csf_expert_matmul, a, device, "csf_expert_matmul")
    finally:
        if own_word:
            _error_lock.release()
    return out
