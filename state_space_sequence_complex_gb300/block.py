"""Binding of the operators around the scan (include/ssdc_block.h): gated scan,
residual norm, 8-bit product. Argument checks and marshalling only; every step
runs in libssdc.so's kernels and there is no fallback.

The classes hold the outputs and workspaces of one problem size, so that a call
allocates nothing and the next call overwrites the last one's outputs: threads that
call at the same time need a plan each.
``gated_scan``, ``residual_norm`` and ``fp8_linear`` are differentiable
(``torch.autograd``, first derivatives) and allocate their outputs. They do not
read the status of a wait between CTAs that gave up, which a plan's ``status()``
does: that waits for the GPU.

A plan's tensors belong to the device it was made for; a call runs there, on that
device's current stream or on ``stream``, whichever device is current. Tensors made on another stream have to be ordered with
it by the caller, as for any kernel.

    from state_space_sequence_complex_gb300 import block
    norm = block.ResidualNorm(M, D, "bf16", out="fp8")
    r, q, scale = norm(x, residual, w)                  # r = x + residual; q, scale: the product's operand
    w_q, w_s = block.Fp8Quantize(N, D, "bf16", scales="blocks")(weight)[:2]
    y = block.Fp8Product(M, N, D)(q, scale, w_q, w_s)   # y = norm(r) weight^T
    scan = block.GatedScan(B, T, C, "bf16")
    h, h_last = scan(x, f, i, h0=state)                 # slices of y work: strides are taken from the tensors
"""
from __future__ import annotations

import ctypes
import struct

import torch
from torch.autograd.function import once_differentiable

from . import ssdc

TYPE_F32, TYPE_BF16, TYPE_E4M3 = 0, 1, 2
SCALE_ROWS, SCALE_BLOCKS = 0, 1
GROUP = 128
STATE_TOKENS = 64

_TYPES = {"fp32": TYPE_F32, "bf16": TYPE_BF16, "fp8": TYPE_E4M3}
_DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}

EXPORTS = ("ssd_gated_scan_states_bytes", "ssd_gated_scan_fwd", "ssd_gated_scan_workspace_bytes", "ssd_gated_scan_fwd_ws", "ssd_gated_scan_step", "ssd_gated_scan_bwd",
           "ssd_residual_norm_fwd", "ssd_residual_norm_bwd_workspace_bytes", "ssd_residual_norm_bwd",
           "ssd_fp8_quantize", "ssd_fp8_matmul_workspace_bytes", "ssd_fp8_matmul", "ssd_block_call")


class ssd_seq(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64)]


class ssd_rows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("ld", ctypes.c_int64)]


class ssd_gated_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("D", ctypes.c_int64), ("type", ctypes.c_int32)]


_lib = None


def load() -> ctypes.CDLL:
    """The library with this header's signatures (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    lib = ssdc.load()
    vp, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    q, r, d = ssd_seq, ssd_rows, ssd_gated_dims
    for name, res, args in (
            ("ssd_gated_scan_states_bytes", sz, [d]),
            ("ssd_gated_scan_fwd", i32, [q, q, q, vp, vp, d, q, vp, vp, vp, vp]),
            ("ssd_gated_scan_workspace_bytes", sz, [d]),
            ("ssd_gated_scan_fwd_ws", i32, [q, q, q, vp, vp, d, q, vp, vp, vp, vp, sz, vp]),
            ("ssd_gated_scan_step", i32, [q, q, q, vp, i64, i64, i32, q, vp, vp]),
            ("ssd_gated_scan_bwd", i32, [q, q, q, vp, vp, q, vp, d, q, q, q, vp, vp, vp]),
            ("ssd_residual_norm_fwd", i32, [r, r, vp, f32, i64, i64, i32, r, i32, r, vp, vp, vp]),
            ("ssd_residual_norm_bwd_workspace_bytes", sz, [i64, i64]),
            ("ssd_residual_norm_bwd", i32, [r, r, r, vp, vp, i64, i64, i32, r, vp, vp, sz, vp]),
            ("ssd_fp8_quantize", i32, [r, i64, i64, i32, i32, r, vp, r, vp, vp]),
            ("ssd_fp8_matmul_workspace_bytes", sz, [i64, i64, i64]),
            ("ssd_fp8_matmul", i32, [r, vp, r, vp, i32, i64, i64, i64, i32, r, vp, sz, vp]),
            ("ssd_block_call", i32, [i32, vp, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _lib = lib
    return lib


# ---- argument checks


def _type(dtype):
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be 'bf16' or 'fp32', not {dtype!r}")
    return _TYPES[dtype]


def _sizes(**sizes):
    for k, v in sizes.items():
        if v <= 0:
            raise ValueError(f"{k} must be positive, not {v}")


# What a call's tensors have to be is kept as (dtype, shape, device index) and compared as a whole;
# for one token or a few these checks are as long as the launch.


def _refuse(name, t, like):
    dtype, shape, index = like
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    want = "the CPU" if index < 0 else f"cuda:{index}"
    raise ValueError(f"{name} must be on {want}, not {t.device}")


def _dense(name, t, like):
    """The address of a dense tensor, or 0 for None."""
    if t is None:
        return 0
    if (t.dtype, t.shape, t.get_device()) != like:
        _refuse(name, t, like)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(name, t, like):
    """The address and row stride of a matrix with contiguous rows; zeros for None."""
    if t is None:
        return 0, 0
    if (t.dtype, t.shape, t.get_device()) != like:
        _refuse(name, t, like)
    ld, one = t.stride()
    if one != 1 and like[1][1] != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), ld


def _seq(name, t, like):
    """The address and the batch and token strides of a (B, T, D) tensor with contiguous channels; zeros for None."""
    if t is None:
        return 0, 0, 0
    if (t.dtype, t.shape, t.get_device()) != like:
        _refuse(name, t, like)
    sb, st, one = t.stride()
    if one != 1 and like[1][2] != 1:
        raise ValueError(f"{name} must have contiguous channels")
    return t.data_ptr(), sb, st


class _Call:
    """One of the library's calls with its arguments as a block of words (``ssd_block_call``), one of its own for
    each call: the interpreter's lock is given up around the library."""

    __slots__ = ("name", "number", "fn", "pack", "index", "several")

    def __init__(self, name, number, words, index):
        self.name, self.number, self.index = name, number, index
        self.several = index >= 0 and torch.cuda.device_count() > 1
        self.fn = load().ssd_block_call
        self.pack = struct.Struct(f"{words}q").pack

    def __call__(self, stream, *words):
        # the library launches on the current device: make it the plan's, whose addresses and stream these are
        if self.several and torch._C._cuda_getDevice() != self.index:
            with torch.cuda.device(self.index):
                return self(stream, *words)
        if stream is not None:
            stream = stream.cuda_stream
        elif self.index >= 0:
            stream = torch._C._cuda_getCurrentRawStream(self.index)
        rc = self.fn(self.number, self.pack(*words), stream)
        if rc:
            _raise(rc, self.name)


def _index(device):
    return -1 if device.type == "cpu" else device.index


def _device(device):
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def _status(plan, stream):
    if plan.device.type == "cpu":
        return ssdc.ssd_complex_status(plan.workspace, stream)
    with torch.cuda.device(plan.device):
        return ssdc.ssd_complex_status(plan.workspace, stream)


def _raise(rc, what):
    raise ssdc.SSDCError(rc, what)


def fp8_pitch(n: int) -> int:
    """Bytes of a row of n 8-bit values: the next multiple of 16."""
    return -(-n // 16) * 16


def fp8_groups(n: int) -> int:
    return -(-n // GROUP)


def fp8_empty(rows: int, cols: int, device="cuda"):
    """An uninitialised (rows, cols) e4m3 operand whose rows start 16-byte aligned."""
    store = torch.empty(rows, fp8_pitch(cols), dtype=torch.uint8, device=device)
    return store.view(torch.float8_e4m3fn)[:, :cols]


# ---- gated scan


class GatedScan:
    """h_t = c_t h_{t-1} + v_t for every channel (``ssd_gated_scan_fwd_ws``), with
    a_t = sigmoid(f_t), c_t = a_t (0 where ``reset`` marks the first token of a
    document), v_t = sigmoid(i_t) x_t, or (1 - a_t) x_t with ``input_gate`` False.
    ``__call__`` takes (B, T, D) tensors with contiguous channels, an optional
    initial state (B, D) float32 (this object's own ``h_last`` continues the last
    call in place) and optional marks (B, T) uint8, and returns ``(h, h_last)``.
    With ``keep_states`` a call also fills ``states``, which the backward pass
    takes."""

    def __init__(self, B, T, D, dtype="bf16", input_gate=True, keep_states=False, device="cuda"):
        _sizes(B=B, T=T, D=D)
        self.device = _device(device)
        self.dims = ssd_gated_dims(int(B), int(T), int(D), _type(dtype))
        self.dtype, self.input_gate = _DTYPES[dtype], bool(input_gate)
        if load().ssd_gated_scan_states_bytes(self.dims) == 0:
            _raise(ssdc.SSDC_ERR_UNSUPPORTED, "GatedScan")
        self.shape, self.state_shape, self.mark_shape = (B, T, D), (B, D), (B, T)
        self.h = torch.empty(self.shape, dtype=self.dtype, device=self.device)
        self.h_last = torch.empty(self.state_shape, dtype=torch.float32, device=self.device)
        self.states = None
        if keep_states:
            self.states = torch.empty((B, -(-T // STATE_TOKENS), D), dtype=torch.float32, device=self.device)
        self.workspace = torch.zeros(64, dtype=torch.int32, device=self.device)
        nbytes = load().ssd_gated_scan_workspace_bytes(self.dims)
        self.joints = torch.empty(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None
        self._like = self.dtype, torch.Size(self.shape), _index(self.device)
        self._state = torch.float32, torch.Size(self.state_shape), self._like[2]
        self._marks = torch.uint8, torch.Size(self.mark_shape), self._like[2]
        self._dims = B, T, D, self.dims.type
        self._h = _seq("h", self.h, self._like)
        self._kept = (self.h_last.data_ptr(), 0 if self.states is None else self.states.data_ptr(), self.workspace.data_ptr(),
                      0 if self.joints is None else self.joints.data_ptr(), nbytes)
        self._call = _Call("ssd_gated_scan_fwd_ws", 7, 23, self._like[2])

    def __call__(self, x, f, i=None, h0=None, reset=None, out=None, stream=None):
        """``out``: where h goes instead of this object's ``h``, a (B, T, D) tensor
        with contiguous channels that shares no element with an input."""
        if (i is not None) != self.input_gate:
            raise ValueError("i must be given exactly when the plan has an input gate")
        like = self._like
        h, h_out = (self.h, self._h) if out is None else (out, _seq("out", out, like))
        self._call(stream, *_seq("x", x, like), *_seq("f", f, like), *_seq("i", i, like),
                   _dense("h0", h0, self._state), _dense("reset", reset, self._marks), *self._dims, *h_out, *self._kept)
        return h, self.h_last

    def status(self, stream=None) -> int:
        return _status(self, stream)


class GatedScanBackward:
    """The gradients of ``GatedScan`` (``ssd_gated_scan_bwd``). ``__call__`` takes
    the forward pass's inputs, the ``states`` it kept, ``dh`` and optionally
    ``dh_last``, and returns a dict: ``dx``, ``df``, ``di`` (with an input gate) and
    ``dh0``."""

    def __init__(self, B, T, D, dtype="bf16", input_gate=True, device="cuda"):
        _sizes(B=B, T=T, D=D)
        self.device = _device(device)
        self.dims = ssd_gated_dims(int(B), int(T), int(D), _type(dtype))
        self.dtype, self.input_gate = _DTYPES[dtype], bool(input_gate)
        if load().ssd_gated_scan_states_bytes(self.dims) == 0:
            _raise(ssdc.SSDC_ERR_UNSUPPORTED, "GatedScanBackward")
        self.shape, self.state_shape, self.mark_shape = (B, T, D), (B, D), (B, T)
        self.states_shape = (B, -(-T // STATE_TOKENS), D)
        names = ("dx", "df", "di") if input_gate else ("dx", "df")
        self.grads = {k: torch.empty(self.shape, dtype=self.dtype, device=self.device) for k in names}
        self.workspace = torch.zeros(64, dtype=torch.int32, device=self.device)
        self.grads["dh0"] = torch.empty(self.state_shape, dtype=torch.float32, device=self.device)
        self._like = self.dtype, torch.Size(self.shape), _index(self.device)
        self._state = torch.float32, torch.Size(self.state_shape), self._like[2]
        self._states = torch.float32, torch.Size(self.states_shape), self._like[2]
        self._marks = torch.uint8, torch.Size(self.mark_shape), self._like[2]
        self._dims = B, T, D, self.dims.type
        g = self.grads
        self._out = (*_seq("dx", g["dx"], self._like), *_seq("df", g["df"], self._like),
                     *_seq("di", g.get("di"), self._like), g["dh0"].data_ptr(), self.workspace.data_ptr())
        self._call = _Call("ssd_gated_scan_bwd", 2, 30, self._like[2])

    def __call__(self, x, f, i, states, dh, dh_last=None, reset=None, stream=None):
        if (i is not None) != self.input_gate:
            raise ValueError("i must be given exactly when the plan has an input gate")
        like = self._like
        self._call(stream, *_seq("x", x, like), *_seq("f", f, like), *_seq("i", i, like),
                   _dense("states", states, self._states), _dense("reset", reset, self._marks), *_seq("dh", dh, like),
                   _dense("dh_last", dh_last, self._state), *self._dims, *self._out)
        return dict(self.grads)

    def status(self, stream=None) -> int:
        return _status(self, stream)


class GatedScanStep:
    """One token of B sequences (``ssd_gated_scan_step``). ``__call__`` takes (B, D)
    tensors with contiguous channels and the state (B, D) float32, and returns
    ``(h, state)``. The new state goes to this object's ``state``, or to
    ``state_out``; passing the state itself there updates it in place."""

    def __init__(self, B, D, dtype="bf16", input_gate=True, device="cuda"):
        _sizes(B=B, D=D)
        self.device = _device(device)
        self.type, self.dtype, self.input_gate = _type(dtype), _DTYPES[dtype], bool(input_gate)
        if load().ssd_gated_scan_states_bytes(ssd_gated_dims(int(B), 1, int(D), self.type)) == 0:
            _raise(ssdc.SSDC_ERR_UNSUPPORTED, "GatedScanStep")
        self.shape = (B, D)
        self.h = torch.empty(self.shape, dtype=self.dtype, device=self.device)
        self.state = torch.empty(self.shape, dtype=torch.float32, device=self.device)
        self._like = self.dtype, torch.Size(self.shape), _index(self.device)
        self._state = torch.float32, torch.Size(self.shape), self._like[2]
        self._rest, self._own = (B, D, self.type, self.h.data_ptr(), D, 0), self.state.data_ptr()
        self._call = _Call("ssd_gated_scan_step", 1, 17, self._like[2])

    def __call__(self, x, f, i, state, state_out=None, stream=None):
        if (i is not None) != self.input_gate:
            raise ValueError("i must be given exactly when the plan has an input gate")
        like = self._like
        to = self._own if state_out is None else _dense("state_out", state_out, self._state)
        self._call(stream, *_rows("x", x, like), 0, *_rows("f", f, like), 0, *_rows("i", i, like), 0,
                   _dense("state", state, self._state), *self._rest, to)
        return self.h, self.state if state_out is None else state_out


# ---- residual norm


class ResidualNorm:
    """r = x + residual, y = w r / sqrt(mean(r^2) + eps) over M rows of D features
    (``ssd_residual_norm_fwd``). ``out`` is y's type: ``"bf16"``, ``"fp32"`` or
    ``"fp8"``. ``__call__`` takes (M, D) tensors with contiguous rows (``residual``
    may be None) and the weights (D) float32 (None: ones). It returns ``(r, y)``,
    or for ``"fp8"`` ``(r, q, scale)`` with scale (ceil(D / 128), M): the operand
    that ``Fp8Product`` takes. ``rstd`` holds 1 / sqrt(mean(r^2) + eps) for the
    backward pass."""

    def __init__(self, M, D, dtype="bf16", out="fp8", eps=1e-5, device="cuda"):
        _sizes(M=M, D=D)
        self.device = _device(device)
        self.type, self.dtype, self.shape, self.eps = _type(dtype), _DTYPES[dtype], (M, D), float(eps)
        if out not in _TYPES:
            raise ValueError(f"out must be 'bf16', 'fp32' or 'fp8', not {out!r}")
        if D > 32768:
            _raise(ssdc.SSDC_ERR_UNSUPPORTED, "ResidualNorm")
        self.out_type = _TYPES[out]
        self.r = torch.empty(self.shape, dtype=self.dtype, device=self.device)
        self.rstd = torch.empty(M, dtype=torch.float32, device=self.device)
        self.scale = None
        if out == "fp8":
            self.y = fp8_empty(M, D, self.device)
            self.scale = torch.empty((fp8_groups(D), M), dtype=torch.float32, device=self.device)
        else:
            self.y = torch.empty(self.shape, dtype=_DTYPES[out], device=self.device)
        self._like = self.dtype, torch.Size(self.shape), _index(self.device)
        self._weights = torch.float32, torch.Size((D,)), self._like[2]
        self._rest = (struct.unpack("I", struct.pack("f", self.eps))[0], M, D, self.type, self.r.data_ptr(), D,
                      self.out_type, self.y.data_ptr(), self.y.stride(0),
                      0 if self.scale is None else self.scale.data_ptr(), self.rstd.data_ptr())
        self._result = (self.r, self.y) if self.scale is None else (self.r, self.y, self.scale)
        self._call = _Call("ssd_residual_norm_fwd", 3, 16, self._like[2])

    def __call__(self, x, residual=None, w=None, stream=None):
        like = self._like
        self._call(stream, *_rows("x", x, like), *_rows("residual", residual, like), _dense("w", w, self._weights),
                   *self._rest)
        return self._result


class ResidualNormBackward:
    """The gradients of ``ResidualNorm`` (``ssd_residual_norm_bwd``). ``__call__``
    takes dy, the forward pass's ``r``, ``w`` and ``rstd``, and the gradient ``dr``
    of r itself (None: zero), and returns ``(dx, dw)``; dx is the gradient of x and
    of the residual."""

    def __init__(self, M, D, dtype="bf16", device="cuda"):
        _sizes(M=M, D=D)
        self.device = _device(device)
        self.type, self.dtype, self.shape = _type(dtype), _DTYPES[dtype], (M, D)
        nbytes = load().ssd_residual_norm_bwd_workspace_bytes(M, D)
        if nbytes == 0:
            _raise(ssdc.SSDC_ERR_UNSUPPORTED, "ResidualNormBackward")
        self.dx = torch.empty(self.shape, dtype=self.dtype, device=self.device)
        self.dw = torch.empty(D, dtype=torch.float32, device=self.device)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self._like = self.dtype, torch.Size(self.shape), _index(self.device)
        self._weights, self._rstd = (torch.float32, torch.Size((D,)), self._like[2]), (torch.float32, torch.Size((M,)), self._like[2])
        self._rest = (M, D, self.type, self.dx.data_ptr(), D, self.dw.data_ptr(), self.workspace.data_ptr(), nbytes)
        self._call = _Call("ssd_residual_norm_bwd", 4, 16, self._like[2])

    def __call__(self, dy, r, w, rstd, dr=None, stream=None):
        like = self._like
        self._call(stream, *_rows("dy", dy, like), *_rows("dr", dr, like), *_rows("r", r, like),
                   _dense("w", w, self._weights), _dense("rstd", rstd, self._rstd), *self._rest)
        return self.dx, self.dw


# ---- 8-bit product


class Fp8Quantize:
    """The 8-bit operands of an (M, K) tensor (``ssd_fp8_quantize``). ``scales`` is
    ``"rows"`` (one for each row and 128 columns: scale (ceil(K / 128), M)) or
    ``"blocks"`` (one for each 128 x 128: (ceil(M / 128), ceil(K / 128))).
    ``__call__`` returns ``(q, scale)``, and with ``transposed`` ``(q, scale, qt,
    scale_t)`` with the operand of the transposed tensor; ``direct`` False leaves
    out q."""

    def __init__(self, M, K, dtype="bf16", scales="rows", direct=True, transposed=False, device="cuda"):
        _sizes(M=M, K=K)
        if scales not in ("rows", "blocks"):
            raise ValueError(f"scales must be 'rows' or 'blocks', not {scales!r}")
        if not direct and not transposed:
            raise ValueError("direct, transposed or both")
        self.device = _device(device)
        self.type, self.dtype, self.shape = _type(dtype), _DTYPES[dtype], (M, K)
        self.scales = SCALE_BLOCKS if scales == "blocks" else SCALE_ROWS
        MB, KB = fp8_groups(M), fp8_groups(K)
        f32 = dict(dtype=torch.float32, device=self.device)
        self.q = self.scale = self.qt = self.scale_t = None
        if direct:
            self.q = fp8_empty(M, K, self.device)
            self.scale = torch.empty((MB, KB) if self.scales else (KB, M), **f32)
        if transposed:
            self.qt = fp8_empty(K, M, self.device)
            self.scale_t = torch.empty((KB, MB) if self.scales else (MB, K), **f32)
        self._like = self.dtype, torch.Size(self.shape), _index(self.device)
        rows = lambda t: (0, 0) if t is None else (t.data_ptr(), t.stride(0))
        ptr = lambda t: 0 if t is None else t.data_ptr()
        self._rest = (M, K, self.type, self.scales, *rows(self.q), ptr(self.scale), *rows(self.qt), ptr(self.scale_t))
        self._result = tuple(t for t in (self.q, self.scale, self.qt, self.scale_t) if t is not None)
        self._call = _Call("ssd_fp8_quantize", 5, 12, self._like[2])

    def __call__(self, x, stream=None):
        self._call(stream, *_rows("x", x, self._like), *self._rest)
        return self._result


class Fp8Product:
    """C = A B^T from 8-bit operands (``ssd_fp8_matmul``): a (M, K) with row scales
    (ceil(K / 128), M), b (N, K) with block scales (ceil(N / 128), ceil(K / 128)), or
    with row scales (ceil(K / 128), N) where ``b_scales`` is ``"rows"``. Operand rows
    start 16-byte aligned (``fp8_empty``, ``Fp8Quantize``, ``ResidualNorm``). Returns
    C (M, N) in ``out`` (``"bf16"`` or ``"fp32"``); its rows start 16-byte aligned too,
    so it is not contiguous where N is no multiple of 8 (bf16) or 4 (fp32)."""

    def __init__(self, M, N, K, out="bf16", b_scales="blocks", device="cuda"):
        _sizes(M=M, N=N, K=K)
        if b_scales not in ("rows", "blocks"):
            raise ValueError(f"b_scales must be 'rows' or 'blocks', not {b_scales!r}")
        self.device = _device(device)
        self.type, self.sizes = _type(out), (M, N, K)
        self.b_scales = SCALE_BLOCKS if b_scales == "blocks" else SCALE_ROWS
        nbytes = load().ssd_fp8_matmul_workspace_bytes(M, N, K)
        if nbytes == 0:
            _raise(ssdc.SSDC_ERR_UNSUPPORTED, "Fp8Product")
        KB = fp8_groups(K)
        self.a_shape, self.a_scale_shape, self.b_shape = (M, K), (KB, M), (N, K)
        self.b_scale_shape = (fp8_groups(N), KB) if self.b_scales else (KB, N)
        per = 8 if out == "bf16" else 4
        self.c = torch.empty((M, -(-N // per) * per), dtype=_DTYPES[out], device=self.device)[:, :N]
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        index, f8, f32 = _index(self.device), torch.float8_e4m3fn, torch.float32
        size = torch.Size
        self._a, self._b = (f8, size(self.a_shape), index), (f8, size(self.b_shape), index)
        self._a_scale, self._b_scale = (f32, size(self.a_scale_shape), index), (f32, size(self.b_scale_shape), index)
        self._rest = (self.b_scales, M, N, K, self.type, self.c.data_ptr(), self.c.stride(0), self.workspace.data_ptr(), nbytes)
        self._call = _Call("ssd_fp8_matmul", 6, 15, index)

    def __call__(self, a, a_scale, b, b_scale, stream=None):
        self._call(stream, *_rows("a", a, self._a), _dense("a_scale", a_scale, self._a_scale), *_rows("b", b, self._b),
                   _dense("b_scale", b_scale, self._b_scale), *self._rest)
        return self.c

    def status(self, stream=None) -> int:
        return _status(self, stream)


class Fp8Linear:
    """A linear layer's training step in 8-bit products: y = x w^T, dx = dy w,
    dw = dy^T x, for x (M, K) and w (N, K). ``forward`` quantises x and w (both ways
    round, in one pass over each) and keeps them for ``backward``, which quantises
    dy. The rounding to 8 bits is taken as the identity by the gradients."""

    def __init__(self, M, N, K, dtype="bf16", device="cuda"):
        self.x_q = Fp8Quantize(M, K, dtype, transposed=True, device=device)
        self.w_q = Fp8Quantize(N, K, dtype, scales="blocks", transposed=True, device=device)
        self.dy_q = Fp8Quantize(M, N, dtype, transposed=True, device=device)
        self.y = Fp8Product(M, N, K, dtype, device=device)
        self.dx = Fp8Product(M, K, N, dtype, device=device)
        self.dw = Fp8Product(N, K, M, dtype, b_scales="rows", device=device)

    def forward(self, x, w, stream=None):
        x_q, x_s, _, _ = self.x_q(x, stream)
        w_q, w_s, _, _ = self.w_q(w, stream)
        return self.y(x_q, x_s, w_q, w_s, stream)

    def backward(self, dy, stream=None):
        """``(dx, dw)`` for the x and w of the last ``forward``."""
        q, s, qt, st = self.dy_q(dy, stream)
        dx = self.dx(q, s, self.w_q.qt, self.w_q.scale_t, stream)
        return dx, self.dw(qt, st, self.x_q.qt, self.x_q.scale_t, stream)


# ---- differentiable forms (once: a gradient of a gradient is an error)


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, f, i, h0, reset):
        name = _dtype_name(x)
        plan = GatedScan(*x.shape, name, input_gate=i is not None, keep_states=True, device=x.device)
        h, last = plan(x, f, i, h0=h0, reset=reset)
        ctx.save_for_backward(x, f, i, plan.states, reset)
        ctx.with_h0 = h0 is not None
        return h, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dh_last):
        x, f, i, states, reset = ctx.saved_tensors
        dh = torch.zeros_like(x) if dh is None else _unit_last(dh)
        plan = GatedScanBackward(*x.shape, _dtype_name(x), input_gate=i is not None, device=x.device)
        g = plan(x, f, i, states, dh, dh_last=None if dh_last is None else dh_last.contiguous(), reset=reset)
        return g["dx"], g["df"], g.get("di"), g["dh0"] if ctx.with_h0 else None, None


def _dtype_name(t):
    for k, v in _DTYPES.items():
        if t.dtype is v:
            return k
    raise TypeError(f"tensors must be bfloat16 or float32, not {t.dtype}")


def _unit_last(t):
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def gated_scan(x, f, i=None, h0=None, reset=None):
    """Differentiable ``GatedScan``: returns new ``(h, h_last)``."""
    return _GatedScan.apply(x, f, i, h0, reset)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, w, eps):
        name = _dtype_name(x)
        plan = ResidualNorm(*x.shape, name, out=name, eps=eps, device=x.device)
        r, y = plan(x, residual, w)
        ctx.save_for_backward(r, w, plan.rstd)
        ctx.with_residual = residual is not None
        return r, y

    @staticmethod
    @once_differentiable
    def backward(ctx, dr, dy):
        r, w, rstd = ctx.saved_tensors
        dy = torch.zeros_like(r) if dy is None else _unit_last(dy)
        plan = ResidualNormBackward(*r.shape, _dtype_name(r), device=r.device)
        dx, dw = plan(dy, r, w, rstd, None if dr is None else _unit_last(dr))
        return dx, dx if ctx.with_residual else None, None if w is None else dw, None


def residual_norm(x, residual=None, w=None, eps=1e-5):
    """Differentiable ``ResidualNorm`` in the inputs' type: returns new ``(r, y)``."""
    return _ResidualNorm.apply(x, residual, w, eps)


class _Fp8Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        (M, K), N, name = x.shape, w.shape[0], _dtype_name(x)
        x_q, x_s, x_qt, x_st = Fp8Quantize(M, K, name, transposed=True, device=x.device)(x)
        w_q, w_s, w_qt, w_st = Fp8Quantize(N, K, name, scales="blocks", transposed=True, device=x.device)(w)
        ctx.save_for_backward(x_qt, x_st, w_qt, w_st)
        ctx.sizes = M, N, K, name
        return Fp8Product(M, N, K, name, device=x.device)(x_q, x_s, w_q, w_s)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x_qt, x_st, w_qt, w_st = ctx.saved_tensors
        M, N, K, name = ctx.sizes
        with_x, with_w = ctx.needs_input_grad
        grads = Fp8Quantize(M, N, name, direct=with_x, transposed=with_w, device=dy.device)(_unit_last(dy))
        dx = Fp8Product(M, K, N, name, device=dy.device)(*grads[:2], w_qt, w_st) if with_x else None
        dw = Fp8Product(N, K, M, name, b_scales="rows", device=dy.device)(*grads[-2:], x_qt, x_st) if with_w else None
        return dx, dw


def fp8_linear(x, w):
    """Differentiable x w^T in 8-bit products (``Fp8Linear``): returns a new (M, N) tensor
    (laid out as ``Fp8Product``'s)."""
    return _Fp8Linear.apply(x, w)
