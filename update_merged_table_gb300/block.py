"""The dense block between a lookup and its gradient, over ragged groups of rows.

``GroupedLinear`` (matrix products whose weights differ by row segment),
``GatedNorm`` (the norm after a block with its gate and residual scale, the
residual sum and the next block's norm) and ``Packed8`` (activations kept in
8 bits for the backward) marshal their arguments to the calls of the same
names in ``include/mt.h``.  Groups are runs of rows: a batch's feature segments, or the
tokens sorted by expert.

Outputs and workspaces are allocated on the stream the call runs on
(``stream``, by default the current one); a handle may be used from several
streams, each with its own workspace.
"""
from __future__ import annotations

import ctypes
import dataclasses
import threading

import torch

from . import MT_BF16, MT_EINVAL, MT_F32, MTError, _check, load_library

__all__ = ["Packed8", "pack8", "unpack8", "GroupedLinear", "GatedNorm", "NormParams", "NormForward", "NormGrads"]

MAX_GROUPS = 1024
MAX_BLOCK_DIM = 8192
PACK_BLOCK = 32
_KINDS = {"rms": 0, "layer": 1}
_GATES = {"none": 0, "linear": 1, "sigmoid": 2, "silu": 3}
_DTYPES = {"f32": MT_F32, "bf16": MT_BF16}


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("exps", ctypes.c_void_p)]


class _GatedNorm(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("dim", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("kind", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("eps", ctypes.c_float), ("offsets", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("post_weight", ctypes.c_void_p), ("post_bias", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("pre_weight", ctypes.c_void_p), ("pre_bias", ctypes.c_void_p)]


_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
_CODES = {torch.float32: MT_F32, torch.bfloat16: MT_BF16}
_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream


def _dtype_code(t):
    code = _CODES.get(t)
    if code is None:
        raise TypeError("rows must be float32 or bfloat16")
    return code


def _rows_2d(t, what: str, width: int, n: int, dtype, device) -> int:
    """The row stride of a row tensor: a CUDA tensor [n, width] of this dtype whose columns are contiguous and whose
    rows do not overlap."""
    try:
        shape, (ld, step) = t.shape, t.stride()
    except (AttributeError, ValueError):
        raise (ValueError if torch.is_tensor(t) else TypeError)(f"{what} must be a 2-D CUDA tensor") from None
    if shape[0] == n and shape[1] == width and step == 1 and ld >= width and t.dtype is dtype and t.device == device:
        return ld
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")
    if tuple(shape) != (n, width):
        raise ValueError(f"{what} must be [{n}, {width}], not {list(shape)}")
    if width > 1 and step != 1:
        raise ValueError(f"the columns of {what} must be contiguous")
    if n <= 1:
        return max(width, ld)
    if ld < width:
        raise ValueError(f"the rows of {what} overlap")
    return ld


def _count(t, what: str) -> int:
    """Rows of a tensor that may be a row tensor (the rest is checked by _rows_2d)."""
    if not torch.is_tensor(t):
        raise TypeError(f"{what} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D CUDA tensor")
    return t.shape[0]


def _cuda(t, what: str):
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return t.device


class _On:
    """The stream a call runs on: its device made current, and torch allocating on it."""

    __slots__ = ("ctx", "index")

    def __init__(self, device, stream):
        self.index = device.index
        if stream is not None:
            if stream.device.index != self.index:
                raise ValueError(f"the stream is on {stream.device}, not on {device}")
            self.ctx = torch.cuda.stream(stream)
        elif _current_device() != self.index:
            self.ctx = torch.cuda.device(device)
        else:
            self.ctx = None

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return _raw_stream(self.index)

    def __exit__(self, *a):
        if self.ctx is not None:
            self.ctx.__exit__(*a)


class Packed8:
    """Rows kept in 8 bits: ``codes`` int8 [n, d] and ``exps`` uint8 [n, ceil(d / 32)], both contiguous.

    Column j of a row stands for ``codes[j] * 2**(exps[j // 32] - 127)``, NaN where the exponent byte is 255;
    every such value is exact in bfloat16.  ``pack8`` and ``GatedNorm.forward`` make them; ``unpack8`` and the
    backward passes read them."""

    __slots__ = ("codes", "exps")

    def __init__(self, codes, exps):
        if codes.dim() != 2 or codes.dtype != torch.int8 or not codes.is_cuda or not codes.is_contiguous():
            raise ValueError("codes must be a contiguous int8 CUDA tensor [n, d]")
        if exps.dtype != torch.uint8 or not exps.is_contiguous() or exps.device != codes.device \
                or tuple(exps.shape) != (codes.shape[0], -(-codes.shape[1] // PACK_BLOCK)):
            raise ValueError("exps must be a contiguous uint8 CUDA tensor [n, ceil(d / 32)]")
        self.codes, self.exps = codes, exps

    @property
    def shape(self):
        return self.codes.shape

    @property
    def device(self):
        return self.codes.device

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.exps.numel()


def _new_packed(n: int, d: int, device) -> Packed8:
    p = Packed8.__new__(Packed8)
    p.codes = torch.empty((n, d), dtype=torch.int8, device=device)
    p.exps = torch.empty((n, -(-d // PACK_BLOCK)), dtype=torch.uint8, device=device)
    return p


def _width_ok(d: int, what: str):
    if not 1 <= d <= MAX_BLOCK_DIM:
        raise ValueError(f"{what} must have 1 to {MAX_BLOCK_DIM} columns")


def pack8(x, out: Packed8 | None = None, stream=None) -> Packed8:
    """The 8-bit form of the rows x [n, d] (float32 or bfloat16; rows may be strided)."""
    n = _count(x, "x")
    d, device = x.shape[1], _cuda(x, "x")
    _width_ok(d, "x")
    dt = _dtype_code(x.dtype)
    ld = _rows_2d(x, "x", d, n, x.dtype, device)
    with _On(device, stream) as s:
        if out is None:
            out = _new_packed(n, d, device)
        elif out.shape != x.shape or out.device != device:
            raise ValueError("out has another shape or device")
        _check(load_library().mt_pack8(x.data_ptr(), ld, n, d, dt, out.codes.data_ptr(), out.exps.data_ptr(), s),
               "mt_pack8")
    return out


def unpack8(p: Packed8, dtype=None, out=None, stream=None):
    """The values p stands for, as rows of `dtype` (bfloat16 by default, which holds them exactly)."""
    n, d = p.codes.shape
    _width_ok(d, "p")
    device = p.codes.device
    if out is not None:
        if dtype is not None and out.dtype != dtype:
            raise TypeError("out has another dtype")
        dtype = out.dtype
    elif dtype is None:
        dtype = torch.bfloat16
    dt = _dtype_code(dtype)
    with _On(device, stream) as s:
        ld = d
        if out is None:
            out = torch.empty((n, d), dtype=dtype, device=device)
        else:
            ld = _rows_2d(out, "out", d, n, dtype, device)
        _check(load_library().mt_unpack8(p.codes.data_ptr(), p.exps.data_ptr(), n, d, dt, out.data_ptr(), ld, s),
               "mt_unpack8")
    return out


# Status words of the handles: one zeroed buffer per device, a word (16 bytes apart) to each handle, so that making a
# handle neither allocates nor waits.
_STATUS_WORDS = 1024
_status_pool = {}
_status_lock = threading.Lock()


def _status_word(device):
    with _status_lock:
        buf, used = _status_pool.get(device, (None, _STATUS_WORDS))
        if used == _STATUS_WORDS:
            buf, used = torch.zeros(4 * _STATUS_WORDS, dtype=torch.int32, device=device), 0
            torch.cuda.current_stream(device).synchronize()  # a handle's first call may come on any stream
        _status_pool[device] = (buf, used + 1)
    return buf[4 * used: 4 * used + 1]


class _Handle:
    """What the block operators keep: their device, a status word and a workspace per stream."""

    def __init__(self, device):
        self.lib = load_library()
        self.device = torch.device(device) if device is not None else torch.device("cuda", _current_device())
        if self.device.index is None:
            self.device = torch.device("cuda", _current_device())
        self._status = _status_word(self.device)
        self._status_ptr = self._status.data_ptr()
        self._ws = {}

    def _workspace(self, stream: int, nbytes: int):
        buf = self._ws.get(stream)
        if buf is None or buf.numel() < nbytes:
            if torch.cuda.is_current_stream_capturing():
                # graphs captured earlier may hold the old buffer's address
                raise RuntimeError("the workspace would have to grow during CUDA graph capture; call "
                                   "reserve_workspace() on this stream with the largest batch before capturing")
            buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
            self._ws[stream] = buf
        return buf

    def _offsets(self, offsets, groups: int):
        if not torch.is_tensor(offsets) or offsets.dtype is not torch.int64 or offsets.device != self.device \
                or offsets.shape != (groups + 1,) or not offsets.is_contiguous():
            raise TypeError(f"offsets must be a contiguous int64 CUDA tensor [{groups + 1}] on {self.device}")
        return offsets.data_ptr()

    def error(self, clear: bool = False) -> int:
        """First error a call found on the device (MT_EINVAL: bad offsets), 0 if none; waits for the device."""
        torch.cuda.synchronize(self.device)
        e = int(self._status.item())
        if clear:
            self._status.zero_()
            torch.cuda.synchronize(self.device)
        return e


class GroupedLinear(_Handle):
    """Matrix products grouped by row segment: ``y_i = W_g x_i`` for the rows i of group g.

    num_groups: 1 to 1024; in_dim, out_dim: 1 to 8192; dtype of x, W, y, dy and dx: "bf16" or "f32"."""

    def __init__(self, num_groups: int, in_dim: int, out_dim: int, dtype: str = "bf16", device=None):
        if dtype not in _DTYPES:
            raise ValueError('dtype must be "f32" or "bf16"')
        if not 1 <= num_groups <= MAX_GROUPS or not 1 <= in_dim <= MAX_BLOCK_DIM or not 1 <= out_dim <= MAX_BLOCK_DIM:
            raise MTError(MT_EINVAL, "GroupedLinear")
        super().__init__(device)
        self.num_groups, self.in_dim, self.out_dim = num_groups, in_dim, out_dim
        self.dtype = dtype
        self.torch_dtype = _TORCH[dtype]
        self._dt = _DTYPES[dtype]
        self._w_shape = (num_groups, out_dim, in_dim)

    def _weight(self, w):
        if w.shape != self._w_shape or w.dtype is not self.torch_dtype or w.device != self.device \
                or not w.is_contiguous():
            raise ValueError(f"weight must be a contiguous {self.torch_dtype} CUDA tensor "
                             f"[{self.num_groups}, {self.out_dim}, {self.in_dim}]")
        return w.data_ptr()

    def forward(self, x, weight, offsets, out=None, stream=None):
        """y [n, out_dim] of x [n, in_dim], weight [num_groups, out_dim, in_dim] and offsets int64 CUDA
        [num_groups + 1]; rows in no group give zeros."""
        n = _count(x, "x")
        ldx = _rows_2d(x, "x", self.in_dim, n, self.torch_dtype, self.device)
        w, off = self._weight(weight), self._offsets(offsets, self.num_groups)
        with _On(self.device, stream) as s:
            if out is None:
                out = torch.empty((n, self.out_dim), dtype=self.torch_dtype, device=self.device)
                ldy = self.out_dim
            else:
                ldy = _rows_2d(out, "out", self.out_dim, n, self.torch_dtype, self.device)
            _check(self.lib.mt_group_linear_forward(x.data_ptr(), ldx, w, off, self.num_groups, n, self.in_dim,
                                                    self.out_dim, self._dt, out.data_ptr(), ldy, self._status_ptr, s),
                   "mt_group_linear_forward")
        return out

    def backward(self, dy, x, weight, offsets, want_dx: bool = True, want_dw: bool = True, out_dx=None, out_dw=None,
                 stream=None):
        """(dx [n, in_dim], dw fp32 [num_groups, out_dim, in_dim]) of dy [n, out_dim]; x: the forward's input, plain
        or ``Packed8`` (None without want_dw)."""
        n = _count(dy, "dy")
        lddy = _rows_2d(dy, "dy", self.out_dim, n, self.torch_dtype, self.device)
        if not want_dx and not want_dw:
            raise ValueError("nothing to compute")
        w = self._weight(weight) if want_dx else None
        off = self._offsets(offsets, self.num_groups)
        rows = None
        if want_dw:
            if isinstance(x, Packed8):
                if tuple(x.shape) != (n, self.in_dim) or x.device != self.device:
                    raise ValueError(f"x must be [{n}, {self.in_dim}] on {self.device}")
                rows = _Rows(None, 0, x.codes.data_ptr(), x.exps.data_ptr())
            else:
                ldx = _rows_2d(x, "x", self.in_dim, n, self.torch_dtype, self.device)
                rows = _Rows(x.data_ptr(), ldx, None, None)
        dx = dw = None
        lddx = self.in_dim
        with _On(self.device, stream) as s:
            if want_dx:
                dx = out_dx
                if dx is None:
                    dx = torch.empty((n, self.in_dim), dtype=self.torch_dtype, device=self.device)
                else:
                    lddx = _rows_2d(dx, "out_dx", self.in_dim, n, self.torch_dtype, self.device)
                if n == 0 and not want_dw:
                    return dx, None
            ws_ptr, ws_len = None, 0
            if want_dw:
                shape = self._w_shape
                dw = out_dw
                if dw is None:
                    dw = torch.empty(shape, dtype=torch.float32, device=self.device)
                elif tuple(dw.shape) != shape or dw.dtype != torch.float32 or not dw.is_contiguous() \
                        or dw.device != self.device:
                    raise ValueError(f"out_dw must be a contiguous float32 CUDA tensor {list(shape)}")
                ws = self._workspace(s, self.lib.mt_group_linear_workspace_bytes(n, self.num_groups, self.in_dim,
                                                                                 self.out_dim))
                ws_ptr, ws_len = ws.data_ptr(), ws.numel()
            # an empty batch has no dx rows to point at: only dw is asked for
            _check(self.lib.mt_group_linear_backward(
                dy.data_ptr(), lddy, ctypes.byref(rows) if rows is not None else None, w, off, self.num_groups, n,
                self.in_dim, self.out_dim, self._dt, dx.data_ptr() if want_dx and n else None, lddx,
                dw.data_ptr() if want_dw else None, self._status_ptr, ws_ptr, ws_len, s), "mt_group_linear_backward")
        return dx, dw

    def reserve_workspace(self, n: int, stream=None):
        """Allocate, on this stream, the workspace a backward over n rows needs (before a CUDA graph capture)."""
        with _On(self.device, stream) as s:
            self._workspace(s, self.lib.mt_group_linear_workspace_bytes(n, self.num_groups, self.in_dim,
                                                                                 self.out_dim))


@dataclasses.dataclass
class NormParams:
    """Parameters of a ``GatedNorm`` (or their gradients): fp32 CUDA tensors [num_groups, dim] ([dim] for one
    group), None where there is none.  post_* and scale: the norm after the block; pre_*: the next block's norm."""
    post_weight: "object" = None
    post_bias: "object" = None
    scale: "object" = None
    pre_weight: "object" = None
    pre_bias: "object" = None


@dataclasses.dataclass
class NormForward:
    z: "object"                # residual stream [n, dim]
    h: "object"                # next block's normed input [n, dim], or None
    packed: dict               # checkpoints asked for: "y", "u", "z", "h" -> Packed8


@dataclasses.dataclass
class NormGrads:
    dx: "object"
    dy: "object"               # None without y
    du: "object"               # None without a gate
    params: NormParams         # fp32 [num_groups, dim], None where the parameter is


_PARAMS = ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias")


class GatedNorm(_Handle):
    """The norm after a block with its gate and residual scale, the residual sum, and the next block's norm::

        z = x + scale * (post_weight * norm(y) + post_bias) * act(u)
        h = pre_weight * norm(z) + pre_bias

    kind: "rms" or "layer" (both norms); gate: "none" (no u), "linear" (act(u) = u), "sigmoid" or "silu"; dim: 1 to
    8192; dtype of the rows: "bf16" or "f32".  Each group of rows has its own parameters (num_groups: 1 to 1024)."""

    def __init__(self, dim: int, num_groups: int = 1, kind: str = "rms", gate: str = "silu", eps: float = 1e-6,
                 dtype: str = "bf16", device=None):
        if kind not in _KINDS or gate not in _GATES or dtype not in _DTYPES:
            raise ValueError("unknown kind, gate or dtype")
        if not 1 <= dim <= MAX_BLOCK_DIM or not 1 <= num_groups <= MAX_GROUPS or not 0.0 < eps <= 1e30:
            raise MTError(MT_EINVAL, "GatedNorm")
        super().__init__(device)
        self.dim, self.num_groups, self.kind, self.gate, self.eps, self.dtype = dim, num_groups, kind, gate, eps, dtype
        self.torch_dtype = _TORCH[dtype]
        self._p_shapes = ((num_groups, dim), (dim,)) if num_groups == 1 else ((num_groups, dim),)
        self._codes = (_DTYPES[dtype], _KINDS[kind], _GATES[gate])

    def _config(self, n: int, params: NormParams, offsets) -> _GatedNorm:
        c = _GatedNorm(n, self.dim, self.num_groups, *self._codes, self.eps, None, self._status_ptr)
        if offsets is not None:
            c.offsets = self._offsets(offsets, self.num_groups)
        elif self.num_groups != 1:
            raise ValueError("several groups need offsets")
        for name in _PARAMS:
            t = getattr(params, name)
            if t is None:
                continue
            if t.dtype is not torch.float32 or t.device != self.device or t.shape not in self._p_shapes \
                    or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 CUDA tensor [{self.num_groups}, {self.dim}]")
            setattr(c, name, t.data_ptr())
        return c

    def _plain(self, t, what: str, n: int):
        if t is None:
            return _Rows()
        ld = _rows_2d(t, what, self.dim, n, self.torch_dtype, self.device)
        return _Rows(t.data_ptr(), ld, None, None)

    def _saved(self, t, what: str, n: int):
        if isinstance(t, Packed8):
            if tuple(t.shape) != (n, self.dim) or t.device != self.device:
                raise ValueError(f"{what} must be [{n}, {self.dim}] on {self.device}")
            return _Rows(None, 0, t.codes.data_ptr(), t.exps.data_ptr())
        return self._plain(t, what, n)

    def _parts(self, y, u, params: NormParams):
        """Which parts there are, checked against the parameters."""
        if (y is None) != (params.post_weight is None):
            raise ValueError("y and post_weight come together")
        if (u is None) != (self.gate == "none" or y is None):
            raise ValueError('u is given exactly with y and a gate other than "none"')
        if y is None and (params.post_bias is not None or params.scale is not None):
            raise ValueError("post_bias and scale need y")
        if params.pre_weight is None and params.pre_bias is not None:
            raise ValueError("pre_bias needs pre_weight")
        if y is None and params.pre_weight is None:
            raise ValueError("nothing to compute")

    def forward(self, x, y=None, u=None, params: NormParams = None, offsets=None, pack="", out_z=None, out_h=None,
                stream=None) -> NormForward:
        """One pass over the rows x, y, u [n, dim].  Without y, z is x itself.  pack: the letters of the checkpoints to
        write, any of "yuzh" (``packed`` holds them by letter)."""
        params = params if params is not None else NormParams()
        self._parts(y, u, params)
        n = _count(x, "x")
        rx = self._plain(x, "x", n)
        ry, ru = self._plain(y, "y", n), self._plain(u, "u", n)
        c = self._config(n, params, offsets)
        if y is None:
            c.gate = 0
        has_h = params.pre_weight is not None
        with _On(self.device, stream) as s:
            z = x
            rz, rh = _Rows(), _Rows()
            if y is not None:
                z = out_z if out_z is not None else torch.empty((n, self.dim), dtype=self.torch_dtype,
                                                                device=self.device)
                rz = self._plain(z, "out_z", n) if out_z is not None else _Rows(z.data_ptr(), self.dim)
            elif out_z is not None:
                raise ValueError("without y there is no z to write")
            h = None
            if has_h:
                h = out_h if out_h is not None else torch.empty((n, self.dim), dtype=self.torch_dtype,
                                                                device=self.device)
                rh = self._plain(h, "out_h", n) if out_h is not None else _Rows(h.data_ptr(), self.dim)
            elif out_h is not None:
                raise ValueError("without pre_weight there is no h to write")
            packed = {}
            for name in pack:
                there = {"y": y is not None, "u": u is not None, "z": True, "h": has_h}.get(name)
                if not there:
                    raise ValueError(f"there is no {name!r} to pack")
                p = packed[name] = _new_packed(n, self.dim, self.device)
                r = {"y": ry, "u": ru, "z": rz, "h": rh}[name]
                r.codes, r.exps = p.codes.data_ptr(), p.exps.data_ptr()
            if n:
                _check(self.lib.mt_gated_norm_forward(ctypes.byref(c), ctypes.byref(rx), ctypes.byref(ry),
                                                      ctypes.byref(ru), ctypes.byref(rz), ctypes.byref(rh), s),
                       "mt_gated_norm_forward")
        return NormForward(z, h, packed)

    def backward(self, dz, dh, y=None, u=None, z=None, params: NormParams = None, offsets=None, out_dx=None,
                 out_dy=None, out_du=None, stream=None) -> NormGrads:
        """Gradients from dz [n, dim] (None: zero) and dh (None without pre_weight).  y, u, z: the forward's, each
        plain or ``Packed8``; z is needed with pre_weight only.  out_dy and out_du may be column slices of one
        tensor (the gradient of a product that made y and u side by side)."""
        params = params if params is not None else NormParams()
        self._parts(y, u, params)
        has_h = params.pre_weight is not None
        if has_h != (dh is not None):
            raise ValueError("dh and pre_weight come together")
        if has_h and z is None:
            raise ValueError("the gradient of the next block's norm needs z")
        lead = dh if has_h else dz
        if lead is None:
            raise ValueError("dz is needed without pre_weight")
        n = _count(lead, "dh" if has_h else "dz")
        rdz, rdh = self._plain(dz, "dz", n), self._plain(dh, "dh", n)
        ry, ru, rz = self._saved(y, "y", n), self._saved(u, "u", n), self._saved(z if has_h else None, "z", n)
        c = self._config(n, params, offsets)
        if y is None:
            c.gate = 0
        with _On(self.device, stream) as s:
            def rows(out, what):
                if out is not None:
                    return out, self._plain(out, what, n)
                t = torch.empty((n, self.dim), dtype=self.torch_dtype, device=self.device)
                return t, _Rows(t.data_ptr(), self.dim)

            dx, rdx = rows(out_dx, "out_dx")
            dy, rdy = rows(out_dy, "out_dy") if y is not None else (None, _Rows())
            du, rdu = rows(out_du, "out_du") if u is not None else (None, _Rows())
            there = [k for k in _PARAMS if getattr(params, k) is not None]
            sums = torch.empty((len(there), self.num_groups, self.dim), dtype=torch.float32, device=self.device)
            grads = dict(zip(there, sums.unbind(0)))
            ws = self._workspace(s, self.lib.mt_gated_norm_workspace_bytes(n, self.dim, self.num_groups))
            _check(self.lib.mt_gated_norm_backward(
                ctypes.byref(c), ctypes.byref(rdz), ctypes.byref(rdh), ctypes.byref(ry), ctypes.byref(ru),
                ctypes.byref(rz), ctypes.byref(rdx), ctypes.byref(rdy), ctypes.byref(rdu),
                *(grads[k].data_ptr() if k in grads else None for k in _PARAMS), ws.data_ptr(), ws.numel(), s),
                "mt_gated_norm_backward")
        return NormGrads(dx, dy, du, NormParams(**grads))

    def reserve_workspace(self, n: int, stream=None):
        """Allocate, on this stream, the workspace a backward over n rows needs (before a CUDA graph capture)."""
        with _On(self.device, stream) as s:
            self._workspace(s, self.lib.mt_gated_norm_workspace_bytes(n, self.dim, self.num_groups))
