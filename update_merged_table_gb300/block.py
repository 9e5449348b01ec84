"""The dense block between a lookup and its gradient, over ragged groups of rows.

``GroupedLinear`` (matrix products whose weights differ by row segment),
``GatedNorm`` (the norm after a block with its gate and residual scale, the
residual sum and the next block's norm) and ``Packed8`` (activations kept in
8 bits for the backward) marshal their arguments to the calls of the same
names in ``include/mt.h``.  Groups are runs of rows: a batch's feature segments, or the
tokens sorted by expert.

Outputs and workspaces are allocated on the stream the call runs on
(``stream``, by default the current one); a handle may be used from several
streams, each with its own workspace.  A call captured in a CUDA graph takes
its workspace from the graph's memory, like its outputs: nothing has to be
reserved, and the graph may be replayed on any stream, beside other calls of
the handle.  A graph writes errors to its handle's status word: keep the handle
as long as the graph.
"""
from __future__ import annotations

import dataclasses
import importlib.util
import ctypes
import os
import threading

import torch

from . import LIB_PATH, MT_BF16, MT_EINVAL, MT_F32, MTError, load_library

__all__ = ["Packed8", "pack8", "unpack8", "GroupedLinear", "GatedNorm", "NormParams", "NormForward", "NormGrads"]

MAX_GROUPS = 1024
MAX_BLOCK_DIM = 8192
PACK_BLOCK = 32
_KINDS = {"rms": 0, "layer": 1}
_GATES = {"none": 0, "linear": 1, "sigmoid": 2, "silu": 3}
_DTYPES = {"f32": MT_F32, "bf16": MT_BF16}
_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
_CODES = {torch.float32: MT_F32, torch.bfloat16: MT_BF16}
_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream


def _capturing(device) -> bool:
    """Whether the device's current stream is being captured."""
    if _current_device() == device.index:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(device):
        return torch.cuda.is_current_stream_capturing()


def _load_native():
    """The module that checks and marshals a call in one native step (built beside libmt.so)."""
    lib = load_library()
    path = os.path.join(os.path.dirname(LIB_PATH), "_mt_block.so")
    if not os.path.exists(path):
        raise RuntimeError(f"the Python module is not built: {path} is missing (run update_merged_table_gb300.build_lib.build())")
    spec = importlib.util.spec_from_file_location("_mt_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    names = ("mt_pack8", "mt_unpack8", "mt_group_linear_forward", "mt_group_linear_backward", "mt_gated_norm_forward",
             "mt_gated_norm_backward")
    mod.init(*(ctypes.cast(getattr(lib, k), ctypes.c_void_p).value for k in names), MTError, torch.OutOfMemoryError)
    return mod


class _Unloaded:
    """Stands for the native module until its first use: the names of this one need no built library."""

    def __getattr__(self, name):
        global _native
        _native = _load_native()
        return getattr(_native, name)


_native = _Unloaded()


class _On:
    """The stream a call runs on made current (and its device), so that torch allocates on it too."""

    __slots__ = ("ctx",)

    def __init__(self, device, stream):
        if stream.device.index != device.index:
            raise ValueError(f"the stream is on {stream.device}, not on {device}")
        self.ctx = torch.cuda.stream(stream)

    def __enter__(self):
        self.ctx.__enter__()

    def __exit__(self, *a):
        self.ctx.__exit__(*a)


def _on(device, stream, f, *args):
    """f(*args) on the given stream, or on the current one."""
    if stream is None:
        return f(*args)
    with _On(device, stream):
        return f(*args)


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


def _packed(codes, exps) -> Packed8:
    p = Packed8.__new__(Packed8)
    p.codes, p.exps = codes, exps
    return p


def pack8(x, out: Packed8 | None = None, stream=None) -> Packed8:
    """The 8-bit form of the rows x [n, d] (float32 or bfloat16; rows may be strided)."""
    c, e = (None, None) if out is None else (out.codes, out.exps)
    c, e = _native.pack8(x, c, e) if stream is None else _on(x.device, stream, _native.pack8, x, c, e)
    return _packed(c, e) if out is None else out


def unpack8(p: Packed8, dtype=None, out=None, stream=None):
    """The values p stands for, as rows of `dtype` (bfloat16 by default, which holds them exactly)."""
    if dtype is None:
        dtype = torch.bfloat16 if out is None else out.dtype
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("rows must be float32 or bfloat16")
    if stream is None:
        return _native.unpack8(p.codes, p.exps, code, out)
    return _on(p.device, stream, _native.unpack8, p.codes, p.exps, code, out)


def _plain_or_packed(t):
    return (t.codes, t.exps) if isinstance(t, Packed8) else t


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


def _rows_of(t, what: str) -> int:
    if not torch.is_tensor(t):
        raise TypeError(f"{what} must be a CUDA tensor")
    return t.shape[0] if t.dim() == 2 else 0  # anything but rows is refused by the call


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

    def _workspace(self, nbytes: int):
        """The workspace of the current stream; under capture one of the graph's own (a kept one may be replaced by a larger
        one later, and its memory reused, while the graph still holds its address)."""
        if _capturing(self.device):
            return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        stream = _raw_stream(self.device.index)
        buf = self._ws.get(stream)
        if buf is None or buf.numel() < nbytes:
            buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
            self._ws[stream] = buf
        return buf

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
        self._cfg = (num_groups, in_dim, out_dim, _DTYPES[dtype], self.device.index, self._status_ptr)

    def forward(self, x, weight, offsets, out=None, stream=None):
        """y [n, out_dim] of x [n, in_dim], weight [num_groups, out_dim, in_dim] and offsets int64 CUDA
        [num_groups + 1]; rows in no group give zeros."""
        if stream is None:
            return _native.linear_forward(*self._cfg, x, weight, offsets, out)
        return _on(self.device, stream, _native.linear_forward, *self._cfg, x, weight, offsets, out)

    def backward(self, dy, x, weight, offsets, want_dx: bool = True, want_dw: bool = True, out_dx=None, out_dw=None,
                 stream=None):
        """(dx [n, in_dim], dw fp32 [num_groups, out_dim, in_dim]) of dy [n, out_dim]; x: the forward's input, plain
        or ``Packed8`` (None without want_dw)."""
        if not want_dx and not want_dw:
            raise ValueError("nothing to compute")
        if stream is not None:
            return _on(self.device, stream, self.backward, dy, x, weight, offsets, want_dx, want_dw, out_dx, out_dw)
        ws = self._reserved(_rows_of(dy, "dy")) if want_dw else None
        return _native.linear_backward(*self._cfg, dy, _plain_or_packed(x), weight, offsets, out_dx, out_dw, int(want_dx),
                                       int(want_dw), ws)

    def _reserved(self, n: int):
        return self._workspace(self.lib.mt_group_linear_workspace_bytes(n, self.num_groups, self.in_dim, self.out_dim))

    def reserve_workspace(self, n: int, stream=None):
        """Allocate, on this stream, the workspace a backward over n rows needs, so that calls up to that size do not."""
        _on(self.device, stream, self._reserved, n)


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
        self._cfg = (num_groups, dim, _DTYPES[dtype], _KINDS[kind], _GATES[gate], eps, self.device.index, self._status_ptr)

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
        has_h = params.pre_weight is not None
        if y is None and out_z is not None:
            raise ValueError("without y there is no z to write")
        if not has_h and out_h is not None:
            raise ValueError("without pre_weight there is no h to write")
        bits = 0
        for name in pack:
            if not {"y": y is not None, "u": u is not None, "z": True, "h": has_h}.get(name):
                raise ValueError(f"there is no {name!r} to pack")
            bits |= 1 << "yuzh".index(name)
        args = (*self._cfg, params.post_weight, params.post_bias, params.scale, params.pre_weight, params.pre_bias, offsets,
                x, y, u, out_z, out_h, bits)
        r = _native.norm_forward(*args) if stream is None else _on(self.device, stream, _native.norm_forward, *args)
        packed = {}
        if bits:
            names = [k for i, k in enumerate("yuzh") if bits >> i & 1]
            packed = {k: _packed(r[2 + 2 * i], r[3 + 2 * i]) for i, k in enumerate(names)}
        return NormForward(r[0] if y is not None else x, r[1], packed)

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
        if stream is not None:
            return _on(self.device, stream, self.backward, dz, dh, y, u, z, params, offsets, out_dx, out_dy, out_du)
        ws = self._reserved(_rows_of(lead, "dh" if has_h else "dz"))
        r = _native.norm_backward(*self._cfg, params.post_weight, params.post_bias, params.scale, params.pre_weight,
                                  params.pre_bias, offsets, dz, dh, _plain_or_packed(y), _plain_or_packed(u),
                                  _plain_or_packed(z), out_dx, out_dy, out_du, ws)
        return NormGrads(r[0], r[1], r[2], NormParams(*r[3:]))

    def _reserved(self, n: int):
        return self._workspace(self.lib.mt_gated_norm_workspace_bytes(n, self.dim, self.num_groups))

    def reserve_workspace(self, n: int, stream=None):
        """Allocate, on this stream, the workspace a backward over n rows needs, so that calls up to that size do not."""
        _on(self.device, stream, self._reserved, n)
