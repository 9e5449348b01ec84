"""Losses of rows against a vocabulary whose logits are never kept.

``CrossEntropy`` (softmax cross entropy) and ``Distillation`` (the divergence
from a teacher that is known by its top logits) marshal their arguments to
``mt_vocab_loss_*`` of ``include/mt.h``.  The vocabulary is any row tensor: the
items' weights, or the table's rows of distinct IDs, whose gradient then goes to
``Table.backward_adam`` with that lookup; targets index its rows, and a row whose
target is negative (what a lookup's ``inverse`` has for an invalid ID) takes no
part.  IDs that come several times, such as a batch's items, are looked up without
their rows first: that lookup's ``unique_keys[:U]`` (their low 56 bits) are the IDs
of a second one whose ``rows`` are the vocabulary, and its ``inverse`` the targets.
(``rows`` of the first would have one row a position, which ``inverse`` does not
index.)

The losses come per row, and so do their weights in the backward: ``dloss`` of
1 / n makes a mean.  Between forward and backward nothing is kept but each row's
log sum (``lse``); a backward holds up to 4 GiB of the logits' gradient at a
time (or 512 bytes a row, fp32 1536, where that is more).  Streams, graphs and errors as in ``block``: calls run on the current stream
or on ``stream``, a captured call's workspace belongs to its graph, and targets
outside the vocabulary are latched in the handle's status word (``error()``).
"""
from __future__ import annotations

import dataclasses

from . import MT_EINVAL, MTError, block
from .block import _DTYPES, _TORCH, MAX_BLOCK_DIM, _Handle, _on

__all__ = ["CrossEntropy", "Distillation", "LossForward"]

MAX_VOCAB = (1 << 31) - 4096
MAX_TOP = 1024


@dataclasses.dataclass
class LossForward:
    loss: "object"   # fp32 [n], 0 where the row takes no part
    lse: "object"    # fp32 [n], log sum of the exponentials of the row's logits; what the backward takes


class _VocabLoss(_Handle):
    def __init__(self, what, vocab, dim, top, scale, smoothing, z_loss, dtype, device):
        if dtype not in _DTYPES:
            raise ValueError('dtype must be "f32" or "bf16"')
        if not 1 <= vocab <= MAX_VOCAB or not 1 <= dim <= MAX_BLOCK_DIM or not 0.0 < scale <= 1e30 \
                or not 0.0 <= smoothing < 1.0 or not 0.0 <= z_loss <= 1e30:
            raise MTError(MT_EINVAL, what)
        super().__init__(device)
        self.vocab, self.dim, self.scale, self.dtype = vocab, dim, scale, dtype
        self.torch_dtype = _TORCH[dtype]
        self._cfg = (vocab, dim, _DTYPES[dtype], top, float(scale), float(smoothing), float(z_loss), self.device.index,
                     self._status_ptr)

    def _forward(self, x, weight, targets, teacher, out_loss, out_lse, stream):
        args = (*self._cfg, x, weight, targets, teacher, out_loss, out_lse)
        return LossForward(*(block._native.vocab_forward(*args) if stream is None else _on(self.device, stream, block._native.vocab_forward, *args)))

    def _backward(self, dloss, x, weight, targets, teacher, lse, want_dx, want_dw, out_dx, out_dw, stream):
        if not want_dx and not want_dw:
            raise ValueError("nothing to compute")
        args = (*self._cfg, dloss, lse, x, weight, targets, teacher, out_dx, out_dw, int(want_dx), int(want_dw))
        return block._native.vocab_backward(*args) if stream is None else _on(self.device, stream, block._native.vocab_backward, *args)


class CrossEntropy(_VocabLoss):
    """Softmax cross entropy of rows x [n, dim] against a vocabulary of rows w [vocab, dim]::

        z_iv = scale * (x_i . w_v),  lse_i = log sum_v exp z_iv
        loss_i = lse_i - (1 - smoothing) * z_i,target - smoothing / vocab * sum_v z_iv + z_loss * lse_i^2

    vocab: 1 to 2^31 - 4096; dim: 1 to 8192; scale > 0; smoothing in [0, 1); z_loss >= 0; dtype of x, w and the
    gradients: "bf16" or "f32"."""

    def __init__(self, vocab: int, dim: int, scale: float = 1.0, smoothing: float = 0.0, z_loss: float = 0.0,
                 dtype: str = "bf16", device=None):
        super().__init__("CrossEntropy", vocab, dim, 0, scale, smoothing, z_loss, dtype, device)
        self.smoothing, self.z_loss = smoothing, z_loss

    def forward(self, x, weight, targets, out_loss=None, out_lse=None, stream=None) -> LossForward:
        """targets: int32 or int64 CUDA [n]; negative: the row takes no part (loss and lse 0)."""
        return self._forward(x, weight, targets, None, out_loss, out_lse, stream)

    def backward(self, dloss, x, weight, targets, lse, want_dx: bool = True, want_dw: bool = True, out_dx=None, out_dw=None,
                 stream=None):
        """(dx [n, dim], dw [vocab, dim]), both in the handle's dtype, of dloss fp32 [n] and the forward's lse."""
        return self._backward(dloss, x, weight, targets, None, lse, want_dx, want_dw, out_dx, out_dw, stream)


class Distillation(_VocabLoss):
    """The divergence of rows x [n, dim] from a teacher that is known by its top_k logits a row, over a vocabulary of
    rows w [vocab, dim]::

        z_iv = scale * (x_i . w_v),  lse_i = log sum_v exp z_iv
        t_ik = softmax over the row's k of scale * logits_ik
        loss_i = sum_k t_ik * (log t_ik - z_i,ids_ik) + lse_i

    scale is one over the temperature.  top_k: 1 to 1024; the rest as for ``CrossEntropy``."""

    def __init__(self, vocab: int, dim: int, top_k: int, scale: float = 1.0, dtype: str = "bf16", device=None):
        if not 1 <= top_k <= MAX_TOP:
            raise MTError(MT_EINVAL, "Distillation")
        super().__init__("Distillation", vocab, dim, top_k, scale, 0.0, 0.0, dtype, device)
        self.top_k = top_k

    def forward(self, x, weight, ids, logits, out_loss=None, out_lse=None, stream=None) -> LossForward:
        """ids: int32 or int64 CUDA [n, top_k]; logits: fp32 or bf16 CUDA [n, top_k].  A pair whose id is negative or whose
        logit is -inf is not there; a row without any takes no part."""
        return self._forward(x, weight, ids, logits, out_loss, out_lse, stream)

    def backward(self, dloss, x, weight, ids, logits, lse, want_dx: bool = True, want_dw: bool = True, out_dx=None, out_dw=None,
                 stream=None):
        """(dx [n, dim], dw [vocab, dim]), both in the handle's dtype, of dloss fp32 [n] and the forward's lse."""
        return self._backward(dloss, x, weight, ids, logits, lse, want_dx, want_dw, out_dx, out_dw, stream)
