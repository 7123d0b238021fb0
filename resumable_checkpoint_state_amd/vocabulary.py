"""The two ends of a model at its vocabulary, in training: a thin binding of the
output head's losses (head_loss, head_distill) and of the embedding's gradient
(embed_grad).

Argument marshalling only, as in the rest of the package: everything is computed
in the HIP kernels of csrc/head.hip and csrc/embed.hip.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _check, _stream, lib

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_INDEX_TYPES = {torch.int32: 0, torch.int64: 1}
MAX_BYTES = 4 << 30


class _Head(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("grad_hidden", ctypes.c_void_p), ("grad_weight", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("hidden_stride", ctypes.c_int64), ("weight_stride", ctypes.c_int64),
                ("grad_hidden_stride", ctypes.c_int64), ("grad_weight_stride", ctypes.c_int64),
                ("type", ctypes.c_int32), ("grad_weight_type", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("mean", ctypes.c_int32),
                ("scale", ctypes.c_float), ("losses", ctypes.c_void_p), ("loss", ctypes.c_void_p),
                ("limit", ctypes.c_int64), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_int64)]


def _on_device(t, name: str, dev: int, types) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in types:
        kinds = ", ".join(str(k).removeprefix("torch.") for k in types)
        raise TypeError(f"{name} must be a tensor of type {kinds}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}; the library works on the current device "
                         f"(cuda:{dev}): use torch.cuda.device(...)")


def _matrix(t, name: str, dev: int, types, shape=None) -> tuple[torch.Tensor, int]:
    """t as rows of its last dimension, and the stride between them."""
    _on_device(t, name, dev, types)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dim() == 0 or t.shape[-1] == 0:
        raise ValueError(f"{name} has shape {tuple(t.shape)}: it has no columns")
    t, cols = t.detach(), t.shape[-1]
    if t.dim() != 2:
        try:
            t = t.view(-1, cols)
        except RuntimeError:
            raise TypeError(f"{name} must have rows at one stride") from None
    rows = t.shape[0]
    stride = t.stride(0) if rows > 1 else cols
    if (cols > 1 and t.stride(1) != 1) or stride < cols:
        raise TypeError(f"{name} must have contiguous rows that do not overlap")
    return t, stride


def _table(t, name: str, dev: int, types, dim: int) -> tuple[torch.Tensor, int]:
    """As _matrix, of a matrix of the vocabulary."""
    _on_device(t, name, dev, types)
    if t.dim() != 2 or t.shape[1] != dim or t.shape[0] == 0:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected (vocab, {dim})")
    return _matrix(t, name, dev, types)


def _packed(t, name: str, dev: int, types, shape) -> torch.Tensor:
    _on_device(t, name, dev, types)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise TypeError(f"{name} must be contiguous")
    return t.detach()


def _stream_context(stream):
    """Allocations inside belong to the stream that will use them."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        if int(stream) == torch.cuda.current_stream().cuda_stream:
            return contextlib.nullcontext()
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else \
            torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _head(call, name, entries, hidden, weight, grad_hidden, grad_weight, accumulate, reduction, scale,
          losses, out, max_bytes, stream):
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    h, hs = _matrix(hidden, "hidden", dev, _TYPES)
    w, ws = _table(weight, "weight", dev, (hidden.dtype,), h.shape[1])
    if reduction not in ("mean", "sum"):
        raise ValueError(f"reduction is {reduction!r}, expected 'mean' or 'sum'")
    lead = hidden.shape[:-1]
    a = _Head(hidden=h.data_ptr(), weight=w.data_ptr(), rows=h.shape[0], vocab=w.shape[0],
              dim=h.shape[1], hidden_stride=hs, weight_stride=ws, type=_TYPES[h.dtype],
              accumulate=bool(accumulate), mean=reduction == "mean", scale=float(scale),
              limit=int(max_bytes))
    if grad_hidden is not None:
        g, a.grad_hidden_stride = _matrix(grad_hidden, "grad_hidden", dev, (hidden.dtype,),
                                          hidden.shape)
        a.grad_hidden = g.data_ptr()
    if grad_weight is not None:
        g, a.grad_weight_stride = _matrix(grad_weight, "grad_weight", dev, _TYPES, weight.shape)
        a.grad_weight, a.grad_weight_type = g.data_ptr(), _TYPES[g.dtype]
    if losses is not None:
        a.losses = _packed(losses, "losses", dev, (torch.float32,), lead).data_ptr()
    need = lib().rcs_head_workspace(ctypes.byref(a), entries)
    _check(int(need) if need < 0 else 0, "rcs_head_workspace")
    with _stream_context(stream):
        if out is None:
            out = torch.empty(1, dtype=torch.float32, device=h.device)
        else:
            _packed(out, "out", dev, (torch.float32,), torch.Size([1]))
        work = torch.empty(need, dtype=torch.uint8, device=h.device)
        a.loss, a.workspace, a.workspace_bytes = out.data_ptr(), work.data_ptr(), need
        _check(call(ctypes.byref(a), _stream(stream)), name)
    return out


def head_loss(hidden, weight, targets, *, grad_hidden=None, grad_weight=None,
              accumulate: bool = True, reduction: str = "mean", scale: float = 1.0,
              ignore_index: int = -100, losses=None, out=None, max_bytes: int = MAX_BYTES,
              stream=None) -> torch.Tensor:
    """Softmax cross entropy of the output head hidden @ weight.T against the
    targets, without the logits, and its gradients; asynchronous on stream.

    hidden (..., dim) and weight (vocab, dim): float32, bfloat16 or float16, both
    of one type, rows contiguous and at one stride. targets (...): int32 or int64.
    Rows whose target is ignore_index have no loss and take no part; any other
    target outside the vocabulary makes the row's loss and the gradients NaN.

    grad_hidden, of hidden's shape and type, is written; grad_weight, of weight's
    shape and any of the three types, is added to (written with
    accumulate=False). Both are those of scale times the loss; without them only
    the loss is computed. reduction: "mean" over the rows that have a loss, or
    "sum". losses: float32 (...), receives each row's loss. Returns the loss, a
    1-element float32 tensor (out, if given); it is 0 if no row has one.

    max_bytes: what the call may take for the exponentials of the logits at a
    time (more rows than that are done in groups), besides the rest of its
    workspace, which comes from torch's allocator for the stream."""
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    _on_device(targets, "targets", dev, _INDEX_TYPES)
    t = _packed(targets, "targets", dev, _INDEX_TYPES, hidden.shape[:-1])

    def call(a, s):
        return lib().head_loss(a, t.data_ptr(), _INDEX_TYPES[t.dtype], int(ignore_index), s)

    return _head(call, "head_loss", 0, hidden, weight, grad_hidden, grad_weight, accumulate,
                 reduction, scale, losses, out, max_bytes, stream)


def head_distill(hidden, weight, indices, logits, *, temperature: float = 1.0, grad_hidden=None,
                 grad_weight=None, accumulate: bool = True, reduction: str = "mean",
                 scale: float = 1.0, losses=None, out=None, max_bytes: int = MAX_BYTES,
                 stream=None) -> torch.Tensor:
    """The divergence from a teacher's top logits to the head's softmax, at a
    temperature and times its square, with its gradients; asynchronous on stream.

    indices (..., entries), int32 or int64: the columns of the teacher's logits
    (..., entries), of any of the three types; at most 1,024 entries. The
    teacher's distribution is the softmax of logits / temperature over the row's
    entries, the student's that of hidden @ weight.T / temperature over the whole
    vocabulary. Entries with a negative index or a logit of -inf are not there,
    and a row without entries has no loss; an index that is not in the vocabulary
    makes the row's loss and the gradients NaN. The rest as for head_loss."""
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    _on_device(indices, "indices", dev, _INDEX_TYPES)
    if indices.dim() == 0:
        raise ValueError("indices has no entries")
    entries = indices.shape[-1]
    i = _packed(indices, "indices", dev, _INDEX_TYPES, hidden.shape[:-1] + (entries,))
    g = _packed(logits, "logits", dev, _TYPES, indices.shape)

    def call(a, s):
        return lib().head_distill(a, i.data_ptr(), _INDEX_TYPES[i.dtype], g.data_ptr(),
                                  _TYPES[g.dtype], entries, float(temperature), s)

    return _head(call, "head_distill", entries, hidden, weight, grad_hidden, grad_weight, accumulate,
                 reduction, scale, losses, out, max_bytes, stream)


def embed_grad(rows, tokens, grad, *, scale: float = 1.0, stream=None) -> None:
    """grad[tokens[...]] += scale * rows[...], the gradient of an embedding lookup,
    in an order that depends on the arguments alone; asynchronous on stream.

    rows (..., dim): the gradient of what was looked up; grad (vocab, dim): of the
    matrix (of tokens or of positions); each float32, bfloat16 or float16, with
    contiguous rows at one stride. tokens (...): int32 or int64; those outside
    [0, vocab) add nothing. Each token's rows are added up in float32 and rounded
    once to grad's type."""
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    r, rs = _matrix(rows, "rows", dev, _TYPES)
    g, gs = _table(grad, "grad", dev, _TYPES, r.shape[1])
    t = _packed(tokens, "tokens", dev, _INDEX_TYPES, rows.shape[:-1])
    count, (vocab, dim) = r.shape[0], g.shape
    need = lib().rcs_embed_workspace(count, vocab, dim)
    _check(int(need) if need < 0 else 0, "rcs_embed_workspace")
    with _stream_context(stream):
        work = torch.empty(need, dtype=torch.uint8, device=g.device)
        _check(lib().embed_grad(r.data_ptr(), rs, _TYPES[r.dtype], count, t.data_ptr(),
                                _INDEX_TYPES[t.dtype], g.data_ptr(), gs, _TYPES[g.dtype], vocab,
                                dim, float(scale), work.data_ptr(), need, _stream(stream)),
               "embed_grad")
