"""The update over a list of tensors: a thin binding of the rcs_list calls.

Argument marshalling only, as in the rest of the package: the norm, the update
and the conversions run in the HIP kernels of csrc/list.inl.
"""
from __future__ import annotations

import ctypes
from collections.abc import Sequence

import torch

from . import _check, _norm_out, _stream, lib

BLOCK = 128  # elements that share a block exponent (RCS_LIST_BLOCK)
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_FLAT_TYPES = (torch.float32, torch.bfloat16)


class _Tensor(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("exps", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("wd", ctypes.c_float), ("w_type", ctypes.c_int32),
                ("g_type", ctypes.c_int32), ("copy_type", ctypes.c_int32)]


def _check_tensor(t, name: str, dev: int, types) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in types or not t.is_contiguous():
        kinds = ", ".join(str(k).removeprefix("torch.") for k in types)
        raise TypeError(f"{name} must be a contiguous tensor of type {kinds}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}; the library works on the current device "
                         f"(cuda:{dev}): use torch.cuda.device(...)")


def _checked(t, name: str, dev: int, types=_TYPES) -> torch.Tensor:
    """A detached alias of t (it keeps the memory alive, whatever becomes of t)."""
    _check_tensor(t, name, dev, types)
    return t.detach()


class AdamWList:
    """Clip and AdamW over many tensors at once, with the state it needs.

    params: the weights, a sequence of contiguous float32, bfloat16 or float16
    tensors (views at any offset are fine; none may overlap another). grads:
    their gradients, of the same shapes and of any of these types; None where a
    tensor has none (it is then left alone; its gradients, once bound, have
    grad_dtype, or the weights' own type). The list works on the memory that
    the tensors have now and keeps it alive.

    state_bits: 32 holds both moments in float32 (the flat tensors m and v, in
    list order); 8 holds them in 8 bits with an exponent for each BLOCK
    elements (m, v and exps, each tensor's part filled up to whole blocks).
    Both start at zero. wd: the weight decay, one number or one a tensor.
    copies: bfloat16 or float16 copies of float32 weights (None where there is
    none), written with every update. seed: of the random bits by which 8-bit
    moments are rounded, which are a function of seed, t and the element's
    place in the list.

    Calls of one list must not overlap on the device. A captured graph that
    holds calls of a list must not be replayed after its close(), which is also
    what becomes of a list that nothing refers to any more.
    """

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor | None],
                 state_bits: int = 32, wd: float | Sequence[float] = 0.0,
                 copies: Sequence[torch.Tensor | None] | None = None, seed: int = 0,
                 grad_dtype: torch.dtype | None = None):
        self._h = None
        params, grads = list(params), list(grads)
        count = len(params)
        if count == 0:
            raise ValueError("the list has no tensors")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits is {state_bits!r}, expected 8 or 32")
        wds = [float(wd)] * count if isinstance(wd, (int, float)) else [float(x) for x in wd]
        copies = [None] * count if copies is None else list(copies)
        for name, x in (("grads", grads), ("wd", wds), ("copies", copies)):
            if len(x) != count:
                raise ValueError(f"{name} has {len(x)} entries, expected {count}")
        dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
        self._params = [_checked(p, f"params[{k}]", dev) for k, p in enumerate(params)]
        if grad_dtype is not None and grad_dtype not in _TYPES:
            raise TypeError(f"grad_dtype is {grad_dtype}")
        self._gtypes = [grad_dtype or p.dtype if g is None else getattr(g, "dtype", None)
                        for p, g in zip(self._params, grads)]
        self._grads = self._checked_grads(grads, dev)
        self._captured: list[list[torch.Tensor | None]] = []  # bound by graphs
        self._copies = []
        for k, (c, p) in enumerate(zip(copies, self._params)):
            if c is not None:
                c = _checked(c, f"copies[{k}]", dev, (torch.bfloat16, torch.float16))
                if p.dtype != torch.float32:
                    raise TypeError(f"copies[{k}] is a copy of {p.dtype} weights")
                if c.shape != p.shape:
                    raise ValueError(f"copies[{k}] has shape {tuple(c.shape)}, expected "
                                     f"{tuple(p.shape)}")
            self._copies.append(c)
        self.state_bits, self.seed = state_bits, int(seed)
        self.n = sum(p.numel() for p in self._params)
        if self.n == 0:
            raise ValueError("the list has no elements")
        where = torch.device("cuda", dev)
        if state_bits == 32:
            self.m = torch.zeros(self.n, device=where)
            self.v = torch.zeros(self.n, device=where)
            self.exps = None
        else:
            blocks = sum(-(-p.numel() // BLOCK) for p in self._params)
            self.m = torch.zeros(blocks * BLOCK, dtype=torch.uint8, device=where)
            self.v = torch.zeros(blocks * BLOCK, dtype=torch.uint8, device=where)
            self.exps = torch.zeros(blocks, 2, dtype=torch.uint8, device=where)
        # the first use may be on another stream than the zeros are written on
        torch.cuda.current_stream().synchronize()
        rows, at = (_Tensor * count)(), 0
        size = 4 if state_bits == 32 else 1
        for k, (p, g, c) in enumerate(zip(self._params, self._grads, self._copies)):
            n = p.numel()
            rows[k] = _Tensor(
                p.data_ptr(), None if g is None else g.data_ptr(), self.m.data_ptr() + size * at,
                self.v.data_ptr() + size * at,
                None if self.exps is None else self.exps.data_ptr() + 2 * (at // BLOCK),
                None if c is None else c.data_ptr(), n, wds[k], _TYPES[p.dtype],
                _TYPES[self._gtypes[k]], 0 if c is None else _TYPES[c.dtype])
            at += n if state_bits == 32 else -(-n // BLOCK) * BLOCK
        h = ctypes.c_void_p()
        _check(lib().rcs_list_create(rows, count, state_bits, ctypes.byref(h)), "rcs_list_create")
        self._h = h
        self._payload: torch.Tensor | None = None

    def _checked_grads(self, grads, dev: int) -> list[torch.Tensor | None]:
        out = []
        for k, (g, p, kind) in enumerate(zip(grads, self._params, self._gtypes)):
            if g is not None:
                g = _checked(g, f"grads[{k}]", dev)
                if g.dtype != kind:
                    raise TypeError(f"grads[{k}] has type {g.dtype}, expected {kind}")
                if g.shape != p.shape:
                    raise ValueError(f"grads[{k}] has shape {tuple(g.shape)}, expected "
                                     f"{tuple(p.shape)}")
            out.append(g)
        return out

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise ValueError("the list is closed")
        return self._h

    def bind_grads(self, grads: Sequence[torch.Tensor | None], stream=None) -> None:
        """Other gradients of the same shapes and types (None: the tensor has
        none), from the stream's next call on. The list lets go of those before:
        keep them while work that uses them is under way on another stream
        than their own. A captured call binds at each replay of its graph, and
        until the first one nothing has changed: the list keeps both the
        gradients from before it and, until close(), those of the graph."""
        h, grads = self.handle, list(grads)
        if len(grads) != len(self._params):
            raise ValueError(f"grads has {len(grads)} entries, expected {len(self._params)}")
        new = self._checked_grads(grads, torch.cuda.current_device())
        ptrs = (ctypes.c_void_p * len(new))(*[None if g is None else g.data_ptr() for g in new])
        s = _stream(stream)
        captured = lib().rcs_stream_capturing(s)
        _check(lib().rcs_list_bind_grads(h, ptrs, len(new), s), "rcs_list_bind_grads")
        if captured:
            self._captured.append(new)
        else:
            self._grads = new

    def step(self, t: int, lr: float, clip: float, grad_scale: float = 1.0, beta1: float = 0.9,
             beta2: float = 0.999, eps: float = 1e-8, norm_out: torch.Tensor | None = None,
             stream=None) -> None:
        """Update t of the whole list in place (asynchronous on stream): one
        global norm of the gradients times grad_scale, one clip factor, AdamW on
        every tensor that has a gradient. norm_out: optional 1-element float64
        device or pinned host tensor that receives the pre-clip norm."""
        np_ = None if norm_out is None else _norm_out(norm_out).data_ptr()
        _check(lib().adamw_clip_step_list(self.handle, int(t), float(lr), float(clip),
                                          float(grad_scale), float(beta1), float(beta2),
                                          float(eps), self.seed & 0xFFFFFFFF, np_,
                                          _stream(stream)), "adamw_clip_step_list")

    def grad_norm(self, out: torch.Tensor | None = None, grad_scale: float = 1.0,
                  stream=None) -> torch.Tensor:
        """Pre-clip global L2 norm of the gradients times grad_scale, into a
        1-element float64 tensor."""
        h, out = self.handle, _norm_out(out)
        _check(lib().grad_global_norm_list(h, float(grad_scale), out.data_ptr(),
                                           _stream(stream)), "grad_global_norm_list")
        return out

    def _flat(self, w, m, v) -> list:
        """Pointer and type of each of three flat arrays (or None)."""
        dev, out = torch.cuda.current_device(), []
        for name, x in (("w", w), ("m", m), ("v", v)):
            if x is None:
                out += (None, 0)
                continue
            _check_tensor(x, name, dev, _FLAT_TYPES)
            if x.numel() != self.n:
                raise ValueError(f"{name} has {x.numel()} elements, expected {self.n}")
            out += (x.data_ptr(), _TYPES[x.dtype])
        return out

    def export_state(self, w=None, m=None, v=None, stream=None) -> None:
        """Writes the weights and moments, in list order, to flat float32 or
        bfloat16 tensors of n elements (None: left out). What 8 bits hold is
        exact in either type."""
        _check(lib().rcs_list_export(self.handle, *self._flat(w, m, v), _stream(stream)),
               "rcs_list_export")

    def import_state(self, w=None, m=None, v=None, stream=None) -> None:
        """Reads them back: weights rounded to their types (copies written
        too), 8-bit moments to the nearest value they can hold (m and v then
        come together)."""
        _check(lib().rcs_list_import(self.handle, *self._flat(w, m, v), _stream(stream)),
               "rcs_list_import")

    def payload_buffer(self) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """Flat float32 w, m and v, the payload of a step file: one allocation
        of 12 bytes an element, made at the first call and kept."""
        if self._payload is None:
            self._payload = torch.empty(3 * self.n, device=self.m.device)
            # the first use may be on another stream than this allocation's
            torch.cuda.current_stream().synchronize()
        w, m, v = self._payload.split(self.n)
        return w, m, v

    def payload(self, stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """The list's state in payload_buffer(), for ckpt_pack or CkptWriter."""
        out = self.payload_buffer()
        self.export_state(*out, stream=stream)
        return out

    def close(self) -> None:
        """Frees the list's description; the tensors stay."""
        if self._h is not None:
            h, self._h = self._h, None
            _check(lib().rcs_list_destroy(h), "rcs_list_destroy")
            self._captured.clear()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
