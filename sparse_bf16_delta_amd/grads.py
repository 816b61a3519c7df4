"""The gradients of a parameter list before the optimizer step: their global
norm, and clipping by it (the trainer side of a sync, just before the step
whose two snapshots diff_many compares).

  grad_norm(grads)                 -- the norm of all tensors together
  clip_grads_(grads, max_norm)     -- times min(1, max_norm / (norm + 1e-6))
  grad_total(grads)                -- what ranks holding shards add up first
  ClipPlan(grads)                  -- the same, every step, for gradients that
                                      stay in their tensors

Gradients are bfloat16, float16 or float32, mixed freely, each contiguous and
all on one device; the norm is a float32 scalar on that device, and nothing is
read back unless asked.  No call records an autograd graph, and every call may
be captured into a HIP graph.
"""
from __future__ import annotations

import ctypes
import math
from typing import Sequence

import torch

from ._abi import (DELTA_BF16, DELTA_FP16, DELTA_FP32, DELTA_NORM_2, DELTA_NORM_INF, DeltaError,
                   check, load)
from .ops import _device

_DTYPES = {torch.bfloat16: DELTA_BF16, torch.float16: DELTA_FP16, torch.float32: DELTA_FP32}


def _stream(device: torch.device) -> int:
    """The current stream's handle: 0.1 us, where current_stream(device), which
    builds an object for it, takes 2 us of a small call's 10."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _kind(norm_type) -> int:
    norm_type = float(norm_type)
    if norm_type == 2.0:
        return DELTA_NORM_2
    if norm_type == math.inf:
        return DELTA_NORM_INF
    raise ValueError(f"norm_type {norm_type}: expected 2 or infinity")


def _max_norm(max_norm) -> float:
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"max_norm {max_norm}: expected a number >= 0")
    return max_norm


def _grad(t, what: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{what}: unsupported dtype {t.dtype}; expected bfloat16, float16 or "
                         "float32")
    if t.device.type != "cuda":
        raise ValueError(f"{what}: must be on a GPU, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    return t


class _List:
    """The host arrays of a checked list."""

    def __init__(self, grads, outs=None):
        grads = list(grads)
        if not grads:
            raise ValueError("empty gradient list")
        for p, g in enumerate(grads):
            _grad(g, f"grads[{p}]")
            if g.device != grads[0].device:
                raise ValueError(f"grads[{p}] on another device")
        if outs is not None:
            outs = list(outs)
            if len(outs) != len(grads):
                raise ValueError("outs and grads differ in length")
            for p, (o, g) in enumerate(zip(outs, grads)):
                _grad(o, f"outs[{p}]")
                if o.dtype != g.dtype or o.numel() != g.numel() or o.device != g.device:
                    raise ValueError(f"outs[{p}] must match grads[{p}] in dtype, numel and device")
        self.grads, self.outs, self.device = grads, outs, grads[0].device
        self.nparams = k = len(grads)
        self.gptrs = (ctypes.c_void_p * k)(*[g.data_ptr() for g in grads])
        self.optrs = None if outs is None else (ctypes.c_void_p * k)(*[o.data_ptr() for o in outs])
        self.nums = (ctypes.c_int64 * k)(*[g.numel() for g in grads])
        self.dtypes = (ctypes.c_int32 * k)(*[_DTYPES[g.dtype] for g in grads])
        self.ws_bytes = load().grad_workspace_size(k)

    def workspace(self):
        # not shared between calls: a captured call keeps its own
        return torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)

    def store(self, ws):
        check(load().grad_list_store(self.nparams, self.gptrs, self.optrs, self.nums, self.dtypes,
                                     ws.data_ptr(), self.ws_bytes, _stream(self.device)))

    def norm(self, kind, total, norm, ws, stored):
        with _device(self.device):  # the library works on the current device
            check(load().grad_norm_many(self.nparams, self.gptrs, self.nums, self.dtypes, kind,
                                        None if total is None else total.data_ptr(),
                                        None if norm is None else norm.data_ptr(), ws.data_ptr(),
                                        self.ws_bytes, stored, _stream(self.device)))

    def clip(self, kind, total, max_norm, norm, ws, stored):
        with _device(self.device):
            check(load().grad_clip_many(self.nparams, self.gptrs, self.optrs, self.nums,
                                        self.dtypes, kind,
                                        None if total is None else total.data_ptr(), max_norm,
                                        norm.data_ptr(), ws.data_ptr(), self.ws_bytes, stored,
                                        _stream(self.device)))


def _given_total(total, device):
    if total is None:
        return None
    if (not isinstance(total, torch.Tensor) or total.dtype != torch.float64 or total.numel() != 1
            or total.device != device):
        raise ValueError("total must be one float64 value on the gradients' device")
    return total


# from here on a number is infinite in float32 (half a step above the largest)
_FLOAT32_END = 2.0 ** 128 - 2.0 ** 103


def _raise_if_nonfinite(total, kind):
    """Whether the norm of `total` is, in float32: a sum of squares can be
    finite in float64 where its root is not."""
    norm = total.item()
    if kind == DELTA_NORM_2:
        norm = math.sqrt(norm) if norm >= 0.0 else math.nan
    if not abs(norm) < _FLOAT32_END:
        raise DeltaError(1, f"the gradients' norm is {norm}")


def grad_norm(grads: Sequence[torch.Tensor], norm_type: float = 2.0) -> torch.Tensor:
    """The norm (2 or infinity) of all gradients together, as a float32 scalar
    tensor.  A NaN among them makes it NaN, an infinity infinite."""
    kind = _kind(norm_type)
    lst = _List(grads)
    norm = torch.empty((), dtype=torch.float32, device=lst.device)
    lst.norm(kind, None, norm, lst.workspace(), 0)
    return norm


def grad_total(grads: Sequence[torch.Tensor], norm_type: float = 2.0) -> torch.Tensor:
    """This rank's part of a norm over several ranks' shards, as a float64
    scalar tensor: the sum of squares (all-reduce it with SUM), or for the
    infinity norm the largest magnitude (MAX).  Then clip_grads_(...,
    total=...) clips every rank's shards by the same factor."""
    kind = _kind(norm_type)
    lst = _List(grads)
    total = torch.empty((), dtype=torch.float64, device=lst.device)
    lst.norm(kind, total, None, lst.workspace(), 0)
    return total


def clip_grads_(grads: Sequence[torch.Tensor], max_norm: float, norm_type: float = 2.0,
                outs: Sequence[torch.Tensor] | None = None, total: torch.Tensor | None = None,
                error_if_nonfinite=False) -> torch.Tensor:
    """Multiplies every gradient by min(1, max_norm / (norm + 1e-6)), in place
    or into `outs`, and returns the norm before clipping (a float32 scalar
    tensor).  total: a grad_total result to clip by instead of this list's.
    error_if_nonfinite: waits for the norm, and raises before anything is
    written when it is infinite or NaN; without it such a norm gives a factor
    of 0 or NaN, and the caller skips the step."""
    kind, max_norm = _kind(norm_type), _max_norm(max_norm)
    lst = _List(grads, outs)
    total = _given_total(total, lst.device)
    norm = torch.empty((), dtype=torch.float32, device=lst.device)
    ws = lst.workspace()
    if error_if_nonfinite:
        if total is None:
            total = torch.empty((), dtype=torch.float64, device=lst.device)
            lst.norm(kind, total, None, ws, 0)
        _raise_if_nonfinite(total, kind)
    lst.clip(kind, total, max_norm, norm, ws, 0)
    return norm


class ClipPlan:
    """grad_norm and clip_grads_ over a fixed list: the table, the partial
    results and the norm are allocated once, outside any capture.  The runs of one plan share them,
    so they must follow one another (on one stream, or ordered by events);
    what a run returns is the plan's own scalar, and the next run overwrites
    it.

    The plan is made for these tensors: it keeps them alive and works at their
    addresses.  A step that makes new gradient tensors leaves it with the old
    ones, and torch's zero_grad() does so unless it is called with
    set_to_none=False (or the gradients live in buffers of the trainer's own).
    Pass the step's gradients as `grads`: others than the plan's are refused, on
    the host, before anything is enqueued."""

    def __init__(self, grads: Sequence[torch.Tensor],
                 outs: Sequence[torch.Tensor] | None = None, norm_type: float = 2.0):
        self._kind = _kind(norm_type)
        self._list = _List(grads, outs)
        lst = self._list
        self.device, self.nparams = lst.device, lst.nparams
        self._what = [(g.data_ptr(), g.numel(), g.dtype) for g in lst.grads]
        with torch.cuda.device(self.device):
            self.ws = lst.workspace()
            self._norm = torch.empty((), dtype=torch.float32, device=self.device)
            self._total = torch.empty((), dtype=torch.float64, device=self.device)
            lst.store(self.ws)
            # runs may come on any stream
            torch.cuda.current_stream(self.device).synchronize()

    def _same(self, grads):
        """Refuses gradients that are not where the plan's are."""
        if grads is None:
            return
        grads = list(grads)
        if len(grads) != self.nparams:
            raise ValueError(f"{len(grads)} gradients, the plan was made for {self.nparams}")
        for p, (g, want) in enumerate(zip(grads, self._what)):
            if (not isinstance(g, torch.Tensor) or not g.is_contiguous()
                    or (g.data_ptr(), g.numel(), g.dtype) != want):
                raise ValueError(f"grads[{p}] is not the tensor that the plan was made for: keep "
                                 "the gradients (zero_grad(set_to_none=False)), or make a new "
                                 "plan")

    def norm(self, grads: Sequence[torch.Tensor] | None = None) -> torch.Tensor:
        """Enqueue the norm alone; nothing is written to the gradients."""
        self._same(grads)
        self._list.norm(self._kind, None, self._norm, self.ws, 1)
        return self._norm

    def total(self, grads: Sequence[torch.Tensor] | None = None) -> torch.Tensor:
        """Enqueue this rank's part of a norm over ranks (see grad_total)."""
        self._same(grads)
        self._list.norm(self._kind, self._total, None, self.ws, 1)
        return self._total

    def run(self, max_norm: float, total: torch.Tensor | None = None,
            grads: Sequence[torch.Tensor] | None = None) -> torch.Tensor:
        """Enqueue the clip; returns the norm before it without syncing.  grads:
        this step's, which must be the plan's."""
        self._same(grads)
        self._list.clip(self._kind, _given_total(total, self.device), _max_norm(max_norm),
                        self._norm, self.ws, 1)
        return self._norm
