"""The sampler's 4-bit replica of its bf16 snapshots, in MXFP4 (blocks of 32
values along the last dimension, one power of two per block, E2M1 elements).

  mxfp4_quantize(t) / mxfp4_quantize_many(ts)      -- the replica
  mxfp4_dequantize(q) / mxfp4_dequantize_many(qs)  -- the values it stands for
  mxfp4_apply_many_(snaps, quants, idx, val, offsets)
                       -- apply_many_ and the replica's update in one pass
  mxfp4_matmul(x, w)   -- Q(x) Q(w)^T: the product that a sampler makes of it
  Mxfp4Plan(snaps)     -- replica and deltas of a fixed list, every sync

Only blocks that a delta touches are quantised again, so a replica follows a
sparse sync at a fraction of what making it costs.  Every call may be captured
into a graph.
"""
from __future__ import annotations

import ctypes
import math
from typing import Sequence

import torch

from ._abi import check, load
from .grads import _DTYPES, _grad, _stream
from .ops import _bits, _device, _raise_on_violations, _violations

BLOCK = 32


def _row_shape(shape):
    """(rows, cols) of a tensor: everything but the last dimension, and that."""
    shape = tuple(int(s) for s in shape)
    if not shape:
        raise ValueError("a tensor without dimensions has no rows to cut into blocks")
    return math.prod(shape[:-1]), shape[-1]


def _blocks(cols: int) -> int:
    return (cols + BLOCK - 1) // BLOCK


class Mxfp4:
    """A tensor in MXFP4: `codes` uint8 [..., 16 * ceil(cols / 32)] (two
    elements to a byte, the even one in the low half), `scales` uint8
    [..., ceil(cols / 32)] (byte e is 2^(e - 127), 255 is NaN), and the
    logical `shape`."""

    __slots__ = ("codes", "scales", "shape", "rows", "cols")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, shape):
        self.shape = tuple(int(s) for s in shape)
        self.rows, self.cols = _row_shape(self.shape)
        n = self.rows * _blocks(self.cols)
        for t, want, what in ((codes, 16 * n, "codes"), (scales, n, "scales")):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or not t.is_contiguous():
                raise ValueError(f"{what}: expected a contiguous uint8 tensor")
            if t.numel() != want:
                raise ValueError(f"{what}: {t.numel()} bytes, a tensor of shape {self.shape} has "
                                 f"{want}")
        if codes.device != scales.device:
            raise ValueError("codes and scales on different devices")
        self.codes, self.scales = codes, scales

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def numel(self) -> int:
        return self.rows * self.cols

    def __repr__(self):
        return f"Mxfp4(shape={self.shape}, device={self.device})"


def mxfp4_empty(shape, device) -> Mxfp4:
    """An uninitialised replica of a tensor of `shape`."""
    _, cols = _row_shape(shape)
    lead, b = tuple(shape[:-1]), _blocks(cols)
    return Mxfp4(torch.empty(lead + (16 * b,), dtype=torch.uint8, device=device),
                 torch.empty(lead + (b,), dtype=torch.uint8, device=device), shape)


class _List:
    """The host arrays of a checked list of tensors and their replicas."""

    def __init__(self, tensors, quants, bf16_only=False):
        if not tensors:
            raise ValueError("empty parameter list")
        if len(tensors) != len(quants):
            raise ValueError("the lists of tensors and replicas differ in length")
        dev = tensors[0].device if isinstance(tensors[0], torch.Tensor) else None
        for p, (t, q) in enumerate(zip(tensors, quants)):
            _grad(t, f"tensors[{p}]")
            if bf16_only and t.dtype != torch.bfloat16:
                raise ValueError(f"tensors[{p}]: a replica follows bfloat16 snapshots, got {t.dtype}")
            if not isinstance(q, Mxfp4):
                raise TypeError(f"replica {p}: expected an Mxfp4, got {type(q).__name__}")
            if _row_shape(t.shape) != (q.rows, q.cols):
                raise ValueError(f"replica {p} has shape {q.shape}, its tensor {tuple(t.shape)}")
            if t.device != dev or q.device != dev:
                raise ValueError(f"parameter {p} on another device")
        self.device, self.nparams = dev, len(tensors)
        k = self.nparams
        self.keep = (list(tensors), list(quants))
        self.xs = (ctypes.c_void_p * k)(*[t.data_ptr() for t in tensors])
        self.dtypes = (ctypes.c_int32 * k)(*[_DTYPES[t.dtype] for t in tensors])
        self.rows = (ctypes.c_int64 * k)(*[q.rows for q in quants])
        self.cols = (ctypes.c_int64 * k)(*[q.cols for q in quants])
        self.codes = (ctypes.c_void_p * k)(*[q.codes.data_ptr() for q in quants])
        self.scales = (ctypes.c_void_p * k)(*[q.scales.data_ptr() for q in quants])
        self.ws_bytes = load().mxfp4_workspace_size(k)

    def workspace(self):
        # not shared between calls: a captured call keeps its own
        return torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)

    def store(self, ws):
        check(load().mxfp4_list_store(self.nparams, self.xs, self.dtypes, self.rows, self.cols,
                                      self.codes, self.scales, ws.data_ptr(), self.ws_bytes,
                                      _stream(self.device)))

    def quantize(self, ws, stored):
        with _device(self.device):  # the library works on the current device
            check(load().mxfp4_quantize_many(self.nparams, self.xs, self.dtypes, self.rows,
                                             self.cols, self.codes, self.scales, ws.data_ptr(),
                                             self.ws_bytes, stored, _stream(self.device)))

    def dequantize(self, xs, dtypes, ws):
        with _device(self.device):
            check(load().mxfp4_dequantize_many(self.nparams, self.codes, self.scales, self.rows,
                                               self.cols, xs, dtypes, ws.data_ptr(),
                                               self.ws_bytes, _stream(self.device)))

    def apply(self, idx, val, offsets, max_nnz, violations, ws, stored):
        dev = self.device
        if (not isinstance(idx, torch.Tensor) or idx.dtype != torch.int32 or idx.device != dev
                or not idx.is_contiguous()):
            raise ValueError("idx must be a contiguous int32 tensor on the snapshots' device")
        _bits(val, "val")
        if val.numel() != idx.numel() or val.device != dev:
            raise ValueError("idx and val must have equal length on the snapshots' device")
        if (not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int64
                or offsets.numel() != self.nparams + 1 or offsets.device != dev
                or not offsets.is_contiguous()):
            raise ValueError("offsets must be a contiguous int64[nparams+1] on the snapshots' "
                             "device")
        if violations is not None and (violations.dtype != torch.int64 or
                                       violations.device != dev):
            raise ValueError("violations must be an int64 tensor on the snapshots' device")
        # the kernels never read past the buffers
        m = idx.numel() if max_nnz is None else min(int(max_nnz), idx.numel())
        with _device(dev):
            check(load().mxfp4_apply_many(
                self.nparams, self.xs, self.rows, self.cols, self.codes, self.scales,
                idx.data_ptr(), val.data_ptr(), offsets.data_ptr(), m,
                None if violations is None else violations.data_ptr(), ws.data_ptr(),
                self.ws_bytes, stored, _stream(dev)))


def mxfp4_quantize_many(tensors: Sequence[torch.Tensor],
                        outs: Sequence[Mxfp4] | None = None) -> list[Mxfp4]:
    """The replicas of a list of bfloat16, float16 or float32 tensors, new or
    written into `outs`."""
    tensors = list(tensors)
    for p, t in enumerate(tensors):
        _grad(t, f"tensors[{p}]")
    outs = [mxfp4_empty(t.shape, t.device) for t in tensors] if outs is None else list(outs)
    lst = _List(tensors, outs)
    lst.quantize(lst.workspace(), 0)
    return outs


def mxfp4_quantize(t: torch.Tensor, out: Mxfp4 | None = None) -> Mxfp4:
    """One tensor's replica."""
    _grad(t, "t")
    out = mxfp4_empty(t.shape, t.device) if out is None else out
    lst = _List([t], [out])
    lst.quantize(lst.workspace(), 0)
    return out


def _check_quants(quants):
    for p, q in enumerate(quants):
        if not isinstance(q, Mxfp4):
            raise TypeError(f"replica {p}: expected an Mxfp4, got {type(q).__name__}")
        if q.device.type != "cuda":
            raise ValueError(f"replica {p}: must be on a GPU, got {q.device}")
    if not quants:
        raise ValueError("empty parameter list")


def _new_values(quants, dtype):
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}; expected bfloat16, float16 or float32")
    return [torch.empty(q.shape, dtype=dtype, device=q.device) for q in quants]


def mxfp4_dequantize_many(quants: Sequence[Mxfp4], outs: Sequence[torch.Tensor] | None = None,
                          dtype: torch.dtype = torch.bfloat16) -> list[torch.Tensor]:
    """The values that replicas stand for, as new tensors of `dtype` or
    written into `outs` (of their own types).  Exact in bfloat16 and float32."""
    quants = list(quants)
    _check_quants(quants)
    outs = _new_values(quants, dtype) if outs is None else list(outs)
    lst = _List(outs, quants)
    lst.dequantize(lst.xs, lst.dtypes, lst.workspace())
    return outs


def mxfp4_dequantize(q: Mxfp4, dtype: torch.dtype = torch.bfloat16,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that one replica stands for."""
    return mxfp4_dequantize_many([q], None if out is None else [out], dtype)[0]


def mxfp4_apply_many_(snaps: Sequence[torch.Tensor], quants: Sequence[Mxfp4], idx: torch.Tensor,
                      val: torch.Tensor, offsets: torch.Tensor, max_nnz: int | None = None,
                      check_indices=False):
    """apply_many_ on the bf16 snapshots, and in the same pass every block that
    the delta touches quantised again, so that `quants` is the replica of the
    updated snapshots (it must be that of the snapshots before).  Returns
    (snaps, quants)."""
    snaps, quants = list(snaps), list(quants)
    lst = _List(snaps, quants, bf16_only=True)
    v = _violations(lst.device, check_indices)
    lst.apply(idx, val, offsets, max_nnz, v, lst.workspace(), 0)
    _raise_on_violations(v)
    return snaps, quants


def _no_graph(t, what: str):
    if isinstance(t, torch.Tensor) and t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} requires a gradient, and mxfp4_matmul has none: detach it, or "
                         "call under torch.no_grad()")


def mxfp4_matmul(x: torch.Tensor | Mxfp4, w: Mxfp4, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """y = Q(x) Q(w)^T with both sides in MXFP4, accumulated in float32 and
    rounded once.  w: a replica of shape [n, k].  x: a contiguous bfloat16,
    float16 or float32 tensor [..., k], quantised in the call exactly as
    mxfp4_quantize does, or an Mxfp4 [..., k].  Returns [..., n] in out_dtype
    (default: x's type, bfloat16 for an Mxfp4), or writes `out`.  A sampler's
    product, without a gradient: an x (or out) that requires one is refused
    where gradients are recorded; detach it, or call under torch.no_grad()."""
    if not isinstance(w, Mxfp4):
        raise TypeError(f"w: expected an Mxfp4, got {type(w).__name__}")
    if len(w.shape) != 2:
        raise ValueError(f"w: expected a replica of shape [n, k], got {w.shape}")
    n, k = w.shape
    given = isinstance(x, Mxfp4)
    _no_graph(x, "x")
    _no_graph(out, "out")
    if not given:
        _grad(x, "x")
        if x.dim() == 0:
            raise ValueError("x: expected at least one dimension")
    shape = x.shape
    if shape[-1] != k:
        raise ValueError(f"x has rows of {shape[-1]} values, w of {k}")
    dev = w.codes.device
    if dev.type != "cuda":
        raise ValueError(f"w: must be on a GPU, got {dev}")
    if x.device != dev:
        raise ValueError("x and w on different devices")
    m = math.prod(shape[:-1])
    if out is None:
        dtype = out_dtype if out_dtype is not None else torch.bfloat16 if given else x.dtype
        if dtype not in _DTYPES:
            raise ValueError(f"unsupported dtype {dtype}; expected bfloat16, float16 or float32")
        out = torch.empty((*shape[:-1], n), dtype=dtype, device=dev)
    else:
        _grad(out, "out")
        dtype = out.dtype
        if (tuple(out.shape) != (*shape[:-1], n) or out.device != dev
                or out_dtype not in (None, dtype)):
            raise ValueError(f"out must be {(*shape[:-1], n)} on {dev}, of out_dtype if that is "
                             "given")
    lib = load()
    with _device(dev):  # the library works on the current device
        # the workspace is not shared between calls: a captured call keeps its own
        size = (lib.mxfp4_matmul_workspace_size if given else
                lib.mxfp4_linear_workspace_size)(m, n, k)
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        work = None if ws is None else ws.data_ptr()
        if given:
            check(lib.mxfp4_matmul(m, n, k, x.codes.data_ptr(), x.scales.data_ptr(),
                                   w.codes.data_ptr(), w.scales.data_ptr(), out.data_ptr(),
                                   _DTYPES[dtype], work, size, _stream(dev)))
        else:
            check(lib.mxfp4_linear(m, n, k, x.data_ptr(), _DTYPES[x.dtype], w.codes.data_ptr(),
                                   w.scales.data_ptr(), out.data_ptr(), _DTYPES[dtype], work,
                                   size, _stream(dev)))
    return out


class Mxfp4Plan:
    """A sampler's fixed list: the resident bf16 snapshots and their replica,
    `quants`, with the tables of both sides built once, outside any capture.
    The runs of one plan share them, so they must follow one another (on one stream, or ordered by
    events)."""

    def __init__(self, snaps: Sequence[torch.Tensor], quants: Sequence[Mxfp4] | None = None):
        """quants: an existing replica of `snaps`; without one, the plan's is
        undefined until the first quantize().  No tensor may appear twice."""
        snaps = list(snaps)
        for p, t in enumerate(snaps):
            _grad(t, f"snaps[{p}]")
        self.quants = ([mxfp4_empty(t.shape, t.device) for t in snaps] if quants is None
                       else list(quants))
        self._list = _List(snaps, self.quants)
        self.device, self.nparams = self._list.device, self._list.nparams
        self._bf16 = all(t.dtype == torch.bfloat16 for t in snaps)
        self._shapes = [(q.cols, q.numel()) for q in self.quants]
        with torch.cuda.device(self.device):
            self.ws = self._list.workspace()
            self._out_ws = self._list.workspace()  # dequantize()'s table
            self._list.store(self.ws)
            # runs may come on any stream
            torch.cuda.current_stream(self.device).synchronize()

    def quantize(self) -> list[Mxfp4]:
        """Enqueue making the whole replica from the snapshots."""
        self._list.quantize(self.ws, 1)
        return self.quants

    def apply(self, idx: torch.Tensor, val: torch.Tensor, offsets: torch.Tensor,
              max_nnz: int | None = None, violations: torch.Tensor | None = None):
        """Enqueue applying a diff_many-layout delta to the snapshots and the
        replica; returns without syncing.  As in ApplyPlan.run, entries j <
        min(offsets[nparams], max_nnz) are applied, and the true count as
        max_nnz (where idx is a larger buffer) picks the right kernel."""
        if not self._bf16:
            raise ValueError("a replica follows deltas of bfloat16 snapshots only")
        self._list.apply(idx, val, offsets, max_nnz, violations, self.ws, 1)
        return self.quants

    def dequantize(self, outs: Sequence[torch.Tensor] | None = None,
                   dtype: torch.dtype = torch.bfloat16) -> list[torch.Tensor]:
        """Enqueue writing the replica's values (see mxfp4_dequantize_many)."""
        outs = _new_values(self.quants, dtype) if outs is None else list(outs)
        if len(outs) != self.nparams:
            raise ValueError("the lists of tensors and replicas differ in length")
        dev, xs, dtypes = self.device, [], []
        for p, (t, (cols, numel)) in enumerate(zip(outs, self._shapes)):
            if (not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES or t.device != dev
                    or not t.is_contiguous() or t.numel() != numel or t.dim() == 0
                    or t.shape[-1] != cols):
                # the long way, which says what is wrong
                _List(outs, self.quants)
                raise ValueError(f"tensors[{p}] does not fit its replica")
            xs.append(t.data_ptr())
            dtypes.append(_DTYPES[t.dtype])
        k = self.nparams
        self._list.dequantize((ctypes.c_void_p * k)(*xs), (ctypes.c_int32 * k)(*dtypes),
                              self._out_ws)
        return outs
