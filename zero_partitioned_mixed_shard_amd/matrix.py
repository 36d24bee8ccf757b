"""Steps of whole matrices (the zero_orthogonalize and zero_muon_* calls of
``include/zero_shard.h``): orthogonalisation by Newton-Schulz products, and the Muon step
of an owner's matrices.

    plan = zero_matrix_plan(updates, out=results)           # 2-D tensors
    ws = torch.empty(zero_matrix_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    zero_orthogonalize(plan, ws)

    plan = zero_muon_plan([(offset, rows, cols), ...])      # of a flat shard
    zero_muon_step(master, momentum, param16, grad16, plan, zero_muon_hparams(lr=3e-4), res, ws)

Calls are asynchronous on the current stream of the plan's device (or ``stream``),
allocate nothing and can be captured in a graph (build the plan before the capture, and
keep it and what the calls use for as long as the graph is replayed).  They do not tell
torch's allocator what they use on which stream: where a call runs on another stream than
a tensor's own, keep the plan, the tensors and the workspace until it is done.  (Of
a plan that goes before, its own table stays for torch's streams; its tensors need not.)
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import numpy as np

from . import (RESULT_BYTES, ZERO_BF16, ZERO_FP16, ZERO_FP32, ZERO_MUON_ASPECT, ZERO_MUON_NONE,
               ZERO_MUON_RMS, ZERO_OK, _check, _lib, zero_newton_schulz)
from .tensors import _Table

_ENTRY = np.dtype([("src", np.uint64), ("dst", np.uint64), ("rows", np.int64), ("cols", np.int64),
                   ("src_ld", np.int64), ("dst_ld", np.int64), ("src_dtype", np.int32),
                   ("dst_dtype", np.int32)])
_SCALINGS = {None: ZERO_MUON_NONE, "none": ZERO_MUON_NONE, "aspect": ZERO_MUON_ASPECT,
             "rms": ZERO_MUON_RMS}


class zero_matrix_plan_t(ctypes.Structure):
    _fields_ = [("n_matrices", ctypes.c_int64), ("numel", ctypes.c_int64),
                ("extent", ctypes.c_int64), ("table_bytes", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_int64), ("kind", ctypes.c_int32),
                ("precise", ctypes.c_int32)]


class _Plan(_Table):
    """A list of matrices with its table on the host and on the device."""

    def _build(self, list_p, n: int, precise: bool, device, init, table) -> None:
        import torch
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("device tensors expected")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        # neither in a capture on the plan's device, whose stream it waits for, nor in
        # one on the current device, which an allocation may break
        capturing = torch.cuda.is_current_stream_capturing()
        with torch.cuda.device(device):
            if capturing or torch.cuda.is_current_stream_capturing():
                raise RuntimeError("build the plan before the capture")
        self.c = zero_matrix_plan_t()
        _check(init(list_p, n, int(precise), ctypes.byref(self.c)), init.__name__)
        self._host = np.zeros(self.c.table_bytes, dtype=np.uint8)
        _check(table(list_p, ctypes.byref(self.c), self._host.ctypes.data), table.__name__)
        self.device, self.precise = device, bool(precise)
        self.parts = 2 if precise else 1        # fp16 parts of a product's factors
        self.n_matrices, self.numel, self.extent = n, self.c.numel, self.c.extent
        self.workspace_bytes = int(self.c.workspace_bytes)
        with torch.cuda.device(device):
            stream = torch.cuda.current_stream(device)
            self.table = torch.from_numpy(self._host).to(device)
            # complete before any stream's calls; the calls then need no events
            stream.synchronize()
            self._streams = {stream.cuda_stream}
        self._args = (ctypes.byref(self.c), self._host.ctypes.data, self.table.data_ptr())

    def _buffer(self, t, dtypes, count: int, name: str) -> int:
        if t.device != self.device or t.dtype not in dtypes or not t.is_contiguous() or \
                t.is_neg() or t.numel() < count:
            raise ValueError(f"{name}: {count} contiguous elements of {dtypes} on {self.device}")
        return t.data_ptr()

    def _workspace(self, ws):
        if ws.device != self.device or not ws.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {self.device}")
        if ws.nbytes < self.workspace_bytes or (self.workspace_bytes and ws.data_ptr() % 256):
            raise ValueError(f"workspace: {self.workspace_bytes} bytes, 256-byte aligned")
        return ws.data_ptr(), ws.nbytes

    def _call(self, fn, args, stream) -> None:
        """fn(*args, stream) with the plan's device current."""
        import torch
        if stream is None:
            raw = torch.cuda.current_stream(self.device).cuda_stream
        elif isinstance(stream, int):
            raw = stream
        else:
            if stream.device != self.device:
                raise ValueError(f"a stream of {self.device} expected")
            raw = stream.cuda_stream
        if raw not in self._streams:
            self._keep_table(raw, stream)
        with torch.cuda.device(self.device):
            rc = fn(*args, raw)
        if rc != ZERO_OK:
            _check(rc, fn.__name__)


class zero_matrix_plan(_Plan):
    """The plan of a list of matrices.

    tensors   2-D device tensors of one device, torch.float32, float16 or bfloat16, with
              rows or columns of consecutive elements (blocks of rows or columns of a
              larger matrix, and transposes, are fine); empty ones are allowed
    out       where the results go: a tensor of the same shape for each, of any of the
              types; None: the tensors themselves.  A matrix with consecutive rows needs
              a result with consecutive rows, a transposed one a transposed one.
    precise   results to 32 bits, at three times the matrix work; None: where some
              result is float32.  Of float16 results, whose own rounding (2e-4) is finer
              than the faster products' (2e-4 to 1e-3, of low rank more), None takes the
              same products (`parts` is 2 then, `precise` False); False leaves them to
              the faster ones
    device    by default the tensors' (needed for an empty list)

    The plan keeps the tensors and holds their addresses.  Results that overlap each
    other, or another's matrix, raise ZeroError.  Building one waits for the current
    stream.
    """

    def __init__(self, tensors: Sequence, out: Optional[Sequence] = None,
                 precise: Optional[bool] = None, device=None):
        import torch
        types = {torch.float32: ZERO_FP32, torch.float16: ZERO_FP16, torch.bfloat16: ZERO_BF16}
        tensors = list(tensors)
        outs = tensors if out is None else list(out)
        if len(outs) != len(tensors):
            raise ValueError("out: one tensor for each tensor")
        if not all(isinstance(t, torch.Tensor) for t in tensors + outs):
            raise TypeError("tensors expected")
        if device is None:
            device = tensors[0].device if tensors else "cuda"
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        entries = np.zeros(max(1, len(tensors)), dtype=_ENTRY)
        for k, (t, y) in enumerate(zip(tensors, outs)):
            for x in (t, y):
                if x.device != device:
                    raise ValueError(f"tensors on {device} expected")
                if x.layout is not torch.strided or x.is_neg():
                    raise ValueError("tensors must be strided (not sparse) and hold their own "
                                     "values (no negated views)")
                if x.dtype not in types:
                    raise TypeError(f"float32, float16 or bfloat16 tensors expected, got {x.dtype}")
                if x.dim() != 2:
                    raise ValueError("2-D tensors expected")
            if t.shape != y.shape:
                raise ValueError("out: the tensor's shape")
            a, b = _rows(t), _rows(y)
            both = a & b
            if not both:
                raise ValueError("matrices need rows or columns of consecutive elements, the "
                                 "same in tensor and out")
            if "rows" in both:
                rows, cols, lds = t.shape[0], t.shape[1], (t.stride(0), y.stride(0))
            else:       # the transpose's result is the result's transpose
                rows, cols, lds = t.shape[1], t.shape[0], (t.stride(1), y.stride(1))
            if rows <= 1:
                lds = (cols, cols)
            entries[k] = (t.data_ptr(), y.data_ptr(), rows, cols, *lds, types[t.dtype],
                          types[y.dtype])
        two = precise
        if precise is None:
            precise = any(y.dtype == torch.float32 for y in outs)
            two = precise or any(y.dtype == torch.float16 for y in outs)
        self.tensors, self.out = tensors, outs
        self._build(entries.ctypes.data, len(tensors), two, device, _lib.zero_matrix_plan_init,
                    _lib.zero_matrix_plan_table)
        self.precise = bool(precise)


def _rows(t) -> set:
    """What of the matrix is consecutive in memory: its rows, its columns, or both."""
    r, c = t.shape
    if r == 0 or c == 0:
        return {"rows", "cols"}
    found = set()
    if (t.stride(1) == 1 or c == 1) and (t.stride(0) >= c or r == 1):
        found.add("rows")
    if (t.stride(0) == 1 or r == 1) and (t.stride(1) >= r or c == 1):
        found.add("cols")
    return found


class zero_muon_plan(_Plan):
    """The plan of matrices of a flat shard: (offset, rows, cols) of each, as elements of
    the shard's buffers.  precise: zero_matrix_plan's, here by default False (an update
    that is off by 1e-3 of itself, of low rank by a few times that, moves a weight by as
    much of its step)."""

    def __init__(self, matrices: Sequence, precise: bool = False, device="cuda"):
        self.matrices = [(int(o), int(r), int(c)) for o, r, c in matrices]
        ranges = np.array(self.matrices or [(0, 0, 0)], dtype=np.int64)
        self._build(ranges.ctypes.data, len(self.matrices), precise, device,
                    _lib.zero_muon_plan_init, _lib.zero_muon_plan_table)


def zero_matrix_workspace_bytes(plan: _Plan) -> int:
    return plan.workspace_bytes


class zero_muon_hparams(ctypes.Structure):
    """lr, momentum, weight_decay, max_grad_norm (<= 0: no clipping), nesterov, scaling
    ("rms": updates times 0.2 sqrt(max(rows, cols)), as large as AdamW's; "aspect": times
    sqrt(max(1, rows / cols)); None) and the products' coefficients ns."""
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("max_grad_norm", ctypes.c_float),
                ("nesterov", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("ns", zero_newton_schulz)]

    def __init__(self, lr: float = 3e-4, momentum: float = 0.95, weight_decay: float = 0.1,
                 max_grad_norm: float = 0.0, nesterov: bool = True, scaling="rms",
                 ns: Optional[zero_newton_schulz] = None):
        if scaling not in _SCALINGS:
            raise ValueError("scaling: 'rms', 'aspect' or None")
        super().__init__(lr, momentum, weight_decay, max_grad_norm, int(bool(nesterov)),
                         _SCALINGS[scaling], zero_newton_schulz() if ns is None else ns)


def zero_orthogonalize(plan: zero_matrix_plan, workspace, ns: Optional[zero_newton_schulz] = None,
                       stream=None) -> None:
    """out = orth(tensor) for every matrix of the plan."""
    if not isinstance(plan, zero_matrix_plan):
        raise TypeError("a zero_matrix_plan expected")
    ns = zero_newton_schulz() if ns is None else ns
    plan._call(_lib.zero_orthogonalize,
               (*plan._args, ctypes.byref(ns), *plan._workspace(workspace)), stream)


def zero_muon_step(master, momentum, param16, grad16, plan: zero_muon_plan, hp: zero_muon_hparams,
                   res, workspace, stream=None) -> None:
    """The Muon step of the plan's matrices; res as for zero_adamw_step."""
    import torch
    if not isinstance(plan, zero_muon_plan):
        raise TypeError("a zero_muon_plan expected")
    codes = {torch.float16: ZERO_FP16, torch.bfloat16: ZERO_BF16}
    if grad16.dtype not in codes or param16.dtype != grad16.dtype:
        raise TypeError("param16 and grad16 must share a 16-bit type")
    if res.device != plan.device or res.nbytes < RESULT_BYTES or not res.is_contiguous():
        raise ValueError(f"res must be a tensor of at least 16 bytes on {plan.device}")
    n, f32, f16 = plan.extent, (torch.float32,), (grad16.dtype,)
    plan._call(_lib.zero_muon_step,
               (plan._buffer(master, f32, n, "master"), plan._buffer(momentum, f32, n, "momentum"),
                plan._buffer(param16, f16, n, "param16"), plan._buffer(grad16, f16, n, "grad16"),
                codes[grad16.dtype], *plan._args, ctypes.byref(hp), res.data_ptr(),
                *plan._workspace(workspace)), stream)
