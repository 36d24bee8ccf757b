"""Operators over tables of gradient tensors (the zero_tensor_* calls of
``include/zero_shard.h``): a plan built once over a list of tensors, then their
norm, clipping and accumulation.

    acc = zero_tensor_plan(grads, out=accumulators)     # 16-bit -> fp32
    zero_tensor_accumulate(acc, overwrite=True)         # first micro-batch
    ...
    zero_tensor_accumulate(acc, res=res, workspace=ws)  # last one, with the norm
    bucket = zero_tensor_plan(accumulators, out=pieces_of_a_flat_buffer)
    zero_tensor_clip(bucket, 1.0, res)                  # clipped, unscaled, 16-bit

(zero_adamw_step unscales and clips by its own result: give it one with inv_scale 1 and
no max_grad_norm after that clip, or leave the clip to it and cast the accumulators with
a result that has inv_scale 1 and max_norm 0.)

Calls are asynchronous on the current stream of the plan's device (or
``stream``), allocate nothing and can be captured in a graph (build the plan
before the capture and keep it, and the tensors' memory, for as long as the
graph is replayed).  A plan holds addresses: where gradients are allocated anew
(``zero_grad(set_to_none=True)``), build a new one.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import numpy as np

from . import (RESULT_BYTES, ZERO_BF16, ZERO_FP16, ZERO_FP32, ZERO_NORM_L2, ZERO_NORM_MAX, ZERO_OK,
               _check, _ctl, _lib)

_ENTRY = np.dtype([("src", np.uint64), ("dst", np.uint64), ("numel", np.int64),
                   ("src_dtype", np.int32), ("dst_dtype", np.int32)])
_KINDS = {"l2": ZERO_NORM_L2, "max": ZERO_NORM_MAX}


class zero_tensor_plan_t(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int64), ("numel", ctypes.c_int64),
                ("bytes", ctypes.c_int64), ("n_pieces", ctypes.c_int64),
                ("n_runs", ctypes.c_int64), ("n_rests", ctypes.c_int64),
                ("head_bytes", ctypes.c_int64), ("table_bytes", ctypes.c_int64),
                ("writable", ctypes.c_int32), ("fp32_out", ctypes.c_int32),
                ("even16", ctypes.c_int32), ("largest", ctypes.c_int32)]


def _order(t):
    """The strides of a tensor whose elements fill its memory, dimensions of
    one element left out (None: contiguous); raises where there are gaps or
    overlaps."""
    if t.is_contiguous():
        return None
    dims = [(st, n) for st, n in zip(t.stride(), t.shape) if n != 1]
    at = 1
    for st, n in sorted(dims):
        if st != at:
            raise ValueError("tensors must be dense: their elements fill their memory in some "
                             "order of the dimensions")
        at *= n
    return tuple(st for st, _ in dims)


class zero_tensor_plan:
    """The plan and device table of a list of tensors.

    tensors   device tensors of one device, each torch.float32, float16 or
              bfloat16 and dense (contiguous, or a permutation of the dimensions
              of a contiguous tensor); empty ones are allowed
    out       where the calls that write put their results: one tensor for each,
              of as many elements and the same order in memory, of any of the
              types; None: the tensors themselves
    device    the table's device (by default the tensors'; needed for an empty
              list)

    The plan keeps the tensors.  A plan over tensors that overlap can be read only:
    the calls that write raise ZeroError.  Building one waits for the current stream.

    Calls do not tell torch's allocator what they use on which stream: where a call
    runs on another stream than a tensor's own, keep the plan, and the call's res,
    norms, workspace and ctl, until that call is done.
    """

    def __init__(self, tensors: Sequence, out: Optional[Sequence] = None, device=None):
        import torch
        types = {torch.float32: ZERO_FP32, torch.float16: ZERO_FP16, torch.bfloat16: ZERO_BF16}
        tensors = list(tensors)
        outs = tensors if out is None else list(out)
        n = len(tensors)
        if len(outs) != n:
            raise ValueError("out: one tensor for each tensor")
        if not all(isinstance(t, torch.Tensor) for t in tensors + ([] if out is None else outs)):
            raise TypeError("tensors expected (leave parameters without a gradient out of the list)")
        if device is None:
            device = tensors[0].device if tensors else "cuda"
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("device tensors expected")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        # neither in a capture on the plan's device, whose stream it works on and waits
        # for, nor in one on the current device, which an allocation may break
        capturing = torch.cuda.is_current_stream_capturing()
        with torch.cuda.device(device):
            if capturing or torch.cuda.is_current_stream_capturing():
                raise RuntimeError("build the plan before the capture")
        # a pass per property: lists of thousands of tensors are common
        sides = []
        for side in ((tensors,) if out is None else (tensors, outs)):
            if any(t.layout is not torch.strided or t.is_neg() for t in side):
                raise ValueError("tensors must be strided (not sparse) and hold their own values "
                                 "(no negated views)")
            if any(t.get_device() != device.index for t in side):
                raise ValueError(f"tensors on {device} expected")
            codes = [types.get(t.dtype) for t in side]
            if None in codes:
                bad = side[codes.index(None)].dtype
                raise TypeError(f"float32, float16 or bfloat16 tensors expected, got {bad}")
            sides.append(([t.data_ptr() for t in side], [t.numel() for t in side], codes,
                          [None if t.is_contiguous() else _order(t) for t in side]))
        _, numels, _, orders = sides[0]
        if sides[-1][1] != numels or sides[-1][3] != orders or \
                any(o is not None and t.shape != y.shape for o, t, y in zip(orders, tensors, outs)):
            raise ValueError("out: as many elements as the tensor, in the same order")
        entries = np.zeros(max(1, n), dtype=_ENTRY)
        if n:
            entries["src"], entries["numel"], entries["src_dtype"] = sides[0][:3]
            entries["dst"], entries["dst_dtype"] = sides[-1][0], sides[-1][2]
        self.c = zero_tensor_plan_t()
        _check(_lib.zero_tensor_plan_init(entries.ctypes.data, n, ctypes.byref(self.c)),
               "zero_tensor_plan_init")
        head = np.empty(self.c.head_bytes, dtype=np.uint8)
        _check(_lib.zero_tensor_plan_head(entries.ctypes.data, ctypes.byref(self.c),
                                          head.ctypes.data), "zero_tensor_plan_head")
        self.tensors, self.out, self.device, self._index = tensors, outs, device, device.index
        self.n_tensors, self.numel = n, self.c.numel
        self.workspace_bytes = int(_lib.zero_tensor_workspace_bytes(ctypes.byref(self.c)))
        with torch.cuda.device(device):
            stream = torch.cuda.current_stream(device)
            self.table = torch.empty(self.c.table_bytes, dtype=torch.uint8, device=device)
            self.table[:self.c.head_bytes].copy_(torch.from_numpy(head))
            self._args = (ctypes.byref(self.c), self.table.data_ptr())
            _check(_lib.zero_tensor_plan_expand(*self._args, stream.cuda_stream),
                   "zero_tensor_plan_expand")
            # complete before any stream's calls; the calls then need no events
            stream.synchronize()
            self._streams = {stream.cuda_stream}

    def _call(self, fn, args, stream) -> None:
        """fn(plan, table, *args, stream) with the plan's device current."""
        import torch
        if stream is None:
            # torch.cuda.current_stream(device).cuda_stream without the object (1.9 us
            # of a call's 7)
            raw = torch._C._cuda_getCurrentRawStream(self._index)
        elif isinstance(stream, int):
            raw = stream
        else:
            if stream.device != self.device:
                raise ValueError(f"a stream of {self.device} expected")
            raw = stream.cuda_stream
        if raw not in self._streams:
            self._keep_table(raw, stream)
        if torch._C._cuda_getDevice() == self._index:
            rc = fn(*self._args, *args, raw)
        else:
            with torch.cuda.device(self.device):
                rc = fn(*self._args, *args, raw)
        if rc != ZERO_OK:
            _check(rc, fn.__name__)

    def _keep_table(self, raw: int, stream) -> None:
        """On a call's first use of a stream: the table is the plan's own, so its memory
        stays until that stream is done.  Only for torch's streams, which live for ever:
        the record is used when the table is freed, and a stream of the caller's making
        may have been destroyed by then (and its handle be another stream's)."""
        import torch
        if raw == 0:
            stream = torch.cuda.default_stream(self.device)
        elif stream is None or isinstance(stream, int):
            stream = torch.cuda.current_stream(self.device)
        # a handle that is not the current stream's, or a stream around a handle, whose
        # id the handle is, is the caller's
        if stream.cuda_stream == raw and (raw == 0 or stream.stream_id != raw):
            self.table.record_stream(stream)
            self._streams.add(raw)

    def _buffer(self, t, nbytes: int, name: str) -> int:
        if t.device != self.device:
            raise ValueError(f"{name} must be a tensor on {self.device}")
        ptr = t.data_ptr()
        if t.nbytes < nbytes or ptr % 8 or not t.is_contiguous():
            raise ValueError(f"{name}: {nbytes} contiguous bytes, 8-byte aligned")
        return ptr

    def _norms(self, norms) -> Optional[int]:
        import torch
        if norms is None:
            return None
        if norms.device != self.device or norms.dtype != torch.float32 or \
                not norms.is_contiguous() or norms.numel() < self.n_tensors:
            raise ValueError(f"norms: float32[{self.n_tensors}] on {self.device}, contiguous")
        return norms.data_ptr() or None

    def _norm_args(self, inv_scale, ctl_dev, res, norms):
        """The norm calls' arguments from inv_scale to norms."""
        if ctl_dev is not None and ctl_dev.device != self.device:
            raise ValueError(f"ctl must be a tensor on {self.device}")
        return (float(inv_scale), None if ctl_dev is None else _ctl(ctl_dev),
                self._buffer(res, RESULT_BYTES, "res"), self._norms(norms))

    def _workspace(self, workspace):
        return self._buffer(workspace, self.workspace_bytes, "workspace"), workspace.nbytes


def _kind(kind) -> int:
    code = _KINDS.get(kind)
    if code is None:
        raise ValueError(f"kind: one of {sorted(_KINDS)}")
    return code


def zero_tensor_workspace_bytes(plan: zero_tensor_plan) -> int:
    return plan.workspace_bytes


def zero_tensor_norm(plan: zero_tensor_plan, inv_scale: float, res, workspace, kind: str = "l2",
                     norms=None, accumulate: bool = False, ctl_dev=None, stream=None) -> None:
    """res: one zero_step_result (16 bytes); norms: float32[n_tensors] for each
    tensor's own norm, or None; kind: 'l2' or 'max'."""
    plan._call(_lib.zero_tensor_norm,
               (_kind(kind), *plan._norm_args(inv_scale, ctl_dev, res, norms),
                *plan._workspace(workspace), int(bool(accumulate))), stream)


def zero_tensor_clip(plan: zero_tensor_plan, max_norm: float, res, norms=None,
                     stream=None) -> None:
    """By the norm in res, or with norms each tensor by its own."""
    plan._call(_lib.zero_tensor_clip,
               (float(max_norm), plan._buffer(res, RESULT_BYTES, "res"), plan._norms(norms)),
               stream)


def zero_tensor_clip_norm(plan: zero_tensor_plan, max_norm: float, inv_scale: float, res,
                          workspace, kind: str = "l2", norms=None, per_tensor: bool = False,
                          ctl_dev=None, stream=None) -> None:
    """zero_tensor_norm, then zero_tensor_clip (per_tensor: each tensor by its
    own norm, which norms receives)."""
    if per_tensor and norms is None:
        raise ValueError("per_tensor needs norms")
    inv, ctl, res_p, norms_p = plan._norm_args(inv_scale, ctl_dev, res, norms)
    plan._call(_lib.zero_tensor_clip_norm,
               (_kind(kind), float(max_norm), inv, ctl, res_p, norms_p, int(bool(per_tensor)),
                *plan._workspace(workspace)), stream)


def zero_tensor_accumulate(plan: zero_tensor_plan, weight: float = 1.0, overwrite: bool = False,
                           res=None, workspace=None, inv_scale: float = 1.0, kind: str = "l2",
                           norms=None, accumulate: bool = False, ctl_dev=None,
                           stream=None) -> None:
    """out = out + weight * tensor (overwrite: out = weight * tensor); with res
    and workspace also the norm of out, in the same pass."""
    if res is None:
        if norms is not None or workspace is not None or ctl_dev is not None or accumulate:
            raise ValueError("the norm needs res and workspace")
        plan._call(_lib.zero_tensor_accumulate, (float(weight), int(bool(overwrite))), stream)
        return
    if workspace is None:
        raise ValueError("the norm needs res and workspace")
    plan._call(_lib.zero_tensor_accumulate_norm,
               (float(weight), int(bool(overwrite)), _kind(kind),
                *plan._norm_args(inv_scale, ctl_dev, res, norms),
                *plan._workspace(workspace), int(bool(accumulate))), stream)


def zero_tensor_accumulate_norm(plan: zero_tensor_plan, inv_scale: float, res, workspace,
                                weight: float = 1.0, overwrite: bool = False, **norm_args) -> None:
    """zero_tensor_accumulate with its norm (the C call's name)."""
    zero_tensor_accumulate(plan, weight, overwrite, res=res, workspace=workspace,
                           inv_scale=inv_scale, **norm_args)
