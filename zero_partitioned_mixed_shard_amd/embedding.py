"""Rows of the vocabulary table by tokens (the zero_embedding_* calls of
``include/zero_shard.h``): lookup with scaling, and its gradient by sorted tokens.

The table of `vocab` rows of `dim` elements is flat, as the group's buffers hold it, and a
call has a slice of it: elements [begin, begin + numel) (all of it with begin 0).  A
partition cuts through rows; what lies outside the slice gives 0, so the owners' lookups
add up to the whole one, and their gradients lie side by side.

    zero_embedding_lookup(out, ids, param16_slice, vocab, dim, begin=b, scale=s)
    ws = torch.empty(zero_embedding_workspace_bytes(ids.numel(), vocab, dim), dtype=torch.uint8,
                     device="cuda")
    zero_embedding_grad(accumulator_slice, ids, dy, vocab, dim, ws, begin=b, scale=s)

Calls are asynchronous on the current stream of the tensors' device (or ``stream``),
allocate nothing and can be captured in a graph.  They do not tell torch's allocator what
they use on which stream.
"""
from __future__ import annotations

from typing import Optional

from . import ZERO_BF16, ZERO_FP16, ZERO_FP32, ZERO_OK, _check, _lib


def _code(t, name: str) -> int:
    import torch
    codes = {torch.float32: ZERO_FP32, torch.float16: ZERO_FP16, torch.bfloat16: ZERO_BF16}
    if t.dtype not in codes:
        raise TypeError(f"{name}: float32, float16 or bfloat16 expected, got {t.dtype}")
    return codes[t.dtype]


def _ids(ids):
    import torch
    if ids.device.type != "cuda":
        raise ValueError("device tensors expected")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids: int32 or int64 expected, got {ids.dtype}")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    return ids.data_ptr(), ids.element_size(), ids.numel()


def _flat(t, ids, name: str):
    """A contiguous tensor on ids' device: its address, type and elements."""
    if t.device != ids.device or not t.is_contiguous() or t.is_neg():
        raise ValueError(f"{name} must be a contiguous tensor on {ids.device}")
    return t.data_ptr(), _code(t, name), t.numel()


def _token_rows(t, ids, dim: int, name: str):
    """A row of dim consecutive elements for each id: address, distance of rows, type."""
    if t.device != ids.device or t.is_neg():
        raise ValueError(f"{name} must be a tensor on {ids.device}")
    n = ids.numel()
    if tuple(t.shape) not in (tuple(ids.shape) + (dim,), (n, dim)):
        raise ValueError(f"{name}: a row of {dim} elements for each id")
    code = _code(t, name)
    if n == 0 or t.is_contiguous():
        return t.data_ptr(), dim, code
    if t.dim() != 2 or (dim > 1 and t.stride(1) != 1) or (n > 1 and t.stride(0) < dim):
        raise ValueError(f"{name}: rows of consecutive elements that do not overlap")
    return t.data_ptr(), t.stride(0) if n > 1 else dim, code


def _call(fn, args, ids, stream) -> None:
    """fn(*args, stream) with ids' device current."""
    import torch
    if stream is None:
        raw = torch.cuda.current_stream(ids.device).cuda_stream
    elif isinstance(stream, int):
        raw = stream
    else:
        if stream.device != ids.device:
            raise ValueError(f"a stream of {ids.device} expected")
        raw = stream.cuda_stream
    if torch.cuda.current_device() == ids.device.index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(ids.device):
            rc = fn(*args, raw)
    if rc != ZERO_OK:
        _check(rc, fn.__name__)


def zero_embedding_lookup(out, ids, table, vocab: int, dim: int, begin: int = 0,
                          scale: float = 1.0, stream=None) -> None:
    """out[t] = round(scale * W[ids[t]]): 0 where the element lies outside the slice, and
    for ids outside [0, vocab).

    out    a row of dim elements for each id, of any of the types
    ids    int32 or int64, any shape
    table  the slice (contiguous, any shape): its elements are W's from `begin`
    """
    ids_p, id_bytes, n = _ids(ids)
    out_p, out_ld, out_code = _token_rows(out, ids, dim, "out")
    table_p, table_code, count = _flat(table, ids, "table")
    _call(_lib.zero_embedding_lookup,
          (out_p, out_ld, out_code, ids_p, id_bytes, n, table_p, table_code, vocab, dim, begin,
           count, float(scale)), ids, stream)


def zero_embedding_workspace_bytes(n_tokens: int, vocab: int, dim: int) -> int:
    """Bytes for zero_embedding_grad of up to so many tokens (0 for sizes that it refuses)."""
    return int(_lib.zero_embedding_workspace_bytes(n_tokens, vocab, dim))


def zero_embedding_grad(grad, ids, dy, vocab: int, dim: int, workspace, begin: int = 0,
                        scale: float = 1.0, overwrite: bool = False,
                        padding_id: Optional[int] = None, stream=None) -> None:
    """grad = round(grad + scale * sum of dy[t] over the tokens of each row) (overwrite:
    without the old value, and 0 in rows that no token has); ids outside [0, vocab) and
    padding_id give nothing.

    grad  the slice (contiguous, any shape) of the table's gradient, from `begin`
    dy    a row of dim elements for each id, of any of the types
    """
    ids_p, id_bytes, n = _ids(ids)
    dy_p, dy_ld, dy_code = _token_rows(dy, ids, dim, "dy")
    grad_p, grad_code, count = _flat(grad, ids, "grad")
    if workspace.device != ids.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {ids.device}")
    _call(_lib.zero_embedding_grad,
          (grad_p, grad_code, ids_p, id_bytes, n, dy_p, dy_ld, dy_code, vocab, dim, begin, count,
           -1 if padding_id is None else padding_id, float(scale), int(bool(overwrite)),
           workspace.data_ptr(), workspace.nbytes), ids, stream)
