"""Training calls of the vocabulary-sharded layers (C ABI in ``include/vpe_train.h``):
the scaled lookup and the gradient of its table shard, and distillation from a
teacher's top logits over the ranks' shards of the logits.

As in the package itself, functions only marshal arguments: they check
placement, dtype and layout, allocate outputs and workspaces with
``torch.empty`` when none is given, and pass raw device pointers plus the
current HIP stream of the tensors' device to the library.  No autograd graph is
built: outputs do not require gradients, whatever the inputs do, and the
gradient calls are made explicitly.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence

import torch

from . import (VPE_DISTILL_WHOLE_ROWS, _check, _dtype_code, _itype_code, _need_device,
               _same_device, load_library)

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_ITYPES = {torch.int32: 0, torch.int64: 1}

# The current stream's handle by device index, without a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:  # pragma: no cover
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


# The current device's index, without the look at whether one is initialised: the
# tensors of a call are on one.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def enqueue(name: str, index: int, *args) -> None:
    """Call `name` of the library with `args` and device `index`'s current stream,
    that device being the current one meanwhile (kernels are enqueued there)."""
    fn = getattr(load_library(), name)
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _check(name, status)


def placed(names: str, *tensors) -> int:
    """The index of the one HIP device all `tensors` (contiguous) are on; `names`
    are theirs, for the error."""
    index = tensors[0].get_device()
    for t in tensors:
        if index < 0 or t.get_device() != index or not t.is_contiguous():
            for name, each in zip(names.split(), tensors):
                _need_device(name, each)
            _same_device(*tensors)
    return index


def dtype_code(t) -> int:
    code = _DTYPES.get(t.dtype)
    return _dtype_code(t) if code is None else code


def itype_code(t) -> int:
    code = _ITYPES.get(t.dtype)
    return _itype_code(t) if code is None else code


def float_rows(name: str, t, m: int) -> None:
    if t.dtype != torch.float32 or t.numel() != m:
        raise ValueError(f"{name} must be a float32 tensor with one value per row")


def new_workspace(need: int, device):
    return torch.empty(need if need > 16 else 16, dtype=torch.uint8, device=device)


def nbytes(t) -> int:
    return t.numel() * t.element_size()


def apart(name: str, t, *others) -> None:
    """Refuse a `t` (written) that shares bytes with one of the `others`."""
    begin, end = t.data_ptr(), t.data_ptr() + nbytes(t)
    for o in others:
        at, size = o.data_ptr(), nbytes(o)
        if at < end and begin < at + size and size and begin < end:
            raise ValueError(f"{name} must not overlap the call's other tensors")


def vpe_embed_scaled(ids, weight, vocab_start: int, scale: float, out=None):
    """vpe_embed with every owned row times `scale` (fp32 product, one rounding)."""
    if weight.dim() != 2:
        raise ValueError("weight must be [shard_rows, dim]")
    rows, dim = weight.shape
    if out is None:
        out = torch.empty((*ids.shape, dim), dtype=weight.dtype, device=weight.device)
    else:
        if out.dtype != weight.dtype or out.numel() != ids.numel() * dim:
            raise ValueError("out must have the weight's dtype and ids.numel() * dim elements")
        apart("out", out, ids, weight)
    index = placed("ids weight out", ids, weight, out)
    enqueue("vpe_embed_scaled", index, ids.data_ptr(), itype_code(ids), ids.numel(),
            weight.data_ptr(), dtype_code(weight), rows, dim, int(vocab_start), scale,
            out.data_ptr())
    return out


@functools.lru_cache(maxsize=256)
def vpe_embed_grad_workspace(n: int, shard_rows: int, dim: int) -> int:
    """Bytes of workspace vpe_embed_grad needs for n ids; as much serves fewer."""
    b = ctypes.c_int64()
    _check("vpe_embed_grad_workspace", load_library().vpe_embed_grad_workspace(
        n, shard_rows, dim, ctypes.byref(b)))
    return b.value


def vpe_embed_grad(ids, grad_out, vocab_start: int, shard_rows: int, scale: float = 1.0,
                   grad_weight=None, accumulate: bool = False, workspace=None, dtype=None):
    """Gradient of the (scaled) lookup with respect to the shard, [shard_rows, dim].

    ids [*] and grad_out [*, dim] are the lookup's ids and the gradient of its
    output.  The result goes to `grad_weight` (added to it when `accumulate`),
    or to a new tensor of `dtype` (grad_out's when None).  Rows of positions
    whose id lies outside the shard add nothing.  A `grad_weight` or `workspace`
    that overlaps another tensor of the call is refused.
    """
    if grad_out.dim() < 1 or grad_out.shape[:-1] != ids.shape:
        raise ValueError("grad_out must be [*ids.shape, dim]")
    dim, n = grad_out.shape[-1], ids.numel()
    if grad_weight is None:
        if accumulate:
            raise ValueError("accumulate needs a grad_weight to add to")
        grad_weight = torch.empty((shard_rows, dim), dtype=dtype or grad_out.dtype,
                                  device=grad_out.device)
    else:
        if dtype is not None and dtype != grad_weight.dtype:
            raise ValueError("dtype differs from grad_weight's")
        if grad_weight.shape != (shard_rows, dim):
            raise ValueError("grad_weight must be [shard_rows, dim]")
        apart("grad_weight", grad_weight, ids, grad_out)
    if workspace is not None:
        apart("workspace", workspace, ids, grad_out, grad_weight)
    else:
        workspace = new_workspace(vpe_embed_grad_workspace(n, int(shard_rows), dim), grad_out.device)
    index = placed("ids grad_out grad_weight workspace", ids, grad_out, grad_weight, workspace)
    enqueue("vpe_embed_grad", index, ids.data_ptr(), itype_code(ids), n, grad_out.data_ptr(),
            dtype_code(grad_out), dim, int(vocab_start), int(shard_rows), scale,
            grad_weight.data_ptr(), dtype_code(grad_weight), bool(accumulate),
            workspace.data_ptr(), nbytes(workspace))
    return grad_weight


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------
def _teacher(teacher_ids, teacher, teacher_lse, m: Optional[int]):
    """Checked (ids, itype, teacher, dtype, k, teacher_lse) arguments, and the rows."""
    if teacher_ids.dim() != 2 or teacher_ids.shape != teacher.shape:
        raise ValueError("teacher_ids and teacher must both be [m, k]")
    rows, k = teacher_ids.shape
    if m is not None and rows != m:
        raise ValueError("the teacher's entries must have one row per row of logits")
    lse = None
    if teacher_lse is not None:
        float_rows("teacher_lse", teacher_lse, rows)
        placed("teacher_ids teacher_lse", teacher_ids, teacher_lse)
        lse = teacher_lse.data_ptr()
    return (teacher_ids.data_ptr(), itype_code(teacher_ids), teacher.data_ptr(),
            dtype_code(teacher), k, lse), rows


def logits_shard(name: str, logits, shard_rows: Optional[int], col_offset: int):
    """(rows, ld, columns of the shard) of a [m, ld] buffer; all columns from
    col_offset on when shard_rows is None."""
    if logits.dim() != 2:
        raise ValueError(f"{name} must be [m, ld]")
    m, ld = logits.shape
    return m, ld, int(ld - col_offset if shard_rows is None else shard_rows)


@functools.lru_cache(maxsize=256)
def vpe_distill_workspace(m: int, shard_rows: int) -> int:
    """Bytes of workspace that serve vpe_distill_shard for m rows and for fewer (it
    needs none if with_lse is False, or from VPE_DISTILL_WHOLE_ROWS rows on)."""
    b = ctypes.c_int64()
    _check("vpe_distill_workspace", load_library().vpe_distill_workspace(
        m, shard_rows, ctypes.byref(b)))
    return b.value


def vpe_distill_shard(logits, teacher_ids, teacher, vocab_start: int, vocab: int,
                      temperature: float = 1.0, teacher_lse=None,
                      shard_rows: Optional[int] = None, col_offset: int = 0, shard_lse=None,
                      shard_dot=None, workspace=None, with_lse: bool = True):
    """One shard's part of the distillation loss: (shard_lse, shard_dot), float32 [m].

    logits [m, ld] hold the shard [vocab_start, vocab_start + shard_rows) of a
    vocabulary of `vocab` at columns col_offset.. (all the rest of the row when
    shard_rows is None).  teacher_ids, teacher [m, k]: the teacher's top entries,
    ids outside [0, vocab) being padding.  With with_lse False only the entries'
    logits are read and shard_lse is None (temperature 1 after
    vpe_lmhead_logsumexp, which gives the same shard_lse).
    """
    m, ld, rows = logits_shard("logits", logits, shard_rows, col_offset)
    entries, _ = _teacher(teacher_ids, teacher, teacher_lse, m)
    if shard_dot is None:
        shard_dot = torch.empty(m, dtype=torch.float32, device=logits.device)
    else:
        float_rows("shard_dot", shard_dot, m)
    if with_lse:
        if shard_lse is None:
            shard_lse = torch.empty_like(shard_dot)
        else:
            float_rows("shard_lse", shard_lse, m)
        if workspace is None and m < VPE_DISTILL_WHOLE_ROWS:
            workspace = new_workspace(vpe_distill_workspace(m, rows), logits.device)
        given = () if workspace is None else (workspace,)
        index = placed("logits teacher_ids teacher shard_dot shard_lse workspace", logits,
                       teacher_ids, teacher, shard_dot, shard_lse, *given)
        tail = (shard_lse.data_ptr(), shard_dot.data_ptr(),
                *((workspace.data_ptr(), nbytes(workspace)) if given else (None, 0)))
    elif shard_lse is not None:
        raise ValueError("shard_lse given with with_lse=False")
    else:
        index = placed("logits teacher_ids teacher shard_dot", logits, teacher_ids, teacher,
                       shard_dot)
        tail = (None, shard_dot.data_ptr(), None, 0)
    enqueue("vpe_distill_shard", index, logits.data_ptr(), ld, int(col_offset), m, rows,
            dtype_code(logits), int(vocab_start), int(vocab), temperature, *entries, *tail)
    return shard_lse, shard_dot


def vpe_distill_loss(shard_lse: Sequence, shard_dot: Sequence, teacher_ids, teacher, vocab: int,
                     temperature: float = 1.0, teacher_lse=None, loss=None, lse=None):
    """(loss, lse) per row, float32 [m], from the shards' parts in shard order."""
    n = len(shard_lse)
    if n == 0 or n != len(shard_dot):
        raise ValueError("need one shard_lse and one shard_dot per shard")
    entries, m = _teacher(teacher_ids, teacher, teacher_lse, None)
    if loss is None:
        loss = torch.empty(m, dtype=torch.float32, device=teacher.device)
    if lse is None:
        lse = torch.empty(m, dtype=torch.float32, device=teacher.device)
    for t in (*shard_lse, *shard_dot, loss, lse):
        float_rows("shard_lse, shard_dot, loss and lse each", t, m)
    index = placed("teacher_ids teacher loss lse" + " shard_lse" * n + " shard_dot" * n,
                   teacher_ids, teacher, loss, lse, *shard_lse, *shard_dot)
    array = ctypes.c_void_p * n
    enqueue("vpe_distill_loss", index, array(*[t.data_ptr() for t in shard_lse]),
            array(*[t.data_ptr() for t in shard_dot]), n, m, int(vocab), temperature,
            *entries, loss.data_ptr(), lse.data_ptr())
    return loss, lse


def vpe_distill_grad(logits, lse, grad_loss, teacher_ids, teacher, vocab_start: int, vocab: int,
                     temperature: float = 1.0, teacher_lse=None,
                     shard_rows: Optional[int] = None, col_offset: int = 0, grad_logits=None,
                     grad_col_offset: Optional[int] = None):
    """Gradient of sum(grad_loss * loss) with respect to the shard's logits.

    lse [m] is vpe_distill_loss's, grad_loss [m] the gradient of each row's
    loss.  The result is written at columns grad_col_offset.. (col_offset when
    None) of grad_logits [m, ld], which may be the logits themselves, or to a
    new [m, shard_rows] tensor.
    """
    m, ld, rows = logits_shard("logits", logits, shard_rows, col_offset)
    entries, _ = _teacher(teacher_ids, teacher, teacher_lse, m)
    float_rows("lse", lse, m)
    float_rows("grad_loss", grad_loss, m)
    if grad_logits is None:
        if grad_col_offset:
            raise ValueError("grad_col_offset needs a grad_logits buffer")
        grad_logits = torch.empty((m, rows), dtype=logits.dtype, device=logits.device)
        grad_col_offset = 0
    else:
        if (grad_logits.dim() != 2 or grad_logits.shape[0] != m
                or grad_logits.dtype != logits.dtype):
            raise ValueError("grad_logits must be [m, ld] of the logits' dtype")
        grad_col_offset = col_offset if grad_col_offset is None else grad_col_offset
    index = placed("logits teacher_ids teacher lse grad_loss grad_logits", logits, teacher_ids,
                   teacher, lse, grad_loss, grad_logits)
    enqueue("vpe_distill_grad", index, logits.data_ptr(), ld, int(col_offset), m, rows,
            dtype_code(logits), int(vocab_start), int(vocab), temperature, *entries, lse.data_ptr(),
            grad_loss.data_ptr(), grad_logits.data_ptr(), grad_logits.shape[1],
            int(grad_col_offset))
    return grad_logits
