"""Training calls of the vocabulary-sharded layers (C ABI in ``include/vpe_train.h``):
the scaled lookup and the gradient of its table shard, and distillation from a
teacher's top logits over the ranks' shards of the logits.

As in the package itself, functions only marshal arguments: they check
placement, dtype and layout, allocate outputs and workspaces with
``torch.empty`` when none is given, and pass raw device pointers plus the
current HIP stream of the tensors' device to the library.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _check, _dtype_code, _itype_code, _need_device, _same_device, load_library

# The current stream's handle by device index, without a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:  # pragma: no cover
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def enqueue(name: str, device, *args) -> None:
    """Call `name` of the library with `args` and the device's current stream, the
    device being the current one meanwhile (kernels are enqueued there)."""
    fn = getattr(load_library(), name)
    if device.index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device.index))
    if status:
        _check(name, status)


def workspace_for(need: int, workspace, device):
    """The caller's workspace (its size is checked by the library), or a new one."""
    if workspace is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    _need_device("workspace", workspace)
    return workspace


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def vpe_embed_scaled(ids, weight, vocab_start: int, scale: float, out=None):
    """vpe_embed with every owned row times `scale` (fp32 product, one rounding)."""
    _need_device("ids", ids)
    _need_device("weight", weight)
    if weight.dim() != 2:
        raise ValueError("weight must be [shard_rows, dim]")
    rows, dim = weight.shape
    if out is None:
        out = torch.empty((*ids.shape, dim), dtype=weight.dtype, device=weight.device)
    else:
        _need_device("out", out)
    if out.dtype != weight.dtype or out.numel() != ids.numel() * dim:
        raise ValueError("out must have the weight's dtype and ids.numel() * dim elements")
    _same_device(ids, weight, out)
    enqueue("vpe_embed_scaled", weight.device, ids.data_ptr(), _itype_code(ids), ids.numel(),
            weight.data_ptr(), _dtype_code(weight), rows, dim, int(vocab_start), float(scale),
            out.data_ptr())
    return out


def vpe_embed_grad_workspace(n: int, shard_rows: int, dim: int) -> int:
    """Bytes of workspace vpe_embed_grad needs for n ids."""
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
    whose id lies outside the shard add nothing.
    """
    _need_device("ids", ids)
    _need_device("grad_out", grad_out)
    if grad_out.dim() < 1 or tuple(grad_out.shape[:-1]) != tuple(ids.shape):
        raise ValueError("grad_out must be [*ids.shape, dim]")
    dim, n = grad_out.shape[-1], ids.numel()
    if grad_weight is None:
        if accumulate:
            raise ValueError("accumulate needs a grad_weight to add to")
        grad_weight = torch.empty((shard_rows, dim), dtype=dtype or grad_out.dtype,
                                  device=grad_out.device)
    else:
        _need_device("grad_weight", grad_weight)
        if dtype is not None and dtype != grad_weight.dtype:
            raise ValueError("dtype differs from grad_weight's")
        if tuple(grad_weight.shape) != (shard_rows, dim):
            raise ValueError("grad_weight must be [shard_rows, dim]")
    itype, dt, gdt = _itype_code(ids), _dtype_code(grad_out), _dtype_code(grad_weight)
    need = vpe_embed_grad_workspace(n, shard_rows, dim)
    workspace = workspace_for(need, workspace, grad_out.device)
    _same_device(ids, grad_out, grad_weight, workspace)
    enqueue("vpe_embed_grad", grad_out.device, ids.data_ptr(), itype, n, grad_out.data_ptr(), dt,
            dim, int(vocab_start), shard_rows, float(scale), grad_weight.data_ptr(), gdt,
            int(accumulate), workspace.data_ptr(), _nbytes(workspace))
    return grad_weight


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------
def _float_rows(name: str, t, m: int):
    _need_device(name, t)
    if t.dtype != torch.float32 or t.numel() != m:
        raise ValueError(f"{name} must be a float32 tensor with one value per row")
    return t


def _teacher(teacher_ids, teacher, teacher_lse, m: Optional[int]):
    """Checked (rows, k, itype, dtype) of a batch of teacher entries."""
    _need_device("teacher_ids", teacher_ids)
    _need_device("teacher", teacher)
    if teacher_ids.dim() != 2 or teacher_ids.shape != teacher.shape:
        raise ValueError("teacher_ids and teacher must both be [m, k]")
    if m is not None and teacher_ids.shape[0] != m:
        raise ValueError("the teacher's entries must have one row per row of logits")
    if teacher_lse is not None:
        _float_rows("teacher_lse", teacher_lse, teacher_ids.shape[0])
        _same_device(teacher_ids, teacher_lse)
    _same_device(teacher_ids, teacher)
    return (*teacher_ids.shape, _itype_code(teacher_ids), _dtype_code(teacher))


def logits_shard(name: str, logits, shard_rows: Optional[int], col_offset: int):
    """(rows, columns of the shard) of a [m, ld] buffer; all columns from
    col_offset on when shard_rows is None."""
    _need_device(name, logits)
    if logits.dim() != 2:
        raise ValueError(f"{name} must be [m, ld]")
    return logits.shape[0], logits.shape[1] - col_offset if shard_rows is None else shard_rows


def vpe_distill_workspace(m: int, shard_rows: int) -> int:
    """Bytes of workspace vpe_distill_shard needs (may be 0)."""
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
    m, rows = logits_shard("logits", logits, shard_rows, col_offset)
    _, k, itype, tdt = _teacher(teacher_ids, teacher, teacher_lse, m)
    dt = _dtype_code(logits)
    if shard_dot is None:
        shard_dot = torch.empty(m, dtype=torch.float32, device=logits.device)
    _float_rows("shard_dot", shard_dot, m)
    if with_lse:
        if shard_lse is None:
            shard_lse = torch.empty(m, dtype=torch.float32, device=logits.device)
        _float_rows("shard_lse", shard_lse, m)
        need = vpe_distill_workspace(m, rows)
        if workspace is not None or need > 0:
            workspace = workspace_for(need, workspace, logits.device)
    elif shard_lse is not None:
        raise ValueError("shard_lse given with with_lse=False")
    _same_device(*(t for t in (logits, teacher, shard_dot, shard_lse, workspace) if t is not None))
    enqueue("vpe_distill_shard", logits.device, logits.data_ptr(), logits.shape[1], int(col_offset),
            m, rows, dt, int(vocab_start), int(vocab), float(temperature), teacher_ids.data_ptr(),
            itype, teacher.data_ptr(), tdt, k, None if teacher_lse is None else
            teacher_lse.data_ptr(), None if shard_lse is None else shard_lse.data_ptr(),
            shard_dot.data_ptr(), None if workspace is None else workspace.data_ptr(), 0 if
            workspace is None else _nbytes(workspace))
    return shard_lse, shard_dot


def vpe_distill_loss(shard_lse: Sequence, shard_dot: Sequence, teacher_ids, teacher, vocab: int,
                     temperature: float = 1.0, teacher_lse=None, loss=None, lse=None):
    """(loss, lse) per row, float32 [m], from the shards' parts in shard order."""
    lses, dots = list(shard_lse), list(shard_dot)
    if not lses or len(lses) != len(dots):
        raise ValueError("need one shard_lse and one shard_dot per shard")
    m, k, itype, tdt = _teacher(teacher_ids, teacher, teacher_lse, None)
    for i, (a, b) in enumerate(zip(lses, dots)):
        _float_rows(f"shard_lse[{i}]", a, m)
        _float_rows(f"shard_dot[{i}]", b, m)
    if loss is None:
        loss = torch.empty(m, dtype=torch.float32, device=teacher.device)
    if lse is None:
        lse = torch.empty(m, dtype=torch.float32, device=teacher.device)
    _float_rows("loss", loss, m)
    _float_rows("lse", lse, m)
    _same_device(teacher, loss, lse, *lses, *dots)
    n = len(lses)
    lp = (ctypes.c_void_p * n)(*[t.data_ptr() for t in lses])
    dp = (ctypes.c_void_p * n)(*[t.data_ptr() for t in dots])
    enqueue("vpe_distill_loss", teacher.device, lp, dp, n, m, int(vocab), float(temperature),
            teacher_ids.data_ptr(), itype, teacher.data_ptr(), tdt, k, None if teacher_lse is None
            else teacher_lse.data_ptr(), loss.data_ptr(), lse.data_ptr())
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
    m, rows = logits_shard("logits", logits, shard_rows, col_offset)
    _, k, itype, tdt = _teacher(teacher_ids, teacher, teacher_lse, m)
    dt = _dtype_code(logits)
    _float_rows("lse", lse, m)
    _float_rows("grad_loss", grad_loss, m)
    if grad_logits is None:
        if grad_col_offset:
            raise ValueError("grad_col_offset needs a grad_logits buffer")
        grad_logits = torch.empty((m, rows), dtype=logits.dtype, device=logits.device)
        grad_col_offset = 0
    else:
        _need_device("grad_logits", grad_logits)
        if (grad_logits.dim() != 2 or grad_logits.shape[0] != m
                or grad_logits.dtype != logits.dtype):
            raise ValueError("grad_logits must be [m, ld] of the logits' dtype")
        grad_col_offset = col_offset if grad_col_offset is None else grad_col_offset
    _same_device(logits, lse, grad_loss, teacher, grad_logits)
    enqueue("vpe_distill_grad", logits.device, logits.data_ptr(), logits.shape[1], int(col_offset),
            m, rows, dt, int(vocab_start), int(vocab), float(temperature), teacher_ids.data_ptr(),
            itype, teacher.data_ptr(), tdt, k, None if teacher_lse is None else
            teacher_lse.data_ptr(), lse.data_ptr(), grad_loss.data_ptr(), grad_logits.data_ptr(),
            grad_logits.shape[1], int(grad_col_offset))
    return grad_logits
