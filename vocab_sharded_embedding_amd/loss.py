"""Loss and gradient calls of a training step's head (C ABI in
``include/vpe_loss.h``): softmax cross entropy straight from the LM head's
shards, without keeping the logits, and its gradients; the LM head's backward
from a given gradient of the logits; the global gradient norm, and clipping.
Argument marshalling only, as in the package itself; no autograd graph is built.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence

import torch

from . import _check, load_library
from .training import (apart, dtype_code, enqueue, float_rows, itype_code, nbytes,
                       new_workspace, placed)


def _workspace(name: str, *sizes) -> int:
    b = ctypes.c_int64()
    _check(name, getattr(load_library(), name)(*sizes, ctypes.byref(b)))
    return b.value


@functools.lru_cache(maxsize=256)
def vpe_lmhead_xent_workspace(m: int, dim: int, shard_rows: int, dtype: int) -> int:
    """Bytes of workspace that serve vpe_lmhead_xent for m rows and for fewer
    (`dtype`: VPE_F32 or VPE_BF16)."""
    return _workspace("vpe_lmhead_xent_workspace", m, dim, shard_rows, dtype)


@functools.lru_cache(maxsize=256)
def vpe_lmhead_xent_grad_workspace(m: int, dim: int, shard_rows: int, dtype: int) -> int:
    """Bytes of workspace that serve vpe_lmhead_xent_grad for m rows and for fewer."""
    return _workspace("vpe_lmhead_xent_grad_workspace", m, dim, shard_rows, dtype)


@functools.lru_cache(maxsize=256)
def vpe_lmhead_grad_workspace(m: int, dim: int, shard_rows: int, dtype: int) -> int:
    """Bytes of workspace that serve vpe_lmhead_grad for m rows and for fewer."""
    return _workspace("vpe_lmhead_grad_workspace", m, dim, shard_rows, dtype)


def _head(x, weight):
    """Checked (rows, width, shard rows, dtype code) of hidden rows and a shard."""
    if x.dim() != 2 or weight.dim() != 2 or x.shape[1] != weight.shape[1]:
        raise ValueError("x must be [m, dim] and weight [shard_rows, dim]")
    if x.dtype != weight.dtype:
        raise TypeError("x and weight must share a dtype")
    return x.shape[0], x.shape[1], weight.shape[0], dtype_code(x)


def _row_targets(targets, m: int) -> int:
    if targets.numel() != m:
        raise ValueError("targets must hold one id per row of x")
    return itype_code(targets)


def _float_out(name: str, t, m: int, device, *inputs):
    if t is None:
        return torch.empty(m, dtype=torch.float32, device=device)
    float_rows(name, t, m)
    apart(name, t, *inputs)
    return t


def vpe_lmhead_xent(x, weight, targets, vocab_start: int, vocab: int, shard_lse=None,
                    target_logit=None, workspace=None):
    """One shard's part of the cross entropy: (shard_lse, target_logit), float32 [m].

    x [m, dim] are hidden rows, weight [shard_rows, dim] the shard [vocab_start,
    vocab_start + shard_rows) of a vocabulary of `vocab`, targets [m] ids of the
    whole vocabulary; a row whose target lies outside it (such as -100) takes no
    part, whatever it holds.  The logits are not kept.
    """
    m, dim, rows, dt = _head(x, weight)
    it = _row_targets(targets, m)
    shard_lse = _float_out("shard_lse", shard_lse, m, x.device, x, weight, targets)
    target_logit = _float_out("target_logit", target_logit, m, x.device, x, weight, targets,
                              shard_lse)
    if workspace is None:
        workspace = new_workspace(vpe_lmhead_xent_workspace(m, dim, rows, dt), x.device)
    else:
        apart("workspace", workspace, x, weight, targets, shard_lse, target_logit)
    index = placed("x weight targets shard_lse target_logit workspace", x, weight, targets,
                   shard_lse, target_logit, workspace)
    enqueue("vpe_lmhead_xent", index, x.data_ptr(), m, dim, weight.data_ptr(), rows, dt,
            int(vocab_start), int(vocab), targets.data_ptr(), it, shard_lse.data_ptr(),
            target_logit.data_ptr(), workspace.data_ptr(), nbytes(workspace))
    return shard_lse, target_logit


def vpe_xent_loss(shard_lse: Sequence, target_logit: Sequence, targets, vocab: int, loss=None,
                  lse=None):
    """(loss, lse) per row, float32 [m], from the shards' parts in shard order; both
    0 for a row without a target."""
    n, m = len(shard_lse), targets.numel()
    if n == 0 or n != len(target_logit):
        raise ValueError("need one shard_lse and one target_logit per shard")
    parts = (*shard_lse, *target_logit)
    for t in parts:
        float_rows("shard_lse and target_logit each", t, m)
    given = []
    if loss is None:
        loss = torch.empty(m, dtype=torch.float32, device=targets.device)
    else:
        given.append(("loss", loss))
    if lse is None:
        lse = torch.empty(m, dtype=torch.float32, device=targets.device)
    else:
        given.append(("lse", lse))
    for name, t in given:
        float_rows(name, t, m)
        apart(name, t, targets, lse if t is loss else loss,
              *[p for p in parts if p.data_ptr() != t.data_ptr()])
    index = placed("targets loss lse" + " part" * len(parts), targets, loss, lse, *parts)
    array = ctypes.c_void_p * n
    enqueue("vpe_xent_loss", index, array(*[t.data_ptr() for t in shard_lse]),
            array(*[t.data_ptr() for t in target_logit]), n, m, int(vocab), targets.data_ptr(),
            itype_code(targets), loss.data_ptr(), lse.data_ptr())
    return loss, lse


def _gradients(x, weight, inputs, grad_x, x_dtype, with_x, grad_weight, weight_dtype, with_weight,
               accumulate):
    """(grad_x, grad_weight) to write, each None where it is not wanted."""
    if not with_x and not with_weight:
        raise ValueError("neither gradient is wanted")
    out = []
    for name, t, like, dtype, wanted in (("grad_x", grad_x, x, x_dtype, with_x),
                                         ("grad_weight", grad_weight, weight, weight_dtype,
                                          with_weight)):
        if not wanted:
            if t is not None or dtype is not None:
                raise ValueError(f"{name} or its dtype given, but not wanted")
        elif t is None:
            if accumulate and name == "grad_weight":
                raise ValueError("accumulate needs a grad_weight to add to")
            t = torch.empty(like.shape, dtype=dtype or like.dtype, device=like.device)
        else:
            if dtype is not None and dtype != t.dtype:
                raise ValueError(f"dtype differs from {name}'s")
            if t.shape != like.shape:
                raise ValueError(f"{name} must have the shape {tuple(like.shape)}")
            apart(name, t, *inputs, *[o for o in out if o is not None])
        out.append(t)
    if accumulate and not with_weight:
        raise ValueError("accumulate needs a grad_weight to add to")
    return out


def _pointer_and_code(t):
    return (None, 0) if t is None else (t.data_ptr(), dtype_code(t))


def vpe_lmhead_xent_grad(x, weight, targets, lse, grad_loss, vocab_start: int, vocab: int,
                         grad_x=None, grad_weight=None, accumulate: bool = False, x_dtype=None,
                         weight_dtype=None, with_x: bool = True, with_weight: bool = True,
                         workspace=None):
    """One shard's gradients of sum(grad_loss * loss): (grad_x, grad_weight).

    lse [m] is vpe_xent_loss's, grad_loss [m] the gradient of each row's loss.
    grad_x [m, dim] is this shard's part (the shards' parts sum to the whole),
    grad_weight [shard_rows, dim] the shard's (added to with `accumulate`).  Each
    is written to the given tensor, or to a new one of x_dtype, weight_dtype (x's
    and weight's when None); with_x or with_weight False leaves one out (None).
    """
    m, dim, rows, dt = _head(x, weight)
    it = _row_targets(targets, m)
    float_rows("lse", lse, m)
    float_rows("grad_loss", grad_loss, m)
    inputs = (x, weight, targets, lse, grad_loss)
    grad_x, grad_weight = _gradients(x, weight, inputs, grad_x, x_dtype, with_x, grad_weight,
                                     weight_dtype, with_weight, accumulate)
    outs = [t for t in (grad_x, grad_weight) if t is not None]
    if workspace is None:
        workspace = new_workspace(vpe_lmhead_xent_grad_workspace(m, dim, rows, dt), x.device)
    else:
        apart("workspace", workspace, *inputs, *outs)
    index = placed("x weight targets lse grad_loss workspace" + " gradient" * len(outs), *inputs,
                   workspace, *outs)
    enqueue("vpe_lmhead_xent_grad", index, x.data_ptr(), m, dim, weight.data_ptr(), rows, dt,
            int(vocab_start), int(vocab), targets.data_ptr(), it, lse.data_ptr(),
            grad_loss.data_ptr(), *_pointer_and_code(grad_x), *_pointer_and_code(grad_weight),
            bool(accumulate), workspace.data_ptr(), nbytes(workspace))
    return grad_x, grad_weight


def vpe_lmhead_grad(grad_logits, x, weight, col_offset: int = 0, grad_x=None, grad_weight=None,
                    accumulate: bool = False, x_dtype=None, weight_dtype=None,
                    with_x: bool = True, with_weight: bool = True, workspace=None):
    """Backward of vpe_lmhead: (grad_x, grad_weight) from the gradient of the logits.

    grad_logits [m, ld] hold the shard's columns at col_offset.., such as
    vpe_distill_grad writes them.  The rest as vpe_lmhead_xent_grad.
    """
    m, dim, rows, dt = _head(x, weight)
    if grad_logits.dim() != 2 or grad_logits.shape[0] != m or grad_logits.dtype != x.dtype:
        raise ValueError("grad_logits must be [m, ld] of x's dtype")
    inputs = (grad_logits, x, weight)
    grad_x, grad_weight = _gradients(x, weight, inputs, grad_x, x_dtype, with_x, grad_weight,
                                     weight_dtype, with_weight, accumulate)
    outs = [t for t in (grad_x, grad_weight) if t is not None]
    if workspace is None:
        workspace = new_workspace(vpe_lmhead_grad_workspace(m, dim, rows, dt), x.device)
    else:
        apart("workspace", workspace, *inputs, *outs)
    index = placed("grad_logits x weight workspace" + " gradient" * len(outs), *inputs, workspace,
                   *outs)
    enqueue("vpe_lmhead_grad", index, grad_logits.data_ptr(), grad_logits.shape[1],
            int(col_offset), x.data_ptr(), m, dim, weight.data_ptr(), rows, dt,
            *_pointer_and_code(grad_x), *_pointer_and_code(grad_weight), bool(accumulate),
            workspace.data_ptr(), nbytes(workspace))
    return grad_x, grad_weight


# ---------------------------------------------------------------------------
# clipping
# ---------------------------------------------------------------------------
class _Table:
    """`tensors` as C arrays of pointers, element counts and dtypes, with the lists
    they were made of and their device's index."""

    def __init__(self, tensors: Sequence):
        n = self.n = len(tensors)
        self.index = placed("gradient " * n, *tensors)
        self.at = [t.data_ptr() for t in tensors]
        self.sizes = [t.numel() for t in tensors]
        kinds = [dtype_code(t) for t in tensors]
        self.bytes = [c * (2 if k else 4) for c, k in zip(self.sizes, kinds)]
        self.args = ((ctypes.c_void_p * n)(*self.at), (ctypes.c_int64 * n)(*self.sizes),
                     (ctypes.c_int32 * n)(*kinds), n)


def vpe_grad_sumsq_workspace(counts: Sequence[int]) -> int:
    """Bytes of workspace vpe_grad_sumsq needs for tensors of `counts` elements."""
    n = len(counts)
    return _workspace("vpe_grad_sumsq_workspace", (ctypes.c_int64 * n)(*counts), n)


def vpe_grad_sumsq(tensors: Sequence, sumsq=None, workspace=None):
    """Sum of the squares of all elements of `tensors` (float32 or bfloat16, at
    least one), as a float64 tensor [1]."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("need at least one tensor")
    table = _Table(tensors)
    device = tensors[0].device
    given = []
    if sumsq is None:
        sumsq = torch.empty(1, dtype=torch.float64, device=device)
    elif sumsq.dtype != torch.float64 or sumsq.numel() != 1:
        raise ValueError("sumsq must be a float64 tensor of one element")
    else:
        apart("sumsq", sumsq, *tensors)
        given.append(sumsq)
    if workspace is None:
        need = ctypes.c_int64()
        _check("vpe_grad_sumsq_workspace", load_library().vpe_grad_sumsq_workspace(
            table.args[1], table.n, ctypes.byref(need)))
        workspace = new_workspace(need.value, device)
    else:
        apart("workspace", workspace, sumsq, *tensors)
        given.append(workspace)
    if given:
        placed("gradient" + " sumsq_or_workspace" * len(given), tensors[0], *given)
    enqueue("vpe_grad_sumsq", table.index, *table.args, sumsq.data_ptr(), workspace.data_ptr(),
            nbytes(workspace))
    return sumsq


def _refuse_overlaps(table, out_at, sumsq, norm) -> None:
    """Refuse an output (at out_at, as large as its tensor; or `norm`) that shares
    bytes with another one, with `sumsq`, or with a tensor other than being the whole
    of its own."""
    spans = [(o, o + n, True) for o, n in zip(out_at, table.bytes)]
    if out_at is not table.at:
        spans += [(t, t + n, False) for t, o, n in zip(table.at, out_at, table.bytes) if t != o]
    spans += [(t.data_ptr(), t.data_ptr() + nbytes(t), False) for t in sumsq]
    spans.append((norm.data_ptr(), norm.data_ptr() + 4, True))
    spans.sort()
    # in order of their first bytes: the furthest end of what came before, of the
    # outputs alone and of everything
    written = read = 0
    for begin, end, is_out in spans:
        if begin == end:
            continue
        if begin < written or (is_out and begin < read):
            raise ValueError("an output of vpe_grad_clip must be its own tensor, or apart from "
                             "the call's other tensors, and norm apart from all of them")
        read = max(read, end)
        if is_out:
            written = max(written, end)


def vpe_grad_clip(tensors: Sequence, sumsq: Sequence, max_norm: float,
                  out: Optional[Sequence] = None, norm=None):
    """`tensors` times min(1, max_norm / (norm + 1e-6)), norm the root of the sum of
    the ranks' `sumsq` (vpe_grad_sumsq, one per rank); in place, or into `out` (of
    the tensors' sizes and types).  Returns the norm, a float32 tensor [1]."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("need at least one tensor")
    if len(sumsq) == 0:
        raise ValueError("need at least one rank's sumsq")
    for s in sumsq:
        if s.dtype != torch.float64 or s.numel() != 1:
            raise ValueError("sumsq must be float64 tensors of one element")
    table = _Table(tensors)
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=tensors[0].device)
    else:
        float_rows("norm", norm, 1)
    out_at, targets = table.at, table.args[0]
    if out is not None:
        out = list(out)
        if len(out) != table.n:
            raise ValueError("out must hold one tensor per gradient")
        for o, t, n in zip(out, tensors, table.sizes):
            if o.dtype != t.dtype or o.numel() != n:
                raise ValueError("each of out must have its gradient's dtype and size")
        placed("gradient" + " out" * len(out), tensors[0], *out)
        out_at = [o.data_ptr() for o in out]
        targets = (ctypes.c_void_p * table.n)(*out_at)
    _refuse_overlaps(table, out_at, sumsq, norm)
    n = len(sumsq)
    placed("gradient norm" + " sumsq" * n, tensors[0], norm, *sumsq)
    enqueue("vpe_grad_clip", table.index, *table.args, targets,
            (ctypes.c_void_p * n)(*[s.data_ptr() for s in sumsq]), n, float(max_norm),
            norm.data_ptr())
    return norm
