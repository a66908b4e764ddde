"""Beam search over the vocabulary-sharded logits (C ABI in ``include/vpe_beam.h``):
selection over beams and vocabulary per shard, the merge of the shards' picks,
and the reordering of per-beam states.  Argument marshalling only, as in the
package itself.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import torch

from . import _check, _dtype_code, _need_device, _same_device, load_library
from .training import _float_rows, _nbytes, enqueue, logits_shard, workspace_for


def vpe_beam_select_workspace(n_seqs: int, beams: int, shard_rows: int, picks: int) -> int:
    """Bytes of workspace vpe_beam_select needs."""
    b = ctypes.c_int64()
    _check("vpe_beam_select_workspace", load_library().vpe_beam_select_workspace(
        n_seqs, beams, shard_rows, picks, ctypes.byref(b)))
    return b.value


def vpe_beam_select(logits, lse, scores, beams: int, picks: int, vocab_start: int, vocab: int,
                    shard_rows: Optional[int] = None, col_offset: int = 0, keys=None,
                    workspace=None):
    """Each sequence's `picks` best (beam, token) candidates over one shard's tokens,
    as keys int64 [n_seqs, picks] (uint64 bits; merged by vpe_beam_merge).

    logits [n_seqs * beams, ld] hold the shard at columns col_offset.. (all the
    rest of the row when shard_rows is None); lse and scores float32 hold, per
    row, the log-sum-exp over the whole vocabulary and the beam's accumulated
    log-probability.
    """
    m, rows = logits_shard("logits", logits, shard_rows, col_offset)
    if beams < 1 or m % beams != 0:
        raise ValueError("logits must have `beams` rows per sequence")
    n = m // beams
    dt = _dtype_code(logits)
    _float_rows("lse", lse, m)
    _float_rows("scores", scores, m)
    need = vpe_beam_select_workspace(n, beams, rows, picks)
    if keys is None:
        keys = torch.empty((n, picks), dtype=torch.int64, device=logits.device)
    _need_device("keys", keys)
    if keys.dtype != torch.int64 or keys.numel() != n * picks:
        raise ValueError("keys must be an int64 tensor [n_seqs, picks] (uint64 keys)")
    workspace = workspace_for(need, workspace, logits.device)
    _same_device(logits, lse, scores, keys, workspace)
    enqueue("vpe_beam_select", logits.device, logits.data_ptr(), logits.shape[1], int(col_offset),
            dt, n, beams, rows, int(vocab_start), int(vocab), lse.data_ptr(), scores.data_ptr(),
            picks, keys.data_ptr(), workspace.data_ptr(), _nbytes(workspace))
    return keys


def vpe_beam_merge(keys: Sequence, vocab: int):
    """(scores float32, parents int64, tokens int64), each [n_seqs, picks], best
    first: the shards' picks merged."""
    parts = list(keys)
    if not parts:
        raise ValueError("need at least one shard's keys")
    for i, t in enumerate(parts):
        _need_device(f"keys[{i}]", t)
        if t.dtype != torch.int64 or t.dim() != 2 or t.shape != parts[0].shape:
            raise ValueError("keys must be int64 tensors [n_seqs, picks] of one shape")
    _same_device(*parts)
    n, picks = parts[0].shape
    device = parts[0].device
    score = torch.empty((n, picks), dtype=torch.float32, device=device)
    parent = torch.empty((n, picks), dtype=torch.int64, device=device)
    token = torch.empty((n, picks), dtype=torch.int64, device=device)
    arr = (ctypes.c_void_p * len(parts))(*[t.data_ptr() for t in parts])
    enqueue("vpe_beam_merge", device, arr, len(parts), n, picks, int(vocab), score.data_ptr(),
            parent.data_ptr(), token.data_ptr())
    return score, parent, token


def vpe_beam_reorder(state, parents, beams: int, dim: int = 0, out=None):
    """A per-beam state with its rows taken from the parents' rows.

    Dimension `dim` of `state` (any dtype) holds n_seqs * beams rows; parents
    int64 [n_seqs, beams_out] (rows may be strided, e.g. the first columns of
    vpe_beam_merge's) names each new beam's old one.  The result has n_seqs *
    beams_out rows there; a parent outside [0, beams) gives zeros.
    """
    _need_device("state", state)
    if not parents.is_cuda:
        raise ValueError(f"parents must be a HIP device tensor, got device {parents.device}")
    if parents.dtype != torch.int64 or parents.dim() != 2:
        raise ValueError("parents must be int64 [n_seqs, beams_out]")
    n, beams_out = parents.shape
    if beams_out < 1 or beams < 1:
        raise ValueError("need at least one beam")
    if beams_out > 1 and parents.stride(1) != 1:
        raise ValueError("parents must have adjacent columns")
    # a single row has no stride to speak of
    ld = max(parents.stride(0), beams_out) if n <= 1 else parents.stride(0)
    if not 0 <= dim < state.dim() or state.shape[dim] != n * beams:
        raise ValueError("dimension `dim` of state must have n_seqs * beams rows")
    outer = math.prod(state.shape[:dim])
    row_bytes = math.prod(state.shape[dim + 1:]) * state.element_size()
    shape = (*state.shape[:dim], n * beams_out, *state.shape[dim + 1:])
    if out is None:
        out = torch.empty(shape, dtype=state.dtype, device=state.device)
    else:
        _need_device("out", out)
        if tuple(out.shape) != shape or out.dtype != state.dtype:
            raise ValueError(f"out must be {shape} of the state's dtype")
    _same_device(state, parents, out)
    if row_bytes == 0:
        return out
    enqueue("vpe_beam_reorder", state.device, state.data_ptr(), outer, n, beams, row_bytes,
            parents.data_ptr(), ld, beams_out, out.data_ptr())
    return out
