"""Beam search over the vocabulary-sharded logits (C ABI in ``include/vpe_beam.h``):
selection over beams and vocabulary per shard, the merge of the shards' picks,
and the reordering of per-beam states.  Argument marshalling only, as in the
package itself.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Sequence

import torch

from . import _check, load_library
from .training import (dtype_code, enqueue, float_rows, logits_shard, nbytes, new_workspace,
                       placed)


@functools.lru_cache(maxsize=256)
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
    beams, picks = int(beams), int(picks)
    m, ld, rows = logits_shard("logits", logits, shard_rows, col_offset)
    if beams < 1 or m % beams != 0:
        raise ValueError("logits must have `beams` rows per sequence")
    n = m // beams
    float_rows("lse", lse, m)
    float_rows("scores", scores, m)
    if workspace is None:
        workspace = new_workspace(vpe_beam_select_workspace(n, beams, rows, picks), logits.device)
    if keys is None:
        keys = torch.empty((n, picks), dtype=torch.int64, device=logits.device)
    elif keys.dtype != torch.int64 or keys.numel() != n * picks:
        raise ValueError("keys must be an int64 tensor [n_seqs, picks] (uint64 keys)")
    index = placed("logits lse scores keys workspace", logits, lse, scores, keys, workspace)
    enqueue("vpe_beam_select", index, logits.data_ptr(), ld, int(col_offset),
            dtype_code(logits), n, beams, rows, int(vocab_start), int(vocab), lse.data_ptr(),
            scores.data_ptr(), picks, keys.data_ptr(), workspace.data_ptr(), nbytes(workspace))
    return keys


def vpe_beam_merge(keys: Sequence, vocab: int):
    """(scores float32, parents int64, tokens int64), each [n_seqs, picks], best
    first: the shards' picks merged."""
    if len(keys) == 0:
        raise ValueError("need at least one shard's keys")
    first = keys[0]
    for t in keys:
        if t.dtype != torch.int64 or t.dim() != 2 or t.shape != first.shape:
            raise ValueError("keys must be int64 tensors [n_seqs, picks] of one shape")
    index = placed("keys " * len(keys), *keys)
    n, picks = first.shape
    score = torch.empty((n, picks), dtype=torch.float32, device=first.device)
    parent, token = torch.empty_like(first), torch.empty_like(first)
    array = (ctypes.c_void_p * len(keys))(*[t.data_ptr() for t in keys])
    enqueue("vpe_beam_merge", index, array, len(keys), n, picks, int(vocab), score.data_ptr(),
            parent.data_ptr(), token.data_ptr())
    return score, parent, token


def vpe_beam_reorder(state, parents, beams: int, dim: int = 0, out=None):
    """A per-beam state with its rows taken from the parents' rows.

    Dimension `dim` of `state` (any dtype) holds n_seqs * beams rows; parents
    int64 [n_seqs, beams_out] (rows may be strided, e.g. the first columns of
    vpe_beam_merge's) names each new beam's old one.  The result has n_seqs *
    beams_out rows there; a parent outside [0, beams) gives zeros.
    """
    if parents.dtype != torch.int64 or parents.dim() != 2:
        raise ValueError("parents must be int64 [n_seqs, beams_out]")
    n, beams_out = parents.shape
    if beams_out < 1 or beams < 1:
        raise ValueError("need at least one beam")
    ld, step = parents.stride()
    if beams_out > 1 and step != 1:
        raise ValueError("parents must have adjacent columns")
    if n <= 1:  # a single row has no stride to speak of
        ld = max(ld, beams_out)
    shape = state.shape
    if not 0 <= dim < len(shape) or shape[dim] != n * beams:
        raise ValueError("dimension `dim` of state must have n_seqs * beams rows")
    to = shape if beams_out == beams else (*shape[:dim], n * beams_out, *shape[dim + 1:])
    if out is None:
        out = (torch.empty_like(state) if to is shape
               else torch.empty(to, dtype=state.dtype, device=state.device))
    elif out.shape != to or out.dtype != state.dtype:
        raise ValueError(f"out must be {tuple(to)} of the state's dtype")
    index = placed("state out", state, out)
    if parents.get_device() != index:
        raise ValueError(f"parents must be on the state's device, got {parents.device}")
    size = nbytes(state)
    if size != 0:
        outer = math.prod(shape[:dim]) if dim else 1
        enqueue("vpe_beam_reorder", index, state.data_ptr(), outer, n, int(beams),
                size // (outer * n * int(beams)), parents.data_ptr(), ld, beams_out,
                out.data_ptr())
    return out
