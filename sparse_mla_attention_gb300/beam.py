"""Beam search: the torch-facing wrapper of smla_beam_select (marshalling only).

The parents that it returns are rows for ``cache_reorder``, which moves the cached sequences along.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from .api import Workspace, _current_device, _need
from .cache import _raw_stream, _size_of

_TYPES = {torch.float32: _lib.SMLA_F32, torch.bfloat16: _lib.SMLA_BF16, torch.float16: _lib.SMLA_F16}
_sizes = {}


def beam_select(logits: torch.Tensor, scores: torch.Tensor, n: Optional[int] = None,
                done: Optional[torch.Tensor] = None, eos: int = -1, workspace: Optional[Workspace] = None,
                out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None
                ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The n best continuations of each group of beams: (parents, tokens, scores), each [B, n], best first.

    logits [B*K, V] float32, bfloat16 or float16 (rows may be any stride apart, a row's values lie side by side);
    scores [B, K] float32. Candidate v of beam k scores scores[b,k] + log_softmax(logits[b*K+k])[v]; a beam that is
    ``done`` [B, K] bool has the one candidate ``eos``, with its score as it is. Equal scores: the lower beam, then the
    larger logit, then the lower token (candidates of beams with different logits that are closer than 1e-5, as a rule 1e-7, may change
    places: smla_beam_select). Scores that are not finite are never taken; where fewer than n candidates are left the rest is
    (-1, -1, -inf). parents are row numbers b * K + k, tokens and parents int32. n is K if not given. Only enqueues work.
    """
    _need(scores, "scores", torch.float32, 2)
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _TYPES:
        raise TypeError("logits must be a float32, bfloat16 or float16 tensor")
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [B*K, V] with a row's values side by side")
    B, K = scores.shape
    rows, V = logits.shape
    index, device = scores.get_device(), scores.device
    if logits.get_device() != index:
        raise ValueError(f"logits must be on {device}, got {logits.device}")
    if rows != B * K or K < 1 or V < 1:
        raise ValueError("logits must have a row for each beam")
    n = K if n is None else int(n)
    p_done = None
    if done is not None:
        _need(done, "done", torch.bool, 2)
        if done.shape != scores.shape or done.get_device() != index:
            raise ValueError("done must have the shape and device of scores")
        if not 0 <= eos < V:
            raise ValueError("done needs eos in [0, V)")
        p_done = done.data_ptr()
    size = _size_of(_sizes, (B, K, V, n), "smla_beam_workspace_size", B, K, V, n)
    ws = (workspace or Workspace(device)).get(size)
    if ws.get_device() != index:
        raise ValueError(f"workspace must be on {device}, got {ws.device}")
    if out is None:
        out = (torch.empty((B, n), dtype=torch.int32, device=device),
               torch.empty((B, n), dtype=torch.int32, device=device),
               torch.empty((B, n), dtype=torch.float32, device=device))
    else:
        for t, dtype in zip(out, (torch.int32, torch.int32, torch.float32)):
            _need(t, "out", dtype, 2)
            if t.shape != (B, n) or t.get_device() != index:
                raise ValueError("out must be (parents, tokens, scores), each [B, n], on the device of scores")
    parents, tokens, best = out
    args = (logits.data_ptr(), _TYPES[logits.dtype], logits.stride(0) if rows > 1 else V, scores.data_ptr(), p_done, eos,
            parents.data_ptr(), tokens.data_ptr(), best.data_ptr(), B, K, V, n, ws.data_ptr(), ws.numel(),
            _raw_stream(index))
    fn = _lib.load().smla_beam_select
    if _current_device() == index:
        code = fn(*args)
    else:
        with torch.cuda.device(index):
            code = fn(*args)
    if code != _lib.SMLA_OK:
        raise _lib.SmlaError(code, "smla_beam_select")
    return parents, tokens, best
