"""Penalties for repeated tokens, biases and grammar masks on logits before they are
sampled from (smp_process_logits, a handle-free call of include/smp.h).  Argument
marshalling only; the conventions are scoring.py's.
"""
import math

import torch

from .binding import _DTYPES, _check, load_library
from .scoring import _F32, _I32, _bitmask, _current_device, _matrix, _need, _raw_stream, _width


def process_logits(logits, history=None, lengths=None, prompt_lengths=None, repetition=None, presence=None,
                   frequency=None, bias_ids=None, bias=None, bitmask=None, V=None, dtype=None, in_place=False,
                   out=None, lib=None):
    """smp_process_logits: per row of logits [B, V] (or [B, ld] with ``V``), in this order,

    * repetition penalty (float32 [B]) on every token of the row's history: positive
      logits divided, others multiplied by it;
    * frequency (float32 [B]) times a token's copies among the generated tokens, and presence
      (float32 [B]) if it has any, subtracted;
    * biases added: bias float32 [B, NB] at token ids bias_ids int32 [B, NB] (outside [0, V):
      unused; -inf bans a token);
    * -inf where bitmask (int32 [B, ceil(V/32)]) has a 0.

    history: int32 [B, H], the prompt's tokens first; lengths, prompt_lengths: int32 [B], the
    entries that a row has (None: H) and how many of them are its prompt (None: 0).  H chooses the
    launch: where rows have a few hundred entries, a buffer of at most 2048 (with NB) is up to 3
    times as fast as a longer one.  The result has the logits' dtype, or float32 with
    ``dtype=torch.float32``.  ``in_place`` changes the
    logits themselves and touches nothing else of them.  Returns logits and status.  ``out``
    takes what an earlier call of the same shape returned; columns past V are -inf in a fresh
    result and are not written otherwise.  Rows with an invalid parameter go through unchanged."""
    L = lib or load_library()
    B, ld = _matrix(logits, "logits", _DTYPES)
    V = _width(V, ld, "V")
    dev = logits.get_device()
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return process_logits(logits, history, lengths, prompt_lengths, repetition, presence, frequency, bias_ids,
                                  bias, bitmask, V, dtype, in_place, out, lib)
    dtype = logits.dtype if dtype is None else dtype
    if dtype is not logits.dtype and (dtype is not _F32 or in_place):
        raise ValueError(f"results of {logits.dtype} logits cannot be {dtype}" + (" in place" if in_place else ""))
    hist = ids = b = None
    H = NB = 0
    if history is not None:
        shape = history.shape
        if len(shape) != 2 or shape[0] != B:
            raise ValueError("history must be [B, H]")
        H = shape[1]
        hist = _need(history, "history", dev, _I32, B * H)
    elif lengths is not None or prompt_lengths is not None:
        raise ValueError("lengths and prompt_lengths need a history")
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    if bias is not None:
        shape = bias.shape
        if len(shape) != 2 or shape[0] != B or bias_ids.shape != shape:
            raise ValueError("bias_ids and bias must be [B, NB]")
        NB = shape[1]
        ids, b = _need(bias_ids, "bias_ids", dev, _I32, B * NB), _need(bias, "bias", dev, _F32, B * NB)
    if out is None:
        status = torch.empty(B, dtype=_I32, device=logits.device)
        if in_place:
            result = logits
        else:
            result = torch.empty((B, ld), dtype=dtype, device=logits.device)
            if V < ld:
                result[:, V:].fill_(-math.inf)
        out = dict(logits=result, status=status)
    else:
        result = logits if in_place else out["logits"]
        if in_place:
            out["logits"] = logits
    shape = result.shape
    if len(shape) != 2 or shape[0] != B or shape[1] < V:
        raise ValueError(f"out must be [{B}, at least {V}], got {list(shape)}")
    rc = L.smp_process_logits(logits.data_ptr(), _DTYPES[logits.dtype], B, V, ld, hist, H, H,
                              None if lengths is None else _need(lengths, "lengths", dev, _I32, B),
                              None if prompt_lengths is None else _need(prompt_lengths, "prompt_lengths", dev, _I32, B),
                              None if repetition is None else _need(repetition, "repetition", dev, _F32, B),
                              None if presence is None else _need(presence, "presence", dev, _F32, B),
                              None if frequency is None else _need(frequency, "frequency", dev, _F32, B), ids, b, NB,
                              None if bitmask is None else _bitmask(bitmask, dev, B, V),
                              _need(result, "out", dev, dtype, B * shape[1]), _DTYPES[dtype], shape[1],
                              _need(out["status"], "status", dev, _I32, B), _raw_stream(dev))
    _check(rc, "smp_process_logits")
    return out
