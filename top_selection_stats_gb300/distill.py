"""Distillation from a teacher's top tokens: the divergence of a student's distribution from
them and its gradient with respect to the student's logits (smp_distill_loss and
smp_distill_loss_grad, handle-free calls of include/smp.h).  Argument marshalling only; the
conventions are scoring.py's.  The results carry no autograd history: examples/distill_step.py
has the torch.autograd.Function around the two.
"""
import torch

from .binding import _DTYPES, _check, load_library
from .scoring import _F32, _I32, _bitmask, _current_device, _matrix, _need, _opt, _raw_stream, _width

_KINDS = {"forward": 0, "reverse": 1, "truncated": 2}


def _slots(teacher_ids, B):
    if teacher_ids.dim() != 2 or teacher_ids.shape[0] != B or teacher_ids.shape[1] < 1:
        raise ValueError("teacher_ids must be [B, K], K >= 1")
    return teacher_ids.shape[1]


def distill_loss(logits, teacher_ids, teacher, kind="forward", targets=None, temperature=None, bitmask=None, V=None,
                 out=None, lib=None):
    """smp_distill_loss: per row of the student's logits [B, V] (or [B, ld] with ``V``) the
    divergence of p = softmax(logits / temperature) over the legal tokens from a teacher
    that is known by K <= 256 of its tokens: teacher_ids int32 [B, K] (distinct; -1: unused slot)
    and teacher float32 [B, K] (-inf: probability 0).

    kind "forward" (teacher from student) and "reverse" (student from teacher): `teacher` holds
    log probabilities at the same temperature, for example token_logprobs' top_ids and
    top_logprobs, and all other tokens are one class.  "truncated": `teacher` holds logits, its
    distribution is their softmax at the row's temperature over the slots, nothing outside.

    targets: int32 [B] (-1: none): tokens whose log probability is wanted as well (hard labels
    beside the soft ones).  temperature: float32 [B] or None (1); bitmask: int32 [B,
    ceil(V/32)] or None.  Returns loss, slot_logprobs and slot_grads [B, K], stats [B, 4] (both
    for distill_loss_grad), status and, with targets, logprobs."""
    L = lib or load_library()
    B, ld = _matrix(logits, "logits", _DTYPES)
    V = _width(V, ld, "V")
    dev = logits.get_device()
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return distill_loss(logits, teacher_ids, teacher, kind, targets, temperature, bitmask, V, out, lib)
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {', '.join(_KINDS)}, got {kind!r}")
    K = _slots(teacher_ids, B)
    if teacher.shape != teacher_ids.shape:
        raise ValueError("teacher must have teacher_ids' shape")
    if out is None:
        out = dict(loss=torch.empty(B, dtype=_F32, device=logits.device),
                   slot_logprobs=torch.empty((B, K), dtype=_F32, device=logits.device),
                   slot_grads=torch.empty((B, K), dtype=_F32, device=logits.device),
                   stats=torch.empty((B, 4), dtype=_F32, device=logits.device),
                   status=torch.empty(B, dtype=_I32, device=logits.device))
        if targets is not None:
            out["logprobs"] = torch.empty(B, dtype=_F32, device=logits.device)
    rc = L.smp_distill_loss(logits.data_ptr(), _DTYPES[logits.dtype], B, V, ld, _bitmask(bitmask, dev, B, V),
                            _opt(temperature, "temperature", dev, _F32, B),
                            _need(teacher_ids, "teacher_ids", dev, _I32, B * K),
                            _need(teacher, "teacher", dev, _F32, B * K), K, _KINDS[kind],
                            _opt(targets, "targets", dev, _I32, B), _need(out["loss"], "loss", dev, _F32, B),
                            _need(out["logprobs"], "logprobs", dev, _F32, B) if targets is not None else None,
                            _need(out["slot_logprobs"], "slot_logprobs", dev, _F32, B * K),
                            _need(out["slot_grads"], "slot_grads", dev, _F32, B * K),
                            _need(out["stats"], "stats", dev, _F32, 4 * B),
                            _need(out["status"], "status", dev, _I32, B), _raw_stream(dev))
    _check(rc, "smp_distill_loss")
    return out


def distill_loss_grad(logits, teacher_ids, slot_logprobs, slot_grads, stats, grad_loss=None, targets=None,
                      logprobs=None, grad_logprobs=None, temperature=None, bitmask=None, V=None, out=None, lib=None):
    """smp_distill_loss_grad: the gradient with respect to logits, in their dtype and shape, for
    d / d loss = grad_loss and d / d logprobs = grad_logprobs (float32 [B], either None).
    slot_logprobs, slot_grads, stats and logprobs are the forward call's; targets and logprobs
    are needed with grad_logprobs only.  ``out`` may be logits itself (in place); columns past V
    are zero in a fresh result and are not written in ``out``."""
    L = lib or load_library()
    B, ld = _matrix(logits, "logits", _DTYPES)
    V = _width(V, ld, "V")
    dev = logits.get_device()
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return distill_loss_grad(logits, teacher_ids, slot_logprobs, slot_grads, stats, grad_loss, targets,
                                     logprobs, grad_logprobs, temperature, bitmask, V, out, lib)
    K = _slots(teacher_ids, B)
    if grad_logprobs is not None and (targets is None or logprobs is None):
        raise ValueError("targets and logprobs are required with grad_logprobs")
    if out is None:
        out = torch.empty_like(logits)
        if V < ld:
            out[:, V:].zero_()
    elif out.shape != logits.shape:
        raise ValueError(f"out must have the logits' shape, got {list(out.shape)}")
    rc = L.smp_distill_loss_grad(logits.data_ptr(), _DTYPES[logits.dtype], B, V, ld, _bitmask(bitmask, dev, B, V),
                                 _opt(temperature, "temperature", dev, _F32, B),
                                 _need(teacher_ids, "teacher_ids", dev, _I32, B * K), K,
                                 _need(slot_logprobs, "slot_logprobs", dev, _F32, B * K),
                                 _need(slot_grads, "slot_grads", dev, _F32, B * K),
                                 _need(stats, "stats", dev, _F32, 4 * B),
                                 _opt(grad_loss, "grad_loss", dev, _F32, B), _opt(targets, "targets", dev, _I32, B),
                                 _opt(logprobs, "logprobs", dev, _F32, B),
                                 _opt(grad_logprobs, "grad_logprobs", dev, _F32, B),
                                 _need(out, "out", dev, logits.dtype, B * ld), ld, _raw_stream(dev))
    _check(rc, "smp_distill_loss_grad")
    return out
