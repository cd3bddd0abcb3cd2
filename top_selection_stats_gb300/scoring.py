"""Scoring of given tokens: log probabilities, entropy, rank and alternatives
under the raw distribution, their gradient, and the same straight from hidden
states (the handle-free calls of include/smp.h).  Argument marshalling only.

Every tensor lives on the logits' (the hidden states') CUDA device and is
contiguous; the calls run on that device's current stream.  ``out`` takes what
an earlier call of the same shape returned and writes it again, so a serving
loop allocates nothing (head_logprobs: with ``workspace`` as well).

The results carry no autograd history, whatever the arguments require: a loss
differentiates them through a torch.autograd.Function around token_logprobs and
token_logprobs_grad, as examples/policy_step.py has it.
"""
import torch

from .binding import _DTYPES, _check, load_library


_F32, _I32 = torch.float32, torch.int32
# the current stream's handle and device without the objects around them (a
# microsecond less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _need(t, name, index, dtype, n):
    """The address of a contiguous tensor of n elements of dtype on device index."""
    if t.get_device() == index and t.dtype is dtype and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    raise ValueError(f"{name} must be contiguous")


def _opt(t, name, index, dtype, n):
    return None if t is None else _need(t, name, index, dtype, n)


def _bitmask(t, index, B, V):
    if t is None:
        return None
    if t.shape != (B, (V + 31) // 32):
        raise ValueError("bitmask must be [B, ceil(V/32)]")
    return _need(t, "bitmask", index, _I32, t.numel())


def _matrix(t, name, dtypes):
    if t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"unsupported {name} dtype {t.dtype}")
    return t.shape


def _width(V, ld, name):
    V = ld if V is None else V
    if not 1 <= V <= ld:
        raise ValueError(f"{name} must be in [1, {ld}], got {V}")
    return V


def token_logprobs(logits, targets, temperature=None, bitmask=None, n_top=0, V=None, out=None,
                   lib=None):
    """smp_token_logprobs: per row of logits [B, V] (or [B, ld] with ``V``) the
    log probability of targets[r] (int32 [B]; -1: none) under
    softmax(logits / temperature) over the legal tokens, the entropy, the
    target's rank, and the ``n_top`` (<= 32) most likely tokens.

    temperature: float32 [B] or None (1); bitmask: int32 [B, ceil(V/32)] or
    None.  Returns logprobs, entropy, rank, stats ([B, 2], for
    token_logprobs_grad), status and, with n_top, top_ids and top_logprobs
    [B, n_top]."""
    L = lib or load_library()
    B, ld = _matrix(logits, "logits", _DTYPES)
    V = _width(V, ld, "V")
    dev = logits.get_device()
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return token_logprobs(logits, targets, temperature, bitmask, n_top, V, out, lib)
    tg = _need(targets, "targets", dev, _I32, B)
    tp = _opt(temperature, "temperature", dev, _F32, B)
    bm = _bitmask(bitmask, dev, B, V)
    if n_top < 0:
        raise ValueError("n_top must be >= 0")
    if out is None:
        out = dict(logprobs=torch.empty(B, dtype=_F32, device=logits.device),
                   entropy=torch.empty(B, dtype=_F32, device=logits.device),
                   rank=torch.empty(B, dtype=_I32, device=logits.device),
                   stats=torch.empty((B, 2), dtype=_F32, device=logits.device),
                   status=torch.empty(B, dtype=_I32, device=logits.device))
        if n_top:
            out["top_ids"] = torch.empty((B, n_top), dtype=_I32, device=logits.device)
            out["top_logprobs"] = torch.empty((B, n_top), dtype=_F32, device=logits.device)
    rc = L.smp_token_logprobs(logits.data_ptr(), _DTYPES[logits.dtype], B, V, ld, bm, tp, tg,
                              _need(out["logprobs"], "logprobs", dev, _F32, B),
                              _need(out["entropy"], "entropy", dev, _F32, B),
                              _need(out["rank"], "rank", dev, _I32, B),
                              _need(out["stats"], "stats", dev, _F32, 2 * B),
                              _need(out["status"], "status", dev, _I32, B), n_top,
                              _need(out["top_ids"], "top_ids", dev, _I32, B * n_top) if n_top else None,
                              _need(out["top_logprobs"], "top_logprobs", dev, _F32, B * n_top) if n_top else None,
                              _raw_stream(dev))
    _check(rc, "smp_token_logprobs")
    return out


def token_logprobs_grad(logits, targets, stats, grad_logprobs=None, entropy=None,
                        grad_entropy=None, temperature=None, bitmask=None, V=None, out=None,
                        lib=None):
    """smp_token_logprobs_grad: the gradient with respect to logits, in their
    dtype and shape, for d loss / d logprobs = grad_logprobs and d loss /
    d entropy = grad_entropy (float32 [B], either None).  stats and entropy are
    the forward call's.  ``out`` may be logits itself (in place); columns past
    V are zero in a fresh result and are not written in ``out``.  Logits that start
    inside a 16-byte unit (a slice of rows of odd length) take 2 to 4 times as long
    into a result that does not, a fresh one among them."""
    L = lib or load_library()
    B, ld = _matrix(logits, "logits", _DTYPES)
    V = _width(V, ld, "V")
    dev = logits.get_device()
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return token_logprobs_grad(logits, targets, stats, grad_logprobs, entropy, grad_entropy,
                                       temperature, bitmask, V, out, lib)
    if grad_entropy is not None and entropy is None:
        raise ValueError("entropy is required with grad_entropy")
    if out is None:
        out = torch.empty_like(logits)
        if V < ld:
            out[:, V:].zero_()
    elif out.shape != logits.shape:
        raise ValueError(f"out must have the logits' shape, got {list(out.shape)}")
    rc = L.smp_token_logprobs_grad(logits.data_ptr(), _DTYPES[logits.dtype], B, V, ld,
                                   _bitmask(bitmask, dev, B, V),
                                   _opt(temperature, "temperature", dev, _F32, B),
                                   _need(targets, "targets", dev, _I32, B),
                                   _need(stats, "stats", dev, _F32, 2 * B),
                                   _opt(entropy, "entropy", dev, _F32, B),
                                   _opt(grad_logprobs, "grad_logprobs", dev, _F32, B),
                                   _opt(grad_entropy, "grad_entropy", dev, _F32, B),
                                   _need(out, "out", dev, logits.dtype, B * ld), ld, _raw_stream(dev))
    _check(rc, "smp_token_logprobs_grad")
    return out


def head_logprobs(hidden, weight, targets, temperature=None, D=None, out=None, workspace=None,
                  lib=None):
    """smp_head_logprobs: token_logprobs' logprobs, entropy, stats and status
    for logits = hidden @ weight.T (hidden [N, D], weight [V, D], both bfloat16
    or both float16, row lengths a multiple of 8; with ``D`` only the first D
    columns count), without the logits in memory.  workspace: uint8, at least
    head_workspace(N, V) bytes, the call's own until its work on the stream is done; when
    None, one is allocated for the call and given back to the stream's allocator."""
    L = lib or load_library()
    N, ldh = _matrix(hidden, "hidden", (torch.bfloat16, torch.float16))
    V, ldw = _matrix(weight, "weight", (torch.bfloat16, torch.float16))
    dev = hidden.get_device()
    if weight.dtype != hidden.dtype or weight.get_device() != dev:
        raise ValueError("hidden and weight must have one dtype and one device")
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return head_logprobs(hidden, weight, targets, temperature, D, out, workspace, lib)
    if D is None and ldh != ldw:
        raise ValueError("hidden and weight must have rows of one length, or D given")
    D = _width(D, min(ldh, ldw), "D")
    if ldh % 8 or ldw % 8:
        raise ValueError("rows of hidden and weight must be a multiple of 8 values long")
    tg = _need(targets, "targets", dev, _I32, N)
    tp = _opt(temperature, "temperature", dev, _F32, N)
    if out is None:
        out = dict(logprobs=torch.empty(N, dtype=_F32, device=hidden.device),
                   entropy=torch.empty(N, dtype=_F32, device=hidden.device),
                   stats=torch.empty((N, 2), dtype=_F32, device=hidden.device),
                   status=torch.empty(N, dtype=_I32, device=hidden.device))
    nbytes = L.smp_head_workspace(N, V)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=hidden.device)
    elif (workspace.dtype != torch.uint8 or workspace.get_device() != dev
          or not workspace.is_contiguous() or workspace.numel() < nbytes):
        raise ValueError(f"workspace must be a contiguous uint8 tensor of {nbytes} bytes on cuda:{dev}")
    rc = L.smp_head_logprobs(hidden.data_ptr(), ldh, weight.data_ptr(), ldw,
                             _DTYPES[hidden.dtype], N, V, D, tp, tg,
                             _need(out["logprobs"], "logprobs", dev, _F32, N),
                             _need(out["entropy"], "entropy", dev, _F32, N),
                             _need(out["stats"], "stats", dev, _F32, 2 * N),
                             _need(out["status"], "status", dev, _I32, N), workspace.data_ptr(),
                             workspace.numel(), _raw_stream(dev))
    _check(rc, "smp_head_logprobs")
    return out


def head_workspace(N, V, lib=None):
    """smp_head_workspace: bytes of workspace that head_logprobs needs."""
    return (lib or load_library()).smp_head_workspace(N, V)


def set_scoring_wait_limit(cycles=0, lib=None):
    """smp_set_scoring_wait_limit: bound on each device wait of later token_logprobs,
    head_logprobs and distill_loss calls of the process (SM cycles; 0 = default)."""
    _check((lib or load_library()).smp_set_scoring_wait_limit(int(cycles)), "smp_set_scoring_wait_limit")
