"""GB300-native batched top-k / top-p truncation and sampling.

A thin binding over the C ABI in ``include/smp.h`` (``libsmp.so``, hand-written
sm_103a CUDA).  This module only marshals arguments: torch supplies device
memory and the current stream, every step of the computation runs in the CUDA
kernels.  There is no fallback: if the library is missing, calls raise.
"""
from .binding import (SMP_OK, SMP_ERR_EMPTY, SMP_ERR_NONFINITE, SMP_ERR_INVALID_PARAM,
                      SMP_ERR_TIMEOUT, SMP_ERR_CUDA, SMP_ERR_CAPACITY, PATH_NAMES, Sampler,
                      SmpError, lib_path, load_library, sample_noalloc)
from .distill import distill_loss, distill_loss_grad
from .processing import process_logits
from .scoring import (head_logprobs, head_workspace, set_scoring_wait_limit, token_logprobs,
                      token_logprobs_grad)

__all__ = ["Sampler", "SmpError", "load_library", "lib_path", "sample_noalloc", "token_logprobs",
           "token_logprobs_grad", "head_logprobs", "head_workspace", "set_scoring_wait_limit",
           "process_logits", "distill_loss", "distill_loss_grad", "SMP_OK",
           "SMP_ERR_EMPTY", "SMP_ERR_NONFINITE", "SMP_ERR_INVALID_PARAM", "SMP_ERR_TIMEOUT", "SMP_ERR_CUDA",
           "SMP_ERR_CAPACITY", "PATH_NAMES"]
