"""A scoring call that could not be launched says so once: the next call of the library is
not blamed for it."""
import ctypes

import pytest
import torch

import top_selection_stats_gb300 as lib

pytestmark = pytest.mark.gpu

CAPTURE_RELAXED = 2


def refused_launches(call):
    """What call(stream 0) returns while a stream that synchronises with the legacy stream is
    being captured: CUDA refuses launches into the legacy stream then."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(stream), 0) == 0
    try:
        assert cu.cuStreamBeginCapture_v2(stream, CAPTURE_RELAXED) == 0
        try:
            return call(None)
        finally:
            cu.cuStreamEndCapture(stream, ctypes.byref(graph))  # invalidated by the refusal
            if graph.value:
                cu.cuGraphDestroy(graph)
    finally:
        assert cu.cuStreamDestroy_v2(stream) == 0


def test_next_call_after_a_refused_launch():
    L = lib.load_library()
    B, V, D = 4, 512, 64
    x = torch.randn(B, V, device="cuda")
    t = torch.arange(B, dtype=torch.int32, device="cuda")
    f, i = torch.zeros(2 * B, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    h, w = torch.zeros((B, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(lib.head_workspace(B, V), dtype=torch.uint8, device="cuda")
    grad = torch.empty_like(x)
    p = {k: v.data_ptr() for k, v in dict(x=x, t=t, f=f, i=i, h=h, w=w, ws=ws, grad=grad).items()}
    calls = {
        "token_logprobs": lambda s: L.smp_token_logprobs(p["x"], 0, B, V, V, None, None, p["t"], p["f"], None, None,
                                                         None, p["i"], 0, None, None, s),
        "token_logprobs_grad": lambda s: L.smp_token_logprobs_grad(p["x"], 0, B, V, V, None, None, p["t"], p["f"],
                                                                   None, p["f"], None, p["grad"], V, s),
        "head_logprobs": lambda s: L.smp_head_logprobs(p["h"], D, p["w"], D, 1, B, V, D, None, p["t"], p["f"], None,
                                                       None, p["i"], p["ws"], ws.numel(), s)}
    sampler = lib.Sampler(0, max_batch=8, max_vocab=1024)
    history, penalty = torch.zeros((B, 3), dtype=torch.int32, device="cuda"), torch.full((B,), 1.5, device="cuda")
    torch.cuda.synchronize()
    try:
        for name, call in calls.items():
            assert call(None) == lib.SMP_OK, name  # the arguments are good
            torch.cuda.synchronize()
            assert refused_launches(call) == lib.SMP_ERR_CUDA, name
            y = x.clone()
            sampler.repetition_penalty(y, history, penalty)  # raises when blamed
            torch.cuda.synchronize()
            assert not torch.equal(x, y), name
            assert call(None) == lib.SMP_OK, name
            torch.cuda.synchronize()
    finally:
        sampler.close()
