"""History buffers of a server: far longer than the rows' lengths, with tokens of earlier requests left
behind them, which count nothing.  Bounds and cases are test_gpu_process's."""
import pytest
import torch

import test_gpu_process as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("H", [2048, 2049, 8192, 70000])
def test_long_buffers_short_rows(H, in_place):
    """The bits of a buffer of 500 entries, whichever side of the table's size the longer one is on."""
    c = G.make(20, 40001, H, 9, "bf16", H, pad=3)
    c["history"].random_(0, 40001)
    c["lengths"] = (torch.arange(20, device="cuda") * 26).int()  # 0 to 494
    c["prompt_lengths"] = c["lengths"] // 3
    short = dict(c, history=c["history"][:, :500].contiguous(), x=c["x"].clone())
    want = G.call(short, in_place=in_place)["logits"]
    G.check(dict(c, x=c["x"].clone()), "bf16", in_place=in_place)
    got = G.call(c, in_place=in_place)["logits"]
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
