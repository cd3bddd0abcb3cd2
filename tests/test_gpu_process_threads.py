"""smp_process_logits from several host threads at once, each on a stream of its own: the calls have
no handle and share nothing, so none may be refused or changed by another."""
import threading

import pytest
import torch

import test_gpu_process as G
import top_selection_stats_gb300 as lib

pytestmark = pytest.mark.gpu


class Recorder:
    """Takes the arguments of a call in place of the library."""

    def smp_process_logits(self, *args):
        self.args = args
        return lib.SMP_OK


@pytest.mark.parametrize("shapes", [((150, 32000, 4000, 0), (150, 16000, 4000, 0), (100, 8000, 3000, 0)),
                                    ((150, 32000, 4000, 300), (40, 20000, 1500, 600), (20, 3000, 40, 4))])
def test_calls_at_once(shapes):
    """Shapes whose shared memory differs, most of them in one kernel; the arguments are put together
    before, so that the threads are in the call nearly all the time."""
    cases = [G.make(*s, "bf16", 5) for s in shapes]
    want = [G.call(c)["logits"].clone() for c in cases]
    torch.cuda.synchronize()
    calls, outs, streams = [], [], [torch.cuda.Stream() for _ in cases]
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            outs.append(G.call(c))
            recorder = Recorder()
            G.call(c, out=outs[-1], lib=recorder)
            calls.append(recorder.args)
    torch.cuda.synchronize()
    f = lib.load_library().smp_process_logits
    start, codes = threading.Barrier(len(cases)), [set() for _ in cases]

    def work(i):
        torch.cuda.set_device(0)
        args, seen = calls[i], codes[i]
        start.wait(60)
        for _ in range(6000):
            seen.add(f(*args))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(300)
    torch.cuda.synchronize()
    assert codes == [{lib.SMP_OK}] * len(cases)
    for o, w in zip(outs, want):
        assert torch.equal(o["logits"], w) and not o["status"].any()
