"""spec_process_logits from two host threads at once, with calls whose blocks need much and little shared memory."""
import threading

import pytest
import torch

from speculative_decoding_verification_34_gb300 import specverify as sv
from tests.test_gpu_logits import SENT, call, dev, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [20000, 900])
def test_two_threads_with_calls_of_other_sizes(V):
    ds = [make(51, 2, 3, V, torch.bfloat16, hist=12000, nbias=9, mask=True), make(52, 2, 3, V, torch.bfloat16, hist=2, mask=True)]
    want = [call(d)[0] for d in ds]
    fns, outs = [], []
    for d in ds:
        logits = dev(d["logits"])
        outs.append(torch.full_like(logits, SENT))
        rest = [dev(d[k]) for k in ("history", "committed", "prompt", "drafts", "num", "parents", "rep", "freq", "pres", "bias_ids",
                                    "bias", "mask")]
        fns.append(sv.prepare_process_logits(logits, outs[-1], *rest, stream=torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed = []

    def loop(f):
        try:
            for _ in range(4000):
                f()
        except sv.SpecVerifyError as e:
            failed.append(str(e))

    threads = [threading.Thread(target=loop, args=(f,)) for f in fns]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == []
    for o, w in zip(outs, want):
        assert torch.equal(o.cpu(), w)
