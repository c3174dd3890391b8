"""spec_process_logits where a sequence's marked ids take several windows of the vocabulary (more marks than a block has entries
for, or more ids than its bitmap), and where a batch takes several launches.  Tolerance as in test_gpu_logits.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_logits import SENT, call, check, dev, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,gmax,V,dtype,hist,nbias,mask,tree", [
    (2, 2, 262144, torch.float32, 60, 9, True, False), (2, 2, 262145, torch.bfloat16, 60, 9, False, True),
    (1, 3, 300000, torch.float32, 900, 40, False, False), (2, 1, 786433, torch.bfloat16, 40, 5, True, False),
    (2, 3, 32000, torch.bfloat16, 32768, 3, True, True), (2, 3, 50001, torch.float32, 100000, 30, False, True),
    (3, 0, 13000, torch.bfloat16, 20000, 0, True, False), (3, 0, 16384, torch.bfloat16, 13000, 4, False, False),
    (2, 1, 30000, torch.float32, 10, 14000, True, False), (2, 4, 12289, torch.bfloat16, 12284, 0, True, False),
    (1, 1, 1 << 20, torch.float32, 20000, 2, True, False)])
def test_several_windows(B, gmax, V, dtype, hist, nbias, mask, tree):
    d = make(41, B, gmax, V, dtype, hist, nbias, mask, tree)
    rng = np.random.default_rng(42)
    d["history"] = rng.integers(0, V, d["history"].shape).astype(np.int32)      # ids all over the vocabulary
    d["history"][:, ::7] = d["history"][:, :1]
    if gmax:
        d["drafts"][:, 0] = V - 1
    d["num"][0], d["committed"][0] = gmax, hist
    out, st = call(d)
    assert (st == 0).all()
    check(d, out)
    buf = dev(d["logits"]).clone()
    got, _ = call(d, logits=buf, out=buf)
    check(d, got, behind=d["logits"])


@pytest.mark.parametrize("hist", [12000, 32768, 100000])
@pytest.mark.parametrize("committed", [0, 1, 100])
def test_a_long_history_buffer_with_few_tokens_in_it(hist, committed):
    """Ids behind the committed length mark nothing, whatever the capacity."""
    d = make(43, 2, 3, 20000, torch.bfloat16, hist=hist, nbias=5)
    d["committed"][:] = committed
    d["prompt"][:] = committed // 3
    out, _ = call(d)
    check(d, out)
    short = dict(d, history=np.ascontiguousarray(d["history"][:, :128]))
    assert torch.equal(call(short)[0], out)


@pytest.mark.parametrize("V,in_place", [(3300, False), (3301, False), (3300, True)])
def test_a_batch_of_several_launches(V, in_place):
    """65535 rows fit one launch of the stream: the same 60 sequences many times over come out the same each time."""
    d = make(44, 60, 4, V, torch.bfloat16, nbias=4, mask=True)
    want, _ = call(d)
    check(d, want)
    times = 225                                                         # 13500 sequences of 5 rows
    many = dict(d, B=60 * times, logits=dev(d["logits"]).repeat(times, 1, 1))
    for k in ("history", "committed", "prompt", "drafts", "num", "rep", "freq", "pres", "bias_ids", "bias", "mask"):
        many[k] = dev(d[k]).repeat(times, *(1,) * (d[k].ndim - 1))
    out = many["logits"].clone() if in_place else torch.full_like(many["logits"], SENT)
    got, st = call(many, logits=out if in_place else None, out=out)
    assert (st == 0).all()
    got = got.view(times, 60, 5, V)
    for b in range(60):
        n = int(d["num"][b]) + 1
        assert torch.equal(got[:, b, :n], want[b, :n].expand(times, n, V))
        rest = d["logits"][b, n:] if in_place else torch.full_like(want[b, n:], SENT)
        assert torch.equal(got[:, b, n:], rest.expand(times, 5 - n, V))
