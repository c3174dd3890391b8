"""Calls on streams other than the current one, with workspaces that the binding allocates."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_34_gb300 import specverify as sv
from tests.test_gpu_attention import SENT, Case, dev

pytestmark = pytest.mark.gpu


def handles(s):
    """A stream as callers pass it."""
    return s, s.cuda_stream, torch.cuda.ExternalStream(s.cuda_stream)


def test_attention_on_two_streams_in_turn():
    """Items that all blocks share, on two streams at once: each call has partials of its own."""
    cs = [Case(40 + i, [9000, 90], 4, 8, 2, 128, 32) for i in range(2)]
    want = [c.run()[0] for c in cs]
    args = [(c.q.cuda(), c.gpu, dev(c.table), dev(c.lens)) for c in cs]
    nums = [dev(c.num) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [torch.full((12, *c.q.shape), SENT, dtype=torch.bfloat16, device="cuda") for c in cs]
    torch.cuda.synchronize()
    for k in range(12):
        for a, num, s, out in zip(args, nums, streams, outs):
            sv.spec_verify_attention(*a, out[k], num, stream=handles(s)[k % 3])
            torch.empty(1 << 20, device="cuda").fill_(float("nan"))       # the current stream goes on allocating
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        for k in range(12):
            assert np.array_equal(out[k].float().cpu().numpy(), w)


def test_a_dropped_workspace_is_not_handed_to_the_current_stream(monkeypatch):
    c = Case(42, [300], 4, 8, 2, 128, 32)
    c.run()
    a, num, out = (c.q.cuda(), c.gpu, dev(c.table), dev(c.lens)), dev(c.num), torch.zeros_like(c.q).cuda()
    sizes, alloc = [], sv.alloc_attention_workspace

    def spy(*x):
        t = alloc(*x)
        sizes.append((t.data_ptr(), t.numel()))
        return t

    monkeypatch.setattr(sv, "alloc_attention_workspace", spy)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    sv.spec_verify_attention(*a, out, num, stream=s)
    (ptr, n), = sizes
    mine = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(t.data_ptr() != ptr for t in mine)


def test_verify_on_another_stream_finds_its_workspace_zero():
    """A long row of work on the current stream, then a call on another: its counters start from zero all the same."""
    g = torch.Generator(device="cuda").manual_seed(0)
    l = torch.randn(6, 5, 5000, generator=g, device="cuda")
    toks = torch.randint(0, 5000, (6, 4), generator=g, device="cuda", dtype=torch.int32)
    toks[:, 0] = l[:, 0].argmax(-1)
    want = torch.zeros(6, 5, dtype=torch.int32, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
    sv.spec_verify_greedy(l, toks, None, *want)
    torch.cuda.synchronize()
    s, busy = torch.cuda.Stream(), torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    for k in range(6):
        got = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        torch.cuda.synchronize()
        for _ in range(8):
            busy.add_(1)
        sv.spec_verify_greedy(l, toks, None, *got, stream=handles(s)[k % 3])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
