"""A workspace that the binding allocates for a call belongs to the call's stream, not to the one that is current: else it
may be handed out again while the call's kernels use it, and its zeros may come after them (CPU only: streams are stand-ins)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from speculative_decoding_verification_34_gb300 import specverify as sv


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def allocated(monkeypatch):
    """The handles of the streams that were current when a workspace was allocated."""
    stack, seen = [Stream(0)], []

    @contextlib.contextmanager
    def on(stream):
        stack.append(stream)
        yield
        stack.pop()

    def alloc(*_, **__):
        seen.append(stack[-1].cuda_stream)
        return torch.zeros(64, dtype=torch.uint8)

    cuda = SimpleNamespace(current_stream=lambda *_: stack[-1], stream=on, Stream=Stream, ExternalStream=Stream,
                           default_stream=lambda *_: Stream(0))
    monkeypatch.setattr(sv.torch, "cuda", cuda)
    monkeypatch.setattr(sv, "load_library", lambda *_: SimpleNamespace(**{f: None for f in dir(sv) if f.startswith("spec_")}))
    monkeypatch.setattr(sv, "alloc_workspace", alloc)
    monkeypatch.setattr(sv, "alloc_attention_workspace", alloc)
    return seen


def _calls():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    l, d = torch.zeros(2, 4, 50), torch.zeros(2, 3, 50)
    tok, out, m, f, u = i32(2, 3), i32(2, 4), i32(2), torch.zeros(2), torch.zeros(2, 3)
    cache = SimpleNamespace(head_dim=64, kv_heads=1, tensors=())
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    yield "greedy", lambda **k: sv.spec_verify_greedy(l, tok, None, out, m, **k)
    yield "greedy prepared", lambda **k: sv.prepare_verify_greedy(l, tok, None, out, m, **k)
    yield "sample", lambda **k: sv.spec_verify_sample(l, d, tok, None, f, u, f, out, m, **k)
    yield "sample prepared", lambda **k: sv.prepare_verify_sample(l, d, tok, None, f, u, f, out, m, **k)
    yield "greedy commit", lambda **k: sv.spec_verify_greedy_commit(l, tok, None, out, m, m, **k)
    yield "sample commit", lambda **k: sv.spec_verify_sample_commit(l, d, tok, None, f, u, f, out, m, m, **k)
    yield "truncated", lambda **k: sv.spec_verify_sample_truncated(l, d, tok, None, f, None, None, u, f, out, m, **k)
    yield "tree", lambda **k: sv.spec_verify_tree_greedy(l, tok, tok, None, out, m, **k)
    yield "tree commit", lambda **k: sv.spec_verify_tree_greedy_commit(l, tok, tok, None, out, m, m, **k)
    yield "greedy split", lambda **k: sv.spec_verify_greedy_split(l[:, 0], l[:, 1:], tok, None, out, m, **k)
    yield "attention", lambda **k: sv.spec_verify_attention(q, cache, i32(2, 1), m, q, **k)
    yield "attention prepared", lambda **k: sv.prepare_verify_attention(q, cache, i32(2, 1), m, q, **k)


CALLS = dict(_calls())


@pytest.mark.parametrize("name", CALLS)
def test_workspace_belongs_to_the_calls_stream(allocated, name):
    cases = [(None, 0), (Stream(4096), 4096), (8192, 8192), (SimpleNamespace(cuda_stream=12288), 12288), (0, 0), (1, 0)]
    for stream, want in cases:
        allocated.clear()
        with pytest.raises(ValueError, match="CUDA"):      # (the tensors are on the CPU: nothing is launched)
            CALLS[name](stream=stream)
        assert allocated == [want], stream
    # in a context of another stream, None means that one and 0 the default stream
    for stream, want in ((None, 4096), (0, 0), (Stream(4096), 4096)):
        allocated.clear()
        with sv.torch.cuda.stream(Stream(4096)), pytest.raises(ValueError, match="CUDA"):
            CALLS[name](stream=stream)
        assert allocated == [want], stream


def test_a_given_workspace_is_taken(allocated):
    with pytest.raises(ValueError, match="CUDA"):
        CALLS["greedy"](stream=Stream(4096), workspace=torch.zeros(64, dtype=torch.uint8))
    assert allocated == []
