"""Who holds the scratch of a shared prefix, and for how long, on the host: a stand-in for the library and for
torch's allocator."""
import contextlib
import types

import pytest
import torch

from cross_loop_sparsity_b200 import flashloop as fl


class Scratch:
    def __init__(self, stream):
        self.stream, self.users = stream, []

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, s):
        self.users.append(s)


@pytest.fixture
def engine(monkeypatch):
    state = types.SimpleNamespace(stream="current", capturing=False, made=[])

    @contextlib.contextmanager
    def on(s):
        old, state.stream = state.stream, s
        yield
        state.stream = old

    def empty(*a, **k):
        state.made.append(Scratch(state.stream))
        return state.made[-1]

    calls = types.SimpleNamespace(**{name: (lambda *a: 0) for name in fl._SIG})
    calls.flashloop_share_prefix_scratch_bytes = lambda *a: 4096
    monkeypatch.setattr(fl, "lib", lambda: calls)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.capturing)
    eng = fl.FlashLoop.__new__(fl.FlashLoop)
    eng.c, eng.ctx, eng.workspace = fl.Config(), None, types.SimpleNamespace(device="cuda:0")
    eng._share_scratch, eng._share_kept = None, []
    return eng, state


def side(n):
    return types.SimpleNamespace(cuda_stream=n)


def test_steps_hold_the_scratch_on_their_streams(engine):
    eng, state = engine
    h0 = Scratch(None)
    eng.decode_step(h0, 2)                       # nothing shared: nothing to hold
    eng.share_prefix(2, 5)
    a, b = side(1), side(2)
    for s in (a, None, b):
        eng.decode_step(h0, 2, stream=s)
    first = state.made[0]
    assert first.users == [a, "default", b]
    eng.share_prefix(2, 7)
    eng.decode_step(h0, 2, stream=b)
    assert state.made[1].users == [b] and first.users == [a, "default", b]
    eng.share_prefix(0, 0)
    eng.decode_step(h0, 2, stream=b)
    assert state.made[1].users == [b] and eng._share_scratch is None and len(state.made) == 2


def test_scratch_belongs_to_the_stream_of_the_steps(engine):
    eng, state = engine
    a = side(1)
    eng.share_prefix(2, 5, stream=a)
    eng.share_prefix(2, 5)                       # a context's calls run on the default stream unless told otherwise
    assert [x.stream for x in state.made] == [a, "default"]


def test_a_captured_step_keeps_its_scratch(engine):
    eng, state = engine
    eng.share_prefix(2, 5)
    state.capturing = True
    eng.decode_step(Scratch(None), 2, stream=side(1))
    eng.decode_step(Scratch(None), 2, stream=side(1))
    state.capturing = False
    eng.share_prefix(0, 0)
    assert eng._share_kept == [state.made[0]] and state.made[0].users == []
