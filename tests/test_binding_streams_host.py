"""Whose memory the binding allocates from when a call is given a stream (no GPU: the library and CUDA's streams
are stand-ins that note what happens).

A call's kernels on a given stream do not wait for the current one.  A tensor allocated on the current stream may
be a block that work queued there still uses; so what a call allocates has to come from the given stream's memory,
and an output has to be recorded on the current stream, where the caller uses it, before its block can go elsewhere.
"""
from __future__ import annotations

import types

import pytest
import torch

from xlstm_mlstm_cell_b200 import binding

GIVEN, CALLER, FOREIGN = (types.SimpleNamespace(cuda_stream=0x5100 + i, device="device %d" % i, device_index=i)
                          for i in (-1, -1, 3))   # the stand-ins' tensors are on the CPU, device -1
CALLER.cuda_stream = 0x5200


class Library:
    """Every entry point succeeds and notes the streams among its arguments; every size is 512 bytes."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*a):
            self.streams += [x for x in a if type(x) is int and x in (GIVEN.cuda_stream, CALLER.cuda_stream)]
            return 512 if name.endswith("_size") else 0
        return call


@pytest.fixture
def notes(monkeypatch):
    """Allocations as (tensor, stream current at that moment) and the streams each was recorded on."""
    made, recorded, current = [], {}, [CALLER]

    def set_stream(s):
        current[0] = s

    def noting(make):
        def wrapped(*a, **kw):
            kw.pop("device", None)
            t = make(*a, **kw)
            made.append((t, current[0]))
            return t
        return wrapped

    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, noting(getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "set_stream", set_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.setdefault(id(t), []).append(s))
    lib = Library()
    monkeypatch.setattr(binding, "load", lambda *a: lib)
    monkeypatch.setattr(binding, "_cuda_index", lambda t: t.get_device())
    monkeypatch.setattr(binding, "_stream", lambda *a: current[0].cuda_stream)
    monkeypatch.setattr(binding, "_on", lambda index, call: call(current[0].cuda_stream))
    yield made, recorded, lib.streams
    assert current == [CALLER], "the current stream is not what it was"


def rand(*shape):
    return torch.randn(*shape)


def delta(*lead):
    q, v, g = rand(2, 1, *lead, 16), rand(2, 2, *lead, 24), rand(2, 2, *lead)
    return q, q.clone(), v, g, g.clone()


STATE = (2, 2, 16, 24)
W = torch.ones(16)
OPERATORS = {
    "gdelta_fwd": (lambda **kw: binding.gdelta_fwd(*delta(5), **kw), 3),
    "gdelta_fwd from a state": (lambda **kw: binding.gdelta_fwd(*delta(5), state=rand(*STATE), **kw), 3),
    "gdelta_fwd without the state": (lambda **kw: binding.gdelta_fwd(*delta(5), return_state=False, **kw), 2),
    "gdelta_step": (lambda **kw: binding.gdelta_step(rand(*STATE), *delta(), **kw), 1),
    "gdelta_bwd": (lambda **kw: binding.gdelta_bwd(*delta(5), rand(2, 2, 5, 24), **kw), 6),
    "gdelta_bwd from a state": (lambda **kw: binding.gdelta_bwd(*delta(5), rand(2, 2, 5, 24), state=rand(*STATE), **kw), 7),
    "qknorm_fwd": (lambda **kw: binding.qknorm_fwd(rand(2, 5, 3, 16), rand(2, 5, 1, 16), **kw), 2),
    "qknorm_bwd": (lambda **kw: binding.qknorm_bwd(rand(2, 3, 5, 16), rand(2, 1, 5, 16), rand(2, 5, 3, 16),
                                                   rand(2, 5, 1, 16), q_weight=W, k_weight=W, **kw), 5),
}


def cell(*lead):
    q, v, g = rand(2, 1, *lead, 16), rand(2, 1, *lead, 16), rand(2, 1, *lead)
    return q, q.clone(), v, g, g.clone()


PARTS = rand(3, 2, 1, 16, 16), rand(3, 2, 1, 16), rand(3, 2, 1), rand(3, 2, 1)
CELLS = {
    "fwd": (lambda **kw: binding.fwd(*cell(5), **kw), 5),
    "fwd with an output gate": (lambda **kw: binding.fwd(*cell(5), rand(2, 1, 5, 16), return_state=False, **kw), 2),
    "bwd": (lambda **kw: binding.bwd(*cell(5), None, rand(2, 1, 5, 16), **kw), 6),
    "bwd with an output gate": (lambda **kw: binding.bwd(*cell(5), rand(2, 1, 5, 16), rand(2, 1, 5, 16), **kw), 7),
    "fwd_final_state": (lambda **kw: binding.fwd_final_state(*cell(5)[1:], **kw), 4),
    "log_decay_sum": (lambda **kw: binding.log_decay_sum(rand(2, 1, 5), **kw), 1),
    "state_prefix": (lambda **kw: binding.state_prefix(*PARTS, rank=1, **kw), 3),
    "fwd_noalloc": (lambda **kw: binding.fwd_noalloc(*cell(5), **kw), 4),
    "step": (lambda **kw: binding.step(rand(2, 1, 16, 16), rand(2, 1, 16), rand(2, 1), *cell(), **kw), 1),
    "slstm_fwd": (lambda **kw: binding.slstm_fwd(rand(2, 5, 4, 1, 16), rand(1, 4, 16, 16), **kw), 5),
}


def check_given_stream(call, tensors, notes):
    made, recorded, launched = notes
    call(stream=GIVEN)
    assert len(made) == tensors and launched == [GIVEN.cuda_stream]
    for t, where in made:
        assert where is GIVEN, "allocated on the current stream, used on the given one"
        assert recorded.get(id(t)) == (None if t.dtype == torch.uint8 else [CALLER])   # workspaces are bytes


@pytest.mark.parametrize("name", sorted(OPERATORS))
def test_a_given_streams_call_allocates_from_that_stream(name, notes):
    call, tensors = OPERATORS[name]
    check_given_stream(call, tensors, notes)


@pytest.mark.parametrize("name", sorted(CELLS))
def test_a_given_streams_cell_allocates_from_that_stream(name, notes):
    call, tensors = CELLS[name]
    check_given_stream(call, tensors, notes)


@pytest.mark.parametrize("name", sorted(OPERATORS) + sorted(CELLS))
def test_a_call_on_the_current_stream_allocates_there(name, notes):
    made, recorded, launched = notes
    call, tensors = {**OPERATORS, **CELLS}[name]
    call()
    assert len(made) == tensors and all(where is CALLER for _, where in made) and not recorded
    assert launched == [CALLER.cuda_stream]


@pytest.mark.parametrize("name", sorted(OPERATORS) + sorted(CELLS))
def test_a_stream_of_another_device_is_refused(name, notes):
    made, _, launched = notes
    with pytest.raises(ValueError, match="stream"):
        {**OPERATORS, **CELLS}[name][0](stream=FOREIGN)
    assert not made and not launched
