"""Calls of the delta rule, the norms and the cells on a given stream beside calls on the current one, nothing synchronized in
between: what the binding allocates is shared by no two calls in flight.  The same inputs give the same bits, so
every result is compared exactly with that of a call that ran alone."""
from __future__ import annotations

import pytest
import torch

from xlstm_mlstm_cell_b200 import binding
from xlstm_mlstm_cell_b200.workloads import make_custom

pytestmark = pytest.mark.gpu


def delta(seed, S=640, DV=128):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    q, k = (torch.nn.functional.normalize(r(2, 4, S, 128), dim=-1).bfloat16().cuda() for _ in range(2))
    g, beta = -torch.rand(2, 8, S, generator=gen).cuda(), torch.rand(2, 8, S, generator=gen).cuda()
    return q, k, r(2, 8, S, DV).bfloat16().cuda(), g, beta, r(2, 8, S, DV).bfloat16().cuda()


def norms(seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    w = [(1 + 0.1 * r(128)).cuda() for _ in range(2)]
    return r(2, 4, 900, 128).cuda(), r(2, 2, 900, 128).cuda(), r(2, 900, 4, 128).cuda(), r(2, 900, 2, 128).cuda(), *w


def cells(seed):
    return [x.cuda() for x in make_custom(2, 4, 640, 128, 128, "bf16", seed=seed, ig=(-1.0, 2.0), fg=(4.0, 1.0))]


def cell_fwd(x, **kw):
    return binding.fwd(*x, **kw)


def cell_bwd(x, **kw):
    return binding.bwd(*x, x[2], **kw)


def fwd(x, **kw):
    return binding.gdelta_fwd(*x[:5], **kw)


def bwd(x, **kw):
    return binding.gdelta_bwd(*x[:5], x[5], **kw)[:5]


def norm_fwd(x, **kw):
    return binding.qknorm_fwd(*x[2:], **kw)


def norm_bwd(x, **kw):
    return binding.qknorm_bwd(*x, **kw)


CALLS = [(fwd, delta), (bwd, delta), (norm_fwd, norms), (norm_bwd, norms), (cell_fwd, cells), (cell_bwd, cells)]


@pytest.mark.parametrize("call,make", CALLS)
def test_current_and_given_stream_side_by_side(call, make):
    xs = [make(s) for s in (1, 2)]
    ref = [call(x) for x in xs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        got.append((call(xs[0]), call(xs[1], stream=side)))
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, ref):
            assert all(torch.equal(u, w) for u, w in zip(a, b))


@pytest.mark.parametrize("call,make", CALLS)
def test_outputs_dropped_while_the_call_runs(call, make):
    x = make(3)
    shapes = [(t.shape, t.dtype) for t in call(x)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        call(x, stream=side)   # dropped at once
        kept = [torch.zeros(s, dtype=d, device="cuda") for s, d in shapes]
        torch.cuda.synchronize()
        assert not any(t.any() for t in kept)


@pytest.mark.parametrize("call,make", CALLS)
def test_outputs_dropped_while_the_caller_reads_them(call, make):
    xs = [make(s) for s in (4, 5)]
    ref = call(xs[0])
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    for _ in range(3):
        out = call(xs[0], stream=side)
        here.wait_stream(side)
        torch.cuda._sleep(2_000_000)
        copies = [t.clone() for t in out]
        del out
        later = call(xs[1], stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, ref))
        del later, copies


def test_a_forked_stream_inside_a_captured_graph():
    """Two calls of one graph on its two branches: they replay as they ran alone."""
    xs = [delta(s) for s in (6, 7)]
    ref = [fwd(x) for x in xs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = [fwd(xs[0]), fwd(xs[1], stream=side)]
        here.wait_stream(side)
    for _ in range(3):
        for out in got:
            for t in out:
                t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert all(torch.equal(u, w) for u, w in zip(a, b))
