"""Host-side checks of the delta rule's and the norms' entry points (no GPU): refusals before any launch."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

from xlstm_mlstm_cell_b200 import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20   # an aligned non-NULL address that is never dereferenced
OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def no_device():
    return not torch.cuda.is_available()


def test_every_declared_symbol_is_bound(lib):
    for header, prefix in (("gdelta.h", "gdelta_"), ("qknorm.h", "qknorm_")):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
        names = set(re.findall(r"\b(%s\w+)\s*\(" % prefix, text))
        assert len(names) >= 3
        for name in names:
            assert hasattr(lib, name) and name in binding.SIGNATURES, name


def gd(lib, fn, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, lengths=None, S0=None, do=FAKE, dS=None, dt=1, B=2, NH=2, NHV=4,
             S=70, DK=64, DV=64, o=FAKE, Sf=None, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE, db=FAKE, dS0=None, ws=FAKE,
             wsb=1 << 40, state=FAKE)
    a.update(over)
    p = lambda *names: [None if a[x] is None else ctypes.c_void_p(a[x]) for x in names]   # noqa: E731
    sizes = [a[x] for x in ("dt", "B", "NH", "NHV", "S", "DK", "DV")]
    if fn == "fwd":
        return lib.gdelta_fwd(*p("q", "k", "v", "g", "beta", "lengths"), *sizes, 0.1, *p("S0", "o", "Sf", "ws"), a["wsb"], None)
    if fn == "step":
        return lib.gdelta_step(*p("state", "q", "k", "v", "g", "beta"), *sizes[:4], *sizes[5:], 0.1, *p("o"), None)
    return lib.gdelta_bwd(*p("q", "k", "v", "g", "beta", "lengths", "S0", "do", "dS"), *sizes, 0.1,
                          *p("dq", "dk", "dv", "dg", "db", "dS0", "ws"), a["wsb"], None)


@pytest.mark.parametrize("fn,over,expect", [(f, o, e) for f in ("fwd", "step", "bwd") for o, e in [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID),
    (dict(beta=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(v=FAKE + 2), INVALID), (dict(B=-1), INVALID),
    (dict(NH=0), INVALID), (dict(NHV=3), INVALID), (dict(NHV=0), INVALID), (dict(dt=2), UNSUPPORTED),
    (dict(DK=12), UNSUPPORTED), (dict(DK=136), UNSUPPORTED), (dict(DV=520), UNSUPPORTED), (dict(DV=4), UNSUPPORTED),
    (dict(DK=0), UNSUPPORTED), (dict(B=1 << 29), UNSUPPORTED)]] + [
    ("fwd", dict(B=40000), UNSUPPORTED), ("bwd", dict(B=40000), UNSUPPORTED),
    ("fwd", dict(B=8000, S=1 << 30), UNSUPPORTED), ("bwd", dict(B=8000, S=1 << 30), UNSUPPORTED),
    ("fwd", dict(o=None), INVALID), ("fwd", dict(S0=FAKE + 4), INVALID), ("fwd", dict(Sf=FAKE + 8), INVALID),
    ("fwd", dict(lengths=FAKE + 2), INVALID), ("fwd", dict(S=-1), INVALID), ("fwd", dict(ws=None), WORKSPACE),
    ("fwd", dict(wsb=1000), WORKSPACE), ("fwd", dict(ws=FAKE + 16), INVALID),
    ("step", dict(state=None), INVALID), ("step", dict(state=FAKE + 4), INVALID), ("step", dict(o=None), INVALID),
    ("bwd", dict(do=None), INVALID), ("bwd", dict(dq=None), INVALID), ("bwd", dict(dk=None), INVALID),
    ("bwd", dict(dv=None), INVALID), ("bwd", dict(dg=None), INVALID), ("bwd", dict(db=None), INVALID),
    ("bwd", dict(dS=FAKE + 4), INVALID), ("bwd", dict(dS0=FAKE + 4), INVALID), ("bwd", dict(ws=None), WORKSPACE),
    ("bwd", dict(wsb=1000), WORKSPACE), ("bwd", dict(ws=FAKE + 128), INVALID), ("bwd", dict(S=-2), INVALID),
])
def test_gdelta_refuses(lib, fn, over, expect):
    assert gd(lib, fn, **over) == expect


def test_gdelta_empty_batch_is_a_no_op(lib):
    none = dict(q=None, k=None, v=None, g=None, beta=None, o=None, do=None, dq=None, dk=None, dv=None, dg=None, db=None,
                state=None, ws=None)
    for fn in ("fwd", "step", "bwd"):
        assert gd(lib, fn, B=0, **none) == OK


def test_gdelta_queries(lib):
    assert lib.gdelta_fwd_workspace_size(2, 2, 4, 70, 64, 64, 1) > 0
    assert lib.gdelta_bwd_workspace_size(2, 2, 4, 70, 64, 64, 0) > lib.gdelta_fwd_workspace_size(2, 2, 4, 70, 64, 64, 0)
    assert lib.gdelta_fwd_workspace_size(2, 2, 3, 70, 64, 64, 1) == 0
    assert lib.gdelta_fwd_workspace_size(2, 2, 4, 70, 256, 64, 1) == 0
    assert lib.gdelta_fwd_tensor_path(136, 64, 1) == -1 and lib.gdelta_fwd_tensor_path(64, 64, 0) == 0


@pytest.mark.skipif(not no_device(), reason="needs a machine without a CUDA device")
def test_launch_failures_are_reported(lib):
    for fn in ("fwd", "step", "bwd"):
        assert gd(lib, fn) == CUDA
        assert gd(lib, fn, dt=0) == CUDA
    assert qk(lib, False) == CUDA and qk(lib, True) == CUDA
    assert qk(lib, False, RD=14) == CUDA


def qk(lib, bwd, **over):
    a = dict(q=FAKE, k=FAKE, wq=None, wk=None, inv=FAKE, pos=None, dt=1, B=2, S=3, NHQ=4, NHK=2, D=64, RD=16, kind=0,
             eps=1e-6, inter=0, qo=FAKE, ko=FAKE, dqo=FAKE, dko=FAKE, dwq=FAKE, dwk=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(over)
    st = binding._Strides(3 * 6 * 64, 6 * 64, 64)
    v = lambda x: None if a[x] is None else ctypes.c_void_p(a[x])   # noqa: E731
    mid = [v("wq"), v("wk"), v("inv"), v("pos"), *(a[x] for x in ("dt", "B", "S", "NHQ", "NHK", "D", "RD", "kind")),
           a["eps"], a["inter"]]
    if not bwd:
        return lib.qknorm_fwd(v("q"), st, v("k"), st, *mid, v("qo"), v("ko"), None)
    return lib.qknorm_bwd(v("dqo"), v("dko"), v("q"), st, v("k"), st, *mid, v("qo"), st, v("ko"), st, v("dwq"), v("dwk"),
                          v("ws"), a["wsb"], None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("over,expect", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(qo=None), INVALID), (dict(ko=None), INVALID),
    (dict(inv=None), INVALID), (dict(RD=15), INVALID), (dict(RD=66), INVALID), (dict(RD=-2), INVALID),
    (dict(kind=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(B=-1), INVALID),
    (dict(S=-1), INVALID), (dict(NHQ=-1), INVALID), (dict(dt=5), UNSUPPORTED), (dict(D=12, RD=4), UNSUPPORTED),
    (dict(D=520, RD=0), UNSUPPORTED), (dict(q=FAKE + 1), INVALID), (dict(wq=FAKE + 2), INVALID),
    (dict(pos=FAKE + 2), INVALID),
])
def test_qknorm_refuses(lib, bwd, over, expect):
    assert qk(lib, bwd, **over) == expect


def test_qknorm_refuses_what_only_one_direction_has(lib):
    assert qk(lib, False, qo=FAKE + 8) == INVALID
    assert qk(lib, True, dqo=None) == INVALID
    assert qk(lib, True, dko=FAKE + 8) == INVALID
    assert qk(lib, True, ws=None) == WORKSPACE and qk(lib, True, wsb=64) == WORKSPACE
    assert lib.qknorm_bwd_workspace_size(2, 3, 4, 2, 12) == 0
    assert qk(lib, False, B=0, q=None, qo=None) == OK and qk(lib, False, NHQ=0, NHK=0) == OK


def test_binding_refuses_what_the_abi_cannot_see():
    q = torch.zeros(1, 2, 4, 64)
    g = torch.zeros(1, 2, 4)
    with pytest.raises(ValueError):   # not on a CUDA device
        binding.gdelta_fwd(q, q, q, g, g)
    with pytest.raises(TypeError):
        binding.gdelta_fwd(q.half(), q.half(), q.half(), g, g)
    with pytest.raises(ValueError):
        binding.qknorm_fwd(q, q)
    with pytest.raises(TypeError):
        binding.qknorm_fwd(q.double(), q.double())
