"""GPU parity of the norms' gradients where the vectors' norms are far from one, against the fp64 oracle.

The tolerances are those of tests/test_qknorm_gpu.py: the arithmetic is the same at every scale as long as no
intermediate leaves fp32's exponents, which is what these cases are about.
"""
from __future__ import annotations

import pytest
import torch

from oracle import qknorm as oracle
from tests.parity import assert_close
from xlstm_mlstm_cell_b200 import binding

pytestmark = pytest.mark.gpu

F32, G32, BF16 = 2e-6, 1e-5, 2.0 ** -8


def make(D, RD, dt, scale, seed):
    gen = torch.Generator().manual_seed(700 + seed)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    t = torch.float32 if dt == "f32" else torch.bfloat16
    x = (scale * r(2, 9, 3, D)).to(t).cuda()
    return x, r(2, 3, 9, D).to(t).cuda(), (1 + 0.3 * r(D)).cuda(), (100.0 ** -(torch.arange(0, RD, 2) / RD)).cuda()


def check(x, dy, w, inv, norm, eps):
    extra = BF16 if x.dtype == torch.bfloat16 else 0.0
    kw = dict(q_weight=w, k_weight=w, norm=norm, eps=eps, inv_freq=inv)
    q, k = binding.qknorm_fwd(x, x, **kw)
    got = binding.qknorm_bwd(dy, dy, x, x, **kw)
    torch.cuda.synchronize()
    ref = (x, w, norm, eps, inv, None, False)
    rx, rw = oracle.norm_rotate_grad(dy, *ref)
    assert_close("y", q, oracle.norm_rotate(*ref), F32 + extra)
    assert_close("dx", got[0], rx, G32 + extra)
    assert_close("dw", got[2], rw, G32)
    for a, b in ((q, k), got[:2], got[2:]):
        assert torch.equal(a, b)
    return got[0], rx


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("scale", [1e-17, 1e-13, 1e13, 1e17])
def test_without_eps(scale, norm, dt):
    """r^3 is no fp32 number at any of these scales; the gradient is."""
    check(*make(64, 32, dt, scale, 1), norm, 0.0)
    check(*make(264, 24, dt, scale, 2), norm, 0.0)   # two units a lane


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_vectors_of_zeros_under_a_small_eps(norm, dt):
    """Every vector is zero: dx = r w d with r = eps^-1/2 = 1e15."""
    x, dy, w, inv = make(64, 32, dt, 0.0, 3)
    dx, _ = check(x, dy, w, inv, norm, 1e-30)
    assert torch.isfinite(dx).all() and dx.abs().max() > 1e14


def test_a_zero_vector_among_others():
    x, dy, w, inv = make(64, 32, "f32", 1.0, 4)
    x[:, 4] = 0
    dx, rx = check(x, dy, w, inv, "l2", 1e-30)
    assert_close("dx of the others", dx[:, :4], rx[:, :4], G32)


def test_given_workspace():
    """As large as the query says, whatever it held; one byte less is refused."""
    x, dy, w, inv = make(64, 32, "bf16", 1.0, 5)
    kw = dict(q_weight=w, k_weight=w, inv_freq=inv)
    n = binding.qknorm_bwd_workspace_size(2, 9, 3, 3, 64)
    ref = binding.qknorm_bwd(dy, dy, x, x, **kw)
    got = binding.qknorm_bwd(dy, dy, x, x, workspace=torch.full((n,), 0xff, dtype=torch.uint8, device="cuda"), **kw)
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    with pytest.raises(binding.MlstmError):
        binding.qknorm_bwd(dy, dy, x, x, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"), **kw)
    assert binding.qknorm_bwd_workspace_size(2, 9, 3, 3, 12) == 0
