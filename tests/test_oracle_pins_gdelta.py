"""Pins of the delta rule's and the norms' fp64 oracles (CPU): each against an independent evaluation."""
from __future__ import annotations

import math

import pytest
import torch

from oracle.gdelta import gdelta_bwd, gdelta_fwd
from oracle.qknorm import norm_rotate, norm_rotate_grad


def inputs(B, NH, NHV, S, DK, DV, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)   # noqa: E731
    q, k = r(B, NH, S, DK), r(B, NH, S, DK)
    k = k / k.norm(dim=-1, keepdim=True)
    return (q, k, r(B, NHV, S, DV), -torch.nn.functional.softplus(r(B, NHV, S)), torch.sigmoid(r(B, NHV, S)),
            r(B, NHV, DK, DV), r(B, NHV, S, DV), r(B, NHV, DK, DV))


def test_linear_attention_limit_of_orthonormal_keys():
    """Orthonormal keys predict nothing of one another: S is the plain sum of k v^T, whatever the order."""
    S = 8
    k = torch.linalg.qr(torch.randn(16, S, dtype=torch.float64, generator=torch.Generator().manual_seed(1)))[0].T[None, None]
    v = torch.randn(1, 1, S, 5, dtype=torch.float64, generator=torch.Generator().manual_seed(2))
    one, zero = torch.ones(1, 1, S, dtype=torch.float64), torch.zeros(1, 1, S, dtype=torch.float64)
    o, state = gdelta_fwd(k, k, v, zero, one, scale=1.0)
    assert torch.allclose(state, k.mT @ v, atol=1e-12)
    assert torch.allclose(o, v, atol=1e-12)   # each token reads back its own value


def test_a_repeated_key_replaces_its_value():
    k = torch.nn.functional.normalize(torch.tensor([[1.0, 2.0, -1.0, 0.5]], dtype=torch.float64), dim=-1)
    k = k.expand(6, 4)[None, None].contiguous()
    v = torch.randn(1, 1, 6, 3, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
    one, zero = torch.ones(1, 1, 6, dtype=torch.float64), torch.zeros(1, 1, 6, dtype=torch.float64)
    o, state = gdelta_fwd(k, k, v, zero, one, scale=1.0)
    assert torch.allclose(o, v, atol=1e-12)
    assert torch.allclose(state, k[:, :, -1, :, None] * v[:, :, -1, None, :], atol=1e-12)


def test_transition_matrix_form():
    """S_t = exp(g) (I - beta k k^T) S_{t-1} + beta k v^T, with explicit matrices."""
    q, k, v, g, beta, S0, _, _ = inputs(1, 1, 1, 7, 6, 4, seed=4)
    S = S0[0, 0]
    for t in range(7):
        kt, b = k[0, 0, t], beta[0, 0, t]
        S = math.exp(g[0, 0, t]) * (torch.eye(6, dtype=torch.float64) - b * torch.outer(kt, kt)) @ S + b * torch.outer(kt, v[0, 0, t])
        o, _ = gdelta_fwd(q[:, :, :t + 1], k[:, :, :t + 1], v[:, :, :t + 1], g[..., :t + 1], beta[..., :t + 1], state=S0)
        assert torch.allclose(o[0, 0, t], q[0, 0, t] @ S / math.sqrt(6), atol=1e-12)


def test_lengths_cut_and_split_sequences_agree():
    q, k, v, g, beta, S0, _, _ = inputs(2, 2, 4, 9, 8, 8, seed=5)
    n = torch.tensor([0, 6])
    o, S = gdelta_fwd(q, k, v, g, beta, state=S0, lengths=n)
    assert torch.equal(S[0], S0[0]) and torch.equal(o[0], torch.zeros_like(o[0])) and not o[1, :, 6:].any()
    a, mid = gdelta_fwd(*(x[1:, :, :4] for x in (q, k, v, g, beta)), state=S0[1:])
    b, end = gdelta_fwd(*(x[1:, :, 4:6] for x in (q, k, v, g, beta)), state=mid)
    assert torch.allclose(torch.cat((a, b), 2)[0], o[1, :, :6], atol=1e-13) and torch.allclose(end[0], S[1], atol=1e-13)


@pytest.mark.parametrize("group,lengths", [(1, None), (2, None), (3, (5, 0))])
def test_adjoint_equals_autograd(group, lengths):
    q, k, v, g, beta, S0, do, dS = inputs(2, 2, 2 * group, 9, 8, 16, seed=6 + group)
    n = None if lengths is None else torch.tensor(lengths)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v, g, beta, S0)]
    o, S = gdelta_fwd(*leaves[:5], state=leaves[5], lengths=n)
    ref = torch.autograd.grad((o * do).sum() + (S * dS).sum(), leaves)
    got = gdelta_bwd(q, k, v, g, beta, do, state=S0, dstate=dS, lengths=n, every=4)
    for a, b in zip(got, ref):
        assert torch.allclose(a, b, atol=1e-11, rtol=1e-11)


def test_adjoint_against_differences():
    args = inputs(1, 1, 2, 5, 8, 8, seed=11)
    q, k, v, g, beta, S0, do, dS = args
    got = gdelta_bwd(q, k, v, g, beta, do, state=S0, dstate=dS)

    def loss(x):
        o, S = gdelta_fwd(*x[:5], state=x[5])
        return float((o * do).sum() + (S * dS).sum())

    h = 1e-6
    for i in range(6):
        flat = got[i].reshape(-1)
        for at in range(0, flat.numel(), max(1, flat.numel() // 7)):
            lo, hi = [x.clone() for x in args[:6]], [x.clone() for x in args[:6]]
            lo[i].reshape(-1)[at] -= h
            hi[i].reshape(-1)[at] += h
            assert abs((loss(hi) - loss(lo)) / (2 * h) - float(flat[at])) < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_turns_with_relative_position(interleaved):
    """Rotated queries and keys meet at an angle that depends on the distance of their positions alone."""
    gen = torch.Generator().manual_seed(7)
    q, k = (torch.randn(1, 1, 1, 8, generator=gen) for _ in range(2))
    inv = torch.tensor([1.0, 0.3, 0.02, 0.001])
    at = lambda x, p: norm_rotate(x, None, "l2", 0.0, inv, torch.tensor([[p]]), interleaved)[0, 0, 0]   # noqa: E731
    ref = at(q, 12) @ at(k, 5)
    assert abs(float(ref - at(q, 100012) @ at(k, 100005))) < 1e-9
    assert abs(float(at(q, 3).norm()) - 1) < 1e-12
    assert abs(float(at(q, 0) @ at(k, 0) - torch.nn.functional.cosine_similarity(q.double(), k.double(), -1))) < 1e-12


def test_rotation_by_hand():
    x = torch.tensor([[[[3.0, 4.0, 0.0, 0.0]]]])
    quarter = torch.tensor([math.pi / 2, 0.0])
    rot = lambda i: norm_rotate(x, None, "l2", 0.0, quarter.double(), torch.tensor([[1]]), i)[0, 0, 0]   # noqa: E731
    assert torch.allclose(rot(True), torch.tensor([-0.8, 0.6, 0.0, 0.0], dtype=torch.float64), atol=1e-7)
    assert torch.allclose(rot(False), torch.tensor([0.0, 0.8, 0.6, 0.0], dtype=torch.float64), atol=1e-7)


@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_norm_gradient_formula(norm):
    """dx = r (w d - r^2 x (mean|sum)(w d x)), dw = sum d r x, without a rotation."""
    gen = torch.Generator().manual_seed(8)
    x, w, dy = torch.randn(2, 3, 2, 10, generator=gen).double(), torch.randn(10, generator=gen), torch.randn(2, 2, 3, 10, generator=gen)
    dx, dw = norm_rotate_grad(dy, x, w, norm, 1e-3, None, None, False)
    d, n = dy.double().transpose(1, 2), 10 if norm == "rms" else 1
    r = 1 / torch.sqrt(x.square().sum(-1, keepdim=True) / n + 1e-3)
    ref = r * (w * d - r ** 2 * x * (w * d * x).sum(-1, keepdim=True) / n)
    assert torch.allclose(dx, ref, atol=1e-12) and torch.allclose(dw, (d * r * x).sum((0, 1, 2)), atol=1e-12)
