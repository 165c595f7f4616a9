"""GPU parity of the per-head norms with the rotation (qknorm_fwd, qknorm_bwd) against the fp64 oracle.

Tolerances (relative L2 over a whole tensor).  In float32 a normed value carries the rounding of a sum of
at most 512 squares, a square root, two products and a rotation, fewer than 32 half steps of 2^-24: F32 = 2e-6;
cosines and sines of an angle reduced in float64 are right to 2^-23.  A gradient subtracts two such terms of
like size and a weight's gradient sums them over all vectors: G32 = 1e-5.  A bf16 output is rounded once more,
by at most half a step: BF16 = 2^-8 more.
"""
from __future__ import annotations

import pytest
import torch

from oracle import qknorm as oracle
from tests.parity import assert_close
from xlstm_mlstm_cell_b200 import binding

pytestmark = pytest.mark.gpu

F32, G32, BF16 = 2e-6, 1e-5, 2.0 ** -8


def make(B, S, NHQ, NHK, D, RD, dt, weight, seed=0, pad=0):
    """q and k as slices of one projection (pad: elements between its rows), on the GPU."""
    gen = torch.Generator().manual_seed(500 + seed)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    t = torch.float32 if dt == "f32" else torch.bfloat16
    proj = (2 * r(B, S, (NHQ + NHK + 1) * D + pad)).to(t).cuda()
    heads = proj[..., pad:].unflatten(-1, (NHQ + NHK + 1, D))
    x = dict(q=heads[:, :, :NHQ], k=heads[:, :, NHQ:NHQ + NHK], dq=r(B, NHQ, S, D).to(t).cuda(),
             dk=r(B, NHK, S, D).to(t).cuda(), how={})
    if weight:
        x["how"].update(q_weight=(1 + 0.3 * r(D)).cuda(), k_weight=(1 + 0.3 * r(D)).cuda())
    if RD:
        x["how"]["inv_freq"] = (10000.0 ** -(torch.arange(0, RD, 2) / RD)).cuda()
        x["how"]["positions"] = torch.randint(0, 131072, (B, S), generator=gen, dtype=torch.int32).cuda()
    return x


def ref_args(x, side, **kw):
    h = {**x["how"], **kw}
    return (x[side], h.get(side + "_weight"), h.get("norm", "rms"), h.get("eps", 1e-6), h.get("inv_freq"),
            h.get("positions"), h.get("interleaved", False))


def check(x, **kw):
    extra = BF16 if x["q"].dtype == torch.bfloat16 else 0.0
    q, k = binding.qknorm_fwd(x["q"], x["k"], **x["how"], **kw)
    got = binding.qknorm_bwd(x["dq"], x["dk"], x["q"], x["k"], **x["how"], **kw)
    torch.cuda.synchronize()
    for side, y, dy, dx, dw in (("q", q, x["dq"], got[0], got[2]), ("k", k, x["dk"], got[1], got[3])):
        a = ref_args(x, side, **kw)
        assert_close(side, y, oracle.norm_rotate(*a), F32 + extra)
        rx, rw = oracle.norm_rotate_grad(dy, *a)
        assert_close("d" + side, dx, rx, G32 + extra)
        assert (dw is None) == (rw is None)
        if dw is not None:
            assert_close("weight of " + side, dw, rw, G32)
    return (q, k, *got)


# (B, S, NHQ, NHK, D, RD): a decode step, odd sizes, partial rotations (halves that are no multiple of a vector
# among them), the smallest and largest heads, more tokens than the launch has CTAs
SHAPES = [(1, 1, 1, 1, 8, 8), (64, 1, 16, 4, 128, 128), (2, 37, 5, 2, 80, 40), (3, 7, 3, 3, 128, 64), (1, 9, 2, 1, 512, 512),
          (2, 5, 4, 4, 96, 94), (1, 33, 2, 2, 24, 6), (2, 6, 3, 1, 200, 0), (1, 2000, 3, 1, 64, 32), (2, 3, 1, 7, 256, 2)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_norms(shape, interleaved, dt):
    norm = "l2" if shape[1] % 2 else "rms"
    check(make(*shape, dt, weight=shape[0] != 2, seed=shape[4]), norm=norm, interleaved=interleaved)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [1, 2, 4])
def test_slices_at_any_element(pad, dt):
    """Vectors that start at odd elements: narrower loads, the same values."""
    check(make(2, 11, 3, 2, 64, 32, dt, weight=True, seed=pad, pad=pad))


def test_far_positions_keep_their_angle():
    """One radian per token at position 2^30: the angle is right to its last bits, not to 64 radians."""
    x = make(1, 4, 2, 2, 16, 16, "f32", weight=False, seed=3)
    x["how"]["positions"] = torch.tensor([[1 << 30, (1 << 30) + 1, (1 << 31) - 1, -(1 << 30)]], dtype=torch.int32).cuda()
    check(x)


def test_positions_default_to_the_token_index():
    x = make(2, 9, 2, 1, 32, 32, "f32", weight=False, seed=4)
    x["how"]["positions"] = torch.arange(9, dtype=torch.int32).expand(2, 9).contiguous().cuda()
    a = binding.qknorm_fwd(x["q"], x["k"], **x["how"])
    b = binding.qknorm_fwd(x["q"], x["k"], inv_freq=x["how"]["inv_freq"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_shared_and_strided_inputs():
    """Heads broadcast from one (stride 0), queries and keys of the same storage, a batch-first view."""
    x = make(3, 5, 1, 1, 64, 16, "bf16", weight=True, seed=5)
    one = x["q"]
    x["q"] = one.expand(3, 5, 4, 64)
    x["k"] = one
    x["dq"] = torch.randn(3, 4, 5, 64, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    check(x)
    y = make(3, 5, 2, 2, 64, 16, "f32", weight=True, seed=7)
    y["q"] = y["q"].transpose(0, 1).contiguous().transpose(0, 1)
    check(y)


def test_gradient_into_slices_of_a_projection():
    x = make(2, 13, 3, 2, 48, 20, "bf16", weight=True, seed=8, pad=6)
    ref = binding.qknorm_bwd(x["dq"], x["dk"], x["q"], x["k"], **x["how"])
    d = torch.full((2, 13, 6 * 48 + 6), 7.0, dtype=torch.bfloat16, device="cuda")
    h = d[..., 6:].unflatten(-1, (6, 48))
    got = binding.qknorm_bwd(x["dq"], x["dk"], x["q"], x["k"], out=(h[:, :, :3], h[:, :, 3:5]), **x["how"])
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    assert (d[..., :6] == 7).all() and (h[:, :, 5] == 7).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_zero_and_tiny_vectors(dt):
    """A vector of zeros stays zero and its gradient is finite: eps alone is under the root."""
    x = make(1, 6, 2, 2, 64, 32, dt, weight=True, seed=9)
    x["q"][:, 2] = 0
    x["k"][:, 3] *= 2.0 ** -40
    y = check(x)
    assert not y[0][:, :, 2].any()


def test_no_queries_no_tokens():
    x = make(2, 4, 2, 2, 32, 16, "f32", weight=True, seed=10)
    q, k = binding.qknorm_fwd(x["q"][:, :, :0], x["k"], **x["how"])
    assert q.shape == (2, 0, 4, 32) and torch.equal(k, binding.qknorm_fwd(x["q"], x["k"], **x["how"])[1])
    how = {n: t for n, t in x["how"].items() if n != "positions"}
    got = binding.qknorm_bwd(x["dq"][:, :, :0].contiguous(), x["dk"][:, :, :0].contiguous(), x["q"][:, :0], x["k"][:, :0], **how)
    assert got[0].numel() == 0 and not got[2].any() and not got[3].any()
    got = binding.qknorm_bwd(x["dq"][:, :0].contiguous(), x["dk"], x["q"][:, :, :0], x["k"], **x["how"])
    assert not got[2].any()


def test_same_bits_in_streams_and_graphs():
    x = make(2, 300, 4, 2, 128, 64, "bf16", weight=True, seed=11)
    ref = (*binding.qknorm_fwd(x["q"], x["k"], **x["how"]), *binding.qknorm_bwd(x["dq"], x["dk"], x["q"], x["k"], **x["how"]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*binding.qknorm_fwd(x["q"], x["k"], **x["how"]),
               *binding.qknorm_bwd(x["dq"], x["dk"], x["q"], x["k"], **x["how"]))
    for _ in range(2):
        for t in got:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, got):
            assert torch.equal(a, b)


def test_refusals_of_the_binding():
    x = make(2, 4, 2, 2, 32, 16, "f32", weight=True, seed=12)
    q, k, inv = x["q"], x["k"], x["how"]["inv_freq"]
    for a, kw in [((q, k[:, :3]), {}), ((q, k.bfloat16()), {}), ((q.transpose(2, 3), k), {}), ((q, k), dict(norm="max")),
                  ((q, k), dict(positions=x["how"]["positions"])), ((q, k), dict(inv_freq=torch.ones(17).cuda())),
                  ((q, k), dict(q_weight=torch.ones(16).cuda())),
                  ((q, k), dict(inv_freq=inv, positions=x["how"]["positions"][:, :3]))]:
        with pytest.raises(ValueError):
            binding.qknorm_fwd(*a, **kw)
    with pytest.raises(TypeError):
        binding.qknorm_fwd(q, k, inv_freq=inv, positions=x["how"]["positions"].long())
    with pytest.raises(ValueError):
        binding.qknorm_bwd(x["dq"].transpose(1, 2), x["dk"], q, k)
    with pytest.raises(binding.MlstmError):
        binding.qknorm_fwd(q, k, eps=-1.0)
