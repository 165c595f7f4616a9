"""How far the tensor-core path of the delta rule is from fp64 on its float32 outputs, and on bf16 ones from one
rounding (bf16 inputs; relative L2 over a whole tensor).

h = 2^-24, half a step of fp32.  A tcgen05 MMA cuts its sum off where fp32 ends: on average 0.69 h of the running sum
(half a step 2^-24 over a mantissa between 1 and 2), always towards zero, so that these add up.  The sum grows over the
MMAs of a product, half its final size on average.  A chunk's contribution to the state passes three products: K S in
eight MMAs (4.5 times its size in all), (T - I) Y in four of full size (2.5; those of the second and third parts of
T - I come first and are small), K^T N in four (2.5): 9.5 * 0.69 h = 6.6 h if every one of them acts on all of the result.
The eight roundings of the passes in between are independent, 0.41 h each: 1.2 h.  STATE = 8 h = 4.8e-7, for the state.
Backwards the last product takes Q's tokens too, eight MMAs: 7.9 h and 1.2 h, DSTATE = 10 h = 6.0e-7, for the initial
state's gradient.  The gradients of the gates and of beta multiply what the two walks left, 18 h, in products of eight MMAs of
full size between two additions in registers, 3 h: GATES = 21 h = 1.25e-6.
"""
from __future__ import annotations

import pytest
import torch

from oracle import gdelta as oracle
from tests.parity import assert_close
from xlstm_mlstm_cell_b200 import binding

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
STATE, DSTATE, GATES = 8 * H, 10 * H, 21 * H
BF16 = 2.0 ** -8 / 3 ** 0.5   # the error of one rounding is spread evenly over half a step to either side


def make(B, NH, NHV, S, DK, DV, rate, seed, same=False):
    """Unit queries and keys, gates -rate softplus(N(0, 1)), beta = sigmoid(N(0, 1)), on the GPU.  same: one key per
    head, repeated, with beta 0.97 and nothing forgotten: what is written next is what is there already."""
    gen = torch.Generator().manual_seed(900 + seed)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).bfloat16().cuda()   # noqa: E731
    q, k = unit(r(B, NH, S, DK)), unit(r(B, NH, S, DK))
    g = (-rate * torch.nn.functional.softplus(r(B, NHV, S))).cuda()
    beta = torch.sigmoid(r(B, NHV, S)).cuda()
    if same:
        k = k[:, :, :1].expand_as(k).contiguous()
        g, beta = torch.zeros_like(g), torch.full_like(beta, 0.97)
    v, do = r(B, NHV, S, DV).bfloat16().cuda(), r(B, NHV, S, DV).bfloat16().cuda()
    S0, dS = 0.3 * r(B, NHV, DK, DV).cuda(), 0.3 * r(B, NHV, DK, DV).cuda()
    return (q, k, v, g, beta), do, S0, dS


def moved(x, gen):
    """x in float64, every element off by up to one step of fp32 either way."""
    return x.double() * (1 + (2 * torch.rand(x.shape, generator=gen, device="cuda", dtype=torch.float64) - 1) * 2 * H)


# few heads run as CTAs of 32 value columns, the 40 heads as CTAs of 64
SHAPES = [(2, 4, 8, 500, 128, 128), (5, 4, 8, 500, 128, 128), (2, 2, 4, 500, 64, 128), (40, 1, 2, 300, 64, 64),
          (2, 2, 4, 500, 128, 256), (3, 1, 2, 333, 72, 40)]


@pytest.mark.parametrize("rate", [0.0, 0.02, 0.2, 1.0])
@pytest.mark.parametrize("shape", SHAPES)
def test_state(shape, rate):
    x, _, S0, _ = make(*shape, rate, seed=shape[3])
    assert binding.gdelta_fwd_tensor_path(shape[4], shape[5], torch.bfloat16) == 1
    o, S = binding.gdelta_fwd(*x, state=S0)
    ro, rS = oracle.gdelta_fwd(*x, state=S0)
    torch.cuda.synchronize()
    assert_close("state", S, rS, STATE)
    assert_close("o", o, ro, BF16)


@pytest.mark.parametrize("B", [1, 40])
@pytest.mark.parametrize("DK", [64, 128])
def test_state_of_a_repeated_key(DK, B):
    """The state is what is left of sums that nearly cancel: the bound is four times what fp64 itself makes of inputs
    that are off by up to one step of fp32, one for each product a token's value passes (the system's inverse, K S,
    T Y, K^T N), on top of the rounding of the result."""
    x, _, S0, _ = make(B, 2, 4, 300, DK, 128, 0.0, seed=DK, same=True)
    S = binding.gdelta_fwd(*x, state=S0)[1]
    rS = oracle.gdelta_fwd(*x, state=S0)[1]
    gen = torch.Generator("cuda").manual_seed(1)
    mS = oracle.gdelta_fwd(*(moved(t, gen) for t in x), state=moved(S0, gen))[1]
    torch.cuda.synchronize()
    assert_close("state", S, rS, STATE + 4 * float((mS - rS).norm() / rS.norm()))


NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dstate0")
BOUNDS = (BF16, BF16, BF16, GATES, GATES, DSTATE)


@pytest.mark.parametrize("rate", [0.0, 0.02, 0.2, 1.0])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients(shape, rate):
    x, do, S0, dS = make(*shape, rate, seed=shape[3] + 1)
    got = binding.gdelta_bwd(*x, do, state=S0, dstate=dS)
    ref = oracle.gdelta_bwd(*x, do, state=S0, dstate=dS)
    torch.cuda.synchronize()
    for name, a, b, bound in zip(NAMES, got, ref, BOUNDS):
        assert_close(name, a, b, bound)


@pytest.mark.parametrize("B", [1, 40])
@pytest.mark.parametrize("DK", [64, 128])
def test_gradients_of_a_repeated_key(DK, B):
    """As for the state; seven products stand behind a gradient of a gate: those of the two walks, and its own."""
    x, do, S0, dS = make(B, 2, 4, 300, DK, 128, 0.0, seed=DK + 1, same=True)
    got = binding.gdelta_bwd(*x, do, state=S0, dstate=dS)
    ref = oracle.gdelta_bwd(*x, do, state=S0, dstate=dS)
    gen = torch.Generator("cuda").manual_seed(2)
    off = oracle.gdelta_bwd(*(moved(t, gen) for t in x), moved(do, gen), state=moved(S0, gen), dstate=moved(dS, gen))
    torch.cuda.synchronize()
    for name, a, b, c, bound, products in list(zip(NAMES, got, ref, off, BOUNDS, (7, 7, 4, 7, 7, 4)))[3:]:
        assert_close(name, a, b, bound + products * float((c - b).norm() / b.norm()))
