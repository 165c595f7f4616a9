"""GPU parity of the gated delta rule (gdelta_fwd, gdelta_step, gdelta_bwd) against the fp64 oracle.

Tolerances (relative L2 over a whole tensor).  A float32 output is a sum of float32 products: per chunk
three products of depth at most 128, whose rounding errors add up like a random walk to about
2^-24 sqrt(3 * 128) = 1.2e-6 of the result, and the state carries those of the chunks it remembers;
F32 = 1e-5 leaves room for about seventy chunks' worth.  A gradient multiplies two such results: G32 =
2e-5.  A bf16 output is rounded once more, by at most half a step (2^-8 of every value): BF16 = 2^-8 more.
On the tensor cores the float32 operands enter as bf16 parts whose residue is below 2^-18 of the value,
of the same order, so the bounds are those.
"""
from __future__ import annotations

import pytest
import torch

from oracle import gdelta as oracle
from oracle import qknorm as norm_oracle
from tests.parity import assert_close
from xlstm_mlstm_cell_b200 import binding

pytestmark = pytest.mark.gpu

F32, G32, BF16 = 1e-5, 2e-5, 2.0 ** -8


def tol(x, base=F32):
    return base + (BF16 if x.dtype == torch.bfloat16 else 0.0)


def make(B, NH, NHV, S, DK, DV, dt, seed=0, rate=1.0, key=None):
    """Unit queries and keys, values ~ N(0, 1), gates -rate softplus(N(0, 1)), beta = sigmoid(N(0, 1)), on the GPU."""
    gen = torch.Generator().manual_seed(1000 + seed)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    t = torch.float32 if dt == "f32" else torch.bfloat16
    q, k = r(B, NH, S, DK), r(B, NH, S, DK)
    if key == "same":     # one key, repeated
        k = k[:, :, :1].expand(B, NH, S, DK).contiguous()
    q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    g, beta = -rate * torch.nn.functional.softplus(r(B, NHV, S)), torch.sigmoid(r(B, NHV, S))
    v, do = r(B, NHV, S, DV), r(B, NHV, S, DV)
    S0, dS = r(B, NHV, DK, DV), r(B, NHV, DK, DV)
    c = lambda x, y=t: x.to(y).cuda()   # noqa: E731
    return dict(q=c(q), k=c(k), v=c(v), g=c(g, torch.float32), beta=c(beta, torch.float32), do=c(do),
                S0=c(S0, torch.float32), dS=c(dS, torch.float32))


def args(x):
    return x["q"], x["k"], x["v"], x["g"], x["beta"]


def check_fwd(x, state=False, lengths=None, scale=None, **kw):
    S0 = x["S0"] if state else None
    o, S = binding.gdelta_fwd(*args(x), state=S0, lengths=lengths, scale=scale, **kw)
    ro, rS = oracle.gdelta_fwd(*args(x), state=S0, lengths=lengths, scale=scale)
    torch.cuda.synchronize()
    assert_close("o", o, ro, tol(o))
    assert_close("state", S, rS, F32)
    return o, S


NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dstate0")


def check_bwd(x, state=False, dstate=False, lengths=None, scale=None):
    kw = dict(state=x["S0"] if state else None, dstate=x["dS"] if dstate else None, lengths=lengths, scale=scale)
    got = binding.gdelta_bwd(*args(x), x["do"], **kw)
    ref = oracle.gdelta_bwd(*args(x), x["do"], **kw)
    torch.cuda.synchronize()
    for name, a, b in zip(NAMES, got, ref):
        if a is not None:
            assert_close(name, a, b, tol(a, G32))
    return got


# (B, NH, NHV, S, DK, DV): one token; one short of, exactly and one beyond a chunk; several chunks; head sizes
# from the smallest to the largest, off every tile; one to four value heads per key head
SHAPES = [(1, 1, 1, 1, 8, 8), (2, 1, 3, 63, 64, 64), (1, 2, 2, 64, 128, 128), (3, 1, 2, 65, 128, 64),
          (1, 2, 8, 200, 128, 128), (2, 2, 2, 129, 96, 80), (1, 1, 2, 190, 72, 200), (1, 1, 1, 130, 128, 512),
          (1, 3, 3, 257, 16, 24), (5, 1, 1, 3, 128, 136)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_fwd(shape, dt):
    check_fwd(make(*shape, dt, seed=shape[3]), state=shape[3] % 2 == 1)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_bwd(shape, dt):
    check_bwd(make(*shape, dt, seed=shape[3]), state=shape[3] % 2 == 1, dstate=shape[3] % 3 == 0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [0.0, 1e-3, 4.0, 40.0])
def test_gates_from_keeping_all_to_forgetting_all(rate, dt):
    x = make(1, 2, 4, 150, 64, 64, dt, seed=7, rate=rate)
    check_fwd(x, state=True)
    got = check_bwd(x, state=True, dstate=True)
    assert got[3].abs().max() > 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_full_reset_is_exact(dt):
    """g = -inf empties the memory: the tokens behind it see nothing of those before."""
    x = make(1, 1, 2, 140, 64, 64, dt, seed=8, rate=0.2)
    x["g"][..., 100] = -torch.inf
    o, S = check_fwd(x, state=True)
    y = {n: (t[:, :, 100:].contiguous() if n not in ("S0", "dS") else t) for n, t in x.items()}
    o2, S2 = binding.gdelta_fwd(*args(y))
    assert_close("o behind the reset", o[:, :, 100:], o2.double(), tol(o))
    assert_close("state", S, S2.double(), F32)
    check_bwd(x, state=True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_key_that_repeats(dt):
    """All keys equal and beta near one, nothing forgotten: the triangular system is full of ones, where a
    power series of its inverse would lose everything."""
    x = make(1, 1, 2, 150, 64, 64, dt, seed=9, rate=0.0, key="same")
    x["beta"].fill_(0.97)
    check_fwd(x, state=True)
    check_bwd(x, state=True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_zero_and_negative_writes(dt):
    x = make(1, 1, 2, 100, 64, 64, dt, seed=10, rate=0.3)
    x["beta"][..., ::3] = 0.0
    x["beta"][..., 1::3] *= -0.5
    check_fwd(x, state=True)
    got = check_bwd(x, state=True)
    assert got[4][..., ::3].abs().max() > 0    # a token that writes nothing still has a gradient of beta


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_padding_is_not_read(dt, poison):
    """Whatever stands behind an item's length, also inside its last chunk, changes no bit."""
    x = make(4, 1, 2, 150, 128, 64, dt, seed=12)
    n = torch.tensor([0, 70, 150, 1], dtype=torch.int32, device="cuda")
    o, S = check_fwd(x, state=True, lengths=n)
    got = check_bwd(x, state=True, dstate=True, lengths=n)
    assert torch.equal(S[0], x["S0"][0]) and torch.equal(got[5][0], x["dS"][0])
    for b, m in enumerate(n.tolist()):
        assert not o[b, :, m:].any()
        for y in got[:5]:
            assert not y[b, :, m:].any()
            y[b, :, m:].fill_(7.0)
        for name in ("q", "k", "v", "g", "beta", "do"):
            x[name][b, :, m:] = poison
    o2, S2 = binding.gdelta_fwd(*args(x), state=x["S0"], lengths=n)
    got2 = binding.gdelta_bwd(*args(x), x["do"], state=x["S0"], dstate=x["dS"], lengths=n)
    assert torch.equal(o, o2) and torch.equal(S, S2) and torch.equal(got[5], got2[5])
    for b, m in enumerate(n.tolist()):
        for a, c in zip(got[:5], got2[:5]):
            assert torch.equal(a[b, :, :m], c[b, :, :m]) and not c[b, :, m:].any()


def test_lengths_beyond_the_sequence_are_clamped():
    x = make(2, 1, 1, 66, 64, 64, "bf16", seed=13)
    o, S = binding.gdelta_fwd(*args(x), lengths=torch.tensor([1 << 30, -5], dtype=torch.int32, device="cuda"))
    full, Sf = binding.gdelta_fwd(*args(x))
    assert torch.equal(o[0], full[0]) and torch.equal(S[0], Sf[0]) and not o[1].any() and not S[1].any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_empty_sequence(dt):
    x = make(2, 1, 2, 0, 64, 64, dt)
    o, S = binding.gdelta_fwd(*args(x), state=x["S0"])
    assert o.shape == (2, 2, 0, 64) and torch.equal(S, x["S0"])
    assert not binding.gdelta_fwd(*args(x))[1].any()
    assert torch.equal(binding.gdelta_bwd(*args(x), x["do"], state=x["S0"], dstate=x["dS"])[5], x["dS"])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 8, 8), (3, 2, 4, 128, 128), (2, 1, 3, 96, 40), (1, 2, 2, 128, 512), (40, 4, 16, 64, 64)])
def test_step(shape, dt):
    B, NH, NHV, DK, DV = shape
    x = make(B, NH, NHV, 2, DK, DV, dt, seed=20)
    S = x["S0"].clone()
    for t in range(2):
        tok = [y[:, :, t].contiguous() for y in args(x)]
        o = binding.gdelta_step(S, *tok)
        ro, _ = oracle.gdelta_fwd(*(y[:, :, :t + 1] for y in args(x)), state=x["S0"])
        assert_close("o", o, ro[:, :, t], tol(o))
    assert_close("state", S, oracle.gdelta_fwd(*args(x), state=x["S0"])[1], F32)


def test_prefill_then_steps_equal_one_pass():
    """The run of a serving loop, in place: norms and rotation, prefill, then the same tokens one by one."""
    gen = torch.Generator().manual_seed(30)
    B, S, NH, NHV, D, DV = 2, 75, 2, 4, 64, 128
    proj = torch.randn(B, S, 2 * NH * D + NHV * DV, generator=gen).bfloat16().cuda()
    q, k = proj[..., :NH * D].unflatten(-1, (NH, D)), proj[..., NH * D:2 * NH * D].unflatten(-1, (NH, D))
    v = proj[..., 2 * NH * D:].unflatten(-1, (NHV, DV)).transpose(1, 2).contiguous()
    g = -torch.rand(B, NHV, S, generator=gen).cuda()
    beta = torch.rand(B, NHV, S, generator=gen).cuda()
    inv = (100.0 ** -(torch.arange(0, 32, 2) / 32)).cuda()
    pos = (torch.arange(S, dtype=torch.int32) + 9).expand(B, S).contiguous().cuda()
    how = dict(norm="l2", inv_freq=inv)
    Q, K = binding.qknorm_fwd(q, k, positions=pos, **how)
    rq, rk = (norm_oracle.norm_rotate(x, None, "l2", 1e-6, inv, pos, False) for x in (q, k))
    assert_close("q", Q, rq, BF16 + F32)
    assert_close("k", K, rk, BF16 + F32)
    o, S1 = binding.gdelta_fwd(Q, K, v, g, beta)
    ro, rS = oracle.gdelta_fwd(Q, K, v, g, beta)
    assert_close("o", o, ro, BF16 + F32)
    n = 70
    cut = lambda x: x[:, :, :n].contiguous()   # noqa: E731
    state = torch.zeros(B, NHV, D, DV, device="cuda")
    binding.gdelta_fwd(*(cut(x) for x in (Q, K, v, g, beta)), state=state, state_out=state)
    for t in range(n, S):
        qt, kt = binding.qknorm_fwd(q[:, t:t + 1], k[:, t:t + 1], positions=pos[:, t:t + 1].contiguous(), **how)
        assert torch.equal(qt[:, :, 0], Q[:, :, t]) and torch.equal(kt[:, :, 0], K[:, :, t])
        ot = binding.gdelta_step(state, qt[:, :, 0].contiguous(), kt[:, :, 0].contiguous(), v[:, :, t].contiguous(),
                                 g[:, :, t].contiguous(), beta[:, :, t].contiguous())
        assert_close("o of token %d" % t, ot, ro[:, :, t], BF16 + F32)
    assert_close("state", state, rS, F32)
    assert_close("state of one pass", S1, rS, F32)


def test_training_run_reaches_the_projection():
    """Norms, delta rule and both backward passes: the gradient of the fused projection, written into its
    slices, against autograd through the fp64 definitions."""
    gen = torch.Generator().manual_seed(31)
    B, S, NH, NHV, D, DV = 1, 40, 2, 4, 32, 24
    W = 2 * NH * D + NHV * DV
    proj = torch.randn(B, S, W, generator=gen).cuda()
    wq, wk = (1 + 0.1 * torch.randn(D, generator=gen).cuda() for _ in range(2))
    wk = wk / D ** 0.5
    g = -torch.rand(B, NHV, S, generator=gen).cuda()
    beta = torch.rand(B, NHV, S, generator=gen).cuda()
    do = torch.randn(B, NHV, S, DV, generator=gen).cuda()
    inv = torch.tensor([1.0, 0.1, 0.01, 0.5]).cuda()
    split = lambda p: (p[..., :NH * D].unflatten(-1, (NH, D)), p[..., NH * D:2 * NH * D].unflatten(-1, (NH, D)),   # noqa: E731
                       p[..., 2 * NH * D:].unflatten(-1, (NHV, DV)).transpose(1, 2))
    q, k, v = split(proj)
    how = dict(q_weight=wq, k_weight=wk, inv_freq=inv, interleaved=True)
    Q, K = binding.qknorm_fwd(q, k, **how)
    dQ, dK, dV, dg, db, _ = binding.gdelta_bwd(Q, K, v.contiguous(), g, beta, do)
    dproj = torch.full_like(proj, 7.0)
    dq, dk, dv = split(dproj)
    _, _, dwq, dwk = binding.qknorm_bwd(dQ, dK, q, k, out=(dq, dk), **how)
    dv.copy_(dV)
    leaves = [t.double().requires_grad_(True) for t in (proj, wq, wk, g, beta)]
    pq, pk, pv = split(leaves[0])
    rq = norm_oracle.norm_rotate(pq, leaves[1], "rms", 1e-6, inv, None, True)
    rk = norm_oracle.norm_rotate(pk, leaves[2], "rms", 1e-6, inv, None, True)
    ro, _ = oracle.gdelta_fwd(rq, rk, pv, leaves[3], leaves[4])
    ref = torch.autograd.grad((ro * do.double()).sum(), leaves)
    for name, a, b in zip(("projection", "q_weight", "k_weight", "g", "beta"), (dproj, dwq, dwk, dg, db), ref):
        assert_close(name, a, b, 2 * G32)   # two gradients in a row


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scale_and_large_values(dt):
    x = make(1, 1, 2, 100, 64, 64, dt, seed=40)
    x["v"] *= 4096.0
    x["do"] *= 2.0 ** -10
    check_fwd(x, scale=1.0)
    check_bwd(x, scale=-3.0)


def test_same_inputs_same_bits_and_side_stream():
    x = make(2, 2, 4, 300, 128, 128, "bf16", seed=41)
    a, b = binding.gdelta_fwd(*args(x)), binding.gdelta_bwd(*args(x), x["do"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c, d = binding.gdelta_fwd(*args(x)), binding.gdelta_bwd(*args(x), x["do"])
    side.synchronize()
    for u, w in zip((*a, *b[:5]), (*c, *d[:5])):
        assert torch.equal(u, w)


def test_captured_calls_replay():
    """Forward, step and backward in one CUDA graph, replayed on new values; an eager call in between."""
    x, y = (make(1, 2, 4, 130, 128, 64, "bf16", seed=s) for s in (42, 43))
    st = {n: t.clone() for n, t in x.items()}
    tok = lambda z: [u[:, :, -1].contiguous() for u in args(z)]   # noqa: E731
    step_in = tok(x)
    binding.gdelta_fwd(*args(st)), binding.gdelta_bwd(*args(st), st["do"])   # the first calls set kernel limits
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = binding.gdelta_fwd(*args(st))
        ot = binding.gdelta_step(S, *step_in)
        grads = binding.gdelta_bwd(*args(st), st["do"])
    for z in (x, y, x):
        for n in st:
            st[n].copy_(z[n])
        for u, w in zip(step_in, tok(z)):
            u.copy_(w)
        binding.gdelta_fwd(*args(y))
        graph.replay()
        eo, eS = binding.gdelta_fwd(*args(z))
        eot = binding.gdelta_step(eS, *tok(z))
        eg = binding.gdelta_bwd(*args(z), z["do"])
        torch.cuda.synchronize()
        for u, w in zip((o, S, ot, *grads[:5]), (eo, eS, eot, *eg[:5])):
            assert torch.equal(u, w)


def test_given_outputs_and_workspaces():
    x = make(1, 1, 2, 70, 64, 64, "bf16", seed=44)
    o, S = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    ws = torch.empty(binding.gdelta_workspace_size(1, 1, 2, 70, 64, 64, torch.bfloat16, backward=True), dtype=torch.uint8,
                     device="cuda")
    r = binding.gdelta_fwd(*args(x), o_out=o, state_out=S, workspace=ws)
    assert r[0] is o and r[1] is S and binding.fwd_status(ws) == 0
    assert torch.equal(o, binding.gdelta_fwd(*args(x), return_state=False)[0])
    assert binding.gdelta_fwd(*args(x), return_state=False)[1] is None
    out = tuple(torch.empty_like(t) for t in (*args(x),)) + (torch.empty_like(S),)
    got = binding.gdelta_bwd(*args(x), x["do"], workspace=ws, out=out)
    assert all(a is b for a, b in zip(got, out)) and binding.fwd_status(ws) == 0
    for a, b in zip(got, binding.gdelta_bwd(*args(x), x["do"], state=torch.zeros_like(S))):
        assert torch.equal(a, b)
    with pytest.raises(binding.MlstmError):
        binding.gdelta_fwd(*args(x), workspace=ws[:1024])


def test_refusals_of_the_binding():
    x = make(2, 2, 4, 10, 64, 64, "bf16", seed=45)
    q, k, v, g, beta = args(x)
    bad = [(q.transpose(2, 3), k, v, g, beta), (q, k[:, :, :5], v, g, beta), (q, k, v[:, :, :5], g, beta),
           (q, k, v, g[..., :5], beta), (q, k, v, g, beta.cpu()), (q, k[..., :32], v, g, beta)]
    for a in bad:
        with pytest.raises(ValueError):
            binding.gdelta_fwd(*a)
    for a in [(q, k.float(), v, g, beta), (q, k, v, g.double(), beta), (q, k, v, g, beta.bfloat16())]:
        with pytest.raises(TypeError):
            binding.gdelta_fwd(*a)
    with pytest.raises(TypeError):
        binding.gdelta_fwd(q, k, v, g, beta, lengths=torch.tensor([1, 2], device="cuda"))
    with pytest.raises(ValueError):
        binding.gdelta_fwd(q, k, v, g, beta, state=x["S0"][:1])
    with pytest.raises(binding.MlstmError):   # three value heads on two key heads
        binding.gdelta_fwd(q, k, v[:, :3].contiguous(), g[:, :3].contiguous(), beta[:, :3].contiguous())


@pytest.mark.parametrize("B,NH,NHV,S", [(1, 4, 8, 4096), (40, 2, 4, 320)])
def test_long_and_wide(B, NH, NHV, S):
    """Sixty-four chunks in a row, and more heads than the GPU has SMs; slowly forgetting gates."""
    x = make(B, NH, NHV, S, 128, 128, "bf16", seed=50, rate=0.01)
    check_fwd(x, state=True)
    check_bwd(x, state=True)


@pytest.mark.parametrize("DK,DV,NH,NHV", [(64, 320, 1, 3), (128, 256, 2, 2), (96, 512, 1, 2)])
def test_many_value_columns(DK, DV, NH, NHV):
    """Up to eight stages of 64 value columns in the gradients, several heads of a group, items of every length."""
    x = make(5, NH, NHV, 150, DK, DV, "bf16", seed=60, rate=0.3)
    lengths = torch.tensor([150, 0, 64, 1, 129], dtype=torch.int32, device="cuda")
    check_fwd(x, state=True, lengths=lengths)
    check_bwd(x, state=True, dstate=True, lengths=lengths)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_resets_side_by_side_and_growing_gates(dt):
    """Resets at neighbouring tokens, at a chunk's first and last token, and gates above zero in between."""
    x = make(1, 1, 2, 200, 64, 64, dt, seed=61, rate=0.2)
    x["g"][..., 70:90] = 0.05
    x["g"][..., [0, 10, 11, 12, 63, 64, 127, 128, 199]] = -torch.inf
    check_fwd(x, state=True)
    check_bwd(x, state=True, dstate=True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_nothing_left_in_a_workspace_is_read(dt):
    x = make(3, 1, 2, 150, 64, 64, dt, seed=62)
    lengths = torch.tensor([150, 70, 0], dtype=torch.int32, device="cuda")
    n = binding.gdelta_workspace_size(3, 1, 2, 150, 64, 64, x["q"].dtype, backward=True)
    runs = []
    for fill in (0, 0xff):   # 0xff: NaN of either type
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        a = binding.gdelta_fwd(*args(x), lengths=lengths, workspace=ws)
        ws.fill_(fill)
        runs.append((*a, *binding.gdelta_bwd(*args(x), x["do"], state=x["S0"], lengths=lengths, workspace=ws)))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_states_in_place():
    x = make(2, 2, 4, 100, 128, 64, "bf16", seed=63)
    o, S = binding.gdelta_fwd(*args(x), state=x["S0"])
    own = x["S0"].clone()
    o2, S2 = binding.gdelta_fwd(*args(x), state=own, state_out=own)
    assert S2 is own and torch.equal(S, own) and torch.equal(o, o2)
    ref = binding.gdelta_bwd(*args(x), x["do"], state=x["S0"], dstate=x["dS"])
    d = x["dS"].clone()
    out = tuple(torch.empty_like(t) for t in args(x)) + (d,)
    got = binding.gdelta_bwd(*args(x), x["do"], state=x["S0"], dstate=d, out=out)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


def test_calls_in_flight_on_two_streams():
    """Given streams, workspaces allocated inside: calls run side by side and their memory is not handed on early."""
    xs = [make(2, 2, 2, 300, 128, 128, "bf16", seed=s) for s in (64, 65)]
    ref = [(*binding.gdelta_fwd(*args(x)), *binding.gdelta_bwd(*args(x), x["do"])[:5]) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [(*binding.gdelta_fwd(*args(x), stream=s), *binding.gdelta_bwd(*args(x), x["do"], stream=s)[:5])
               for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert all(torch.equal(u, w) for u, w in zip(a, b))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_step_of_more_heads_than_a_grid_axis_holds(dt):
    x = make(35000, 1, 2, 1, 8, 8, dt, seed=66)
    tok = [t[:, :, 0].contiguous() for t in args(x)]
    S = x["S0"].clone()
    o = binding.gdelta_step(S, *tok)
    ro, rS = oracle.gdelta_fwd(*args(x), state=x["S0"])
    assert_close("o", o, ro[:, :, 0], tol(o))
    assert_close("state", S, rS, F32)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_groups_of_heads_in_one_cta(dt):
    """More chunks than the GPU holds CTAs for: a key head's value heads share one, in preparation and gradients."""
    x = make(40, 1, 3, 130, 16, 72, dt, seed=67, rate=0.3)
    lengths = torch.randint(0, 131, (40,), generator=torch.Generator().manual_seed(68), dtype=torch.int32).cuda()
    check_fwd(x, state=True, lengths=lengths)
    check_bwd(x, state=True, dstate=True, lengths=lengths)


@pytest.mark.parametrize("DV", [48, 136])
def test_tensor_cores_with_groups_in_one_cta(DV):
    x = make(70, 1, 3, 200, 72, DV, "bf16", seed=69, rate=0.3)
    check_fwd(x, state=True)
    check_bwd(x, state=True, dstate=True)
