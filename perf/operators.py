"""What the gated delta rule and the per-head query/key norms are measured on.

``listed()`` gives the measured cases, ``draw(rng)`` one more of the same ranges, ``prepare`` a
case's inputs on the GPU and ``run`` one pass through an operator: in its plain form (elementary
torch operations in float32) or, where ``own`` is true, through the library's entry points.
``exact`` evaluates the definitions token by token in float64 and ``work`` counts the bytes and
operations that a pass cannot do without.

The gated delta rule, per value head with a state S [DK][DV], token by token:
    S <- e^g S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q.
The norms: y = rotate(w * x / sqrt(mean(x^2) + eps)) (or sum instead of mean, "l2"), per head of a
fused projection [B, S, heads, D], written head by head as [B, heads, S, D].
"""
import math

import torch

own = False

CHUNK = 64
BASE = 10000.0


def listed():
    d = dict(DK=128, DV=128, dtype="bf16", state=False, ragged=False)
    return [
        # a short prompt appended to a running conversation: starts from a state, ends inside a chunk
        dict(d, name="gdelta_fwd_resume", op="gdelta_fwd", B=2, NH=4, NHV=8, S=200, state=True),
        # the prefill of one long prompt: the chain over the chunks is what counts
        dict(d, name="gdelta_fwd_long", op="gdelta_fwd", B=1, NH=16, NHV=32, S=16384),
        # a serving batch padded to its longest prompt, more heads than the GPU has SMs
        dict(d, name="gdelta_fwd_padded", op="gdelta_fwd", B=16, NH=8, NHV=16, S=2048, ragged=True),
        # float32 with head sizes that fill no tile
        dict(d, name="gdelta_fwd_f32_odd", op="gdelta_fwd", B=2, NH=6, NHV=6, S=777, DK=96, DV=200, dtype="f32"),
        # a training step's gradients, value heads in pairs over one key head
        dict(d, name="gdelta_bwd_train", op="gdelta_bwd", B=4, NH=8, NHV=16, S=4096),
        # gradients in float32 over three value heads per key head, from a state, odd sizes
        dict(d, name="gdelta_bwd_f32_odd", op="gdelta_bwd", B=1, NH=4, NHV=12, S=333, DK=64, DV=72, dtype="f32",
             state=True),
        # decode: one token for one sequence (latency) and for a full batch (the state's bandwidth)
        dict(d, name="gdelta_step_one", op="gdelta_step", B=1, NH=16, NHV=32),
        dict(d, name="gdelta_step_batch", op="gdelta_step", B=256, NH=16, NHV=32),
        # the norms and the rotation in front of the long prefill, of a decode step, and of training
        dict(name="qknorm_fwd_long", op="qknorm_fwd", B=1, S=16384, NHQ=16, NHK=16, D=128, RD=64, dtype="bf16",
             norm="rms", weight=True, interleaved=False),
        dict(name="qknorm_fwd_decode", op="qknorm_fwd", B=64, S=1, NHQ=16, NHK=16, D=128, RD=128, dtype="bf16",
             norm="rms", weight=True, interleaved=False),
        dict(name="qknorm_bwd_train", op="qknorm_bwd", B=4, S=4096, NHQ=16, NHK=4, D=128, RD=128, dtype="bf16",
             norm="rms", weight=True, interleaved=False),
        # float32 without weights, as the delta rule's unit keys, a partial interleaved rotation, odd sizes
        dict(name="qknorm_bwd_f32_odd", op="qknorm_bwd", B=3, S=501, NHQ=5, NHK=2, D=80, RD=40, dtype="f32",
             norm="l2", weight=False, interleaved=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gdelta_fwd", "gdelta_fwd", "gdelta_bwd", "gdelta_bwd", "gdelta_step", "qknorm_fwd", "qknorm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("qknorm"):
        NHQ, D = _log(rng, 1, 32), 8 * rng.randint(4, 32)
        NHK = rng.randint(1, NHQ)
        # no more elements than the listed training step has
        tokens = 4 * 4096 * 20 * 128 // ((NHQ + NHK) * D * (2 if dtype == "f32" else 1))
        S = _log(rng, 1, min(16384, tokens))
        B = _log(rng, 1, max(1, min(256, tokens // S)))
        return dict(op=op, B=B, S=S, NHQ=NHQ, NHK=NHK, D=D,
                    RD=rng.choice([0, D, 2 * rng.randint(1, D // 2)]), dtype=dtype, norm=rng.choice(["rms", "l2"]),
                    weight=rng.random() < 0.5, interleaved=rng.random() < 0.5)
    NH, group = _log(rng, 1, 16), rng.choice([1, 2, 3, 4])
    c = dict(op=op, NH=NH, NHV=NH * group, DK=rng.choice([128, 128, 64, 8 * rng.randint(2, 16)]),
             DV=rng.choice([128, 128, 256, 8 * rng.randint(2, 32)]), dtype=dtype)
    if op == "gdelta_step":
        return dict(c, B=_log(rng, 1, max(1, 256 * 32 * 128 * 128 // (c["NHV"] * c["DK"] * c["DV"]))), state=False,
                    ragged=False)
    top = (16384 if op == "gdelta_fwd" else 4096) * (16 if dtype == "f32" else 32)
    S = _log(rng, 1, 16384 if op == "gdelta_fwd" else 4096)
    B = _log(rng, 1, max(1, min(32, top * 128 * 128 // (S * c["NHV"] * c["DK"] * c["DV"]))))
    S = min(S, max(1, top * 128 * 128 // (B * c["NHV"] * c["DK"] * c["DV"])))
    return dict(c, B=B, S=S, state=rng.random() < 0.4, ragged=rng.random() < 0.3)


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    c, dt = case, _type(case)
    if c["op"].startswith("qknorm"):
        B, S, NHQ, NHK, D, RD = (c[x] for x in ("B", "S", "NHQ", "NHK", "D", "RD"))
        # one fused projection [q | k | v], of which the operator reads slices
        proj = (1.5 * randn(B, S, (NHQ + 2 * NHK) * D)).to(dt)
        heads = proj.view(B, S, NHQ + 2 * NHK, D)
        st = dict(case=c, q=heads[:, :, :NHQ], k=heads[:, :, NHQ:NHQ + NHK], wq=None, wk=None, inv_freq=None,
                  positions=None)
        if c["weight"]:
            st["wq"], st["wk"] = 1 + 0.2 * randn(D), 1 + 0.2 * randn(D)
        if RD:
            st["inv_freq"] = (BASE ** (-torch.arange(0, RD, 2, dtype=torch.float64, device="cuda") / RD)).float()
            # the place of each sequence in a context of up to 131072 tokens
            first = torch.randint(0, 131072 - S, (B, 1), generator=gen, device="cuda")
            st["positions"] = (first + torch.arange(S, device="cuda")).int()
        if c["op"] == "qknorm_bwd":
            st["dq_out"], st["dk_out"] = randn(B, NHQ, S, D).to(dt), randn(B, NHK, S, D).to(dt)
        return st
    B, NH, NHV, DK, DV = (c[x] for x in ("B", "NH", "NHV", "DK", "DV"))
    T = (c["S"],) if "S" in c else ()
    q, k = randn(B, NH, *T, DK), randn(B, NH, *T, DK)
    # unit queries and keys, forget rates from 0.02 to 2.7 per token, write strengths in (0, 1)
    rate = torch.exp(5 * torch.rand((1, NHV) + (1,) * len(T), generator=gen, device="cuda") - 4)
    st = dict(case=c, scale=DK ** -0.5, q=(q / q.norm(dim=-1, keepdim=True)).to(dt),
              k=(k / k.norm(dim=-1, keepdim=True)).to(dt), v=randn(B, NHV, *T, DV).to(dt),
              g=-rate * torch.nn.functional.softplus(randn(B, NHV, *T)), beta=torch.sigmoid(randn(B, NHV, *T)),
              state=None, lengths=None, do=None)
    if c["state"] or c["op"] == "gdelta_step":
        st["state"] = 0.3 * randn(B, NHV, DK, DV)
    if c["ragged"]:
        n = torch.randint(1, c["S"] + 1, (B,), generator=gen, device="cuda")
        n[0] = c["S"]
        st["lengths"] = n.int()
    if c["op"] == "gdelta_bwd":
        st["do"] = randn(B, NHV, *T, DV).to(dt)
    return st


# ---------------------------------------------------------------- the plain forms

def _live(st):
    """[B, 1, S] truth values: the tokens that are no padding."""
    B, S = st["q"].shape[0], st["q"].shape[2]
    t = torch.arange(S, device="cuda")
    n = torch.full((B,), S, device="cuda") if st["lengths"] is None else st["lengths"]
    return (t[None, :] < n[:, None])[:, None, :]


def _chunks(st):
    """The inputs in float32, padding as zeros, value heads side by side, cut into chunks, and what
    each chunk needs of itself alone: decays, scores and the inverse of its triangular system."""
    c = st["case"]
    B, NH, NHV, S = c["B"], c["NH"], c["NHV"], c["S"]
    n = -(-S // CHUNK)
    live = _live(st)

    def cut(x, heads):
        x = torch.where(live if x.dim() == 3 else live[..., None], x.float(), 0.0)
        x = x.repeat_interleave(NHV // heads, dim=1)
        x = torch.nn.functional.pad(x, ((0, 0) if x.dim() == 4 else ()) + (0, n * CHUNK - S))
        return x.reshape(B, NHV, n, CHUNK, *x.shape[3:])

    w = dict(q=cut(st["q"], NH), k=cut(st["k"], NH), v=cut(st["v"], NHV), g=cut(st["g"], NHV),
             beta=cut(st["beta"], NHV)[..., None])
    if st["do"] is not None:
        w["do"] = cut(st["do"], NHV)
    a = w["g"].cumsum(-1)
    i = torch.arange(CHUNK, device="cuda")
    below = i[:, None] > i[None, :]
    at = below | (i[:, None] == i[None, :])
    w["decay"] = torch.exp(torch.where(at, a[..., :, None] - a[..., None, :], -torch.inf))
    w["kk"] = torch.where(below, w["decay"] * (w["k"] @ w["k"].mT), 0.0)
    w["p"] = w["decay"] * (w["q"] @ w["k"].mT)
    w["in"], w["out"], w["all"] = a.exp()[..., None], (a[..., -1:] - a).exp()[..., None], a[..., -1].exp()[..., None, None]
    # T = (I + kk diag(beta))^-1, a row at a time
    m = w["kk"] * w["beta"].mT
    T = torch.eye(CHUNK, device="cuda").expand(m.shape).clone()
    for r in range(1, CHUNK):
        T[..., r, :r] = -(m[..., r:r + 1, :r] @ T[..., :r, :r])[..., 0, :]
    w["T"] = T
    return w


def _walk(st, w):
    """The states at the chunks' starts, the state after the last, and e = v - S^T k of every token."""
    c = st["case"]
    S = st["state"] if st["state"] is not None else torch.zeros(c["B"], c["NHV"], c["DK"], c["DV"], device="cuda")
    starts, errs = [], []
    for j in range(w["k"].shape[2]):
        starts.append(S)
        k = w["k"][:, :, j]
        e = w["T"][:, :, j] @ (w["v"][:, :, j] - w["in"][:, :, j] * (k @ S))
        S = w["all"][:, :, j] * S + k.mT @ (w["out"][:, :, j] * w["beta"][:, :, j] * e)
        errs.append(e)
    return torch.stack(starts, 2), S, torch.stack(errs, 2)


def _joined(x, S):
    """Chunks [B, H, n, 64, ...] as tokens [B, H, S, ...]."""
    return x.flatten(2, 3)[:, :, :S]


def _plain_fwd(st):
    c, w = st["case"], _chunks(st)
    starts, S, e = _walk(st, w)
    o = st["scale"] * (w["in"] * (w["q"] @ starts) + w["p"] @ (w["beta"] * e))
    o = torch.where(_live(st)[..., None], _joined(o, c["S"]), 0.0)
    return {"o": o.to(_type(c)), "state": S}


def _plain_bwd(st):
    c, w, scale = st["case"], _chunks(st), st["scale"]
    starts, _, e = _walk(st, w)
    u, do = w["beta"] * e, w["do"]
    dS = torch.zeros_like(starts[:, :, 0])
    ends, dvs, dus = [], [], []
    pdo = scale * (w["p"].mT @ do)
    for j in range(w["k"].shape[2] - 1, -1, -1):
        ends.append(dS)
        k, q = w["k"][:, :, j], w["q"][:, :, j]
        du = pdo[:, :, j] + w["out"][:, :, j] * (k @ dS)
        dv = w["T"][:, :, j].mT @ (w["beta"][:, :, j] * du)
        dS = (w["all"][:, :, j] * dS + scale * (q.mT @ (w["in"][:, :, j] * do[:, :, j]))
              - k.mT @ (w["in"][:, :, j] * dv))
        dvs.append(dv)
        dus.append(du)
    ends, dv, du = (torch.stack(x[::-1], 2) for x in (ends, dvs, dus))
    du = du - w["kk"].mT @ dv
    dP = scale * (do @ u.mT)
    dA = -(dv @ u.mT)
    # what every pair of tokens, and every token with the states around its chunk, gives through its decay
    from_start_q, from_start_k = scale * w["in"] * (do @ starts.mT), -w["in"] * (dv @ starts.mT)
    to_end = w["out"] * (u @ ends.mT)
    before = lambda x: torch.nn.functional.pad(x[..., :-1], (1, 0)).cumsum(-1)  # noqa: E731 - the sum over j < t
    i = torch.arange(CHUNK, device="cuda")
    pairs = torch.where(i[:, None] >= i[None, :], before(dP * w["p"] + dA * w["kk"]), 0.0).sum(-2)
    z_in = (from_start_q * w["q"] + from_start_k * w["k"]).sum(-1)
    z_out = (to_end * w["k"]).sum(-1)
    dg = (z_in.flip(-1).cumsum(-1).flip(-1) + before(z_out) + pairs
          + w["all"][..., 0] * (starts * ends).sum((-2, -1))[..., None])
    dP, dA = dP * w["decay"], torch.where(i[:, None] > i[None, :], dA * w["decay"], 0.0)
    dq = from_start_q + dP @ w["k"]
    dk = from_start_k + to_end + dP.mT @ w["q"] + dA @ w["k"] + dA.mT @ w["k"]
    live = _live(st)

    def shared(x):  # the value heads of one key head add up
        x = _joined(x, c["S"]).reshape(c["B"], c["NH"], -1, c["S"], c["DK"]).sum(2)
        return torch.where(live[..., None], x, 0.0).to(_type(c))

    return {"dq": shared(dq), "dk": shared(dk), "dv": torch.where(live[..., None], _joined(dv, c["S"]), 0.0).to(_type(c)),
            "dg": torch.where(live, _joined(dg, c["S"]), 0.0),
            "dbeta": torch.where(live, _joined((du * e).sum(-1), c["S"]), 0.0),
            "dstate": dS if st["state"] is not None else None}


def _plain_step(st):
    c, S = st["case"], st["state"]
    q, k = (st[x].float().repeat_interleave(c["NHV"] // c["NH"], dim=1) for x in ("q", "k"))
    S.mul_(st["g"].exp()[..., None, None])
    u = st["beta"][..., None] * (st["v"].float() - (S * k[..., None]).sum(-2))
    S.add_(k[..., None] * u[..., None, :])
    return {"o": (st["scale"] * (S * q[..., None]).sum(-2)).to(_type(c)), "state": S}


def _angles(st):
    a = st["positions"].double()[:, :, None, None] * st["inv_freq"].double()
    return a.cos().float(), a.sin().float()


def _halves(x, rd, interleaved):
    r = x[..., :rd]
    return (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rd // 2], r[..., rd // 2:])


def _join(a, b, rest, interleaved):
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _inv_norm(x, norm):
    s = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((s / x.shape[-1] if norm == "rms" else s) + 1e-6)


def _plain_norm(st, x, w):
    c, x = st["case"], x.float()
    y = x * _inv_norm(x, c["norm"])
    y = y if w is None else y * w
    if c["RD"]:
        cos, sin = _angles(st)
        a, b = _halves(y, c["RD"], c["interleaved"])
        y = _join(a * cos - b * sin, a * sin + b * cos, y[..., c["RD"]:], c["interleaved"])
    return y.to(_type(c)).transpose(1, 2).contiguous()


def _plain_norm_grad(st, x, w, dy):
    c, x, d = st["case"], x.float(), dy.float().transpose(1, 2)
    if c["RD"]:
        cos, sin = _angles(st)
        a, b = _halves(d, c["RD"], c["interleaved"])
        d = _join(a * cos + b * sin, b * cos - a * sin, d[..., c["RD"]:], c["interleaved"])
    r = _inv_norm(x, c["norm"])
    xh = x * r
    dw = None if w is None else (d * xh).sum((0, 1, 2))
    d = d if w is None else d * w
    s = (d * xh).sum(-1, keepdim=True)
    return (r * (d - xh * (s / x.shape[-1] if c["norm"] == "rms" else s))).to(_type(c)), dw


# ---------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    if own:
        return _own(state)
    if c["op"] == "gdelta_fwd":
        return _plain_fwd(state)
    if c["op"] == "gdelta_bwd":
        return _plain_bwd(state)
    if c["op"] == "gdelta_step":
        return _plain_step(state)
    if c["op"] == "qknorm_fwd":
        return {"q": _plain_norm(state, state["q"], state["wq"]), "k": _plain_norm(state, state["k"], state["wk"])}
    dq, dwq = _plain_norm_grad(state, state["q"], state["wq"], state["dq_out"])
    dk, dwk = _plain_norm_grad(state, state["k"], state["wk"], state["dk_out"])
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}


def _own(st):
    from xlstm_mlstm_cell_b200 import binding
    c = st["case"]
    if c["op"] == "gdelta_fwd":
        o, S = binding.gdelta_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], state=st["state"],
                                  lengths=st["lengths"], scale=st["scale"])
        return {"o": o, "state": S}
    if c["op"] == "gdelta_bwd":
        names = ("dq", "dk", "dv", "dg", "dbeta", "dstate")
        return dict(zip(names, binding.gdelta_bwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["do"],
                                                  state=st["state"], lengths=st["lengths"], scale=st["scale"])))
    if c["op"] == "gdelta_step":
        o = binding.gdelta_step(st["state"], st["q"], st["k"], st["v"], st["g"], st["beta"], scale=st["scale"])
        return {"o": o, "state": st["state"]}
    how = dict(q_weight=st["wq"], k_weight=st["wk"], norm=c["norm"], eps=1e-6, inv_freq=st["inv_freq"],
               positions=st["positions"], interleaved=c["interleaved"])
    if c["op"] == "qknorm_fwd":
        q, k = binding.qknorm_fwd(st["q"], st["k"], **how)
        return {"q": q, "k": k}
    names = ("dq", "dk", "dq_weight", "dk_weight")
    return dict(zip(names, binding.qknorm_bwd(st["dq_out"], st["dk_out"], st["q"], st["k"], **how)))


# ---------------------------------------------------------------- the definitions in 64 bits

def _tokens(st):
    """Per token in float64: q, k, v, e^g, beta (and do) as [heads, ...], padding with beta = 0, e^g = 1, q = 0."""
    c, live = st["case"], _live(st)
    G = c["NHV"] // c["NH"]

    def wide(x):
        x = torch.where(live if x.dim() == 3 else live[..., None], x.double(), 0.0)
        return x.flatten(0, 1)

    q, k = (wide(st[x].repeat_interleave(G, dim=1)) for x in ("q", "k"))
    return q * st["scale"], k, wide(st["v"]), wide(st["g"]).exp(), wide(st["beta"]), st["do"] is not None and wide(st["do"])


def _first_state(st):
    c = st["case"]
    if st["state"] is not None:
        return st["state"].double().flatten(0, 1)
    return torch.zeros(c["B"] * c["NHV"], c["DK"], c["DV"], dtype=torch.float64, device="cuda")


def _token(S, k, v, f, b):
    D = S * f[:, None, None]
    e = v - torch.bmm(k[:, None, :], D)[:, 0]
    return D, e, torch.baddbmm(D, k[:, :, None], (b[:, None] * e)[:, None, :])


def _exact_fwd(st):
    c = st["case"]
    q, k, v, f, b, _ = _tokens(st)
    S, out = _first_state(st), torch.empty_like(v)
    for t in range(c["S"]):
        _, _, S = _token(S, k[:, t], v[:, t], f[:, t], b[:, t])
        out[:, t] = torch.bmm(q[:, t, None, :], S)[:, 0]
    return {"o": out.view(st["v"].shape), "state": S.view(c["B"], c["NHV"], c["DK"], c["DV"])}


def _exact_bwd(st):
    c, seg = st["case"], 64
    q, k, v, f, b, do = _tokens(st)
    S, marks = _first_state(st), []
    for t in range(c["S"]):
        if t % seg == 0:
            marks.append(S)
        _, _, S = _token(S, k[:, t], v[:, t], f[:, t], b[:, t])
    dS = torch.zeros_like(S)
    dq, dk, dv, dg, db = (torch.empty_like(x) for x in (q, k, v, f, b))
    for j in range(len(marks) - 1, -1, -1):
        S, kept = marks[j], []
        for t in range(j * seg, min(c["S"], (j + 1) * seg)):
            D, e, S = _token(S, k[:, t], v[:, t], f[:, t], b[:, t])
            kept.append((t, D, e, S))
        for t, D, e, S in reversed(kept):
            dq[:, t] = st["scale"] * torch.bmm(S, do[:, t, :, None])[..., 0]
            dS = torch.baddbmm(dS, q[:, t, :, None], do[:, t, None, :])
            du = torch.bmm(k[:, t, None, :], dS)[:, 0]
            de = b[:, t, None] * du
            db[:, t] = (du * e).sum(-1)
            dv[:, t] = de
            dk[:, t] = torch.bmm(dS, (b[:, t, None] * e)[..., None])[..., 0] - torch.bmm(D, de[..., None])[..., 0]
            dS = torch.baddbmm(dS, k[:, t, :, None], de[:, None, :], alpha=-1)
            dg[:, t] = (dS * D).sum((-2, -1))
            dS = dS * f[:, t, None, None]
    live, shape = _live(st), (c["B"], c["NHV"], c["S"])

    def rows(x):
        return torch.where(live[..., None], x.view(*shape, -1), 0.0)

    def shared(x):
        return rows(x).view(c["B"], c["NH"], -1, c["S"], c["DK"]).sum(2)

    return {"dq": shared(dq), "dk": shared(dk), "dv": rows(dv), "dg": torch.where(live, dg.view(shape), 0.0),
            "dbeta": torch.where(live, db.view(shape), 0.0),
            "dstate": dS.view(c["B"], c["NHV"], c["DK"], c["DV"]) if st["state"] is not None else None}


def _turns(st):
    """e^(i angle) of every token and pair, complex128."""
    return torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       st["positions"].double()[..., None] * st["inv_freq"].double())[:, :, None, :]


def _turned(x, turn, rd, interleaved):
    """x with its first rd elements, as rd / 2 complex numbers, times `turn`."""
    r = x[..., :rd].unflatten(-1, (-1, 2) if interleaved else (2, -1))
    r = r if interleaved else r.mT
    r = torch.view_as_real(torch.view_as_complex(r.contiguous()) * turn)
    return torch.cat(((r if interleaved else r.mT).flatten(-2), x[..., rd:]), -1)


def _exact_norm(st, x, w, dy=None):
    c, x = st["case"], x.double()
    n = c["D"] if c["norm"] == "rms" else 1
    length = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / n + 1e-6)
    weight = torch.ones(c["D"], dtype=torch.float64, device="cuda") if w is None else w.double()
    if dy is None:
        y = x / length * weight
        return (_turned(y, _turns(st), c["RD"], c["interleaved"]) if c["RD"] else y).transpose(1, 2)
    d = dy.double().transpose(1, 2)
    d = _turned(d, _turns(st).conj(), c["RD"], c["interleaved"]) if c["RD"] else d
    dw = None if w is None else (d * x / length).sum((0, 1, 2))
    d = d * weight
    return d / length - x * (d * x).sum(-1, keepdim=True) / (n * length ** 3), dw


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "gdelta_fwd":
        return _exact_fwd(st)
    if case["op"] == "gdelta_bwd":
        return _exact_bwd(st)
    if case["op"] == "gdelta_step":
        G = case["NHV"] // case["NH"]
        k, q = (st[x].double().repeat_interleave(G, dim=1) for x in ("k", "q"))
        _, _, S = _token(_first_state(st), k.flatten(0, 1), st["v"].double().flatten(0, 1),
                         st["g"].double().exp().flatten(), st["beta"].double().flatten())
        o = st["scale"] * torch.bmm(q.flatten(0, 1)[:, None, :], S)[:, 0]
        return {"o": o.view(st["v"].shape), "state": S.view(st["state"].shape)}
    if case["op"] == "qknorm_fwd":
        return {"q": _exact_norm(st, st["q"], st["wq"]), "k": _exact_norm(st, st["k"], st["wk"])}
    dq, dwq = _exact_norm(st, st["q"], st["wq"], st["dq_out"])
    dk, dwk = _exact_norm(st, st["k"], st["wk"], st["dk_out"])
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}


def work(case):
    c, e = case, 4 if case["dtype"] == "f32" else 2
    if c["op"].startswith("qknorm"):
        rows, D = c["B"] * c["S"] * (c["NHQ"] + c["NHK"]), c["D"]
        side = (4 * c["B"] * c["S"] + 2 * c["RD"] if c["RD"] else 0) + (8 * D if c["weight"] else 0)
        if c["op"] == "qknorm_fwd":  # rows in and out; square, norm, weight, rotation
            return {"bytes": 2 * rows * D * e + side, "flops": rows * (4 * D + 3 * c["RD"])}
        return {"bytes": 3 * rows * D * e + side + (8 * D if c["weight"] else 0), "flops": rows * (11 * D + 3 * c["RD"])}
    B, NH, NHV, DK, DV = (c[x] for x in ("B", "NH", "NHV", "DK", "DV"))
    T = B * c.get("S", 1)
    qk, vv, gates, state = 2 * T * NH * DK * e, T * NHV * DV * e, 8 * T * NHV, 4 * B * NHV * DK * DV
    cell = T * NHV * DK * DV
    if c["op"] == "gdelta_fwd":  # S^T k, k u^T and S^T q of every token; the final state is written
        return {"bytes": qk + 2 * vv + gates + state * (2 if c["state"] else 1), "flops": 6 * cell}
    if c["op"] == "gdelta_step":
        return {"bytes": qk + 2 * vv + gates + 2 * state, "flops": 7 * cell}
    # q, k, v, do and the gates in, their gradients out; the states once more (4), and of every token
    # q do^T, dS^T k, dS u, D de, S do, k de^T (12) and the gate's inner product (2)
    return {"bytes": 2 * qk + 3 * vv + 2 * gates + (2 * state if c["state"] else 0), "flops": 18 * cell}
