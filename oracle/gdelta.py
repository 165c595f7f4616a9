"""fp64 oracle of the gated delta rule, token by token, and the adjoint of that recurrence.

Per batch item, value head and token, with a state S [DK][DV]:
    D = exp(g) S,  e = v - D^T k,  S' = D + beta k e^T,  o = scale S'^T q.
Plain torch operations in float64 on the device of the inputs; no chunks, no code of the library.
"""
from __future__ import annotations

import torch


def _wide(q, k, v, g, beta, lengths):
    """float64, value heads side by side; tokens behind lengths[b] become tokens that change nothing."""
    B, NH, S, DK = q.shape
    G = v.shape[1] // NH
    n = torch.full((B,), S, device=q.device) if lengths is None else lengths.long().clamp(0, S)
    live = (torch.arange(S, device=q.device)[None, :] < n[:, None])[:, None, :]
    w = [torch.where(live[..., None], x.double().repeat_interleave(h, dim=1), 0.0) for x, h in ((q, G), (k, G), (v, 1))]
    return (*w, torch.where(live, g.double(), 0.0).exp(), torch.where(live, beta.double(), 0.0), live)


def _update(S, k, v, f, b):
    D = f[..., None, None] * S
    e = v - torch.einsum("bhij,bhi->bhj", D, k)
    return D, e, D + torch.einsum("bhi,bhj->bhij", k, b[..., None] * e)


def gdelta_fwd(q, k, v, g, beta, state=None, lengths=None, scale=None):
    """(o [B, NHV, S, DV], final state [B, NHV, DK, DV]) in float64."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    Q, K, V, F, Bt, live = _wide(q, k, v, g, beta, lengths)
    S = torch.zeros(*v.shape[:2], q.shape[-1], v.shape[-1], dtype=torch.float64, device=q.device) \
        if state is None else state.double()
    o = torch.zeros_like(V)
    for t in range(q.shape[2]):
        _, _, S = _update(S, K[:, :, t], V[:, :, t], F[:, :, t], Bt[:, :, t])
        o[:, :, t] = scale * torch.einsum("bhij,bhi->bhj", S, Q[:, :, t])
    return torch.where(live[..., None], o, 0.0), S


def gdelta_bwd(q, k, v, g, beta, do, state=None, dstate=None, lengths=None, scale=None, every=64):
    """Gradients of sum(do * o) + sum(dstate * final state): (dq, dk, dv, dg, dbeta, dstate0), float64.

    Runs the sequence backwards from states kept every ``every`` tokens.  With dS the gradient of the
    state after token t (o_t's share included):
        dq = scale S' do,  du = dS^T k,  dbeta = du . e,  dv = beta du,
        dk = dS (beta e) - D dv,  dD = dS - k dv^T,  dg = <dD, D>,  dS <- exp(g) dD.
    """
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    B, NH, T, DK = q.shape
    Q, K, V, F, Bt, live = _wide(q, k, v, g, beta, lengths)
    dO = torch.where(live[..., None], do.double(), 0.0)
    S = torch.zeros(*v.shape[:2], DK, v.shape[-1], dtype=torch.float64, device=q.device) \
        if state is None else state.double()
    dS = torch.zeros_like(S) if dstate is None else dstate.double()
    kept = []
    for t in range(T):
        if t % every == 0:
            kept.append(S)
        _, _, S = _update(S, K[:, :, t], V[:, :, t], F[:, :, t], Bt[:, :, t])
    dq, dk, dv = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
    dg, db = torch.zeros_like(F), torch.zeros_like(F)
    for seg in reversed(range(len(kept))):
        S, run = kept[seg], []
        for t in range(seg * every, min(T, (seg + 1) * every)):
            D, e, S = _update(S, K[:, :, t], V[:, :, t], F[:, :, t], Bt[:, :, t])
            run.append((t, D, e, S))
        for t, D, e, S in reversed(run):
            dq[:, :, t] = scale * torch.einsum("bhij,bhj->bhi", S, dO[:, :, t])
            dS = dS + scale * torch.einsum("bhi,bhj->bhij", Q[:, :, t], dO[:, :, t])
            du = torch.einsum("bhij,bhi->bhj", dS, K[:, :, t])
            db[:, :, t] = (du * e).sum(-1)
            de = Bt[:, :, t, None] * du
            dv[:, :, t] = de
            dk[:, :, t] = torch.einsum("bhij,bhj->bhi", dS, Bt[:, :, t, None] * e) - torch.einsum("bhij,bhj->bhi", D, de)
            dS = dS - torch.einsum("bhi,bhj->bhij", K[:, :, t], de)
            dg[:, :, t] = (dS * D).sum((-2, -1))
            dS = F[:, :, t, None, None] * dS

    def rows(x):
        return torch.where(live[..., None] if x.dim() == 4 else live, x, 0.0)

    def shared(x):
        return rows(x).reshape(B, NH, -1, T, DK).sum(2)

    return shared(dq), shared(dk), rows(dv), rows(dg), rows(db), dS
