"""fp64 oracle of the per-head norms with the position rotation, and of their gradients (autograd).

Plain torch operations in float64 on the device of the inputs; the rotation is a complex product.
"""
from __future__ import annotations

import torch


def norm_rotate(x, weight, norm, eps, inv_freq, positions, interleaved):
    """[B, S, H, D] -> [B, H, S, D] in float64."""
    x = x.double()
    s = x.square().sum(-1, keepdim=True)
    y = x / torch.sqrt((s / x.shape[-1] if norm == "rms" else s) + eps)
    if weight is not None:
        y = y * weight.double()
    if inv_freq is not None and inv_freq.numel():
        B, S, H, D = x.shape
        pos = torch.arange(S, device=x.device).expand(B, S) if positions is None else positions
        ang = pos.double()[:, :, None, None] * inv_freq.double()
        turn = torch.polar(torch.ones_like(ang), ang)
        rd = 2 * inv_freq.numel()
        a, b = (y[..., :rd:2], y[..., 1:rd:2]) if interleaved else (y[..., :rd // 2], y[..., rd // 2:rd])
        z = torch.complex(a, b) * turn
        r = torch.stack((z.real, z.imag), -1).flatten(-2) if interleaved else torch.cat((z.real, z.imag), -1)
        y = torch.cat((r, y[..., rd:]), -1)
    return y.transpose(1, 2)


def norm_rotate_grad(dy, x, weight, norm, eps, inv_freq, positions, interleaved):
    """(dx [B, S, H, D], dweight [D] or None) in float64."""
    x = x.detach().double().requires_grad_(True)
    w = None if weight is None else weight.detach().double().requires_grad_(True)
    y = norm_rotate(x, w, norm, eps, inv_freq, positions, interleaved)
    grads = torch.autograd.grad((y * dy.double()).sum(), [x] if w is None else [x, w])
    return grads[0], None if w is None else grads[1]
