"""The delta rule with one decay per head, the norm with rotation and their backward
passes in 64 bits, token by token, from their definitions (torch tensors on any device)."""
from __future__ import annotations

import torch


def rule(q, k, v, g, beta, scale, state):
    """q, k [T, Hk, K], v [T, Hv, V], g, beta [T, Hv], state [Hv, K, V]; (out, last state,
    the state before each token)."""
    q, k, v, g, beta, S = (x.double() for x in (q, k, v, g, beta, state))
    share = v.shape[1] // k.shape[1]
    q, k = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1)
    outs, before = [], []
    for t in range(v.shape[0]):
        before.append(S)
        S = S * g[t].exp()[:, None, None]
        delta = beta[t][:, None] * (v[t] - (k[t][:, :, None] * S).sum(1))
        S = S + k[t][:, :, None] * delta[:, None, :]
        outs.append(scale * (q[t][:, :, None] * S).sum(1))
    out = torch.stack(outs) if outs else torch.zeros_like(v)
    return out, S, before


def rule_bwd(q, k, v, g, beta, scale, state, dout, dfinal):
    """Gradients of sum(out * dout) + sum(last state * dfinal), by the reversed steps."""
    _, _, before = rule(q, k, v, g, beta, scale, state)
    hk = k.shape[1]
    q, k, v, g, beta, dout, D = (x.double() for x in (q, k, v, g, beta, dout, dfinal))
    share = v.shape[1] // hk
    q, k = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1)
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    for t in reversed(range(v.shape[0])):
        a = g[t].exp()[:, None, None]
        held = before[t] * a
        miss = v[t] - torch.einsum("hkv,hk->hv", held, k[t])
        delta = beta[t][:, None] * miss
        S = held + k[t][:, :, None] * delta[:, None]
        D = D + scale * q[t][:, :, None] * dout[t][:, None]
        dq[t] = scale * torch.einsum("hkv,hv->hk", S, dout[t])
        ddelta = torch.einsum("hkv,hk->hv", D, k[t])
        dk[t] = torch.einsum("hkv,hv->hk", D, delta)
        dv[t] = beta[t][:, None] * ddelta
        db[t] = (ddelta * miss).sum(-1)
        D = D - k[t][:, :, None] * dv[t][:, None]
        dk[t] -= torch.einsum("hkv,hv->hk", held, dv[t])
        dg[t] = (D * held).sum((-2, -1))
        D = D * a
    dq, dk = (x.unflatten(1, (hk, share)).sum(2) for x in (dq, dk))
    return dq, dk, dv, dg, db, D


def turn(x, cos, sin, interleaved, back=False):
    """x [T, H, D]; cos, sin [T, rotary / 2]: each pair times its rotation."""
    half = cos.shape[-1]
    y = x.clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        c, s = cos[:, None, i], -sin[:, None, i] if back else sin[:, None, i]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm(x, kind, eps, weight=None, cos=None, sin=None, interleaved=False):
    x = x.double()
    total = x.square().sum(-1, keepdim=True) / (x.shape[-1] if kind == "rms" else 1)
    y = x / (total + eps).sqrt()
    y = y if weight is None else y * weight.double()
    return y if cos is None else turn(y, cos.double(), sin.double(), interleaved)


def norm_bwd(x, dz, kind, eps, weight=None, cos=None, sin=None, interleaved=False):
    """(dL/dx, dL/dweight) for dL/d(norm's result) = dz."""
    x, dz = x.double(), dz.double()
    if cos is not None:
        dz = turn(dz, cos.double(), sin.double(), interleaved, back=True)
    n = x.shape[-1] if kind == "rms" else 1
    root = (x.square().sum(-1, keepdim=True) / n + eps).sqrt()
    dw = (dz * x / root).sum((0, 1))
    du = dz if weight is None else dz * weight.double()
    return du / root - x * (x * du).sum(-1, keepdim=True) / (n * root ** 3), dw
