"""Linear attention with a decay for each head and rotary positions in float64 on the CPU, token
by token from their definitions.  Gradients come from autograd through the token loop."""
from __future__ import annotations

import math

import torch


def lens_of(cu, B, T):
    if cu is None:
        return [(b * T, T) for b in range(B)]
    cu = [int(x) for x in cu]
    return [(a, b - a) for a, b in zip(cu[:-1], cu[1:])]


def fwd(q, k, v, g, S0=None, cu=None):
    """o [B,T,H,dv], S_T [N,H,dk,dv] (float64, differentiable)."""
    q, k, v, g = (x.to("cpu", torch.float64) for x in (q, k, v, g))
    B, T, _, dk = q.shape
    H, dv = g.shape[-1], v.shape[-1]
    full = lambda x: x.reshape(B * T, *x.shape[2:]).repeat_interleave(H // x.shape[2], 1)  # noqa: E731
    q, k, v = full(q), full(k), full(v)
    al = torch.exp(g.expand(B * T, H) if g.dim() == 1 else g.reshape(B * T, H))
    outs, ends = [], []
    for n, (start, length) in enumerate(lens_of(cu, B, T)):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if S0 is None else S0[n].to("cpu", torch.float64)
        for t in range(start, start + length):
            S = al[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            outs.append((S * q[t][:, :, None]).sum(1))
        ends.append(S)
    o = torch.stack(outs).reshape(B, T, H, dv) if outs else torch.zeros(B, T, H, dv, dtype=torch.float64)
    return o, torch.stack(ends)


def bwd(q, k, v, g, S0=None, cu=None, dO=None, dS_T=None):
    """(dq, dk, dv, dg, dS0) of sum(dO o) + sum(dS_T S_T), float64; dS0 also where S0 is None."""
    leaf = lambda x: x.detach().to("cpu", torch.float64).clone().requires_grad_()  # noqa: E731
    w = [leaf(x) for x in (q, k, v, g)]
    N = len(lens_of(cu, q.shape[0], q.shape[1]))
    s0 = leaf(S0) if S0 is not None else torch.zeros(N, g.shape[-1], q.shape[-1], v.shape[-1],
                                                     dtype=torch.float64, requires_grad=True)
    o, S_T = fwd(*w, s0, cu)
    loss = 0.0 * s0.sum()
    if dO is not None:
        loss = loss + (o * dO.to("cpu", torch.float64)).sum()
    if dS_T is not None:
        loss = loss + (S_T * dS_T.to("cpu", torch.float64)).sum()
    got = torch.autograd.grad(loss, w + [s0], allow_unused=True)
    return [torch.zeros_like(x) if y is None else y for x, y in zip(w + [s0], got)]


def rotary(x, pos, freqs, layout, inverse=False, scale=1.0):
    x = x.to("cpu", torch.float64)
    f = [float(v) for v in freqs]
    n, y = len(f), x.clone()
    p = pos.to("cpu").reshape(-1).tolist()
    xr, yr = x.reshape(len(p), *x.shape[-2:]), y.reshape(len(p), *x.shape[-2:])
    for t, at in enumerate(p):
        for i in range(n):
            a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
            th = -at * f[i] if inverse else at * f[i]
            c, s = math.cos(th), math.sin(th)
            yr[t, :, a] = scale * (xr[t, :, a] * c - xr[t, :, b] * s)
            yr[t, :, b] = scale * (xr[t, :, b] * c + xr[t, :, a] * s)
    return y
