"""fp64 oracle of the gated delta rule and the group norm.

TEST INFRASTRUCTURE: only the tests may import this module; the CUDA library
shares no code with it. The recurrence is followed step by step, forward and
in reverse, from the definitions in numpy float64.
"""
from __future__ import annotations

import numpy as np

from .gated import f64, sigmoid


def _rows(x, i, t, share):
    return x[i, t] if share == 1 else np.repeat(x[i, t], share, 0)


def fwd(q, k, v, g, beta, state=None, scale=None, reset=None, lengths=None):
    """q, k [B,T,Nk,Dk], v [B,T,N,Dv], g, beta [B,T,N], state [B,1,N,Dk,Dv] or
    None -> (o, last, trail), trail what bwd needs."""
    q, k, v, g, beta, state = (f64(x) for x in (q, k, v, g, beta, state))
    B, T, Nk, Dk = q.shape
    N, Dv = v.shape[2:]
    share = N // Nk
    scale = Dk ** -0.5 if scale is None else scale
    o = np.zeros((B, T, N, Dv))
    last = np.zeros((B, 1, N, Dk, Dv))
    trail = []
    for i in range(B):
        S = np.zeros((N, Dk, Dv)) if state is None else state[i, 0].copy()
        n = T if lengths is None else min(max(int(lengths[i]), 0), T)
        steps = []
        for t in range(n):
            marked = (reset is not None and int(reset[i, t])) or False
            kt, qt = _rows(k, i, t, share), _rows(q, i, t, share)
            a = np.where(g[i, t] < -104, 0.0, np.exp(np.maximum(g[i, t], -104)))
            if marked:
                a = np.zeros_like(a)
            D = np.where(a[:, None, None] == 0, 0.0, a[:, None, None] * np.where(a[:, None, None] == 0, 0.0, S))
            e = v[i, t] - np.einsum("nkv,nk->nv", D, kt)
            S = D + kt[:, :, None] * (beta[i, t][:, None] * e)[:, None]
            o[i, t] = scale * np.einsum("nkv,nk->nv", S, qt)
            steps.append((a, D, e, S))
        last[i, 0] = S
        trail.append(steps)
    return o, last, trail


def bwd(q, k, v, g, beta, trail, do=None, dlast=None, scale=None):
    """Gradients of sum(o do) + sum(last dlast): (dq, dk, dv, dg, dbeta, dstate,
    and the two products that each of dq and dk is the sum of)."""
    q, k, v, g, beta, do, dlast = (f64(x) for x in (q, k, v, g, beta, do, dlast))
    B, T, Nk, Dk = q.shape
    N, Dv = v.shape[2:]
    share = N // Nk
    scale = Dk ** -0.5 if scale is None else scale
    dq, dk = np.zeros((B, T, N, Dk)), np.zeros((B, T, N, Dk))
    parts = np.zeros((4, B, T, N, Dk))
    dv, dg, db = np.zeros(v.shape), np.zeros(g.shape), np.zeros(g.shape)
    ds = np.zeros((B, 1, N, Dk, Dv))
    for i in range(B):
        dS = np.zeros((N, Dk, Dv)) if dlast is None else dlast[i, 0].copy()
        for t in reversed(range(len(trail[i]))):
            a, D, e, S = trail[i][t]
            kt, qt = _rows(k, i, t, share), _rows(q, i, t, share)
            d = np.zeros((N, Dv)) if do is None else scale * do[i, t]
            dS = dS + qt[:, :, None] * d[:, None]
            du = np.einsum("nkv,nk->nv", dS, kt)
            u = beta[i, t][:, None] * e
            dv[i, t] = beta[i, t][:, None] * du
            db[i, t] = (du * e).sum(1)
            parts[0, i, t] = np.einsum("nkv,nv->nk", D, d)
            parts[1, i, t] = kt * (u * d).sum(1)[:, None]
            parts[2, i, t] = np.einsum("nkv,nv->nk", dS, u)
            parts[3, i, t] = -np.einsum("nkv,nv->nk", D, dv[i, t])
            dq[i, t] = parts[0, i, t] + parts[1, i, t]
            dk[i, t] = parts[2, i, t] + parts[3, i, t]
            dD = dS - kt[:, :, None] * dv[i, t][:, None]
            dg[i, t] = (D * dD).sum((1, 2))
            dS = a[:, None, None] * dD
        ds[i, 0] = dS
    fold = lambda x: x.reshape(B, T, Nk, share, Dk).sum(3)  # noqa: E731
    return fold(dq), fold(dk), dv, dg, db, ds, parts


def _act(x, activation):
    """(value, slope)"""
    s = sigmoid(x)
    if activation is None:
        return x, np.ones_like(x)
    if activation == "sigmoid":
        return s, s * sigmoid(-x)
    return x * s, s + x * s * sigmoid(-x)


def group_norm(x, groups, weight=None, bias=None, gate=None, activation=None, eps=1e-5, centered=True, dy=None):
    """x [..., C] -> y, or with dy (y, dx, dgate, dweight, dbias, the largest term
    of dx's difference)."""
    x, weight, bias, gate, dy = (f64(t) for t in (x, weight, bias, gate, dy))
    C = x.shape[-1]
    flat = x.reshape(-1, groups, C // groups)
    mean = flat.mean(2, keepdims=True) if centered else 0.0
    r = 1 / np.sqrt(((flat - mean) ** 2).mean(2, keepdims=True) + eps)
    n = (flat - mean) * r
    w = np.ones(C) if weight is None else weight
    t = n.reshape(x.shape) * w + (0 if bias is None else bias)
    a, slope = _act(t if gate is None else gate, activation)
    y = a if gate is None else t * a
    if dy is None:
        return y
    dt = dy * (slope if gate is None else a)
    dgate = None if gate is None else dy * t * slope
    dn = (dt * w).reshape(flat.shape)
    dx = dn - n * (dn * n).mean(2, keepdims=True)
    if centered:
        dx = dx - dn.mean(2, keepdims=True)
    lead = tuple(range(x.ndim - 1))
    return y, (dx * r).reshape(x.shape), dgate, (dt * n.reshape(x.shape)).sum(lead), dt.sum(lead), np.abs(
        dn * r).max(initial=0.0)
