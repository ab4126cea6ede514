"""fp64 oracle of the gated linear scan, the 8-bit activation checkpoints and
the token embedding.

TEST INFRASTRUCTURE: only the tests may import this module; the CUDA library
shares no code with it. Everything is written out step by step (and token by
token) from the definitions in numpy float64.
"""
from __future__ import annotations

import numpy as np

CHUNK = 128  # steps between the states a training forward keeps
BLOCK = 32   # rows that share a scale in an 8-bit checkpoint


def f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        import torch
        a = a.detach().cpu().to(torch.float64).numpy()
    return np.array(a, dtype=np.float64)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def _coeff(a, function):
    """a [G, ...] -> f, u, output factor."""
    if function == "linear":
        return sigmoid(a[1]), sigmoid(a[0]) * a[2], sigmoid(a[3])
    return sigmoid(a[0]), sigmoid(-a[0]) * a[1], np.ones_like(a[0])


def fwd(Wx, b, state, function, reset=None, lengths=None):
    """Wx [B,T,G,N,D], b [G,N,D] or None, state [B,1,N,D] or None -> (h, last,
    states before every step [B,T,N,D])."""
    Wx, b, state = f64(Wx), f64(b), f64(state)
    B, T, G, N, D = Wx.shape
    h = np.zeros((B, T, N, D))
    before = np.zeros((B, T, N, D))
    last = np.zeros((B, 1, N, D))
    for i in range(B):
        c = np.zeros((N, D)) if state is None else state[i, 0].copy()
        n = T if lengths is None else min(max(int(lengths[i]), 0), T)
        for t in range(T):
            before[i, t] = c
            if t >= n:
                continue
            f, u, o = _coeff(Wx[i, t] + (0 if b is None else b), function)
            if reset is not None and int(reset[i, t]):
                c = np.zeros_like(c)
            c = f * c + u
            h[i, t] = o * c
        last[i, 0] = c
    return h, last, before


def bwd(Wx, b, before, function, dh=None, dlast=None, reset=None, lengths=None, packed=False):
    """Gradients (dWx, db, dstate). before: the states fwd met before every
    step. packed: at the values that Wx's 8-bit checkpoint stands for, from
    the exact states at the starts of the chunks."""
    Wx, b, dh, dlast = f64(Wx), f64(b), f64(dh), f64(dlast)
    B, T, G, N, D = Wx.shape
    dWx = np.zeros_like(Wx)
    ds = np.zeros((B, 1, N, D))
    for i in range(B):
        n = T if lengths is None else min(max(int(lengths[i]), 0), T)
        x = Wx[i].copy()
        if packed:
            x[n:] = 0
            x = unpacked(x.reshape(T, -1)).reshape(x.shape) if T else x
        prev, after = np.zeros((T, N, D)), np.zeros((T, N, D))
        c = None
        for t in range(n):
            if t % CHUNK == 0 or c is None:
                c = before[i, t]
            f, u, _ = _coeff(x[t] + (0 if b is None else b), function)
            prev[t] = 0 if reset is not None and int(reset[i, t]) else c
            c = f * prev[t] + u
            after[t] = c
        d = np.zeros((N, D)) if dlast is None else dlast[i, 0].copy()
        for t in reversed(range(n)):
            a = x[t] + (0 if b is None else b)
            g = np.zeros((N, D)) if dh is None else dh[i, t]
            f, _, o = _coeff(a, function)
            d = d + g * o
            if function == "linear":
                s = sigmoid(a[0])
                dWx[i, t, 0] = d * a[2] * s * sigmoid(-a[0])
                dWx[i, t, 1] = d * prev[t] * f * sigmoid(-a[1])
                dWx[i, t, 2] = d * s
                dWx[i, t, 3] = g * after[t] * o * sigmoid(-a[3])
            else:
                dWx[i, t, 0] = d * (prev[t] - a[1]) * f * sigmoid(-a[0])
                dWx[i, t, 1] = d * sigmoid(-a[0])
            d = f * d
            if reset is not None and int(reset[i, t]):
                d = np.zeros_like(d)
        ds[i, 0] = d
    return dWx, dWx.sum((0, 1)), ds


def pack(x):
    """x [rows, cols] -> (q, scale bytes) by the definition, block by block."""
    x = f64(x)
    rows, cols = x.shape
    q = np.zeros((rows, cols), dtype=np.int64)
    sc = np.zeros((-(-rows // BLOCK), cols), dtype=np.int64)
    for k in range(sc.shape[0]):
        v = x[k * BLOCK:(k + 1) * BLOCK]
        for j in range(cols):
            col = v[:, j]
            if not np.isfinite(col).all():
                sc[k, j] = 255
                continue
            top = np.abs(col).max()
            e = -126
            while top > 127 * 2.0 ** e and e < 121:  # 64 * 2^122 would be past the types' range
                e += 1
            sc[k, j] = e + 127
            q[k * BLOCK:(k + 1) * BLOCK, j] = np.clip(np.rint(col / 2.0 ** e), -127, 127)
    return q, sc


def unpack(q, sc):
    scale = np.where(sc == 255, np.nan, 2.0 ** (sc - 127.0))
    return q * np.repeat(scale, BLOCK, axis=0)[:q.shape[0]]


def unpacked(x):
    return unpack(*pack(x))


def embed(ids, W, scale):
    W = f64(W)
    out = np.zeros((len(ids), W.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < W.shape[0]:
            out[i] = scale * W[v]
    return out


def embed_grad(ids, V, dout, scale, padding_idx=None):
    dout = f64(dout)
    dW = np.zeros((V, dout.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < V and v != padding_idx:
            dW[v] += scale * dout[i]
    return dW
