"""fp64 oracle of the linear-attention layer's operators (numpy, no GPU code shared).

The definitions in include/kda.h, token by token: the recurrence with one decay
per head over packed sequences and a pool of states, and the norm of the heads
with its activation.
"""
from __future__ import annotations

import numpy as np


def decays(g, T, Hv):
    """Log decays [T,Hv] from [T,Hv] or [Hv]."""
    return np.broadcast_to(np.asarray(g, np.float64), (T, Hv))


def step(S, q, k, v, g, scale):
    """One token: S [Hv,dk,dv], q, k [Hk,dk], v [Hv,dv], g [Hv] -> (o [Hv,dv], S)."""
    r = v.shape[0] // q.shape[0]
    q, k = np.repeat(q, r, 0), np.repeat(k, r, 0)
    a = np.exp(g)[:, None, None]
    S = np.where(a == 0, 0.0, S * a) + k[:, :, None] * v[:, None, :]
    return scale * np.einsum("hkv,hk->hv", S, q), S


def prefill(q, k, v, g, cu, pool=None, read=None, write=None, interval=0, scale=1.0):
    """Returns (o [T,Hv,dv], pool after the call, rungs [rows,Hv,dk,dv], final states [N,Hv,dk,dv]); rows of o
    that belong to no sequence are NaN."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    T, Hv, dv = v.shape
    dk = q.shape[2]
    g = decays(g, T, Hv)
    o = np.full((T, Hv, dv), np.nan)
    new = None if pool is None else np.array(pool, np.float64)
    rungs, final = [], []
    for n in range(len(cu) - 1):
        S = np.zeros((Hv, dk, dv))
        if pool is not None and read is not None and 0 <= read[n] < len(pool):
            S = np.array(pool[read[n]], np.float64)
        for i, t in enumerate(range(int(cu[n]), int(cu[n + 1]))):
            o[t], S = step(S, q[t], k[t], v[t], g[t], scale)
            if interval and (i + 1) % interval == 0:
                rungs.append(S)
        final.append(S)
        if pool is not None and write is not None and 0 <= write[n] < len(pool):
            new[write[n]] = S
    shape = (Hv, dk, dv)
    return o, new, np.array(rungs).reshape(-1, *shape), np.array(final).reshape(-1, *shape)


def decode(q, k, v, g, pool, read, write, scale=1.0):
    """One token of each sequence: (o [N,Hv,dv], pool after the call)."""
    N = len(q)
    o, new, _, _ = prefill(q, k, v, g, np.arange(N + 1), pool, read, write, scale=scale)
    return o, new


def activation(x, act):
    """act 0 none, 1 SiLU, 2 sigmoid."""
    if act == 0:
        return x
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-x))
        return x * s if act == 1 else s


def head_norm(x, gate=None, weight=None, bias=None, eps=1e-6, center=False, act=1):
    """x, gate [T,H,D], weight, bias [D] or [H,D].  Returns (y, y before the activation)."""
    x = np.asarray(x, np.float64)
    if center:
        x = x - x.mean(-1, keepdims=True)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    if gate is None:
        return activation(y, act), y
    return y * activation(np.asarray(gate, np.float64), act), y
