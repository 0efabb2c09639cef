"""fp64 oracle of the attention-layer operators (numpy, no GPU code shared).

The definitions in include/kda.h, element by element: e4m3 rounding from the
format's grid, the cache as an array of values with a scale per page and head,
attention as an explicit softmax over the keys each row sees.
"""
from __future__ import annotations

import numpy as np

CODE_MAX = 448.0
SCALE_EXP = (-100, 119)


def e4m3_values():
    """The 256 values of e4m3 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f is NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def e4m3_round(x):
    """Nearest e4m3 value, ties to even, saturating at 448; NaN stays."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), CODE_MAX)
    ulp = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.where(np.isnan(x), np.nan, np.copysign(np.minimum(np.rint(a / ulp) * ulp, CODE_MAX), x))


def scale_for(amax):
    """Smallest power of two s with amax <= 448 s, within the limits."""
    if not amax > 0:
        return 2.0 ** SCALE_EXP[0]
    e = int(np.ceil(np.log2(amax) - np.log2(CODE_MAX))) - 1
    while amax > CODE_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** min(max(e, SCALE_EXP[0]), SCALE_EXP[1])


def norm_rope(x, weight, eps, positions=None, table=None, pairs=False):
    """x [T,H,D] -> normalised and rotated; rows of padded tokens come back as NaN."""
    x = np.asarray(x, np.float64)
    T, H, D = x.shape
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if table is None:
        return y
    n_pos, rot = table.shape
    out = y.copy()
    for t in range(T):
        p = int(positions[t])
        if p < 0 or p >= n_pos:
            out[t] = np.nan
            continue
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
            c, s = float(table[p, i]), float(table[p, rot // 2 + i])
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
    return out


class Cache:
    """One of the two halves (keys or values): codes as the numbers they are, and scales."""

    def __init__(self, codes, scale, table):
        self.codes = np.array(codes, np.float64)      # [n_pages, Hk, page, D]
        self.scale = np.array(scale, np.float64)      # [n_pages, Hk]
        self.table = np.asarray(table)
        self.n_pages, self.Hk, self.page, self.D = self.codes.shape

    def pid(self, n, pos):
        b = pos // self.page
        if pos < 0 or b >= self.table.shape[1]:
            return -1
        p = int(self.table[n, b])
        return p if 0 <= p < self.n_pages else -1

    def write(self, x, cu, kv_len):
        x = np.asarray(x, np.float64)
        for n in range(len(kv_len)):
            start = int(kv_len[n]) - int(cu[n + 1] - cu[n])
            by_page = {}
            for t in range(int(cu[n]), int(cu[n + 1])):
                pos = start + t - int(cu[n])
                if self.pid(n, pos) >= 0:
                    by_page.setdefault(pos // self.page, []).append((t, pos % self.page))
            for b, rows in by_page.items():
                pid, first = self.pid(n, b * self.page), rows[0][1]
                for h in range(self.Hk):
                    new = np.stack([x[t, h] for t, _ in rows])
                    finite = np.abs(new[np.isfinite(new)])
                    s = scale_for(finite.max() if finite.size else 0.0)
                    if first > 0:
                        held = self.scale[pid, h]
                        if s > held:
                            self.codes[pid, h, :first] = e4m3_round(self.codes[pid, h, :first] * (held / s))
                        s = max(s, held)
                    self.scale[pid, h] = s
                    for (t, r), v in zip(rows, new):
                        self.codes[pid, h, r] = e4m3_round(v / s)

    def read(self, cu, kv_len, T):
        out = np.zeros((T, self.Hk, self.D))
        for n in range(len(kv_len)):
            for t in range(int(cu[n]), int(cu[n + 1])):
                pos = int(kv_len[n]) - int(cu[n + 1]) + t
                pid = self.pid(n, pos)
                if pid >= 0:
                    out[t] = self.codes[pid, :, pos % self.page] * self.scale[pid][:, None]
        return out


def attn(q, cu, kv_len, keys, values, scale, causal=True, window=0):
    """(o [T,Hq,D], lse [T,Hq], A [T,Hq,D], S [T,Hq]): A = sum of softmax |v| and S = the largest
    sum |scale q_i k_i| over the keys a row sees, for error bounds."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    G = Hq // keys.Hk
    o, A = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, S = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for n in range(len(kv_len)):
        L, new = int(kv_len[n]), int(cu[n + 1] - cu[n])
        pages = [keys.pid(n, j) for j in range(max(L, 0))]
        pos = np.array([j for j in range(max(L, 0)) if pages[j] >= 0], int)
        if not len(pos):
            continue
        ids = np.array([pages[j] for j in pos])
        K = keys.codes[ids, :, pos % keys.page] * keys.scale[ids][:, :, None]      # [keys, Hk, D]
        V = values.codes[ids, :, pos % keys.page] * values.scale[ids][:, :, None]
        for i in range(new):
            p = L - new + i
            see = np.ones(len(pos), bool)
            if causal:
                see &= pos <= p
            if window:
                see &= pos > p - window
            if not see.any():
                continue
            t = int(cu[n]) + i
            for h in range(Hq):
                k, v = K[see, h // G], V[see, h // G]
                s = (k @ q[t, h]) * scale
                m = s.max()
                e = np.exp(s - m)
                w = e / e.sum()
                o[t, h], A[t, h] = w @ v, w @ np.abs(v)
                lse[t, h] = m + np.log(e.sum())
                S[t, h] = (np.abs(k) @ np.abs(q[t, h])).max() * abs(scale)
    return o, lse, A, S
