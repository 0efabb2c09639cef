"""The launch plans of kda_attn (attn_plan in csrc/kda_attn.hip), asked of the built library, and calls
that reach each of them.  Used by test_attn_plans.py (CPU) and test_gpu_attn_plans.py."""
import ctypes as C

import numpy as np

import gated_delta_rule_46_amd.kda as K

CUS = 256


class KvArgs(C.Structure):
    """kda::KvArgs (csrc/kda_attn.h)."""
    _fields_ = [(x, C.c_void_p) for x in ("k_codes", "v_codes", "k_scale", "v_scale", "table")] + \
        [("n_pages", C.c_int64), ("page", C.c_int32), ("width", C.c_int32), ("cu", C.c_void_p), ("kv_len", C.c_void_p),
         ("N", C.c_int32), ("Hk", C.c_int32), ("T", C.c_int64), ("k", C.c_void_p), ("v", C.c_void_p),
         ("k_row", C.c_int64), ("v_row", C.c_int64), ("k_out", C.c_void_p), ("v_out", C.c_void_p)]


class AttnArgs(C.Structure):
    """kda::AttnArgs."""
    _fields_ = [("kv", KvArgs), ("q", C.c_void_p), ("q_row", C.c_int64), ("o", C.c_void_p), ("lse", C.c_void_p),
                ("part", C.c_void_p), ("Hq", C.c_int32), ("scale", C.c_float), ("q_sign", C.c_float)] + \
        [(x, C.c_int32) for x in ("causal", "window", "short_rows", "unit_rows", "workers", "row_units", "row_splits",
                                  "split_tiles", "row_fold")]


_plan = K.LIB["_ZN3kda9attn_planEibiiliilPNS_8AttnArgsE"]
_plan.restype = None
_plan.argtypes = [C.c_int, C.c_bool, C.c_int, C.c_int, C.c_int64, C.c_int, C.c_int, C.c_int64, C.POINTER(AttnArgs)]
_bytes = K.LIB["_ZN3kda18attn_partial_bytesEiRKNS_8AttnArgsE"]
_bytes.restype = C.c_size_t
_bytes.argtypes = [C.c_int, C.POINTER(AttnArgs)]


def plan(dtype, D, N, T, Hq, Hk, max_kv, window=0):
    a = AttnArgs()
    a.window, a.Hq, a.kv.Hk = window, Hq, Hk
    _plan(CUS, dtype == "bf16", D, N, T, Hq, Hk, max_kv, C.byref(a))
    return a


def partial_bytes(a, D):
    return _bytes(D, C.byref(a))


def mode(a):
    """What a call launches: kda_attn.hip's part, then kda_attn_rows.hip's."""
    short = None if a.workers < 0 else \
        f"{a.unit_rows} rows, " + ("whole units" if a.workers == 0 else "shares") + \
        (", all sequences" if a.short_rows > 64 else "")
    if not a.row_units:
        return short, None
    return short, ("parts" if a.row_splits > 1 else "whole") + (", folded" if a.row_fold < a.row_units else "")


def call(name, expect, new, kv, Hq, Hk, D, page, room, dtype="bf16", window=0, pad=0):
    """room: tokens that the table holds per sequence; pad: rows behind the last sequence."""
    return dict(name=name, expect=expect, new=new, kv=kv, Hq=Hq, Hk=Hk, D=D, page=page, room=room, dtype=dtype,
                window=window, pad=pad)


def _kv(new, lo, hi, seed):
    r = np.random.default_rng(seed)
    return [n + int(x) for n, x in zip(new, r.integers(lo, hi, len(new)))]


_MIX8 = [1, 140, 3, 16, 300, 0, 17, 23]                                       # 500 new tokens
_MIX9 = [1, 140, 2, 9, 300, 16, 1, 232]                                       # 701
_MANY = [1] * 60 + [100, 40, 2, 200, 0, 33, 1, 120, 1, 45]                    # 70 sequences, two rounds of probes
_DECODE_AND_CHUNK = [1] * 20 + [225] + [1] * 11                               # 32 sequences, 256 tokens
_ONE_TAKES_ALL = [30] + [0] * 25 + [1] * 9 + [0] * 4 + [1]                    # 40 sequences, 40 tokens

CALLS = [
    call("long prompt", (None, "whole"), [1100], [1100], 64, 8, 128, 64, 1152),
    call("long prompt, heads of 64", (None, "whole"), [1100], [1163], 64, 8, 64, 32, 1184),
    call("long prompt, fp32", (None, "whole"), [1100], [1100], 64, 8, 128, 64, 1152, dtype="f32"),
    call("long prompt, window", (None, "whole"), [1100], [1500], 64, 8, 128, 16, 1536, window=333),
    call("prompt that fits the card", (None, "whole, folded"), [1000], [1000], 32, 8, 128, 64, 1024, pad=5),
    call("prompt that fits the card, heads of 64", (None, "whole, folded"), [1030], [1030], 32, 8, 64, 128, 1152),
    call("prompt that fits the card, fp32", (None, "whole, folded"), [1000], [1001], 32, 8, 128, 64, 1024, dtype="f32"),
    call("whole units of both kernels", ("32 rows, whole units", "whole, folded"), _MIX8, _kv(_MIX8, 0, 390, 1), 32, 2, 128, 64,
         704, pad=1),
    call("whole units of both kernels, fp32", ("16 rows, whole units", "whole, folded"), _MIX8, _kv(_MIX8, 0, 390, 2), 64, 4, 128,
         64, 704, dtype="f32", pad=7),
    call("whole short units, parts of long ones", ("32 rows, whole units", "parts"), _MIX9, _kv(_MIX9, 0, 700, 3), 32, 8, 128, 64,
         1024),
    call("whole short units, parts of long ones, fp32", ("16 rows, whole units", "parts"), _MIX9, _kv(_MIX9, 0, 700, 4), 32, 8,
         128, 64, 1024, dtype="f32"),
    call("many sequences", ("32 rows, shares", "whole"), _MANY, _kv(_MANY, 0, 900, 5), 32, 8, 128, 64, 6400),
    call("many sequences, heads of 64", ("32 rows, shares", "whole"), _MANY, _kv(_MANY, 0, 3000, 6), 32, 8, 64, 16, 12800,
         window=2100),
    call("many sequences, fp32", ("16 rows, shares", "whole"), _MANY, _kv(_MANY, 0, 500, 7), 32, 8, 128, 64, 6400, dtype="f32"),
    call("many sequences that fit the card", ("32 rows, shares", "whole, folded"), _MANY[:64], _kv(_MANY[:64], 0, 600, 8), 32, 8,
         128, 64, 6400, pad=3),
    call("many sequences that fit the card, fp32", ("16 rows, shares", "whole, folded"), _MANY[:64], _kv(_MANY[:64], 0, 600, 15), 32,
         8, 128, 64, 6400, dtype="f32"),
    call("many sequences in whole units", ("32 rows, whole units", "whole"), _MANY, _kv(_MANY, 0, 800, 16), 32, 8, 128, 64, 1024),
    call("many sequences in whole units, fp32", ("16 rows, whole units", "whole"), _MANY, _kv(_MANY, 0, 800, 17), 32, 8, 128, 64, 1024,
         dtype="f32", pad=2),
    call("drafted tokens, whole units", ("32 rows, whole units, all sequences", None), [5] * 64, _kv([5] * 64, 0, 1000, 9), 32, 8,
         128, 64, 1024),
    call("drafted tokens, whole units, heads of 64", ("32 rows, whole units, all sequences", None), [7] * 100,
         _kv([7] * 100, 0, 900, 10), 24, 8, 64, 32, 1024),
    call("a chunk among decoding sequences, T a multiple of N", ("32 rows, shares, all sequences", None), _DECODE_AND_CHUNK,
         _kv(_DECODE_AND_CHUNK, 0, 1500, 11), 32, 8, 128, 64, 12800),
    call("a chunk among decoding sequences, fp32", ("16 rows, shares, all sequences", None), _DECODE_AND_CHUNK,
         _kv(_DECODE_AND_CHUNK, 0, 900, 12), 16, 4, 64, 64, 51200, dtype="f32"),
    call("one sequence takes a decode step's rows", ("16 rows, shares, all sequences", None), _ONE_TAKES_ALL,
         _kv(_ONE_TAKES_ALL, 0, 1500, 13), 32, 8, 128, 64, 12800),
    call("a decode step padded by a row", ("32 rows, shares", "parts"), [1] * 63, _kv([1] * 63, 0, 900, 14), 32, 8, 128, 64, 6400,
         pad=1),
    call("short calls in small units", ("16 rows, whole units, all sequences", None), [1, 9, 4], [300, 9, 77], 8, 2, 64, 16, 304),
]


def plan_of(c):
    new, page = c["new"], c["page"]
    return plan(c["dtype"], c["D"], len(new), sum(new) + c["pad"], c["Hq"], c["Hk"], c["room"] // page * page, c["window"])


def attn(q, cu, kv_len, keys, values, scale, causal=True, window=0):
    """oracle.attention.attn with a matrix product for each sequence and kv head."""
    T, Hq, D = q.shape
    G = Hq // keys.Hk
    o, A = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, S = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for n, L in enumerate(kv_len):
        c0, new = int(cu[n]), int(cu[n + 1] - cu[n])
        ids = np.array([keys.pid(n, j) for j in range(L)], int)
        pos = np.nonzero(ids >= 0)[0] if L > 0 else np.zeros(0, int)
        if not new or not len(pos):
            continue
        ids, at = ids[pos], pos % keys.page
        p = (L - new + np.arange(new))[:, None]
        see = np.ones((new, len(pos)), bool)
        if causal:
            see &= pos <= p
        if window:
            see &= pos > p - window
        see = np.repeat(see, G, 0)                               # rows (token, head of the group)
        for h in range(keys.Hk):
            k = keys.codes[ids, h, at] * keys.scale[ids, h][:, None]
            v = values.codes[ids, h, at] * values.scale[ids, h][:, None]
            rows = q[c0:c0 + new, h * G:(h + 1) * G].reshape(new * G, D)
            s = np.where(see, (rows @ k.T) * scale, -np.inf)
            m = s.max(1, keepdims=True)
            e = np.exp(s - np.where(np.isinf(m), 0, m))
            total = e.sum(1, keepdims=True)
            w = e / np.where(total > 0, total, 1)
            to = (slice(c0, c0 + new), slice(h * G, (h + 1) * G))
            o[to], A[to] = (w @ v).reshape(new, G, D), (w @ np.abs(v)).reshape(new, G, D)
            with np.errstate(divide="ignore"):
                lse[to] = (m + np.log(total)).reshape(new, G)
            S[to] = np.where(see, np.abs(rows) @ np.abs(k).T, 0).max(1).reshape(new, G) * abs(scale)
    return o, lse, A, S
