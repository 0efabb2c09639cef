"""The launch plans of kda_attn: the calls of attn_plans.py reach every one of them (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import oracle.attention as A

pytest.importorskip("gated_delta_rule_46_amd.kda", reason="libkda.so not built (run __graft_entry__.build())")
import attn_plans as P  # noqa: E402

K = P.K


def test_the_plan_struct_is_the_librarys():
    """Its fields lie where the library has them: the partial results counted from them are the workspace."""
    for dtype, D, N, T, Hq, Hk, width, window in (("bf16", 128, 64, 64, 32, 8, 500, 0), ("f32", 64, 5, 300, 8, 2, 40, 100),
                                                  ("bf16", 128, 1, 512, 32, 8, 63, 0), ("bf16", 64, 9, 701, 8, 8, 900, 0)):
        a = P.plan(dtype, D, N, T, Hq, Hk, width * 64, window)
        assert a.row_splits >= 1 and a.unit_rows in (16, 32) and a.workers >= -1
        cfg = K.kda_attn_config(Hq, Hk, D, 1 if dtype == "bf16" else 0)
        cache = K.kda_kv_cache(1 << 20, 1 << 20, 1 << 20, 1 << 20, 4, 64, width, 1 << 20)
        ws = K.LIB.kda_attn_workspace(ctypes.byref(cfg), ctypes.byref(cache), N, T, window)
        assert ws == -(-P.partial_bytes(a, D) // 256) * 256


@pytest.mark.parametrize("c", P.CALLS, ids=[c["name"] for c in P.CALLS])
def test_each_call_has_its_plan(c):
    assert P.mode(P.plan_of(c)) == c["expect"]
    assert len(c["new"]) == len(c["kv"]) and all(n <= k <= c["room"] for n, k in zip(c["new"], c["kv"]))


def test_the_calls_reach_every_plan():
    """Every combination that sizes over the whole range lead to stands in the list, or is one of the plans
    that test_gpu_attn.py's cases take (parts of long units alone, or beside shares of short ones)."""
    seen = {}
    rng = np.random.default_rng(1)
    for _ in range(40000):
        N = int(2 ** rng.uniform(0, 8))
        T = N * int(2 ** rng.uniform(0, 12 if N < 16 else 7)) + (int(rng.integers(0, N)) if rng.random() < 0.5 else 0)
        Hk = int(2 ** rng.integers(0, 4))
        Hq = Hk * int(rng.integers(1, 9))
        keys = int(2 ** rng.uniform(4, 17)) // 16 * 16
        dtype, D = ("bf16", "f32")[rng.integers(0, 2)], (64, 128)[rng.integers(0, 2)]
        seen.setdefault(P.mode(P.plan(dtype, D, N, T, Hq, Hk, keys)), (dtype, D, N, T, Hq, Hk, keys))
    there = {c["expect"] for c in P.CALLS}
    elsewhere = {(None, "parts"), ("32 rows, shares", "parts"), ("16 rows, shares", "parts")}
    assert there <= set(seen)
    missing = {m: x for m, x in seen.items() if m not in there | elsewhere}
    assert not missing, missing


def test_the_matrix_oracle_is_the_oracle():
    rng = np.random.default_rng(2)
    table = np.array([[3, 1, -1], [0, 2, 1]])
    half = [A.Cache(A.e4m3_round(rng.normal(size=(4, 2, 16, 8)) * 40), 2.0 ** rng.integers(-6, -3, (4, 2)), table) for _ in "kv"]
    q = rng.normal(size=(9, 6, 8))
    for kv in ([40, 20], [2, 33]):
        for causal, window in ((True, 0), (True, 5), (False, 0)):
            for x, y in zip(P.attn(q, [0, 5, 9], kv, *half, 0.3, causal, window), A.attn(q, [0, 5, 9], kv, *half, 0.3, causal, window)):
                assert np.allclose(x, y, rtol=1e-12, atol=1e-14)
