"""How linear-attention calls are cut into segments (no GPU): the places of segments, states and pieces that
csrc/kda_lin.hip derives from a sequence's first token alone, and the workspace that follows from T and N."""
import ctypes

import numpy as np
import pytest

K = pytest.importorskip("gated_delta_rule_46_amd.kda", reason="libkda.so not built (run __graft_entry__.build())")


def lengths(rng):
    kind = rng.integers(4)
    n = int(rng.integers(1, 40))
    if kind == 0:
        lens = rng.integers(0, 400, n)
    elif kind == 1:
        lens = np.exp(rng.uniform(0, np.log(5000), n)).astype(int)
    elif kind == 2:
        lens = np.where(rng.random(n) < 0.3, rng.integers(0, 4000, n), 0)
    else:
        lens = 64 * rng.integers(0, 30, n)
    return lens


@pytest.mark.parametrize("seed", range(60))
def test_places_do_not_meet(seed):
    """Stretch c / seg + s of segments with another behind them, slots 2 (c / seg) + s of split sequences: distinct and
    within their buffers, and the search over the first tokens finds the owner of a stretch."""
    rng = np.random.default_rng(seed)
    lens = lengths(rng)
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1]) + int(rng.integers(0, 50))
    seg = 64 * int(rng.integers(1, 12))
    stretches, slots = {}, set()
    for n, ln in enumerate(lens):
        first, segs = int(cu[n]) // seg, max(-(-int(ln) // seg), 1)
        if segs < 2:
            continue
        for s in range(segs - 1):
            assert first + s not in stretches and first + s < T // seg
            stretches[first + s] = (n, s)
        for s in range(segs):
            assert 2 * first + s not in slots and 2 * first + s < 2 * (T // seg)
            slots.add(2 * first + s)
    firsts = cu[:-1] // seg
    for p in range(T // seg):
        n = int(np.searchsorted(firsts, p, side="right")) - 1     # the last sequence that starts in or before it
        ln = int(lens[n])
        s = p - int(firsts[n])
        owns = 0 <= s < max(-(-ln // seg), 1) - 1
        assert owns == (p in stretches) and (not owns or stretches[p] == (n, s))


def workspace(T, N, Hv, dk=128, dv=128, dtype=1):
    c = K.kda_lin_config(1, Hv, dk, dv, dtype, 1.0)
    return K.LIB.kda_lin_prefill_workspace(ctypes.byref(c), T, N)


def test_what_is_cut():
    state = 128 * 128 * 4
    assert workspace(256, 1, 32) == 0 and workspace(0, 1, 32) == 0 and workspace(300, 60, 8) == 0
    assert workspace(8192, 1, 32) >= 3 * 16 * 32 * state              # 16 segments: states twice, what they add
    assert workspace(131072, 1, 32) >= (2 + 4) * 16 * 32 * state      # and in four pieces
    assert workspace(8192, 1, 256) == 0 and workspace(8192, 1, 512) == 0
    # 64 sequences of 64 tokens on average: segments of max(4,096 / 16, 128) = 256, which is not more than 4 x 64, so
    # the call is cut (one of them may be long): 16 stretches, states twice and what they add, two words a head.
    assert workspace(4096, 64, 32) == 16 * 32 * (3 * state + 8)
    assert workspace(4096, 65, 32) == 0                               # 63 on average: not cut, and not ordered below 128
    assert workspace(64 * 128, 64, 1024) == 64 * 4                    # only the order of the sequences
    assert workspace(64 * 128 - 1, 64, 1024) == 0


@pytest.mark.parametrize("Hv", [1, 3, 8, 32, 100, 512, 65535])
def test_workspace_is_bounded(Hv):
    """No call asks for more than 2 GiB and some of the states of 512 workgroups, whatever its length."""
    for T in (1, 64, 257, 1000, 4096, 100000, (1 << 26) // Hv):
        if T * Hv > 1 << 26:
            continue
        for N in (1, 2, 17, 1024):
            if N * Hv <= 1 << 20:
                assert workspace(T, N, Hv) <= 512 * 8 * 128 * 128 * 4 + (1 << 24)


def test_where_cutting_begins():
    """Six of the shortest segments for bf16 heads of 128 columns, four for others; half as many again, of the length
    halfway between the mean and all tokens, where there are several sequences."""
    for dk, dv, dtype, fewest in ((128, 128, 1, 6), (64, 128, 1, 6), (128, 64, 1, 4), (64, 64, 1, 4), (128, 128, 0, 4)):
        T = fewest * 128                                              # 32 heads: segments of 4 x 32 tokens at least
        assert workspace(T - 1, 1, 32, dk, dv, dtype) == 0 < workspace(T, 1, 32, dk, dv, dtype)
        assert workspace(2 * T - 1, 2, 32, dk, dv, dtype) == 0 < workspace(2 * T, 2, 32, dk, dv, dtype)
        assert workspace(0, 1, 32, dk, dv, dtype) == 0 == workspace(1, 1, 32, dk, dv, dtype)
