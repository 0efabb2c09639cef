"""GPU tests of the linear-attention layer's prefill in every launch plan: cut into segments, in up to four pieces, taken
longest first, captured, on another stream.  Each test asserts the plan that it is for, from the workspace that the plan
needs.  Tolerances as in test_gpu_linear.py."""
import ctypes

import numpy as np
import pytest

import oracle.linear as R
from test_gpu_linear import HALF, U, Call, dt, f32, i32, i64, rel_l2, say, within
from test_gpu_linear_edges import K, is_cut, workspace  # noqa: F401 (K: the fixture)
from workloads.device import to_numpy_f64

pytestmark = pytest.mark.gpu

UNITS = 512                                                       # two workgroups for each of 256 compute units


def is_ordered(c):
    """Whether the sequences are taken longest first."""
    N, T = len(c.lens), c.q.shape[0]
    return 1 < N <= 1024 and N * c.dims[1] > UNITS and T // N >= 128


def plan_of(K, dtype, T, N, Hk, Hv, dk, dv):
    """(tokens of a segment, pieces) that explain the workspace of an unordered call; None without segments."""
    need = workspace(K, dtype, T, N, Hk, Hv, dk, dv)
    found = []
    for seg in range(64, T + 1, 64):
        stretches = T // seg
        for pieces in range(1, 5):
            words = (2 + pieces) * dk * dv + 1 + pieces + (2 * seg // 64 if pieces > 1 else 0)
            if need == -(-stretches * Hv * words * 4 // 256) * 256 and seg >= -(-T * Hv // UNITS):
                found.append((seg, pieces))
    return found[0] if found else None


# ---------------------------------------------------------------------------
# pieces
# ---------------------------------------------------------------------------
def normal(seed, *shapes):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda") for s in shapes]


def heads_on_device(dtype, T, Hk, Hv, dk, dv, seed):
    return [x.to(dt(dtype)) for x in normal(seed, (T, Hk, dk), (T, Hk, dk), (T, Hv, dv))]


def decays(kind, T, H, seed):
    rng = np.random.default_rng(seed)
    if kind == "slow":                                            # every piece leaves something
        return f32(-1e-3 * 2.0 ** -np.linspace(0, 8, H))
    if kind == "mixed":                                           # of some heads' pieces nothing is left
        return f32(-2.0 ** -np.linspace(2, 14, H) * np.exp(0.5 * rng.normal(size=(T, H))))
    g = np.where(rng.random((T, H)) < 0.001, -60.0, -1e-3 * rng.random((T, H)))
    return f32(g)                                                 # drops now and then


@pytest.mark.parametrize("kind", ["slow", "mixed", "drops"])
@pytest.mark.parametrize("dtype,dk,dv,T,pieces", [("bf16", 128, 128, 16600, 4), ("bf16", 64, 128, 12700, 3),
                                                  ("bf16", 128, 64, 8400, 2), ("f32", 128, 128, 12700, 3),
                                                  ("f32", 64, 64, 16600, 4)])
def test_pieces(K, dtype, dk, dv, T, pieces, kind):
    """Segments of T / 4 tokens and more in up to four pieces.  A state takes 32 tokens a step, each with one rounding of
    the sum, one of the decay and two of the product's terms, and outputs those of their own products (fp32 rows)."""
    import torch
    Hk, Hv, N = 2, 128, 2
    lens = [T - 75, 75]
    seg, p = plan_of(K, dtype, T, N, Hk, Hv, dk, dv)
    say(f"segments of {seg} in {p} pieces")
    assert p == pieces and T // seg >= 3
    q, k, v = heads_on_device(dtype, T, Hk, Hv, dk, dv, 101)
    g = decays(kind, T, Hv, 102)
    pool, = normal(103, (4, Hv, dk, dv))
    pick = [0, 31, 64, 100, 127]
    first = to_numpy_f64(pool[:, pick])
    read, write = [1, -1], [1, 3]
    o, _ = K.kda_lin_prefill(q, k, v, g, i64([0, T - 75, T]), pool, i32(read), i32(write), scale=dk ** -0.5)
    torch.cuda.synchronize()
    f = to_numpy_f64
    qk = [h // (Hv // Hk) for h in pick]
    ref = R.prefill(f(q[:, qk]), f(k[:, qk]), f(v[:, pick]), R.decays(f(g), T, Hv)[:, pick], [0, T - 75, T], first, read,
                    write, scale=dk ** -0.5)
    tol = U * (8 + 4 * (4 * T / 32) ** 0.5)
    for i, h in enumerate(pick):
        e = [rel_l2(f(o[:, h]), ref[0][:, i])] + [rel_l2(f(pool[w, h]), ref[1][w][i]) for w in write]
        say(f"head {h}: o {e[0]:.2e}, states {e[1]:.2e} {e[2]:.2e}")
        assert e[0] <= (HALF["bf16"] if dtype == "bf16" else tol) and max(e[1:]) <= tol
    assert np.array_equal(f(pool[[0, 2]][:, pick]), first[[0, 2]])


# ---------------------------------------------------------------------------
# segments
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [64, 128])
def test_split_heads_of_128_columns(K, dtype, dk):
    c = Call(dtype, [4000, 20], 3, 6, dk, 128, "token", 111)
    assert is_cut(K, c) and not is_ordered(c)
    c.check(K, interval=448)


@pytest.mark.parametrize("gate", ["head", "token", "strong"])
@pytest.mark.parametrize("dk", [64, 128])
def test_grouped_heads_ragged_in_segments(K, dk, gate):
    """Value heads that share q and k; ragged sequences, taken longest first, the long ones cut, with rungs."""
    import torch
    lens = [1, 33, 0, 64, 200, 31, 3100, 7, 90, 257, 65, 12, 700]
    Hk, Hv = 12, 48
    c = Call("bf16", lens, Hk, Hv, dk, 64, gate, 112, pad=2)
    assert is_cut(K, c) and is_ordered(c)
    pick, first = [0, 1, 6, 47], c.pool.clone()
    qk = [h // 4 for h in pick]
    off = np.concatenate([[0], np.cumsum([n // 64 for n in lens])])
    f = to_numpy_f64
    out = torch.full(c.v.shape, 7.0, dtype=c.v.dtype, device="cuda")
    o, rungs = K.kda_lin_prefill(c.q, c.k, c.v, c.g, i64(c.cu), c.pool, i32(c.read), i32(c.write), scale=0.3,
                                 ckpt_interval=64, ckpt_offsets=i64(off), out=out)
    torch.cuda.synchronize()
    live = c.cu[-1]
    assert (f(o)[live:] == 7.0).all()
    args = (f(c.q[:, qk]), f(c.k[:, qk]), f(c.v[:, pick]), R.decays(f(c.g), sum(lens) + 2, Hv)[:, pick], c.cu,
            f(first[:, pick]), c.read, c.write, 64)
    ref = R.prefill(*args, scale=0.3)
    top = R.prefill(*(np.abs(x) if i in (0, 1, 2, 5) else x for i, x in enumerate(args)), scale=0.3)
    half, n = HALF["bf16"], max(lens)
    tol = half * np.abs(ref[0][:live]) + (2 * half + (6 * n + dk + 8) * U) * top[0][:live] + 1e-37
    within("o", f(o[:live, pick]), ref[0][:live], tol)
    Call.states("pool", f(c.pool[:, pick])[c.write], ref[1][c.write], top[1][c.write], n)
    Call.states("rungs", f(rungs[:, pick]), ref[2], top[2], n)
    rest = np.setdiff1d(np.arange(len(first)), c.write)
    assert torch.equal(first[rest], c.pool[rest])


@pytest.mark.parametrize("seed", range(8))
def test_segments_have_places_of_their_own(K, seed):
    """Ragged sequences at random places, some of them empty: each one's outputs and states are right, and the bytes around
    the workspace are left as they were."""
    import torch
    rng = np.random.default_rng(seed)
    dtype = ["bf16", "f32"][seed % 2]
    n = int(rng.integers(3, 12))
    lens = np.where(rng.random(n) < 0.3, 0, np.exp(rng.uniform(0, np.log(900), n))).astype(int)
    lens[int(rng.integers(n))] += 2500
    c = Call(dtype, lens.tolist(), 1, 2, 64, 64, "token", 120 + seed, pad=int(rng.integers(0, 70)))
    assert is_cut(K, c)
    need = workspace(K, dtype, c.q.shape[0], n, *c.dims)
    around = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    c.check(K, interval=128, workspace=around[4096:4096 + need])
    assert (around[:4096] == 0xA5).all() and (around[4096 + need:] == 0xA5).all()


# ---------------------------------------------------------------------------
# several launches in a graph, and on a stream
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,Hk,Hv,dk,dv,lens", [
    ("bf16", 2, 32, 64, 64, [2600] + [300] * 19),                 # the order, states, the carry and the units
    ("bf16", 4, 4, 128, 128, [3000, 90, 0, 5]),                   # states, the carry and the units
    ("f32", 1, 128, 64, 64, [8300, 148]),                         # sums too: two pieces a segment
])
def test_captured_segments_replay(K, dtype, Hk, Hv, dk, dv, lens):
    """Each replay of a captured call of several launches, between eager work, gives what the eager call gives."""
    import torch
    T = sum(lens)
    need = workspace(K, dtype, T, len(lens), Hk, Hv, dk, dv)
    assert need > 4 * Hv * dk * dv * 4                            # states of segments
    q, k, v = heads_on_device(dtype, T, Hk, Hv, dk, dv, 131)
    g = decays("mixed", T, Hv, 132)
    N = len(lens)
    cu, slots = i64(np.concatenate([[0], np.cumsum(lens)])), i32(range(N))
    start, = normal(133, (N, Hv, dk, dv))
    pool = start.clone()
    rungs = torch.zeros((sum(n // 64 for n in lens), Hv, dk, dv), device="cuda")
    off = i64(np.concatenate([[0], np.cumsum([n // 64 for n in lens])]))

    def call():
        return K.kda_lin_prefill(q, k, v, g, cu, pool, slots, slots, scale=0.1, ckpt_interval=64, ckpt_offsets=off,
                                 ckpt_out=rungs)[0]
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        for t in (q, k, v):
            t.mul_(-0.9).add_(0.01 * i)
        results = []
        for replay in (False, True):
            pool.copy_(start)
            rungs.zero_()
            if replay:
                out.zero_()
                graph.replay()
            o = out if replay else call()
            torch.cuda.synchronize()
            results.append([x.clone() for x in (o, pool, rungs)])
        assert all(torch.equal(a, b) for a, b in zip(*results)), f"replay {i}"


def test_segments_on_another_stream(K):
    """A call that allocates its workspace on the stream given, beside another one on the current stream."""
    import torch
    c = Call("bf16", [2000, 33], 2, 4, 128, 64, "token", 141)
    assert is_cut(K, c)
    want, _ = K.kda_lin_prefill(c.q, c.k, c.v, c.g, i64(c.cu))
    cu = i64(c.cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        a, _ = K.kda_lin_prefill(c.q, c.k, c.v, c.g, cu, stream=s)
        b, _ = K.kda_lin_prefill(c.q, c.k, c.v, c.g, cu)
        s.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want)
