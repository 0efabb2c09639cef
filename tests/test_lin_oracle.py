"""CPU tests of the linear-attention layer's operators: the fp64 oracle against closed forms, and the C ABI's
refusals (fake addresses: every call here fails its checks or has nothing to do)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.linear as R

K = pytest.importorskip("gated_delta_rule_46_amd.kda", reason="libkda.so not built (run __graft_entry__.build())")

FAKE, MISALIGNED = 1 << 20, (1 << 20) + 2


# ---------------------------------------------------------------------------
# oracle
# ---------------------------------------------------------------------------
def rows(rng, T, Hk, Hv, dk, dv):
    return rng.normal(size=(T, Hk, dk)), rng.normal(size=(T, Hk, dk)), rng.normal(size=(T, Hv, dv))


def test_prefill_is_the_explicit_sum():
    """o_t = scale (sum_j e^{G_t - G_j} (q_t.k_j) v_j + e^{G_t} S0^T q_t), per sequence and with grouped heads."""
    rng = np.random.default_rng(1)
    T, Hk, Hv, dk, dv, cu = 9, 2, 4, 5, 3, [0, 4, 4, 9]
    q, k, v = rows(rng, T, Hk, Hv, dk, dv)
    g = -rng.random((T, Hv))
    pool = rng.normal(size=(5, Hv, dk, dv))
    o, new, _, final = R.prefill(q, k, v, g, cu, pool, [3, 1, -1], [0, 2, 4], scale=0.7)
    for n, S0 in enumerate((pool[3], pool[1], np.zeros_like(pool[0]))):
        a, b = cu[n], cu[n + 1]
        G = np.cumsum(g[a:b], 0)
        for h in range(Hv):
            for i in range(b - a):
                ref = S0[h].T @ q[a + i, h // 2] * np.exp(G[i, h])
                for j in range(i + 1):
                    ref = ref + np.exp(G[i, h] - G[j, h]) * (q[a + i, h // 2] @ k[a + j, h // 2]) * v[a + j, h]
                assert np.allclose(o[a + i, h], 0.7 * ref)
    assert np.array_equal(new[2], pool[1]) and np.array_equal(new[1], pool[1]) and np.array_equal(new[3], pool[3])
    assert np.array_equal(new[0], final[0]) and np.array_equal(new[4], final[2])


def test_prefill_in_pieces_and_rungs():
    """Chunks resumed from stored states give the whole run; the rungs are its states on the way."""
    rng = np.random.default_rng(2)
    q, k, v = rows(rng, 12, 1, 2, 4, 4)
    g = np.array([-0.3, -1.1])
    o, _, rungs, final = R.prefill(q, k, v, g, [0, 12], interval=5)
    pool = np.zeros((1, 2, 4, 4))
    parts = []
    for a, b in ((0, 5), (5, 10), (10, 12)):
        x, pool, _, _ = R.prefill(q[a:b], k[a:b], v[a:b], g, [0, b - a], pool, [0], [0])
        parts.append(x)
        if b < 12:
            assert np.allclose(pool[0], rungs[b // 5 - 1])
    assert np.allclose(np.concatenate(parts), o) and np.allclose(pool[0], final[0]) and len(rungs) == 2


def test_a_dropped_state_starts_afresh():
    """g = -inf forgets everything before a token, infinities too."""
    rng = np.random.default_rng(3)
    q, k, v = rows(rng, 6, 1, 1, 4, 4)
    g = -rng.random((6, 1))
    g[3] = -np.inf
    o, _, _, S = R.prefill(q, k, v, g, [0, 6])
    o2, _, _, S2 = R.prefill(q[3:], k[3:], v[3:], g[3:], [0, 3])
    assert np.allclose(o[3:], o2) and np.allclose(S, S2)


def test_head_norm_closed_forms():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    y, _ = R.head_norm(x, eps=0.0, act=0)
    assert np.allclose(y, x / 2.5)
    y, _ = R.head_norm(x + 5, eps=0.0, center=True, act=0)
    assert np.allclose(y.mean(), 0) and np.allclose((y * y).mean(), 1)
    z = np.array([[[0.0, 1.0, -1.0, 30.0]]])
    y, n = R.head_norm(x, z, np.full(4, 2.0), np.ones(4), act=2)
    assert np.allclose(y, n / (1 + np.exp(-z)))
    y, n = R.head_norm(x, act=1)
    assert np.allclose(y, n / (1 + np.exp(-n)))


# ---------------------------------------------------------------------------
# refusals of the C ABI
# ---------------------------------------------------------------------------
def err():
    return K.LIB.kda_last_error().decode()


def cfg(Hk=2, Hv=4, dk=128, dv=64, dtype=1, scale=1.0):
    return K.kda_lin_config(Hk, Hv, dk, dv, dtype, scale)


def ptr(x):
    return None if x is None else ctypes.byref(x)


def prefill(c=cfg(), q=FAKE, q_row=256, k=FAKE, k_row=256, v=FAKE, v_row=256, g=FAKE, g_row=4, cu=FAKE, N=2, T=100,
            pool=K.kda_state_pool(FAKE, 4, FAKE, FAKE), o=2 * FAKE, ckpt=None):
    return K.LIB.kda_lin_prefill(ptr(c), q, q_row, k, k_row, v, v_row, g, g_row, cu, N, T, ptr(pool), o, ptr(ckpt),
                                 FAKE, 0, None)


def decode(c=cfg(), N=2, q=FAKE, q_row=256, k=FAKE, k_row=256, v=FAKE, v_row=256, g=FAKE, g_row=4,
           pool=K.kda_state_pool(FAKE, 4, FAKE, FAKE), o=2 * FAKE):
    return K.LIB.kda_lin_decode(ptr(c), N, q, q_row, k, k_row, v, v_row, g, g_row, ptr(pool), o, None)


def norm(dtype=1, T=8, H=4, D=64, x=FAKE, x_row=256, gate=FAKE, gate_row=256, weight=FAKE, bias=FAKE, per_head=0,
         eps=1e-6, center=0, act=1, y=2 * FAKE, y_row=256):
    return K.LIB.kda_head_norm(dtype, T, H, D, x, x_row, gate, gate_row, weight, bias, per_head, eps, center, act, y,
                               y_row, None)


def test_struct_layout():
    pool = K.kda_state_pool.from_buffer_copy(K._pool_bytes(1 << 40, -3, 0, 5))
    assert (pool.states, pool.n_slots, pool.read_idx, pool.write_idx) == (1 << 40, -3, None, 5)
    assert ctypes.sizeof(K.kda_lin_config) == 24 and K.kda_lin_config.scale.offset == 20


@pytest.mark.parametrize("call", [prefill, decode])
def test_rows_and_config_are_checked(call):
    E, U, A = K.KDA_ERR_ARG, K.KDA_ERR_UNSUPPORTED, K.KDA_ERR_ALIGN
    assert call(c=None) == E
    assert call(c=cfg(Hk=0)) == E and call(c=cfg(Hv=-1)) == E
    assert call(c=cfg(Hk=3)) == E and "multiple" in err()
    assert call(c=cfg(dtype=2)) == E
    assert call(c=cfg(dk=96)) == U and call(c=cfg(dv=32)) == U and call(c=cfg(dk=0)) == U
    assert call(c=cfg(Hv=1 << 17)) == U
    assert call(c=cfg(scale=float("inf"))) == E and call(c=cfg(scale=float("nan"))) == E
    assert call(N=-1) == E
    assert call(N=(1 << 18) + 1) == U
    for name in ("q", "k", "v", "g", "o"):
        assert call(**{name: None}) == E and name in err()
        assert call(**{name: MISALIGNED}) == A and name in err()
    for name in ("q_row", "k_row", "v_row"):
        assert call(**{name: 255}) == E and name in err()
        assert call(**{name: 257}) == A and name in err()
        assert call(**{name: (1 << 24) + 8}) == U and name in err()
    assert call(g_row=3) == E and "g_row" in err()
    assert call(g_row=-4) == E
    assert call(g_row=(1 << 24) + 1) == U
    for name in ("q", "k", "v"):
        assert call(o=3 * FAKE, **{name: 3 * FAKE}) == E and "alias" in err()
    assert call(pool=K.kda_state_pool(FAKE, 0, FAKE, FAKE)) == E
    assert call(pool=K.kda_state_pool(None, 4, FAKE, FAKE)) == E
    assert call(pool=K.kda_state_pool(MISALIGNED, 4, FAKE, FAKE)) == A
    assert call(pool=K.kda_state_pool(FAKE, 4, MISALIGNED - 1, FAKE)) == A
    assert call(pool=K.kda_state_pool(FAKE, 4, FAKE, MISALIGNED - 1)) == A


def test_prefill_checks_its_own_arguments():
    E, U, A = K.KDA_ERR_ARG, K.KDA_ERR_UNSUPPORTED, K.KDA_ERR_ALIGN
    assert prefill(T=-1) == E
    assert prefill(T=(1 << 24) + 1) == U
    assert prefill(N=0) == E and "sequence" in err()
    assert prefill(cu=None) == E and prefill(cu=FAKE + 4) == A
    assert prefill(ckpt=K.kda_ckpt(100, FAKE, FAKE)) == E
    assert prefill(ckpt=K.kda_ckpt(0, FAKE, FAKE)) == E
    assert prefill(ckpt=K.kda_ckpt(128, None, FAKE)) == E and "offsets" in err()
    assert prefill(ckpt=K.kda_ckpt(128, FAKE, None)) == E
    assert prefill(ckpt=K.kda_ckpt(128, FAKE, MISALIGNED)) == A
    assert prefill(N=0, T=0, q=None, k=None, v=None, g=None, o=None, cu=None) == K.KDA_OK


def test_decode_needs_a_pool():
    E = K.KDA_ERR_ARG
    assert decode(pool=None) == E
    assert decode(pool=K.kda_state_pool(FAKE, 4, None, FAKE)) == E
    assert decode(pool=K.kda_state_pool(FAKE, 4, FAKE, None)) == E
    assert decode(N=0, q=None, k=None, v=None, g=None, o=None) == K.KDA_OK


def test_workspace_query_of_refused_calls():
    for c, T, N in ((None, 100, 1), (cfg(dk=96), 100, 1), (cfg(), -1, 1), (cfg(), 100, 0)):
        assert K.LIB.kda_lin_prefill_workspace(ptr(c), T, N) == 0


def test_head_norm_is_checked():
    E, U, A = K.KDA_ERR_ARG, K.KDA_ERR_UNSUPPORTED, K.KDA_ERR_ALIGN
    assert norm(dtype=7) == E and norm(T=-1) == E and norm(H=0) == E
    for D in (0, -8, 12, 1032):
        assert norm(D=D, x_row=8192, gate_row=8192, y_row=8192) == U
    assert norm(T=(1 << 24) + 1) == U
    assert norm(H=(1 << 24) + 1, D=64, T=1, x_row=1 << 31, gate_row=1 << 31, y_row=1 << 31) == U
    assert norm(per_head=2) == E and norm(center=-1) == E and norm(act=3) == E
    for eps in (-1e-6, float("inf"), float("nan")):
        assert norm(eps=eps) == E
    for name in ("x_row", "gate_row", "y_row"):
        assert norm(**{name: 248}) == E and norm(**{name: 260}) == A
    for name in ("x", "gate", "weight", "bias", "y"):
        assert norm(**{name: MISALIGNED}) == A
    assert norm(x=None) == E and norm(y=None) == E
    assert norm(y=FAKE, y_row=512) == E and "same row distance" in err()
    assert norm(y=3 * FAKE, gate=3 * FAKE, gate_row=512) == E
    assert norm(T=0, x=None, y=None) == K.KDA_OK


# ---------------------------------------------------------------------------
# refusals of the binding (forms as the calls see them: shape, strides, type, device)
# ---------------------------------------------------------------------------
def form(shape, dtype=torch.bfloat16, strides=None, dev=0):
    t = torch.empty(shape, dtype=dtype)
    return t.shape, t.stride() if strides is None else strides, dtype, dev


F32, I32, I64 = torch.float32, torch.int32, torch.int64
GOOD = dict(q=form((9, 2, 64)), k=form((9, 2, 64)), v=form((9, 4, 128)), g=form((9, 4), F32), cu=form((3,), I64),
            pool=form((5, 4, 64, 128), F32), read=form((2,), I32), write=form((2,), I32), interval=0, offsets=None,
            ckpt=None, out=None, workspace=None, scale=1.0)


def plan(**kw):
    return K._lin_prefill_plan(*{**GOOD, **kw}.values())


def test_prefill_forms():
    assert plan()[5] == [128, 128, 512, 4]
    assert plan(g=form((4,), F32))[5][3] == 0
    assert plan(g=form((9, 4), F32, (0, 1)))[5][3] == 0
    assert plan(q=form((9, 2, 64), strides=(640, 64, 1)), g=form((9, 4), F32, (12, 1)))[5] == [640, 128, 512, 12]
    one = dict(q=form((1, 2, 64)), k=form((1, 2, 64)), v=form((1, 4, 128)), cu=form((2,), I64), read=None, write=None)
    assert plan(**one, g=form((1, 4), F32, (0, 1)))[5] == [128, 128, 512, 4]
    plan(interval=128, offsets=form((3,), I64), ckpt=form((7, 4, 64, 128), F32))


@pytest.mark.parametrize("kw,kind", [
    (dict(q=form((9, 128))), ValueError), (dict(k=form((9, 1, 64))), ValueError), (dict(k=form((8, 2, 64))), ValueError),
    (dict(v=form((9, 4, 128), F32)), TypeError), (dict(q=form((9, 2, 64), torch.float16)), TypeError),
    (dict(q=form((9, 2, 64), strides=(128, 1, 2))), ValueError), (dict(v=form((9, 4, 128), dev=1)), ValueError),
    (dict(q=form((9, 2, 64), dev=-1)), ValueError), (dict(g=form((9, 2), F32)), ValueError),
    (dict(g=form((9, 4), torch.float64)), TypeError), (dict(g=form((9, 4), F32, (1, 9))), ValueError),
    (dict(g=form((3,), F32)), ValueError), (dict(cu=form((3,), I32)), TypeError), (dict(cu=form((0,), I64)), ValueError),
    (dict(pool=form((5, 4, 128, 64), F32)), ValueError), (dict(pool=form((5, 4, 64, 128))), TypeError),
    (dict(read=form((3,), I32)), ValueError), (dict(write=form((2,), I64)), TypeError), (dict(pool=None), ValueError),
    (dict(interval=64), ValueError), (dict(offsets=form((3,), I64)), ValueError),
    (dict(ckpt=form((7, 4, 64, 128), F32)), ValueError), (dict(out=form((9, 4, 64))), ValueError),
    (dict(interval=64, offsets=form((2,), I64)), ValueError),
    (dict(interval=96, offsets=form((3,), I64)), ValueError), (dict(interval=-64, offsets=form((3,), I64)), ValueError),
])
def test_prefill_refuses_forms(kw, kind):
    with pytest.raises(kind):
        plan(**kw)


def test_decode_and_norm_refuse_forms():
    d = dict(q=form((3, 2, 64)), k=form((3, 2, 64)), v=form((3, 4, 128)), g=form((4,), F32), pool=form((5, 4, 64, 128), F32),
             read=form((3,), I32), write=form((3,), I32), out=None, scale=1.0)
    assert K._lin_decode_plan(*d.values())[3] == [128, 128, 512, 0]
    for kw in (dict(pool=None), dict(read=None), dict(write=None), dict(read=form((2,), I32)), dict(out=form((3, 2, 128)))):
        with pytest.raises(ValueError):
            K._lin_decode_plan(*{**d, **kw}.values())
    n = dict(x=form((3, 4, 24)), gate=form((3, 4, 24), strides=(192, 24, 1)), weight=form((24,), F32), bias=None, out=None)
    assert K._head_norm_plan(*n.values())[5] == [96, 192, 96]
    for kw in (dict(x=form((3, 96))), dict(gate=form((3, 4, 16))), dict(weight=form((4, 24), F32), bias=form((24,), F32)),
               dict(weight=form((96,), F32)), dict(out=form((3, 4, 24), strides=(96, 1, 4)))):
        with pytest.raises(ValueError):
            K._head_norm_plan(*{**n, **kw}.values())
    with pytest.raises(TypeError):
        K._head_norm_plan(*{**n, **dict(gate=form((3, 4, 24), F32))}.values())
