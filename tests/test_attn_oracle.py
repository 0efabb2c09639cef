"""Pins of the attention-layer oracle (oracle/attention.py) to facts other than itself, and the
refusals of the new entry points.  No GPU needed, nothing is launched."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.attention as A

K = pytest.importorskip("gated_delta_rule_46_amd.kda",
                        reason="libkda.so not built (run __graft_entry__.build())")

FAKE = 1 << 20
MISALIGNED = FAKE + 2


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------
def test_e4m3_matches_torch_casts():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(A.e4m3_values(), codes.astype(np.float64), equal_nan=True)
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-14, 8, 4000), [0.0, 448.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = np.clip(x.astype(np.float32), -448, 448)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(A.e4m3_round(x), ref)
    assert A.e4m3_round(np.inf) == 448 and A.e4m3_round(-1e9) == -448 and np.isnan(A.e4m3_round(np.nan))


def test_scale_is_the_smallest_power_of_two():
    for amax in (448.0, 448.0001, 449.0, 1.0, 0.875, 0.8750001, 3e38, 1e-20, 7.0):
        s = A.scale_for(amax)
        assert amax <= 448 * s or s == 2.0 ** 119
        assert amax > 448 * (s / 2) or s == 2.0 ** -100
    assert A.scale_for(448.0) == 1.0 and A.scale_for(np.nextafter(448.0, 500)) == 2.0
    assert A.scale_for(0.0) == 2.0 ** -100 and A.scale_for(3.3e38) == 2.0 ** 119


def test_norm_rope_is_a_rotation():
    rng = np.random.default_rng(4)
    x = rng.normal(size=(3, 2, 64))
    ang = rng.uniform(0, 6, size=(5, 16))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for pairs in (False, True):
        y = A.norm_rope(x, None, 0.0, [4, 0, 2], table, pairs)
        assert np.allclose((y * y).mean(-1), 1.0)                       # norm kept by the rotation
        assert np.array_equal(y[..., 32:], A.norm_rope(x, None, 0.0)[..., 32:])
        back = A.norm_rope(y, None, 0.0, [0, 0, 0], np.concatenate([np.cos(ang[:1]), -np.sin(ang[:1])], 1), pairs)
        assert np.allclose(back[1], A.norm_rope(x, None, 0.0)[1])       # the opposite angle undoes it
    e = np.zeros((1, 1, 64))
    e[..., 0] = 1.0
    quarter = np.concatenate([np.zeros((1, 16)), np.ones((1, 16))], 1)
    assert A.norm_rope(e, None, 0.0, [0], quarter)[0, 0].argmax() == 16
    assert A.norm_rope(e, None, 0.0, [0], quarter, True)[0, 0].argmax() == 1


def test_cache_append_equals_one_write_when_the_scale_is_known_first():
    """Token by token equals all at once if the first token holds the maximum; read returns codes x scale."""
    rng = np.random.default_rng(5)
    x = rng.normal(size=(40, 2, 64)).astype(np.float32).astype(np.float64)
    x[0], x[16], x[32] = 9.0, 9.0, 9.0
    table = np.array([[2, 0, 1, -1]])
    mk = lambda: A.Cache(np.zeros((3, 2, 16, 64)), np.ones((3, 2)), table)
    one, many = mk(), mk()
    one.write(x, [0, 40], [40])
    for t in range(40):
        many.write(x[t:t + 1], [0, 1], [t + 1])
    assert np.array_equal(one.codes, many.codes) and np.array_equal(one.scale, many.scale)
    got = one.read([0, 40], [40], 40)
    assert np.abs(got - x).max() <= 9.0 * 2.0 ** -4 and np.array_equal(got[0], np.full((2, 64), 9.0))
    assert not one.read([0, 3], [60], 3).any()                         # absent pages


def test_attn_closed_forms():
    """Equal keys give the mean of the visible values; one visible key gives its value."""
    D, page = 64, 16
    rng = np.random.default_rng(6)
    table = np.array([[1, 0]])
    kc = np.ones((2, 1, page, D))
    vc = A.e4m3_round(rng.normal(size=(2, 1, page, D)))
    keys, vals = A.Cache(kc, np.ones((2, 1)), table), A.Cache(vc, np.full((2, 1), 2.0), table)
    v = np.concatenate([vc[1, 0], vc[0, 0]]) * 2
    q = rng.normal(size=(3, 2, D))
    o, lse, _, _ = A.attn(q, [0, 3], [20], keys, vals, 0.1)
    for i in range(3):
        assert np.allclose(o[i, 0], v[:18 + i].mean(0))
        assert np.allclose(lse[i], 0.1 * q[i].sum(-1) + np.log(18 + i))
    o, lse, _, _ = A.attn(q, [0, 3], [20], keys, vals, 0.1, window=1)
    assert np.allclose(o[:, 1], v[17:20])
    o, lse, _, _ = A.attn(q, [0, 3], [2], keys, vals, 0.1)
    assert not o[0].any() and np.all(lse[0] == -np.inf) and np.allclose(o[1, 0], v[0])


# ---------------------------------------------------------------------------
# refusals of the C ABI
# ---------------------------------------------------------------------------
def err():
    return K.LIB.kda_last_error().decode()


def cfg(Hq=8, Hk=2, D=128, dtype=1):
    return K.kda_attn_config(Hq, Hk, D, dtype)


def cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, n_pages=4, page=64, width=16, table=FAKE):
    return K.kda_kv_cache(k, v, ks, vs, n_pages, page, width, table)


def ref(x):
    return ctypes.byref(x) if x is not None else None


def rotate(c=cfg(), T=4, q=FAKE, q_row=1024, k_row=256, table=FAKE, n_pos=64, rot=128, layout=0, pos=FAKE, q_out=FAKE,
           qo_row=1024, eps=1e-6, w=None):
    return K.LIB.kda_qk_norm_rope(ref(c), T, q, q_row, FAKE, k_row, w, None, eps, table, n_pos, rot, layout, pos, q_out,
                                  qo_row, FAKE, 256, None)


def write(c=cfg(), kc=cache(), N=2, T=8, cu=FAKE, kv=FAKE, k=FAKE, k_row=256):
    return K.LIB.kda_kv_write(ref(c), ref(kc), N, T, cu, kv, k, k_row, FAKE, 256, None)


def read(c=cfg(), kc=cache(), N=2, T=8, k=FAKE):
    return K.LIB.kda_kv_read(ref(c), ref(kc), N, T, FAKE, FAKE, k, FAKE, None)


def attn(c=cfg(), kc=cache(), N=2, T=8, cu=FAKE, q=FAKE, q_row=1024, scale=0.1, causal=1, window=0, o=FAKE + 4096,
         lse=None, ws=FAKE, wsb=1 << 30):
    return K.LIB.kda_attn(ref(c), ref(kc), N, T, cu, FAKE, q, q_row, scale, causal, window, o, lse, ws, wsb, None)


@pytest.mark.parametrize("call", [rotate, write, read, attn])
def test_attn_config_refusals(call):
    assert call(c=None) == K.KDA_ERR_ARG and "cfg" in err()
    assert call(c=cfg(Hq=0)) == K.KDA_ERR_ARG
    assert call(c=cfg(Hk=-1)) == K.KDA_ERR_ARG
    assert call(c=cfg(Hq=7)) == K.KDA_ERR_ARG and "multiple" in err()
    assert call(c=cfg(dtype=2)) == K.KDA_ERR_ARG
    assert call(c=cfg(D=96)) == K.KDA_ERR_UNSUPPORTED
    assert call(T=-1) == K.KDA_ERR_ARG
    assert call(T=1 << 28) == K.KDA_ERR_UNSUPPORTED and "2^24" in err()
    assert call(T=(1 << 24) - 1) == K.KDA_ERR_UNSUPPORTED and "2^26" in err()
    assert call(T=0) == K.KDA_OK and err() == ""


@pytest.mark.parametrize("call", [write, read, attn])
def test_cache_refusals(call):
    assert call(kc=None) == K.KDA_ERR_ARG and "cache" in err()
    assert call(N=-1) == K.KDA_ERR_ARG
    assert call(N=0) == K.KDA_ERR_ARG
    assert call(N=1 << 23) == K.KDA_ERR_UNSUPPORTED and "2^20" in err()
    assert call(N=0, T=0) == K.KDA_OK
    for page in (0, 8, 48, 256):
        assert call(kc=cache(page=page)) == K.KDA_ERR_UNSUPPORTED
    assert call(kc=cache(n_pages=0)) == K.KDA_ERR_ARG
    assert call(kc=cache(width=0)) == K.KDA_ERR_ARG
    assert call(kc=cache(width=1 << 26)) == K.KDA_ERR_UNSUPPORTED
    assert call(kc=cache(k=None)) == K.KDA_ERR_ARG
    assert call(kc=cache(v=FAKE + 8)) == K.KDA_ERR_ALIGN
    assert call(kc=cache(ks=None)) == K.KDA_ERR_ARG
    assert call(kc=cache(vs=MISALIGNED)) == K.KDA_ERR_ALIGN
    assert call(kc=cache(table=MISALIGNED)) == K.KDA_ERR_ALIGN


def test_rotate_refusals():
    assert rotate(q=None) == K.KDA_ERR_ARG and rotate(q=MISALIGNED) == K.KDA_ERR_ALIGN
    assert rotate(q_row=1000) == K.KDA_ERR_ARG and "q_row" in err()
    assert rotate(q_row=1028) == K.KDA_ERR_ALIGN
    assert rotate(layout=2) == K.KDA_ERR_ARG
    assert rotate(rot=24) == K.KDA_ERR_UNSUPPORTED and rotate(rot=256) == K.KDA_ERR_UNSUPPORTED
    assert rotate(rot=0) == K.KDA_ERR_UNSUPPORTED
    assert rotate(n_pos=0) == K.KDA_ERR_ARG
    assert rotate(pos=None) == K.KDA_ERR_ARG and rotate(pos=FAKE + 4) == K.KDA_ERR_ALIGN
    assert rotate(eps=-1.0) == K.KDA_ERR_ARG and rotate(eps=float("nan")) == K.KDA_ERR_ARG
    assert rotate(w=MISALIGNED) == K.KDA_ERR_ALIGN
    assert rotate(q_row=2048) == K.KDA_ERR_ARG and "in place" in err()


def test_write_read_refusals():
    assert write(k=None) == K.KDA_ERR_ARG and write(k=MISALIGNED) == K.KDA_ERR_ALIGN
    assert write(k_row=128) == K.KDA_ERR_ARG and write(k_row=260) == K.KDA_ERR_ALIGN
    assert write(cu=None) == K.KDA_ERR_ARG and write(kv=FAKE + 4) == K.KDA_ERR_ALIGN
    assert read(k=None) == K.KDA_ERR_ARG and read(k=MISALIGNED) == K.KDA_ERR_ALIGN


def test_attn_refusals():
    assert attn(scale=float("inf")) == K.KDA_ERR_ARG and attn(scale=-3e38) == K.KDA_ERR_ARG
    assert attn(causal=2) == K.KDA_ERR_ARG and attn(window=-1) == K.KDA_ERR_ARG
    assert attn(q=None) == K.KDA_ERR_ARG and attn(o=MISALIGNED) == K.KDA_ERR_ALIGN
    assert attn(o=FAKE) == K.KDA_ERR_ARG and "alias" in err()
    assert attn(lse=MISALIGNED) == K.KDA_ERR_ALIGN
    assert attn(cu=FAKE + 4) == K.KDA_ERR_ALIGN
    need = K.LIB.kda_attn_workspace(ref(cfg()), ref(cache(width=64)), 2, 8, 0)
    assert need > 0 and need % 256 == 0
    big = cache(width=64)
    assert attn(kc=big, ws=None) == K.KDA_ERR_WORKSPACE and attn(kc=big, wsb=need - 1) == K.KDA_ERR_WORKSPACE
    assert attn(kc=big, ws=FAKE + 8) == K.KDA_ERR_ALIGN
    assert K.LIB.kda_attn_workspace(ref(cfg()), ref(cache(width=64)), 2, 0, 0) == 0
    assert K.LIB.kda_attn_workspace(None, ref(cache(width=64)), 2, 8, 0) == 0
    # a unit per workgroup: no parts
    assert K.LIB.kda_attn_workspace(ref(cfg()), ref(cache(width=8)), 2, 8, 0) == 0
    assert K.LIB.kda_attn_workspace(ref(cfg()), ref(cache(width=64)), 2, 8, 100) == 0


def test_attn_struct_layouts():
    assert ctypes.sizeof(K.kda_attn_config) == 16 and ctypes.sizeof(K.kda_kv_cache) == 56
    assert K.kda_kv_cache.page.offset == 40 and K.kda_kv_cache.table.offset == 48


def test_binding_refuses_host_tensors_and_bad_layouts():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        K.kda_qk_norm_rope(x, x)
    f = K._form
    with pytest.raises(ValueError, match="contiguous"):
        K._rows(f(x.transpose(0, 1).contiguous().transpose(0, 1)), "q", 4, 64, x.dtype, -1)
    with pytest.raises(ValueError, match="shape"):
        K._rows(f(x), "q", 4, 128, x.dtype, -1)
    with pytest.raises(ValueError, match="shape"):
        K._rows(f(x), "q", 4, 64, x.dtype, -1, 3)
    with pytest.raises(TypeError, match="dtype"):
        K._rows(f(x), "q", 4, 64, torch.float32, -1)
    wide = torch.zeros((4, 6, 64), dtype=torch.bfloat16)
    assert K._rows(f(wide[:, 2:4]), "k", 4, 64, x.dtype, -1) == 384
    assert K._rows(f(wide[:1, 2:4]), "k", 1, 64, x.dtype, -1) == 384
    K._dense(f(wide[:1, 2:4]), "w", (1, 2, 64), x.dtype, -1)
    for bad in (wide[:, 2:4], wide.transpose(1, 2)):
        with pytest.raises(ValueError, match="contiguous"):
            K._dense(f(bad), "w", bad.shape, x.dtype, -1)
    with pytest.raises(ValueError, match="required"):
        K._dense(None, "w", (4,), x.dtype, -1)

    def cache(k=torch.uint8, table=(1, 4), scale=(3, 2)):
        return K.KVCache(torch.zeros((3, 2, 16, 64), dtype=k), torch.zeros((3, 2, 16, 64), dtype=torch.uint8),
                         torch.ones(scale), torch.ones(3, 2), torch.zeros(table, dtype=torch.int32)).form()
    assert K._cache_sizes(cache(), 1, 2, 64, -1) == (3, 16, 4)
    with pytest.raises(TypeError, match="uint8"):
        K._cache_sizes(cache(k=torch.float32), 1, 2, 64, -1)
    with pytest.raises(ValueError, match="cache.table"):
        K._cache_sizes(cache(), 2, 2, 64, -1)
    with pytest.raises(ValueError, match="k_scale"):
        K._cache_sizes(cache(scale=(3, 1)), 1, 2, 64, -1)
    with pytest.raises(ValueError, match="cache.k"):
        K._cache_sizes(cache(), 1, 4, 64, -1)
    with pytest.raises(ValueError, match="cu_seqlens"):
        K._sequences(f(torch.zeros((2, 2), dtype=torch.int64)), f(torch.zeros(1, dtype=torch.int64)), -1)
    with pytest.raises(TypeError, match="kv_len"):
        K._sequences(f(torch.zeros(2, dtype=torch.int64)), f(torch.zeros(1, dtype=torch.int32)), -1)
