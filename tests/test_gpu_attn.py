"""GPU tests of the attention-layer operators against the fp64 oracle (oracle/attention.py).

Tolerances follow from the arithmetic and are elementwise:
  * the cache is exact: scales are powers of two, codes are rounded once;
  * norm and rotation: fp32 arithmetic (D/2 + 16 roundings of 2^-24 along the sum of squares, square
    root, products) relative to the two values of a pair, and half a step of the output type;
  * attention: half a step of the output type (2^-8 bf16, 2^-24 fp32) on the result, half a bf16 step
    (bf16 rows) on each probability, hence on A = sum p |v|, and twice the error d of a score's fp32
    arithmetic on A; d = 2^-24 (D + 8) max_j sum_i |scale q_i k_ij| + (keys + 16) 2^-24.
"""
import sys

import numpy as np
import pytest

import oracle.attention as A
from workloads.device import to_numpy_f64

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def say(msg):
    print(f"[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def K():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_46_amd.kda as kda
    return kda


def dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def dev(x, dtype=None):
    import torch
    t = torch.as_tensor(np.asarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def i64(x):
    return dev(np.asarray(x, np.int64))


def within(name, got, ref, tol):
    bad = ~(np.abs(got - ref) <= tol)
    bad &= ~((np.isnan(got) & np.isnan(ref)) | (np.isinf(ref) & (got == ref)))
    worst = float(np.nanmax(np.where(tol > 0, np.abs(got - ref) / np.where(tol > 0, tol, 1), 0.0))) if got.size else 0.0
    say(f"{name}: worst error / tolerance {worst:.3f}")
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: " \
        f"{got[tuple(np.argwhere(bad)[0])]} against {ref[tuple(np.argwhere(bad)[0])]}"


# ---------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------
def rope_table(n_pos, rot, base=10000.0):
    f = base ** (-np.arange(rot // 2) / (rot // 2))
    a = np.arange(n_pos)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rotate_case(K, dtype, T, Hq, Hk, D, rot, pairs, seed, weights=True, in_place=False, packed=True, pad=()):
    import torch
    rng = np.random.default_rng(seed)
    qkv = dev(rng.normal(size=(T, Hq + 2 * Hk, D)) * 2, dt(dtype))
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    pos = rng.integers(0, 500, T)
    for i, p in pad:
        pos[i] = p
    table = rope_table(500, rot) if rot else None
    w = [dev((1 + 0.3 * rng.normal(size=D)).astype(np.float32)) if weights else None for _ in "qk"]
    ref = [A.norm_rope(to_numpy_f64(x), None if y is None else to_numpy_f64(y), 1e-6, pos, table, pairs)
           for x, y in ((q, w[0]), (k, w[1]))]
    keep = [to_numpy_f64(x) for x in (q, k)]
    kw = dict(q_out=q, k_out=k) if in_place else dict(q_out=torch.full_like(q.contiguous(), 7.0),
                                                      k_out=torch.full_like(k.contiguous(), 7.0))
    rest = qkv[:, Hq + Hk:].clone()
    got = K.kda_qk_norm_rope(q, k, i64(pos) if rot else None, None if table is None else dev(table), q_weight=w[0],
                             k_weight=w[1], layout=K.KDA_ROPE_PAIRS if pairs else K.KDA_ROPE_HALVES, **kw)
    torch.cuda.synchronize()
    assert torch.equal(rest, qkv[:, Hq + Hk:])
    for name, g, r, old in zip("qk", got, ref, keep):
        g = to_numpy_f64(g)
        left = np.isnan(r).all((1, 2))
        assert np.array_equal(g[left], old[left] if in_place else np.full_like(g[left], 7.0)), "a padded row changed"
        g, r = g[~left], r[~left]
        pair = np.zeros_like(r)
        if rot:
            x = r[..., :rot]
            if pairs:
                y = np.repeat(np.hypot(x[..., 0::2], x[..., 1::2]), 2, -1)
            else:
                y = np.concatenate([np.hypot(x[..., :rot // 2], x[..., rot // 2:])] * 2, -1)
            pair[..., :rot] = y
        within(name, g, r, HALF[dtype] * np.abs(r) + (D / 2 + 16) * 2.0 ** -24 * np.maximum(np.abs(r), 2 * pair) + 1e-37)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot,pairs", [(128, 128, False), (128, 128, True), (128, 48, False), (128, 16, True),
                                         (64, 64, False), (64, 32, True), (64, 16, False), (128, 0, False)])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (5, 6, 3), (67, 32, 8)])
def test_rotate(K, dtype, D, rot, pairs, T, Hq, Hk):
    say(f"rotate {dtype} D={D} rot={rot} pairs={pairs} T={T} Hq={Hq} Hk={Hk}")
    rotate_case(K, dtype, T, Hq, Hk, D, rot, pairs, 100 + T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotate_in_place_padding_and_plain_rows(K, dtype):
    say(f"rotate in place {dtype}")
    rotate_case(K, dtype, 9, 5, 5, 64, 64, False, 7, in_place=True, pad=((0, -1), (4, 500), (8, 1 << 40)))
    say("rotate plain rows, no weights, padded tokens")
    rotate_case(K, dtype, 9, 3, 1, 128, 64, True, 8, weights=False, packed=False, pad=((3, -5),))


def test_rotate_non_finite_stays_in_its_head(K):
    import torch
    say("rotate with NaN, inf and a zero row")
    q = torch.randn(4, 3, 64, device="cuda")
    k = torch.randn(4, 3, 64, device="cuda")
    q[0, 1, 5], q[1, 0, 9], k[2, 1] = float("nan"), float("inf"), 0.0
    qo, ko = K.kda_qk_norm_rope(q, k, i64([0, 1, 2, 3]), dev(rope_table(8, 64)))
    torch.cuda.synchronize()
    assert torch.isnan(qo[0, 1]).all() and torch.isfinite(qo[0, [0, 2]]).all() and torch.isfinite(qo[1, 1:]).all()
    assert (ko[2, 1] == 0).all() and torch.isfinite(ko).all()


def test_rotate_infinity_stays_in_its_dim_where_nothing_rotates(K):
    import torch
    say("rotate with an infinity among the dims behind rot, pairs")
    q, k = torch.randn(2, 2, 64, device="cuda"), torch.randn(2, 1, 64, device="cuda")
    q[0, 1, 40] = float("inf")
    qo, _ = K.kda_qk_norm_rope(q, k, i64([3, 5]), dev(rope_table(8, 32)), layout=K.KDA_ROPE_PAIRS)
    torch.cuda.synchronize()
    rest = [i for i in range(64) if i != 40]           # x / inf = 0
    assert torch.isnan(qo[0, 1, 40]) and (qo[0, 1, rest] == 0).all() and torch.isfinite(qo[1]).all()


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------
class Model:
    """A cache on the GPU and its oracle, written and read together."""

    def __init__(self, K, dtype, Hk, D, page, n_pages, table, seed=1):
        import torch
        self.K, self.dtype, self.Hk, self.D = K, dtype, Hk, D
        rng = np.random.default_rng(seed)
        codes = [rng.integers(0, 256, (n_pages, Hk, page, D)).astype(np.uint8) for _ in "kv"]    # what was there before
        scale = [2.0 ** rng.integers(-5, 5, (n_pages, Hk)).astype(np.float32) for _ in "kv"]
        self.table = np.asarray(table, np.int32)
        self.gpu = K.KVCache(*[dev(x) for x in codes], *[dev(x) for x in scale], dev(self.table))
        vals = A.e4m3_values()
        self.keys, self.values = (A.Cache(vals[c], s, self.table) for c, s in zip(codes, scale))

    def write(self, k, v, cu, kv_len, T=None):
        """k, v: device rows."""
        import torch
        self.K.kda_kv_write(k, v, i64(cu), i64(kv_len), self.gpu)
        torch.cuda.synchronize()
        self.keys.write(to_numpy_f64(k), cu, kv_len)
        self.values.write(to_numpy_f64(v), cu, kv_len)
        self.check()

    def check(self, void=None):
        """Codes and scales of the whole cache, the untouched and stale parts among them."""
        import torch
        for g, s, m in ((self.gpu.k, self.gpu.k_scale, self.keys), (self.gpu.v, self.gpu.v_scale, self.values)):
            assert np.array_equal(to_numpy_f64(s), m.scale)
            got = A.e4m3_values()[g.view(torch.uint8).cpu().numpy()]
            assert np.array_equal(got, m.codes, equal_nan=True)

    def rows(self, rng, T, spread=1.0):
        x = rng.normal(size=(T, 2 * self.Hk, self.D)) * np.exp(spread * rng.normal(size=(T, 2 * self.Hk, 1)))
        x = dev(x, dt(self.dtype))
        return x[:, :self.Hk], x[:, self.Hk:]


def tables(n_seq, width, rng, extra=2):
    n = n_seq * width + extra
    return rng.permutation(n)[:n_seq * width].reshape(n_seq, width).astype(np.int32), n


def cum(x):
    return [0] + list(np.cumsum(x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hk,D", [(1, 64), (3, 128)])
def test_cache_write_in_steps(K, dtype, page, Hk, D):
    """Prompts, chunks that end inside pages, single tokens, an empty and an absent sequence; the maximum
    grows and shrinks, so scales grow inside pages."""
    say(f"cache write {dtype} page={page} Hk={Hk} D={D}")
    rng = np.random.default_rng(page + D)
    tab, n_pages = tables(4, 5, rng)
    tab[3, 1:] = -1
    m = Model(K, dtype, Hk, D, page, n_pages, tab)
    kv = np.zeros(4, int)
    for new in ([page + 3, 0, 1, 5], [1, 1, 1, 1], [page, 7, 2 * page + 1, 0], [1, 0, 1, 1], [5, 60, 1, page]):
        kv = kv + new
        k, v = m.rows(rng, sum(new))
        m.write(k, v, cum(new), kv)
    back = np.minimum(kv, page + 9)
    gk, gv = K.kda_kv_read(i64(cum(back)), i64(kv), m.gpu, int(back.sum()), dt(dtype))
    assert np.array_equal(to_numpy_f64(gk), m.keys.read(cum(back), kv, int(back.sum())))
    assert np.array_equal(to_numpy_f64(gv), m.values.read(cum(back), kv, int(back.sum())))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_special_values(K, dtype):
    """Zeros, infinities, NaN, the largest and the smallest numbers, code ties."""
    say(f"cache special values {dtype}")
    rng = np.random.default_rng(2)
    m = Model(K, dtype, 2, 64, 16, 8, [[3, 1, 7, 0, 2]])
    big = 3.3e38
    rows = rng.normal(size=(70, 4, 64))
    rows[0:16] = 0
    rows[3, 0, 5], rows[4, 1, 6], rows[5, 2, 7] = np.nan, np.inf, -np.inf
    rows[16:32, 0] *= 1e-38
    rows[16:32, 1] *= 1e-30
    rows[20, 2, 3], rows[21, 3, 4] = big, -big
    rows[32:48] = np.round(rows[32:48] * 64) / 16                        # many ties of the code grid
    rows[48, :, 0] = 448.0
    rows[49, :, 1] = 449.0 if dtype == "f32" else 450.0
    x = dev(rows, dt(dtype))
    k, v = x[:, :2], x[:, 2:]
    m.write(k[:40], v[:40], [0, 40], [40])
    m.write(k[40:49], v[40:49], [0, 9], [49])
    m.write(k[49:50], v[49:50], [0, 1], [50])                            # a scale that just has to grow
    m.write(k[50:], v[50:], [0, 20], [70])
    m.write(k[:3], v[:3], [0, 3], [36])                                  # an earlier position again: rows behind are void


def test_cache_padding_and_bad_places(K):
    """Rows behind the last sequence, positions past the table or below zero, pages outside the pool."""
    import torch
    say("cache padding")
    rng = np.random.default_rng(9)
    tab = [[5, 99, -7, 2], [0, 1, 3, 4]]
    m = Model(K, "bf16", 2, 64, 16, 6, tab)
    for new, kv in (([40, 3], [64, 3]), ([5, 30], [70, 66]), ([7, 2], [4, 0]), ([2, 9], [1 << 40, 12]), ([1, 1], [-3, 13])):
        k, v = m.rows(rng, sum(new) + 6)
        m.write(k, v, cum(new), kv)
        T = sum(new) + 6
        out = [torch.full((T, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        K.kda_kv_read(i64(cum(new)), i64(kv), m.gpu, T, k_out=out[0], v_out=out[1])
        torch.cuda.synchronize()
        for got, c in zip(out, (m.keys, m.values)):
            assert np.array_equal(to_numpy_f64(got)[:sum(new)], c.read(cum(new), kv, sum(new)), equal_nan=True)
            assert (got[sum(new):] == 3.0).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def plain_model(K, dtype, Hk, D, page, kv, seed, width=None, nan_tail=True):
    """A filled cache: normal codes up to each kv_len; the rest of the pool holds NaN codes and wild scales."""
    rng = np.random.default_rng(seed)
    need = [max(0, -(-max(n, 0) // page)) for n in kv]
    width = max(max(need), 1) if width is None else width
    n_pages = sum(need) + 2
    order = rng.permutation(n_pages)
    tab = np.full((len(kv), width), -1, np.int32)
    at = 0
    for n, b in enumerate(need):
        tab[n, :b] = order[at:at + b]
        at += b
    m = Model(K, dtype, Hk, D, page, n_pages, tab, seed)
    import torch
    for half in ("k", "v"):
        codes = np.full((n_pages, Hk, page, D), 0x7F if nan_tail else 0, np.uint8)
        scale = np.full((n_pages, Hk), np.nan if nan_tail else 1.0, np.float32)
        for n, L in enumerate(kv):
            for b in range(need[n]):
                r = min(page, L - b * page)
                x = torch.from_numpy(rng.normal(size=(Hk, r, D)) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
                codes[tab[n, b], :, :r] = x.view(torch.uint8).numpy()
                scale[tab[n, b]] = 2.0 ** rng.integers(-8, -4, Hk)
        setattr(m.gpu, half, dev(codes))
        setattr(m.gpu, half + "_scale", dev(scale))
        c = A.Cache(A.e4m3_values()[codes], scale, tab)
        if half == "k":
            m.keys = c
        else:
            m.values = c
    return m, rng


def attn_check(K, m, dtype, q, cu, kv, scale, causal=True, window=0, name="o", **kw):
    import torch
    o, lse = K.kda_attn(q, i64(cu), i64(kv), m.gpu, scale=scale, causal=causal, window=window, want_lse=True, **kw)
    torch.cuda.synchronize()
    attn_compare(m, dtype, q, cu, kv, scale, causal, window, o, lse, name)
    return o, lse


def attn_compare(m, dtype, q, cu, kv, scale, causal, window, o, lse, name="o"):
    T, _, D = q.shape
    ro, rl, RA, S = A.attn(to_numpy_f64(q), cu, kv, m.keys, m.values, scale, causal, window)
    used = cu[-1]
    d = (2.0 ** -24 * (D + 8) * S + (max(list(kv) + [0]) + 16) * 2.0 ** -24)
    p = HALF[dtype] if dtype == "bf16" else 2.0 ** -24
    tol = HALF[dtype] * np.abs(ro) + (p + 2 * d[..., None]) * RA * (1 + 2.0 ** -7) + 1e-37
    within(name, to_numpy_f64(o)[:used], ro[:used], tol[:used])
    within(name + " lse", to_numpy_f64(lse)[:used], rl[:used],
           d[:used] + 2.0 ** -22 * np.abs(np.where(np.isinf(rl), 0, rl))[:used])


def queries(rng, T, Hq, D, dtype, packed=True):
    x = dev(rng.normal(size=(T, Hq + 3, D)) * 2, dt(dtype))
    return x[:, :Hq] if packed else x[:, :Hq].contiguous()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,page,Hk,G", [(128, 64, 2, 4), (64, 16, 1, 1), (128, 32, 1, 7), (64, 128, 3, 2), (128, 16, 1, 16),
                                         (64, 64, 1, 24)])
@pytest.mark.parametrize("wide", [False, True])
def test_attn_decode(K, dtype, D, page, Hk, G, wide):
    """One new token per sequence: lengths 0, 1, around tiles and pages, long ones; a capacity that
    makes the call split its units and one that does not."""
    say(f"attn decode {dtype} D={D} page={page} Hk={Hk} G={G} wide={wide}")
    kv = [1, 63, 64, 65, 0, 17, 200, 300] + ([2500, 777] if wide else [])
    m, rng = plain_model(K, dtype, Hk, D, page, kv, 11 + D + G, width=None if wide else 512 // page)
    attn_check(K, m, dtype, queries(rng, len(kv), Hk * G, D, dtype), cum([1] * len(kv)), kv, 0.3 * D ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,page,Hk,G", [(128, 64, 2, 4), (64, 16, 2, 1), (128, 128, 1, 3), (64, 32, 1, 8)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (False, 0), (False, 33), (True, 1), (True, 2000)])
@pytest.mark.parametrize("room", [0, 20000])
def test_attn_rows(K, dtype, D, page, Hk, G, causal, window, room):
    """Packed sequences of many lengths, an empty one, one whose new tokens are all it has; a table for
    just these lengths (a workgroup per unit) and a wide one (shares that cut units)."""
    say(f"attn rows {dtype} D={D} page={page} Hk={Hk} G={G} causal={causal} window={window} room={room}")
    new = [1, 33, 0, 150, 2, 64]
    kv = [40, 33, 20, 411, 130, 700]
    m, rng = plain_model(K, dtype, Hk, D, page, kv, 5 + D + G + window, width=room // page or None)
    attn_check(K, m, dtype, queries(rng, sum(new), Hk * G, D, dtype), cum(new), kv, D ** -0.5, causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,page,Hk,G", [(128, 64, 1, 4), (64, 16, 2, 2), (128, 128, 1, 3), (64, 32, 1, 8), (128, 16, 1, 1)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (False, 0), (True, 7)])
def test_attn_prompts(K, dtype, D, page, Hk, G, causal, window):
    """Prompts and chunks long enough for units of 128 rows beside short ones and an empty sequence."""
    say(f"attn prompts {dtype} D={D} page={page} Hk={Hk} G={G} causal={causal} window={window}")
    new = [1, 300, 0, 65, 620, 3]
    kv = [40, 300, 20, 411, 1500, 130]
    m, rng = plain_model(K, dtype, Hk, D, page, kv, 6 + D + G + window, width=6400 // page)
    attn_check(K, m, dtype, queries(rng, sum(new), Hk * G, D, dtype), cum(new), kv, D ** -0.5, causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,kv,window", [(33, 33, 0), (129, 4200, 0), (257, 70, 0), (64, 2100, 200), (5, 1000, 0)])
@pytest.mark.parametrize("room", [0, 50000])
def test_attn_one_sequence(K, dtype, new, kv, window, room):
    """A sequence alone: a prompt, a chunk that is split over the keys, more rows than keys, a window; a
    table for just this length (small calls: units of 16 rows) and a wide one (units of 128,
    of 16 and 32 for the shortest)."""
    say(f"attn one sequence {dtype} new={new} kv={kv} window={window} room={room}")
    m, rng = plain_model(K, dtype, 2, 128, 64, [kv], new, width=room // 64 or None)
    attn_check(K, m, dtype, queries(rng, new, 8, 128, dtype), [0, new], [kv], 0.1, True, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,new,kv", [(400, 1, 30), (400, 4, 2000), (400, 0, 50), (130, 129, 500)])
def test_attn_one_padded_sequence(K, dtype, T, new, kv):
    """A sequence alone in a call padded to more rows: its rows right, the others left as they are."""
    import torch
    say(f"attn one padded sequence {dtype} T={T} new={new} kv={kv}")
    m, rng = plain_model(K, dtype, 2, 128, 64, [kv], 9 + new, width=800)
    q = queries(rng, T, 8, 128, dtype)
    out, lse = torch.full((T, 8, 128), 5.0, dtype=dt(dtype), device="cuda"), torch.full((T, 8), 5.0, device="cuda")
    attn_check(K, m, dtype, q, [0, new], [kv], 0.1, out=out, lse_out=lse)
    assert (out[new:] == 5.0).all() and (lse[new:] == 5.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,page,Hk,G,new", [(128, 64, 2, 4, [5] * 5), (64, 16, 1, 8, [4] * 3), (128, 128, 1, 3, [7] * 4),
                                             (64, 32, 2, 1, [31, 31]), (128, 16, 1, 24, [1] * 6), (64, 64, 1, 1, [18] * 4),
                                             (128, 32, 1, 8, [1, 8, 0, 3, 9, 5]), (64, 64, 2, 4, [16, 2, 17, 4, 8])])
@pytest.mark.parametrize("window", [0, 70])
def test_attn_drafted_tokens(K, dtype, D, page, Hk, G, new, window):
    """A few tokens on each sequence with a large table: 17 to 32 query rows per kv head (units of 32),
    equally many or not, and sequences of just over and under 64 rows side by side."""
    say(f"attn drafts {dtype} D={D} page={page} Hk={Hk} G={G} new={new} window={window}")
    kv = [900, 65, 31, 333, 64, 2000][:len(new)]
    m, rng = plain_model(K, dtype, Hk, D, page, kv, 40 + D + G, width=300000 // page)
    attn_check(K, m, dtype, queries(rng, sum(new), Hk * G, D, dtype), cum(new), kv, D ** -0.5, True, window)


@pytest.mark.parametrize("wide", [False, True])
def test_attn_shared_pages(K, wide):
    """A common prefix: pages that stand in several sequences' tables, and twice in one."""
    say(f"attn shared pages wide={wide}")
    new, kv = [1, 40, 2], [300, 300, 200]
    m, rng = plain_model(K, "bf16", 2, 64, 32, kv, 4, width=200 if wide else 10)
    m.table[1, :6] = m.table[0, :6]
    m.table[2, 3] = m.table[2, 2]
    m.gpu.table = dev(m.table)
    m.keys.table = m.values.table = m.table
    attn_check(K, m, "bf16", queries(rng, sum(new), 4, 64, "bf16"), cum(new), kv, 0.1)


def test_attn_window_argument(K):
    say("attn window beyond 31 bits")
    m, rng = plain_model(K, "bf16", 1, 64, 16, [20], 1)
    q = queries(rng, 1, 1, 64, "bf16")
    for bad in (1 << 31, (1 << 32) + 5, -1):
        with pytest.raises(ValueError, match="window"):
            K.kda_attn(q, i64([0, 1]), i64([20]), m.gpu, window=bad)
    attn_check(K, m, "bf16", q, [0, 1], [20], 0.1, window=(1 << 31) - 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_prompt_queries_of_all_sizes(K, dtype):
    """Query elements from 2^-40 to 2^30 in one row, rows of zeros, NaN and infinite queries."""
    import torch
    say(f"attn query sizes {dtype}")
    new, kv, D = 200, 330, 128
    m, rng = plain_model(K, dtype, 1, D, 64, [kv], 51, width=400)
    q = queries(rng, new, 2, D, dtype).clone()
    attn_check(K, m, dtype, q, [0, new], [kv], 0.0, name="scale 0")
    attn_check(K, m, dtype, q, [0, new], [kv], -0.1, name="negative scale")
    attn_check(K, m, dtype, q, [0, new], [kv], 5.0, name="scores of hundreds")
    q *= torch.exp2(torch.randint(-8, 5, q.shape, device="cuda")).to(q.dtype)
    q[10] = 0
    q[11] *= 2.0 ** -100
    q[12, 0, ::3] *= 2.0 ** -30
    attn_check(K, m, dtype, q, [0, new], [kv], 0.02)
    q[20, 0, 7], q[21, 1, 9], q[22, 0] = float("nan"), float("inf"), float("-inf")
    o, lse = K.kda_attn(q, i64([0, new]), i64([kv]), m.gpu, want_lse=True)
    bad = torch.zeros(new, 2, dtype=torch.bool, device="cuda")
    bad[20, 0] = bad[21, 1] = bad[22, 0] = True
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    assert torch.equal(torch.isnan(lse), bad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_rows_that_see_nothing(K, dtype):
    """kv_len below the new tokens, absent pages, a table that ends early, padded rows: o = 0 and lse =
    -inf for rows without keys, rows behind the last sequence untouched."""
    import torch
    say(f"attn empty rows {dtype}")
    new, kv = [5, 3, 20, 4, 7], [2, 0, 90, 1 << 40, -4]
    m, rng = plain_model(K, dtype, 2, 64, 16, [2, 0, 90, 200, 0], 21, width=13)
    m.table[2, 0:2] = -1                               # the first 32 keys of sequence 2
    m.table[2, 4] = 12345
    m.gpu.table = dev(m.table)
    m.keys.table = m.values.table = m.table
    kv_o = [2, 0, 90, 200, -4]
    q = queries(rng, sum(new) + 4, 6, 64, dtype)
    for causal, window in ((True, 0), (True, 9), (False, 0)):
        out = torch.full((sum(new) + 4, 6, 64), 5.0, dtype=dt(dtype), device="cuda")
        lse = torch.full((sum(new) + 4, 6), 5.0, device="cuda")
        K.kda_attn(q, i64(cum(new)), i64(kv), m.gpu, scale=0.2, causal=causal, window=window, want_lse=True, out=out,
                   lse_out=lse)
        torch.cuda.synchronize()
        assert (out[sum(new):] == 5.0).all() and (lse[sum(new):] == 5.0).all()
        # sequence 3 stands at 2^40: with a window it sees nothing
        s3 = slice(sum(new[:3]), sum(new[:4]))
        if window:
            assert not out[s3].any() and torch.isinf(lse[s3]).all()
        keep = [n for n in range(5) if n != 3]
        rows = np.concatenate([np.arange(sum(new[:n]), sum(new[:n + 1])) for n in keep])
        ref = A.attn(to_numpy_f64(q), cum(new), kv_o, m.keys, m.values, 0.2, causal, window)
        empty = np.isinf(ref[1][rows])
        assert empty.any() and not empty.all()
        got, gl = to_numpy_f64(out)[rows], to_numpy_f64(lse)[rows]
        assert not got[empty].any() and np.all(gl[empty] == -np.inf)
        d = 2.0 ** -24 * 72 * ref[3][rows] + 300 * 2.0 ** -24
        tol = HALF[dtype] * np.abs(ref[0][rows]) + (HALF[dtype] + 2 * d[..., None]) * ref[2][rows] * 1.01 + 1e-37
        within("o", got, ref[0][rows], tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width,len0", [(8, 40), (40, 40), (20000, 14)])
def test_attn_hidden_nan_and_extremes(K, dtype, width, len0):
    """NaN keys and values reach exactly the rows that see them; scores of hundreds, a scale of zero and a
    negative one; units of 16 rows with and without shares, of 32 rows."""
    import torch
    say(f"attn NaN and extremes {dtype} width={width} new={len0}")
    new, kv = [len0, 1], [200, 131]
    m, rng = plain_model(K, dtype, 1, 64, 64, kv, 33, width=width)
    vals = A.e4m3_values()

    def put(half, n, pos, d, code):
        c = m.keys if half == "k" else m.values
        pid = c.pid(n, pos)
        getattr(m.gpu, half)[pid, 0, pos % 64, d] = code
        c.codes[pid, 0, pos % 64, d] = vals[code]
    put("v", 0, 170, 5, 0x7F)                          # seen by rows from position 170 on
    put("v", 0, 171, 9, 0xFF)
    put("k", 0, 190, 3, 0x7F)                          # whole rows from position 190 on
    put("v", 1, 131 - 1, 0, 0x7F)                      # the last key of a full tail
    q = queries(rng, len0 + 1, 4, 64, dtype)
    for causal, window in ((True, 0), (True, 12)):
        o, lse = K.kda_attn(q, i64(cum(new)), i64(kv), m.gpu, scale=0.125, causal=causal, window=window, want_lse=True)
        torch.cuda.synchronize()
        ro, rl, _, _ = A.attn(to_numpy_f64(q), cum(new), kv, m.keys, m.values, 0.125, causal, window)
        assert np.isnan(ro).any() and not np.isnan(ro).all()
        assert np.array_equal(np.isnan(to_numpy_f64(o)), np.isnan(ro))
        assert np.array_equal(np.isnan(to_numpy_f64(lse)), np.isnan(rl))
    m, rng = plain_model(K, dtype, 1, 64, 64, kv, 34, width=width)
    attn_check(K, m, dtype, queries(rng, len0 + 1, 4, 64, dtype), cum(new), kv, 8.0, name="scores of hundreds")
    attn_check(K, m, dtype, queries(rng, len0 + 1, 4, 64, dtype), cum(new), kv, 0.0, name="scale 0")
    attn_check(K, m, dtype, queries(rng, len0 + 1, 4, 64, dtype), cum(new), kv, -0.125, name="negative scale")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 64])
def test_attn_prompt_hidden_nan(K, dtype, page):
    """NaN keys and values in a prompt and its context reach exactly the rows that see them."""
    import torch
    say(f"attn prompt NaN {dtype} page={page}")
    new, kv, D = 150, 300, 128
    m, rng = plain_model(K, dtype, 1, D, page, [kv], 61, width=25600 // page)
    for half, pos, d, code in (("v", 205, 5, 0x7F), ("v", 206, 127, 0xFF), ("k", 280, 3, 0x7F), ("v", 299, 64, 0x7F)):
        c = m.keys if half == "k" else m.values
        pid = c.pid(0, pos)
        getattr(m.gpu, half)[pid, 0, pos % page, d] = code
        c.codes[pid, 0, pos % page, d] = np.nan
    q = queries(rng, new, 4, D, dtype)
    for window in (0, 20):
        o, lse = K.kda_attn(q, i64([0, new]), i64([kv]), m.gpu, window=window, want_lse=True)
        torch.cuda.synchronize()
        ro, rl, _, _ = A.attn(to_numpy_f64(q), [0, new], [kv], m.keys, m.values, D ** -0.5, True, window)
        assert np.isnan(ro).any() and not np.isnan(ro).all()
        assert np.array_equal(np.isnan(to_numpy_f64(o)), np.isnan(ro))
        assert np.array_equal(np.isnan(to_numpy_f64(lse)), np.isnan(rl))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_long_rows(K, dtype):
    """One sequence with a few hundred new tokens over a longer context, and the same call twice: the same bits."""
    import torch
    say(f"attn long rows {dtype}")
    new, kv = [301], [1201]
    m, rng = plain_model(K, dtype, 1, 128, 64, kv, 44, width=400)
    q = queries(rng, 301, 4, 128, dtype)
    o, lse = attn_check(K, m, dtype, q, cum(new), kv, 128 ** -0.5)
    o2, lse2 = K.kda_attn(q, i64(cum(new)), i64(kv), m.gpu, want_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("n", [300, 700])
def test_attn_many_sequences(K, n):
    """More sequences than a workgroup has threads."""
    say(f"attn {n} sequences")
    rng = np.random.default_rng(n)
    kv = [int(x) for x in rng.integers(0, 90, n)]
    kv[5] = 640
    m, rng = plain_model(K, "bf16", 1, 64, 16, kv, n, width=200)
    attn_check(K, m, "bf16", queries(rng, n, 2, 64, "bf16"), cum([1] * n), kv, 0.1)


# ---------------------------------------------------------------------------
# the layer's calls together, streams and graphs
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_layer_prompt_chunks_and_decode(K, dtype):
    """norm + rotation -> cache -> attention: prompts in chunks, then single tokens, on two sequences of
    packed qkv rows; every step against the oracle chain on the same rounded rows."""
    import torch
    say(f"attention layer {dtype}")
    Hq, Hk, D, page = 8, 2, 128, 64
    rng = np.random.default_rng(77)
    tab, n_pages = tables(2, 6, rng)
    m = Model(K, dtype, Hk, D, page, n_pages, tab)
    table = dev(rope_table(512, D))
    w = [dev((1 + 0.2 * rng.normal(size=D)).astype(np.float32)) for _ in "qk"]
    kv = np.zeros(2, int)
    for new in ([100, 37], [64, 130], [1, 1], [1, 1], [3, 0], [1, 1]):
        T = sum(new)
        qkv = dev(rng.normal(size=(T, Hq + 2 * Hk, D)), dt(dtype))
        pos = np.concatenate([np.arange(a, a + b) for a, b in zip(kv, new)])
        kv = kv + new
        q, k = K.kda_qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], i64(pos), table, q_weight=w[0], k_weight=w[1])
        m.write(k, qkv[:, Hq + Hk:], cum(new), kv)
        attn_check(K, m, dtype, q, cum(new), kv, D ** -0.5, name=f"o after {kv.tolist()}")


def test_attn_layer_in_a_captured_graph(K):
    """A captured decode step, replayed as the sequences grow, with eager work and a second graph on the
    same workspace between the replays: always the eager result."""
    import torch
    say("attention layer in a graph")
    Hq, Hk, D, page, N = 8, 2, 128, 64, 3
    rng = np.random.default_rng(5)
    tab, n_pages = tables(N, 40, rng)
    m = Model(K, "bf16", Hk, D, page, n_pages, tab)
    eager = K.KVCache(m.gpu.k.clone(), m.gpu.v.clone(), m.gpu.k_scale.clone(), m.gpu.v_scale.clone(), m.gpu.table)
    start = [600, 64, 5]
    qkv = dev(rng.normal(size=(sum(start), Hq + 2 * Hk, D)), torch.bfloat16)
    for c in (m.gpu, eager):
        K.kda_kv_write(qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], i64(cum(start)), i64(start), c)
    table = dev(rope_table(1024, D))
    x = torch.zeros((N, Hq + 2 * Hk, D), dtype=torch.bfloat16, device="cuda")
    cu, kv, pos = i64(cum([1] * N)), i64(start), i64(start)
    cfg, cc = K._attn_config(Hq, Hk, D, torch.bfloat16), m.gpu.c((n_pages, page, 40))
    ws = torch.empty(K.LIB.kda_attn_workspace(cfg, cc, N, N, 0), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0

    def step(c):
        q, k = K.kda_qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hk], pos, table)
        K.kda_kv_write(k, x[:, Hq + Hk:], cu, kv, c)
        return K.kda_attn(q, cu, kv, c, want_lse=True, workspace=ws)
    side = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = step(m.gpu)
        graphs.append((g, out))
    for i in range(5):
        x.copy_(dev(rng.normal(size=tuple(x.shape)), torch.bfloat16))
        kv.copy_(i64([n + 1 + i for n in start]))
        pos.copy_(i64([n + i for n in start]))
        g, out = graphs[i % 2]
        g.replay()
        got = [t.clone() for t in out]
        ref = step(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), f"replay {i}"
        assert torch.equal(m.gpu.k, eager.k) and torch.equal(m.gpu.v_scale, eager.v_scale)


def test_attn_on_another_stream(K):
    """stream=: the call's allocations and launches are on that stream, behind work that it holds."""
    import torch
    say("attention on another stream")
    m, rng = plain_model(K, "bf16", 2, 64, 64, [900, 40], 3)
    q = queries(rng, 2, 8, 64, "bf16")
    cu, kv = i64([0, 1, 2]), i64([900, 40])
    ref = K.kda_attn(q, cu, kv, m.gpu)
    s = torch.cuda.Stream()
    q2 = torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(4):
            big = big @ big * 1e-4
        q2.copy_(q)
    o = K.kda_attn(q2, cu, kv, m.gpu, stream=s)
    s.synchronize()
    assert torch.equal(o, ref)
