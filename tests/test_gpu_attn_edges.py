"""GPU tests of the attention-layer operators at the ends of their number range, and of empty calls,
against the fp64 oracle (oracle/attention.py).  Tolerances as in test_gpu_attn.py."""
import numpy as np
import pytest

import oracle.attention as A
import test_gpu_attn as G
from test_gpu_attn import dev, dt, i64, say, within
from workloads.device import to_numpy_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_46_amd.kda as kda
    return kda


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot,pairs", [(128, 128, False), (64, 32, True), (128, 0, False)])
@pytest.mark.parametrize("eps", [1e-6, 0.0, 1e-32])
def test_rotate_heads_of_any_magnitude(K, dtype, D, rot, pairs, eps):
    """Heads whose squares overflow or vanish in fp32, among ordinary ones: 2^-133 to 2^125 times normal
    values, one huge element, tiny ones against an eps of their size.

    Tolerance: test_gpu_attn's relative one (the power of two by which a head is scaled is exact), and 2^-120
    for results below the smallest normals (a result is at most sqrt(D) times its weight, a product that falls
    below 2^-126 loses that much at most, three of them per result)."""
    import torch
    say(f"rotate magnitudes {dtype} D={D} rot={rot} pairs={pairs} eps={eps}")
    rng = np.random.default_rng(int(D + rot))
    exps = [0, -133, -126, -110, -75, -64, -52, -50, -48, -40, 40, 60, 62, 63, 64, 90, 120, 125]
    T, Hq, Hk = len(exps), 4, 2
    x = np.clip(rng.normal(size=(T, Hq + Hk, D)), -3, 3) * np.exp2(np.array(exps, float))[:, None, None]
    x[0, 1, 7], x[0, Hq, D - 1] = 3e38, -2e30                     # one huge element among ordinary ones
    x[5, 0] = rng.normal(size=D)                                  # an ordinary head beside tiny ones
    x[12, Hq] = rng.normal(size=D)                                # and beside huge ones
    if eps:
        x[3, 1] = 0
    x = dev(x.astype(np.float32), dt(dtype))
    q, k = x[:, :Hq], x[:, Hq:]
    pos = rng.integers(0, 500, T)
    table = G.rope_table(500, rot) if rot else None
    w = dev((1 + 0.3 * rng.normal(size=D)).astype(np.float32))
    got = K.kda_qk_norm_rope(q, k, i64(pos) if rot else None, None if table is None else dev(table), q_weight=w, k_weight=w,
                             eps=eps, layout=K.KDA_ROPE_PAIRS if pairs else K.KDA_ROPE_HALVES)
    torch.cuda.synchronize()
    eps32 = float(np.float32(eps))
    for name, g, src in zip("qk", got, (q, k)):
        r = A.norm_rope(to_numpy_f64(src), to_numpy_f64(w), eps32, pos, table, pairs)
        assert np.isfinite(r).all()
        pair = np.zeros_like(r)
        if rot:
            y = r[..., :rot]
            pair[..., :rot] = np.repeat(np.hypot(y[..., 0::2], y[..., 1::2]), 2, -1) if pairs else \
                np.concatenate([np.hypot(y[..., :rot // 2], y[..., rot // 2:])] * 2, -1)
        within(name, to_numpy_f64(g), r,
               G.HALF[dtype] * np.abs(r) + (D / 2 + 16) * 2.0 ** -24 * np.maximum(np.abs(r), 2 * pair) + 2.0 ** -120)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 32), (128, 16)])
def test_rotate_infinite_results_behind_the_rotated_dims(K, D, rot, pairs):
    """A dim behind rot whose weight makes it infinite stays an infinity of its sign; its neighbours are as ever."""
    import torch
    say(f"rotate infinite results D={D} rot={rot} pairs={pairs}")
    rng = np.random.default_rng(D)
    x = dev(rng.normal(size=(5, 3, D)).astype(np.float32))
    w = np.ones(D, np.float32)
    w[rot], w[D - 7] = np.inf, -np.inf
    pos, table = rng.integers(0, 500, 5), G.rope_table(500, rot)
    q, k = K.kda_qk_norm_rope(x[:, :2], x[:, 2:], i64(pos), dev(table), q_weight=dev(w), k_weight=dev(w),
                              layout=K.KDA_ROPE_PAIRS if pairs else K.KDA_ROPE_HALVES)
    torch.cuda.synchronize()
    for name, g, src in (("q", q, x[:, :2]), ("k", k, x[:, 2:])):
        r = A.norm_rope(to_numpy_f64(src), w, 1e-6, pos, table, pairs)
        assert np.isinf(r).sum() == 2 * r.shape[0] * r.shape[1] and not np.isnan(r).any()
        fin = np.where(np.isinf(r), 0, r)
        within(name, to_numpy_f64(g), r, G.HALF["f32"] * np.abs(fin) + (D / 2 + 16) * 2.0 ** -24 * (np.abs(fin) + 2 * 2 ** 0.5 * np.abs(
            fin).max(-1, keepdims=True)))
