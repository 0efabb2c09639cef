"""GPU tests of kda_attn in every launch plan (attn_plans.py) and of the long form of kda_kv_read, against
the fp64 oracle.  Outputs start as a sentinel: rows that no workgroup writes, or that one writes past the
last sequence, show.  Tolerances as in test_gpu_attn.py."""
import numpy as np
import pytest

pytest.importorskip("gated_delta_rule_46_amd.kda", reason="libkda.so not built (run __graft_entry__.build())")
import attn_plans as P  # noqa: E402
import test_gpu_attn as G  # noqa: E402
from test_gpu_attn import HALF, cum, dev, dt, i64, say, within  # noqa: E402
from workloads.device import to_numpy_f64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_46_amd.kda as kda
    return kda


@pytest.mark.parametrize("c", P.CALLS, ids=[c["name"] for c in P.CALLS])
def test_attn_plan(K, c):
    import torch
    new, kv, D, dtype = c["new"], c["kv"], c["D"], c["dtype"]
    say(f"attn plan: {c['name']} {P.mode(P.plan_of(c))}")
    if torch.cuda.get_device_properties(0).multi_processor_count != P.CUS:
        pytest.skip(f"the plans are those of a device with {P.CUS} compute units")
    m, rng = G.plain_model(K, dtype, c["Hk"], D, c["page"], kv, len(new) + D, width=c["room"] // c["page"])
    T, used = sum(new) + c["pad"], sum(new)
    q = G.queries(rng, T, c["Hq"], D, dtype)
    out = torch.full((T, c["Hq"], D), 9.0, dtype=dt(dtype), device="cuda")
    lse = torch.full((T, c["Hq"]), 1e4, device="cuda")
    scale = D ** -0.5
    K.kda_attn(q, i64(cum(new)), i64(kv), m.gpu, scale=scale, window=c["window"], want_lse=True, out=out, lse_out=lse)
    torch.cuda.synchronize()
    assert (out[used:] == 9.0).all() and (lse[used:] == 1e4).all(), "rows behind the last sequence changed"
    ro, rl, RA, S = (x[:used] for x in P.attn(to_numpy_f64(q), cum(new), kv, m.keys, m.values, scale, True, c["window"]))
    d = 2.0 ** -24 * (D + 8) * S + (max(kv) + 16) * 2.0 ** -24
    tol = HALF[dtype] * np.abs(ro) + (HALF[dtype] + 2 * d[..., None]) * RA * (1 + 2.0 ** -7) + 1e-37
    within("o", to_numpy_f64(out)[:used], ro, tol)
    within("lse", to_numpy_f64(lse)[:used], rl, d + 2.0 ** -22 * np.abs(np.where(np.isinf(rl), 0, rl)))
    again = torch.full_like(out, -9.0)
    K.kda_attn(q, i64(cum(new)), i64(kv), m.gpu, scale=scale, window=c["window"], out=again)
    assert torch.equal(again[:used], out[:used]), "the same call gives other bits"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,Hk,page", [(128, 1, 64), (64, 3, 16), (128, 2, 128), (64, 1, 32)])
def test_cache_read_of_many_rows(K, dtype, D, Hk, page):
    """16,384 rows and more in one call (16 to a workgroup): sequences of 0 to 5 tokens side by side, long ones,
    more of them than one round of probes, absent pages, tokens past the table and before its start, rows behind
    the last sequence, a last workgroup that is not full.  Bit for bit."""
    import torch
    say(f"cache read of many rows {dtype} D={D} Hk={Hk} page={page}")
    rng = np.random.default_rng(D + page)
    back = [int(x) for x in rng.integers(0, 6, 150)] + [0, 0, 7001, 1, 16, 15, 17, 0, 9173, 3]
    kv = [b + int(x) for b, x in zip(back, rng.integers(0, 40, len(back)))]
    kv[3], kv[40] = back[3] - 2, 1 << 40                           # before the start, past the table
    width = -(-9300 // page)
    pages = 300
    table = rng.integers(0, pages, (len(kv), width)).astype(np.int32)   # pages are only read: shared ones too
    table[5], table[152, ::7], table[158, 3] = -1, pages, -(1 << 31)
    m = G.Model(K, dtype, Hk, D, page, pages, table, seed=D)
    used = sum(back)
    T = used + 5
    assert T >= 16 * 1024 and T % 16
    out = [torch.full((T, Hk, D), 3.0, dtype=dt(dtype), device="cuda") for _ in "kv"]
    K.kda_kv_read(i64(cum(back)), i64(kv), m.gpu, T, dt(dtype), k_out=out[0], v_out=out[1])
    torch.cuda.synchronize()
    pos = np.concatenate([np.arange(b) + L - b for b, L in zip(back, kv)])
    seq = np.repeat(np.arange(len(back)), back)
    there = (pos >= 0) & (pos < width * page)
    pid = np.where(there, table[seq, np.clip(pos // page, 0, width - 1)], -1)
    there &= (pid >= 0) & (pid < pages)
    assert 0 < (~there).sum() < used // 2
    pid = np.where(there, pid, 0)
    for got, c in zip(out, (m.keys, m.values)):
        ref = np.where(there[:, None, None], c.codes[pid, :, pos % page] * c.scale[pid][:, :, None], 0.0)
        assert np.array_equal(to_numpy_f64(got)[:used], ref, equal_nan=True)
        assert (got[used:] == 3.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,Hk,page", [(128, 1, 64), (64, 2, 16)])
def test_cache_write_of_many_sequences(K, dtype, D, Hk, page):
    """More sequences than one round of probes, most with 0 to 5 new tokens, some with many pages."""
    say(f"cache write of many sequences {dtype} D={D} Hk={Hk} page={page}")
    rng = np.random.default_rng(page)
    new = [int(x) for x in rng.integers(0, 6, 90)] + [0, 0, 3 * page + 1, 1, page, 0, 2 * page - 1] + [1] * 50 + [0, 700, 0]
    kv = [b + int(x) for b, x in zip(new, rng.integers(0, 2 * page, len(new)))]
    kv[7] = new[7] + page                                          # starts a page
    table, n_pages = G.tables(len(new), -(-1000 // page), rng)
    m = G.Model(K, dtype, Hk, D, page, n_pages, table)
    k, v = m.rows(rng, sum(new))
    m.write(k, v, cum(new), kv)
