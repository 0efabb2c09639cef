"""GPU tests of kda_attn in every launch plan (attn_plans.py), against
the fp64 oracle.  Outputs start as a sentinel: rows that no workgroup writes, or that one writes past the
last sequence, show.  Tolerances as in test_gpu_attn.py."""
import numpy as np
import pytest

import attn_plans as P
import test_gpu_attn as G
from test_gpu_attn import HALF, cum, dev, dt, i64, say, within
from workloads.device import to_numpy_f64

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
