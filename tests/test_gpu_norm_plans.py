"""GPU tests of the norm of the heads where a lane takes several heads.  Tolerances as in test_gpu_linear.py."""
import pytest

from test_gpu_linear import HALF, U, dt, say
from test_gpu_linear_edges import K  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

NORMS = [  # D, heads and lanes of a head where 1,024 workgroups are full (fp32 heads of 128: one head a lane at any number)
    ("bf16", 128, 4, 16), ("f32", 128, 4, 32), ("bf16", 8, 4, 1), ("bf16", 264, 4, 64), ("f32", 264, 2, 64),
    ("bf16", 1024, 2, 64), ("f32", 520, 2, 64), ("f32", 1024, 2, 64),
]


@pytest.mark.parametrize("center,per_head,gate,act,place", [
    (False, False, True, 1, None), (True, True, False, 1, None), (True, False, True, 2, "x"), (False, True, True, 0, "gate")])
@pytest.mark.parametrize("dtype,D,heads,lanes", NORMS)
def test_norm_with_several_heads_a_lane(K, dtype, D, heads, lanes, center, per_head, gate, act, place):
    """Just above the number of heads from which a lane takes two or four: all heads against fp64, and bit for bit what
    calls of few heads, one a lane, give.  Some heads' squares overflow or vanish in fp32."""
    import torch
    H = 3
    T = (256 // lanes * heads * 1024) // H + 5
    assert T * H >= 256 // lanes * heads * 1024 and T * H % (256 // lanes * heads)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(D + heads)
    x = torch.randn((T, H, D), generator=gen, device="cuda") + 0.3
    for t, e in ((0, 80), (1, -80), (T // 2, 66), (T - 1, -70), (T - 1, 0)):
        x[t, t % H] *= 2.0 ** e
    x = x.to(dt(dtype))
    z = torch.randn((T, 2 * H, D), generator=gen, device="cuda").to(dt(dtype))[:, H:] if gate else None
    shape = (H, D) if per_head else (D,)
    w = 1 + 0.3 * torch.randn(shape, generator=gen, device="cuda")
    b = 0.5 * torch.randn(shape, generator=gen, device="cuda") if center else None
    kw = dict(weight=w, bias=b, eps=1e-6, center=center, activation=act)
    step = 64 // H
    small = torch.cat([K.kda_head_norm(x[t:t + step], None if z is None else z[t:t + step], **kw)
                       for t in [*range(0, 4 * step, step), *range(T - 4 * step, T, step)]])
    X, Z = x.double(), None if z is None else z.double()
    y = K.kda_head_norm(x, z, out={None: None, "x": x, "gate": z}[place], **kw)
    torch.cuda.synchronize()
    assert place is None or y is {"x": x, "gate": z}[place]
    assert torch.equal(torch.cat([y[:4 * step], y[T - 4 * step:]]), small)
    # the definition in 64 bits, and test_gpu_linear.py's tolerance
    mean = X.mean(-1, keepdim=True) if center else 0.0
    sc = 1 / ((X - mean).pow(2).mean(-1, keepdim=True) + kw["eps"]).sqrt()
    inner = (X - mean) * sc * w.double() + (0.0 if b is None else b.double())
    big = X.abs().amax(-1, keepdim=True) * sc * w.double().abs()
    e = (D / 2 + 24) * U * (inner.abs() + (big if center else 0.0) + (0.0 if b is None else b.double().abs()))

    def activation(x):
        return x if act == 0 else torch.sigmoid(x) * (x if act == 1 else 1.0)
    if gate:
        ref = inner * activation(Z)
        tol = e * activation(Z).abs() + 8 * U * ref.abs()
    else:
        ref = activation(inner)
        tol = 1.1 * e + 8 * U * (ref.abs() + inner.abs())
    tol = HALF[dtype] * ref.abs() + tol + 1e-37
    part = ((y.double() - ref).abs() / tol).amax().item()
    say(f"worst error / tolerance {part:.3f}")
    assert part <= 1.0
