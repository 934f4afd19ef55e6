"""The float64 statements the mixer's GPU tests compare with: their gradient formulas
against central differences of their forward forms (no GPU)."""
import pytest
import torch

import mixer_reference as ref

F64 = torch.float64


def _check(f, args, grads, seed):
    """d/de sum(f(args + e v) . weights) against sum(grad . v), for a random direction v of every argument."""
    gen = torch.Generator().manual_seed(seed)
    for i, (x, g) in enumerate(zip(args, grads)):
        v = torch.randn(x.shape, generator=gen, dtype=F64)
        e = 1e-6
        hi, lo = (f(*[a + s * e * v if j == i else a for j, a in enumerate(args)]) for s in (1, -1))
        # central differences: truncation e^2 ~ 1e-12, cancellation 1e-16 |f| / e ~ 1e-9 of |f|
        num, want = (hi - lo) / (2 * e), (g * v).sum()
        assert abs(num - want) <= 1e-6 * (1 + abs(want) + abs(hi)), (i, float(num), float(want))


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu", "softplus"])
def test_activation_derivatives(kind):
    x = torch.linspace(-6, 6, 51, dtype=F64) + 0.01
    v, d = ref.act(x, kind)
    num = (ref.act(x + 1e-6, kind)[0] - ref.act(x - 1e-6, kind)[0]) / 2e-6
    assert torch.allclose(num, d, atol=1e-8)


def test_norm_gradient_formula():
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(5, 7, generator=gen, dtype=F64) for _ in range(2))
    w, b = (torch.randn(7, generator=gen, dtype=F64) for _ in range(2))
    _, mean, rstd = ref.norm_fwd(x, w, b, 1e-5)
    _check(lambda x, w, b: (ref.norm_fwd(x, w, b, 1e-5)[0] * dy).sum(), [x, w, b], ref.norm_bwd(dy, x, w, mean, rstd), 2)


@pytest.mark.parametrize("cu", [None, [0, 1, 1, 4, 9, 10]])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_gradient_formula(cu, W):
    gen = torch.Generator().manual_seed(3)
    B, T, C = (2, 5, 3) if cu is None else (1, 10, 3)
    n = B if cu is None else len(cu) - 1
    r = lambda *s: torch.randn(s, generator=gen, dtype=F64)  # noqa: E731
    x, w, b, st, dy, dst = r(B, T, C), r(C, W), r(C), r(n, W - 1, C), r(B, T, C), r(n, W - 1, C)

    def f(x, w, b, st):
        y, out = ref.conv(x, w, b, cu, st, True)
        return (y * dy).sum() + (out * dst).sum()
    _check(f, [x, w, b, st], ref.conv(x, w, b, cu, st, True, dy, dst), 4)


@pytest.mark.parametrize("cu", [None, [0, 0, 3, 7, 7, 8]])
@pytest.mark.parametrize("gate,sp", [(True, True), (False, False)])
def test_scan_gradient_formula(cu, gate, sp):
    gen = torch.Generator().manual_seed(5)
    B, T, ch, G, N = (2, 4, 4, 2, 3) if cu is None else (1, 8, 4, 2, 3)
    n = B if cu is None else len(cu) - 1
    r = lambda *s: torch.randn(s, generator=gen, dtype=F64)  # noqa: E731
    u, dt, A, Bm, Cm, D = r(B, T, ch), r(B, T, ch), -r(ch, N).exp(), r(B, T, G, N), r(B, T, G, N), r(ch)
    z, bias, h0, dy, dh = r(B, T, ch) if gate else None, r(ch), r(n, ch, N), r(B, T, ch), r(n, ch, N)

    def f(u, dt, A, Bm, Cm, D, bias, h0, z=z):
        y, fin = ref.scan(u, dt, A, Bm, Cm, D, z, bias, sp, h0, cu)
        return (y * dy).sum() + (fin * dh).sum()
    du, ddt, dA, dB, dC, dD, dz, db, dh0 = ref.scan(u, dt, A, Bm, Cm, D, z, bias, sp, h0, cu, dy, dh)
    _check(f, [u, dt, A, Bm, Cm, D, bias, h0], [du, ddt, dA, dB, dC, dD, db, dh0], 6)
    if gate:
        _check(lambda z: f(u, dt, A, Bm, Cm, D, bias, h0, z=z), [z], [dz], 7)
