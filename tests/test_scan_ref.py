"""The float64 forms that the kernels are held to, against differences and one another."""
import numpy as np
import pytest
import scan_ref as ref


def difference(f, base, d, h=1e-5):
    return (f(base + h * d) - f(base - h * d)) / (2 * h)


@pytest.mark.parametrize("kind", ["decay", "sigmoid"])
@pytest.mark.parametrize("T,start", [(1, False), (1, True), (9, True), (23, False)])
def test_scan_gradients(kind, T, start):
    """Central differences: off by h^2 = 1e-10 of the third derivative and 1e-16 / h."""
    rng = np.random.default_rng(T)
    B, D = 2, 3
    x, dh = rng.standard_normal((2, B, T, D))
    gate = rng.standard_normal((B, T, D))
    if kind == "decay":
        gate = 1 / (1 + np.exp(-gate))
    h0 = rng.standard_normal((B, D)) if start else None
    dhT = rng.standard_normal((B, D))

    def loss(x, gate, h0):
        h = ref.scan(x, gate, h0, kind)[0]
        return (h * dh).sum() + (h[:, -1] * dhT).sum()

    got = ref.scan_grad(x, gate, dh, h0, dhT, kind)
    start0 = np.zeros((B, D)) if h0 is None else h0
    for name, base, f in (("dx", x, lambda z: loss(z, gate, h0)),
                          ("dgate", gate, lambda z: loss(x, z, h0)),
                          ("dh0", start0, lambda z: loss(x, gate, z))):
        d = rng.standard_normal(base.shape)
        assert abs((got[name][0] * d).sum() - difference(f, base, d)) < 1e-7, name


def test_sigmoid_is_a_mean():
    """a + b = 1: a constant input is kept, and a gate far out is a switch."""
    a, b = ref.coefficients(np.array([-800.0, -3.0, 0.0, 3.0, 800.0]), "sigmoid")
    assert np.allclose(a + b, 1, atol=1e-15) and a[0] == 0 and b[4] == 0
    h = ref.scan(np.full((1, 50, 4), 2.5), np.random.default_rng(0).standard_normal((1, 50, 4)),
                 np.full((1, 4), 2.5), "sigmoid")[0]
    assert np.allclose(h, 2.5, atol=1e-13)


@pytest.mark.parametrize("weight", [False, True])
def test_layer_norm_gradients(weight):
    rng = np.random.default_rng(5)
    N, D, eps = 4, 16, 1e-5
    x, dy, ds = rng.standard_normal((3, N, D))
    w, b = (rng.standard_normal((2, D)) if weight else (None, None))
    m, r = ref.layer_norm(x, w, b, eps)[2:4]

    def loss(x, w, b):
        return (ref.layer_norm(x, w, b, eps)[0] * dy).sum() + (x * ds).sum()

    got = ref.layer_norm_grad(x, dy, m, r, w, ds)
    d = rng.standard_normal((N, D))
    assert abs((got["dx"][0] * d).sum() - difference(lambda z: loss(z, w, b), x, d)) < 1e-7
    if weight:
        d = rng.standard_normal(D)
        assert abs((got["dw"][0] * d).sum() - difference(lambda z: loss(x, z, b), w, d)) < 1e-7
        assert abs((got["db"][0] * d).sum() - difference(lambda z: loss(x, w, z), b, d)) < 1e-7
