"""The float64 references of the linear attention and norm tests against the
closed forms and against differences (CPU)."""
import linear_ref as ref
import numpy as np
import pytest


def problem(rng, B=2, T=7, Hq=2, H=4, K=3, V=5):
    n = rng.standard_normal
    return (n((B, T, Hq, K)), n((B, T, Hq, K)), n((B, T, H, V)), np.array([0.0, 0.4, 0.9, 1.0]),
            n((B, H, V, K)))


def test_sum_form_and_plain_linear_attention():
    rng = np.random.default_rng(0)
    q, k, v, a, S0 = problem(rng)
    o, S = ref.linear(q, k, v, a, S0, 0.7)
    for b in range(2):
        for h in range(4):
            for t in range(7):
                x = a[h] ** (t + 1) * S0[b, h]
                for s in range(t + 1):
                    x = x + a[h] ** (t - s) * np.outer(v[b, s, h], k[b, s, h // 2])
                assert np.allclose(o[b, t, h], 0.7 * x @ q[b, t, h // 2], atol=1e-12)
            assert np.allclose(S[b, h], x, atol=1e-12)
    # a decay of 1 from nothing: sum of v k^T
    _, S = ref.linear(q, k, v, np.ones(4))
    assert np.allclose(S[0, 1], np.einsum("tv,tk->vk", v[0, :, 1], k[0, :, 0]))


def test_linear_gradient_against_differences():
    rng = np.random.default_rng(1)
    q, k, v, a, S0 = problem(rng)
    do, dST = rng.standard_normal(v.shape), rng.standard_normal(S0.shape)

    def loss(q, k, v, S0):
        o, S = ref.linear(q, k, v, a, S0, 0.7)
        return (o * do).sum() + (S * dST).sum()

    got = ref.linear_grad(q, k, v, a, do, S0, dST, 0.7)
    args = [q, k, v, S0]
    for i in range(4):
        for _ in range(6):
            d = rng.standard_normal(args[i].shape)
            up, dn = list(args), list(args)
            # the loss is linear in each argument alone: the difference is exact
            up[i], dn[i] = args[i] + 0.5 * d, args[i] - 0.5 * d
            assert np.isclose(loss(*up) - loss(*dn), (got[i] * d).sum(), rtol=1e-9, atol=1e-9)


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("pairing", ["half", "adjacent"])
def test_norm_gradient_against_differences(norm, pairing):
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((3, 2, 8)), rng.standard_normal((3, 2, 8))
    w, pos, f = rng.standard_normal(8), np.array([0, 5, 70000]), np.array([1.0, 0.01])
    dx, dw = ref.norm_rotate_grad(x, w, pos, f, dy, norm, pairing, 1e-3)

    def loss(x, w):
        return (ref.norm_rotate(x, w, pos, f, norm, pairing, 1e-3) * dy).sum()

    h = 1e-6
    for _ in range(6):
        d = rng.standard_normal(x.shape)
        assert np.isclose((loss(x + h * d, w) - loss(x - h * d, w)) / (2 * h), (dx * d).sum(),
                          rtol=1e-7, atol=1e-7)
        d = rng.standard_normal(8)
        assert np.isclose((loss(x, w + h * d) - loss(x, w - h * d)) / (2 * h), (dw * d).sum(),
                          rtol=1e-7, atol=1e-7)


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
def test_rotation_keeps_distances_only(pairing):
    """Turned pairs depend on the difference of their positions alone."""
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    f = np.array([1.0, 0.3, 0.01, 1e-4])

    def dot(p, s):
        a = ref.norm_rotate(q, None, np.array([p]), f, "l2", pairing, 0.0)
        b = ref.norm_rotate(k, None, np.array([s]), f, "l2", pairing, 0.0)
        return float((a * b).sum())

    assert np.isclose(dot(10, 3), dot(1007, 1000), atol=1e-9)
    assert not np.isclose(dot(10, 3), dot(10, 4), atol=1e-3)
