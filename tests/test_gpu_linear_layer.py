"""The example layer: norm, rotation, prompt, steps and gradients together."""
import importlib.util
import os

import numpy as np
import pytest

import linear_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    pytest.importorskip("torch")
    spec = importlib.util.spec_from_file_location(
        "linear_layer", os.path.join(ROOT, "examples", "linear_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(layer, w, x, pos):
    """The layer in float64: w by name, x [B, T, dim]."""
    B, T, _ = x.shape
    n = np.cumsum(layer.sizes)
    p = x @ w["w_in"].T
    q = p[..., :n[0]].reshape(B, T, layer.Hq, layer.K)
    k = p[..., n[0]:n[1]].reshape(B, T, layer.Hq, layer.K)
    v = p[..., n[1]:].reshape(B, T, layer.H, layer.V)
    f = layer.inv_freq.cpu().numpy()
    q = ref.norm_rotate(q, w["wq"], pos, f, "rms", "half", 1e-6)
    k = ref.norm_rotate(k, w["wk"], pos, f, "rms", "half", 1e-6)
    o, _ = ref.linear(q, k, v, layer.alpha.double().cpu().numpy(), None, layer.scale)
    return o.reshape(B, T, -1) @ w["w_out"].T


def test_example_layer(example):
    """Float32 runs: forward against float64, a step against the prompt, gradients against
    differences of the float64 layer (central, of third order: h^2 = 1e-8 and 2^-53 / h = 1e-12,
    under the float32 steps of some 500 additions in a row, 500 x 2^-24 = 3e-5)."""
    import torch
    layer = example.LinearAttention(dim=96, heads=4, key_heads=2, key_width=64, value_width=64,
                                    dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(3)
    B, T = 2, 37
    x = torch.randn(B, T, 96, generator=g, device="cuda")
    dy = torch.randn(B, T, 96, generator=g, device="cuda")
    pos = torch.arange(T, device="cuda").repeat(B, 1) + 1000
    y, _ = layer.prompt(x, pos)
    names = ("w_in", "w_out", "wq", "wk")
    w = {n: getattr(layer, n).double().cpu().numpy() for n in names}
    xn, posn, dyn = x.double().cpu().numpy(), pos.cpu().numpy(), dy.double().cpu().numpy()
    want = plain(layer, w, xn, posn)
    assert np.linalg.norm(y.double().cpu().numpy() - want) <= 3e-5 * np.linalg.norm(want)
    # the last token as a step
    _, state = layer.prompt(x[:, :-1].contiguous(), pos[:, :-1].contiguous())
    last = layer.step(x[:, -1].contiguous(), pos[:, -1].contiguous(), state)
    assert np.linalg.norm(last.double().cpu().numpy() - want[:, -1]) <= 3e-5 * np.linalg.norm(want[:, -1])
    grads = layer.gradients(x, pos, dy)
    rng = np.random.default_rng(0)
    for name in names + ("x",):
        base = xn if name == "x" else w[name]
        d = rng.standard_normal(base.shape)
        d /= np.linalg.norm(d)
        h = 1e-4

        def loss(t):
            if name == "x":
                return (plain(layer, w, xn + t * d, posn) * dyn).sum()
            return (plain(layer, dict(w, **{name: base + t * d}), xn, posn) * dyn).sum()

        diff = (loss(h) - loss(-h)) / (2 * h)
        got = grads[name].double().cpu().numpy()
        assert abs((got * d).sum() - diff) <= 6e-5 * np.linalg.norm(got), name


def test_example_runs(example, capsys):
    example.main()
    assert "gradient of w_in" in capsys.readouterr().out
