"""The example block: norm with the sum, recurrence dense, packed and token by
token, and gradients together."""
import importlib.util
import os

import numpy as np
import pytest
import scan_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    pytest.importorskip("torch")
    spec = importlib.util.spec_from_file_location(
        "recurrent_layer", os.path.join(ROOT, "examples", "recurrent_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(w, s, h0=None):
    """The block in float64 from the sum s [B, T, dim] on: (y, last state)."""
    B, T, dim = s.shape
    n = ref.layer_norm(s.reshape(-1, dim), w["norm_w"], w["norm_b"], 1e-5)[0].reshape(s.shape)
    p = n @ w["w_in"].T
    width = w["w_out"].shape[1]
    h, _, _ = ref.scan(p[..., :width], p[..., width:] + w["b_gate"], h0, "sigmoid")
    return h @ w["w_out"].T, h[:, -1]


def test_example_block(example):
    """Float32 runs against float64.  Products over up to 192 values, off by 192 x 2^-24 = 1.2e-5
    of their terms' norm, twice, and the recurrence's and the norm's steps: within 5e-5 of the
    whole.  Gradients against central differences of the float64 block: h^2 = 1e-8 of the third
    derivative, 2^-53 / h = 1e-12, and the float32 steps of three products and two passes, twice
    the forward pass's."""
    import torch
    torch.backends.cuda.matmul.allow_tf32 = False
    block = example.RecurrentBlock(dim=96, width=192, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(3)
    B, T = 2, 137
    x, r, dy, ds = (torch.randn(B, T, 96, generator=g, device="cuda") for _ in range(4))
    names = ("w_in", "w_out", "norm_w", "norm_b", "b_gate")
    w = {n: getattr(block, n).double().cpu().numpy() for n in names}
    num = lambda t: t.double().cpu().numpy()  # noqa: E731
    near = lambda a, b: np.linalg.norm(num(a) - b) <= 5e-5 * np.linalg.norm(b)  # noqa: E731
    y, s, state = block.prompt(x, r)
    assert s.equal(x + r)
    want, last = plain(w, num(s))
    assert near(y, want) and near(state, last)
    # the same in one packed call of unequal parts, from states of their own
    cuts = [0, 50, 50, 51, 137]
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    h0 = torch.randn(4, 192, generator=g, device="cuda")
    yp, sp, hp = block.packed(x[0].contiguous(), r[0].contiguous(), off, h0)
    for i in range(4):
        a, b = cuts[i], cuts[i + 1]
        if a == b:
            assert hp[i].equal(h0[i])
            continue
        wy, wh = plain(w, num(sp[None, a:b]), num(h0[i:i + 1]))
        assert near(yp[a:b], wy[0]) and near(hp[i], wh[0])
    # the last token as a step
    _, _, state = block.prompt(x[:, :-1].contiguous(), r[:, :-1].contiguous())
    yl, _ = block.step(x[:, -1].contiguous(), r[:, -1].contiguous(), state)
    assert near(yl, want[:, -1]) and near(state, last)
    grads = block.gradients(x, r, dy, ds)
    rng = np.random.default_rng(0)
    sn, dyn, dsn = num(x + r), num(dy), num(ds)
    for name in names + ("x",):
        base = sn if name == "x" else w[name]
        d = rng.standard_normal(base.shape)
        d /= np.linalg.norm(d)
        h = 1e-4

        def loss(t):
            if name == "x":
                z = sn + t * d
                return (plain(w, z)[0] * dyn).sum() + (z * dsn).sum()
            return (plain(dict(w, **{name: base + t * d}), sn)[0] * dyn).sum()

        diff = (loss(h) - loss(-h)) / (2 * h)
        got = num(grads[name])
        assert abs((got * d).sum() - diff) <= 1e-4 * np.linalg.norm(got), name


def test_example_runs(example, capsys):
    example.main()
    assert "gradient of norm_w" in capsys.readouterr().out
