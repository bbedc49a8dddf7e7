"""Edges of the norm with rotation on the GPU: no eps, frequencies that are not
finite."""
import linear_ref as ref
import numpy as np
import pytest
from test_gpu_qk_norm import frequencies, pair_size, tensor, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("N,H", [(1, 1), (1, 16), (37, 5), (700, 3)])
def test_gradients_without_eps(torch, N, H, D, norm, dtype):  # noqa: F811
    """Lanes beyond a tile's last row have no norm: they must not reach the weights' gradients.
    Bounds as in test_forward_and_backward."""
    from gated_delta_rule_49_gb300 import binding
    rng = np.random.default_rng(D + N)
    R = D // 2
    q, qn = tensor(torch, rng, (N, H, D), dtype)
    k, kn = tensor(torch, rng, (N, 1, D), dtype)
    dyq, dyqn = tensor(torch, rng, (N, H, D), dtype)
    dyk, dykn = tensor(torch, rng, (N, 1, D), dtype)
    w, wn = tensor(torch, rng, (D,), "fp32")
    posn, fn = np.arange(N) + 3, frequencies(R)
    pos, f = torch.from_numpy(posn).cuda(), torch.from_numpy(fn).cuda()
    got = binding.qk_norm_rotate_backward(q, k, pos, f, dyq, dyk, w, w, norm=norm, eps=0.0)
    y = binding.qk_norm_rotate(q, k, pos, f, w, w, norm=norm, eps=0.0)
    f32, u, c = 2.0 ** -24 * (D / 8 + 20), ref.U[dtype], 1 / D if norm == "rms" else 1.0
    for x, dyn, out, dx, dw, h in ((qn, dyqn, y[0], got[0], got[2], H),
                                   (kn, dykn, y[1], got[1], got[3], 1)):
        want = ref.norm_rotate(x, wn, posn, fn, norm, "half", 0.0)
        size = pair_size(ref.norm_rotate(x, wn, posn, fn[:0], norm, "half", 0.0), R, "half")
        off = np.abs(out.double().cpu().numpy() - want)
        assert (off <= u * np.abs(want) + f32 * (1 + u) * 2 * size).all()
        wantx, wantw = ref.norm_rotate_grad(x, wn, posn, fn, dyn, norm, "half", 0.0)
        r = 1 / np.sqrt(c * (x * x).sum(-1, keepdims=True))
        turned = pair_size(dyn, R, "half")
        g = turned * np.abs(wn)
        mag = r * (g + c * r * r * np.abs(x) * (np.abs(x) * g).sum(-1, keepdims=True))
        off = np.abs(dx.double().cpu().numpy() - wantx)
        assert (off <= u * np.abs(wantx) + f32 * (1 + u) * 3 * mag).all()
        mag = (turned * np.abs(x) * r).reshape(-1, D).sum(0)
        off = np.abs(dw.double().cpu().numpy() - wantw)
        assert (off <= (f32 + 2.0 ** -24 * N * h) * 3 * mag).all()


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_frequencies_that_are_not_finite(torch, bad, pairing):  # noqa: F811
    """Their pair is not a number, at every position (0 too); the other channels keep their bits."""
    from gated_delta_rule_49_gb300 import binding
    x = torch.randn(9, 3, 64, device="cuda")
    pos = torch.arange(9, device="cuda")
    f = torch.from_numpy(frequencies(32)).cuda()
    g = f.clone()
    g[5] = bad
    pair = [5, 21] if pairing == "half" else [10, 11]
    rest = [i for i in range(64) if i not in pair]
    want, _ = binding.qk_norm_rotate(x, None, pos, f, pairing=pairing)
    y, _ = binding.qk_norm_rotate(x, None, pos, g, pairing=pairing)
    assert y[..., pair].isnan().all() and torch.equal(y[..., rest], want[..., rest])
    dx = binding.qk_norm_rotate_backward(x, None, pos, g, x, None, pairing=pairing)[0]
    assert dx.isnan().all()  # through the norm
