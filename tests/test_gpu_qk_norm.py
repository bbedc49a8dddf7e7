"""Norms of queries and keys with the position rotation on the GPU against
float64 (tests/linear_ref.py).  Bounds count the float32 steps: about D/8 + 5
additions and 5 more roundings of the norm, 8 of the product with the weight and the rotation
(whose angle has 2^-25 turns), against the magnitudes of the turned pair."""
import linear_ref as ref
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    from gated_delta_rule_49_gb300 import binding
    binding.load()
    return torch


def tensor(torch, rng, shape, dtype, scale=1.0):
    x = torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32))
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return x.cuda(), x.double().numpy()


def frequencies(R, base=10000.0):
    return np.float32(base) ** (-np.arange(0, R, 2, dtype=np.float32) / np.float32(max(R, 1)))


def pair_size(x, R, pairing):
    """The length of the pair that each channel is turned with (its own size beyond R)."""
    y = np.abs(x).copy()
    i = np.arange(R // 2)
    a, b = (i, i + R // 2) if pairing == "half" else (2 * i, 2 * i + 1)
    n = np.hypot(x[..., a], x[..., b])
    y[..., a] = n
    y[..., b] = n
    return y


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D,R", [(32, 32), (64, 32), (128, 128), (128, 16), (256, 256), (64, 0)])
@pytest.mark.parametrize("norm,pairing", [("rms", "half"), ("l2", "adjacent"), ("rms", "adjacent"),
                                          ("l2", "half")])
@pytest.mark.parametrize("lead,Hq,Hk", [((1,), 1, 1), ((3, 37), 5, 2), ((130,), 16, 16), ((2, 3), 7, 0)])
def test_forward_and_backward(torch, lead, Hq, Hk, D, R, norm, pairing, dtype):
    from gated_delta_rule_49_gb300 import binding
    rng = np.random.default_rng(D + R + Hq)
    q, qn = tensor(torch, rng, lead + (Hq, D), dtype)
    k, kn = tensor(torch, rng, lead + (Hk, D), dtype) if Hk else (None, None)
    dyq, dyqn = tensor(torch, rng, lead + (Hq, D), dtype)
    dyk, dykn = tensor(torch, rng, lead + (Hk, D), dtype) if Hk else (None, None)
    wq, wqn = tensor(torch, rng, (D,), "fp32")
    posn = rng.integers(-5, 200000, lead)
    fn = frequencies(R)
    pos, f = torch.from_numpy(posn).cuda(), torch.from_numpy(fn).cuda()
    if R == 0:
        f = None
    wk, wkn = None, None  # the keys' weight is left out
    yq, yk = binding.qk_norm_rotate(q, k, pos, f, wq, wk, norm=norm, pairing=pairing, eps=EPS)
    got = binding.qk_norm_rotate_backward(q, k, pos, f, dyq, dyk, wq, wk, norm=norm,
                                          pairing=pairing, eps=EPS)
    f32 = 2.0 ** -24 * (D / 8 + 20)
    u = ref.U[dtype]
    rows = int(np.prod(lead))
    for x, xn, w, y, dyn, dx, dw, h in ((q, qn, wqn, yq, dyqn, got[0], got[2], Hq),
                                        (k, kn, wkn, yk, dykn, got[1], got[3], Hk)):
        if x is None:
            assert y is None and dx is None
            continue
        want = ref.norm_rotate(xn, w, posn, fn, norm, pairing, EPS)
        size = pair_size(ref.norm_rotate(xn, w, posn, fn[:0], norm, pairing, EPS), R, pairing)
        off = np.abs(y.double().cpu().numpy() - want)
        assert (off <= u * np.abs(want) + f32 * (1 + u) * 2 * size).all()
        wantx, wantw = ref.norm_rotate_grad(xn, w, posn, fn, dyn, norm, pairing, EPS)
        c = 1 / D if norm == "rms" else 1.0
        r = 1 / np.sqrt(c * (xn * xn).sum(-1, keepdims=True) + EPS)
        g = pair_size(dyn, R, pairing) * (1 if w is None else np.abs(w))
        mag = r * (g + c * r * r * np.abs(xn) * (np.abs(xn) * g).sum(-1, keepdims=True))
        off = np.abs(dx.double().cpu().numpy() - wantx)
        assert (off <= u * np.abs(wantx) + f32 * (1 + u) * 3 * mag).all()
        if w is None:
            assert dw is None
            continue
        mag = (pair_size(dyn, R, pairing) * np.abs(xn) * r).reshape(-1, D).sum(0)
        off = np.abs(dw.double().cpu().numpy() - wantw)
        assert (off <= (f32 + 2.0 ** -24 * rows * h) * 3 * mag).all()


def test_zero_rows(torch):
    """A row of zeros has a norm through eps alone: zero out, gradient eps^-1/2 of the weighted one."""
    from gated_delta_rule_49_gb300 import binding
    q = torch.zeros(2, 3, 64, device="cuda")
    pos = torch.zeros(2, dtype=torch.int64, device="cuda")
    f = torch.ones(16, device="cuda")
    y, _ = binding.qk_norm_rotate(q, None, pos, f, eps=1e-4)
    assert not y.any()
    dy = torch.ones_like(q)
    dx = binding.qk_norm_rotate_backward(q, None, pos, f, dy, None, eps=1e-4)[0]
    assert torch.allclose(dx, torch.full_like(dx, 100.0), rtol=1e-5)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_far_positions(torch, dtype):
    """Positions whose angles float32 cannot tell apart."""
    from gated_delta_rule_49_gb300 import binding
    rng = np.random.default_rng(1)
    posn = np.array([2 ** 31 + 5, 10 ** 12 + 1, 123456789, -(2 ** 33) - 3])
    q, qn = tensor(torch, rng, (4, 2, 64), dtype)
    fn = frequencies(64)
    y, _ = binding.qk_norm_rotate(q, None, torch.from_numpy(posn).cuda(), torch.from_numpy(fn).cuda(), eps=EPS)
    want = ref.norm_rotate(qn, None, posn, fn, "rms", "half", EPS)
    # the angle itself, in float64: 1e12 radians to about 2e-4
    assert np.abs(y.double().cpu().numpy() - want).max() <= 4 * (ref.U[dtype] + 1e-3)


def test_slices_in_place_streams_and_bits(torch):
    from gated_delta_rule_49_gb300 import binding
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(3, 50, 4 * 128 + 2 * 128 + 64, device="cuda").to(dtype)
        q = x[..., :512].unflatten(-1, (4, 128))
        k = x[..., 512:768].unflatten(-1, (2, 128))
        pos = torch.arange(150, device="cuda").view(3, 50)
        f = torch.from_numpy(frequencies(64)).cuda()
        w = torch.rand(128, device="cuda")
        want = binding.qk_norm_rotate(q, k, pos, f, w, w)
        qd, kd = q.contiguous(), k.contiguous()
        got = binding.qk_norm_rotate(qd, kd, pos, f, w, w)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = binding.qk_norm_rotate(qd, kd, pos, f, w, w, out=(qd, kd))
        torch.cuda.current_stream().wait_stream(s)
        assert got[0] is qd and all(torch.equal(a, b) for a, b in zip(got, want))
        dy = [torch.randn_like(t) for t in want]
        one = binding.qk_norm_rotate_backward(q, k, pos, f, *dy, w, w)
        for _ in range(3):
            two = binding.qk_norm_rotate_backward(q, k, pos, f, *dy, w, w)
            assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_many_tokens_and_no_tokens(torch):
    from gated_delta_rule_49_gb300 import binding
    rng = np.random.default_rng(4)
    q, qn = tensor(torch, rng, (9001, 3, 32), "bf16")
    posn = np.arange(9001)
    fn = frequencies(32)
    pos, f = torch.from_numpy(posn).cuda(), torch.from_numpy(fn).cuda()
    w, wn = tensor(torch, rng, (32,), "fp32")
    y, _ = binding.qk_norm_rotate(q, None, pos, f, w)
    want = ref.norm_rotate(qn, wn, posn, fn, "rms", "half", EPS)
    size = pair_size(ref.norm_rotate(qn, wn, posn, fn[:0], "rms", "half", EPS), 32, "half")
    u = ref.U["bf16"]
    assert (np.abs(y.double().cpu().numpy() - want) <= u * np.abs(want) + 1e-5 * size).all()
    y, _ = binding.qk_norm_rotate(q[:0], None, pos[:0], f, w)
    assert y.shape == (0, 3, 32)
    got = binding.qk_norm_rotate_backward(q[:0], None, pos[:0], f, q[:0], None, w)
    assert not got[2].any()
