"""Infinite states and gradients under decays whose product over a run of tokens is 0 in float32,
though none of them is: what the recurrence carries them to is not finite (an infinity or NaN),
all else has the bits that it has without them."""
import pytest
from test_gpu_scan import status, torch  # noqa: F401

pytestmark = pytest.mark.gpu
INF = float("inf")


def small(torch, kind, shape, dtype):  # noqa: F811
    """Gates with decays of about 3e-4 (16 of them: 1e-56) and, in every third channel, 0.9."""
    g = torch.full(shape, -8.0, device="cuda") + 0.1 * torch.randn(shape, device="cuda")
    g[..., ::3] = 2.2
    return torch.sigmoid(g) if kind == "decay" else g.to(dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("kind", ["decay", "sigmoid"])
@pytest.mark.parametrize("shape", [(3, 700, 72), (1, 4000, 64), (5, 40, 64), (300, 64, 64)], ids=str)
def test_dense(torch, shape, kind, dtype):  # noqa: F811
    from gated_delta_rule_49_gb300 import binding
    torch.manual_seed(0)
    B, T, D = shape
    dtype = getattr(torch, dtype)
    x, dh = (torch.randn(shape, device="cuda").to(dtype) for _ in range(2))
    g = small(torch, kind, shape, dtype)
    h0, dhT = torch.randn(2, B, D, device="cuda")
    bad = torch.zeros(B, D, dtype=torch.bool, device="cuda")
    bad[B // 2, 5:9] = bad[0, 12] = True
    sign = torch.where(torch.arange(D, device="cuda") % 2 == 0, INF, -INF).expand(B, D)

    def forward(start, xx=x):
        return binding.scan_prefill(xx, g, start, kind, keep_states=True)

    h, hT, states = forward(h0)
    got, gT, kept = forward(torch.where(bad, sign, h0))
    rows = bad[:, None].expand(shape)
    assert got[~rows].equal(h[~rows]) and gT[~bad].equal(hT[~bad])
    assert not got[rows].isfinite().any() and not gT[bad].isfinite().any()
    rows = bad[:, None].expand(states.shape)
    assert kept[~rows].equal(states[~rows]) and not kept[rows].isfinite().any()
    # from a token on
    t = T // 3
    xx = x.clone()
    xx[:, t][bad] = INF
    got, gT, _ = forward(h0, xx)
    rows = bad[:, None].repeat(1, T, 1)
    rows[:, :t] = False
    assert got[~rows].equal(h[~rows]) and gT[~bad].equal(hT[~bad])
    assert not got[rows].isfinite().any() and not gT[bad].isfinite().any()

    def backward(end, d=dh):
        return binding.scan_backward(x, g, d, h0, end, states, kind, want_dh0=True)

    dx, dg, dh0 = backward(dhT)
    gx, gg, g0 = backward(torch.where(bad, sign, dhT))
    rows = bad[:, None].expand(shape)
    for a, b in ((gx, dx), (gg, dg)):
        assert a[~rows].equal(b[~rows]) and not a[rows].isfinite().any()
    assert g0[~bad].equal(dh0[~bad]) and not g0[bad].isfinite().any()
    d = dh.clone()
    d[:, t][bad] = INF
    gx, gg, g0 = backward(dhT, d)
    rows = bad[:, None].repeat(1, T, 1)
    rows[:, t + 1:] = False
    for a, b in ((gx, dx), (gg, dg)):
        assert a[~rows].equal(b[~rows]) and not a[rows].isfinite().any()
    assert g0[~bad].equal(dh0[~bad]) and not g0[bad].isfinite().any()
    assert status() == binding.GDN_OK


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("kind", ["decay", "sigmoid"])
def test_packed(torch, kind, dtype):  # noqa: F811
    """An infinite state stays in its sequence."""
    from gated_delta_rule_49_gb300 import binding
    torch.manual_seed(1)
    lens, D = [130, 0, 1, 500, 64, 7, 0, 2000], 64
    dtype = getattr(torch, dtype)
    off = torch.tensor([0] + lens).cumsum(0).int().cuda()
    T, B = sum(lens), len(lens)
    x, dh = (torch.randn(T, D, device="cuda").to(dtype) for _ in range(2))
    g = small(torch, kind, (T, D), dtype)
    h0, dhT = torch.randn(2, B, D, device="cuda")
    h, hT, states = binding.scan_prefill(x, g, h0, kind, off, keep_states=True)
    dx, dg, dh0 = binding.scan_backward(x, g, dh, h0, dhT, states, kind, off)
    for i in (0, 1, 3, 5, 7):
        start, end = h0.clone(), dhT.clone()
        start[i, 3:7], end[i, 10:12] = -INF, INF
        mine = torch.zeros(T, D, dtype=torch.bool, device="cuda")
        s = slice(int(off[i]), int(off[i + 1]))
        mine[s, 3:7] = True
        seq = torch.zeros(B, D, dtype=torch.bool, device="cuda")
        seq[i, 3:7] = True
        got, gT, _ = binding.scan_prefill(x, g, start, kind, off)
        assert got[~mine].equal(h[~mine]) and not got[mine].isfinite().any()
        assert gT[~seq].equal(hT[~seq]) and not gT[seq].isfinite().any()
        mine, seq = mine.zero_(), seq.zero_()
        mine[s, 10:12] = seq[i, 10:12] = True
        gx, gg, g0 = binding.scan_backward(x, g, dh, h0, end, states, kind, off)
        for a, b in ((gx, dx), (gg, dg)):
            assert a[~mine].equal(b[~mine]) and not a[mine].isfinite().any()
        assert g0[~seq].equal(dh0[~seq]) and not g0[seq].isfinite().any()
    assert status() == binding.GDN_OK
