"""The layer norm at the widths about which its rows change hands: from one piece of
channels a thread to several, from two rows at a time to one, from weights in shared
memory to registers."""
import pytest
import test_gpu_layer_norm as rows
from test_gpu_scan import status, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [2056, 2560, 4104, 5120, 6144, 6152, 8192, 8200, 12288])
def test_forward_and_backward(torch, D, dtype):  # noqa: F811
    rows.test_forward_and_backward(torch, D, dtype)


@pytest.mark.parametrize("D", [5120, 6152, 8200])
def test_gradients_of_many_rows(torch, D):  # noqa: F811
    """Rows' own gradients bit for bit as in calls of few rows; equal calls, equal sums."""
    from gated_delta_rule_49_gb300 import binding
    N = 2003
    g = torch.Generator(device="cuda").manual_seed(D)
    x, dy, ds = (torch.randn(N, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    w, b = torch.randn(2, D, generator=g, device="cuda")
    stats = binding.layer_norm(x, w, b, want_stats=True)[2]
    for past in (ds, None):
        dx, dw, db = binding.layer_norm_backward(x, dy, stats, w, past, want_db=True)
        for i in range(0, N, 150):
            part = slice(i, i + 150)
            few = binding.layer_norm_backward(x[part], dy[part], stats[part], w,
                                              None if past is None else past[part])[0]
            assert few.equal(dx[part])
        again = binding.layer_norm_backward(x, dy, stats, w, past, want_db=True)
        assert all(p.equal(q) for p, q in zip((dx, dw, db), again))
        # sums of N terms in float32, whatever their order
        n = (x.double() - stats[:, :1]) * stats[:, 1:]
        for got, term in ((dw, dy.double() * n), (db, dy.double())):
            limit = 2.0 ** -24 * (N + 8) * term.abs().sum(0)
            assert ((got - term.sum(0)).abs() <= limit).all()
    assert status() == binding.GDN_OK
