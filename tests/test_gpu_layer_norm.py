"""The layer norm on the GPU against float64, value by value."""
import numpy as np
import pytest
import scan_ref as ref
from test_gpu_scan import close, number, tensor, torch  # noqa: F401

pytestmark = pytest.mark.gpu
WIDTHS = [8, 16, 24, 64, 72, 128, 200, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 5000,
          8192, 8200, 16384]


def problem(torch, rng, N, D, dtype):  # noqa: F811
    """Rows of channels of different sizes about means of their own."""
    size = np.exp(0.5 * rng.standard_normal(D))
    x, xn = tensor(torch, (rng.standard_normal((N, D)) + rng.standard_normal(D)) * size, dtype)
    w, wn = tensor(torch, 1 + 0.2 * rng.standard_normal(D))
    b, bn = tensor(torch, 0.3 * rng.standard_normal(D))
    return x, xn, w, wn, b, bn


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_forward_and_backward(torch, D, dtype):  # noqa: F811
    from gated_delta_rule_49_gb300 import binding
    for N in (1, 2, 37, 1003):
        rng = np.random.default_rng(N + D)
        x, xn, w, wn, b, bn = problem(torch, rng, N, D, dtype)
        res, resn = tensor(torch, rng.standard_normal((N, D)), dtype)
        dy, dyn = tensor(torch, rng.standard_normal((N, D)), dtype)
        ds, dsn = tensor(torch, rng.standard_normal((N, D)), dtype)
        for r, weight, bias in ((None, None, None), (res, w, b), (res, w, None), (None, w, b)):
            y, s, stats = binding.layer_norm(x, weight, bias, r, want_stats=True)
            if r is None:
                assert s is None
                s, sn = x, xn
            else:
                assert s.equal((x.float() + res.float()).to(x.dtype))
                sn = number(s)
            want, err, m, rs, dm, dr = ref.layer_norm(sn, None if weight is None else wn,
                                                      None if bias is None else bn, 1e-5)
            close(y, want, err, dtype)
            close(stats[:, :1], m, dm, "fp32")
            close(stats[:, 1:], rs, dr * rs, "fp32")
            past = None if r is None else ds
            got = binding.layer_norm_backward(s, dy, stats, weight, past, want_db=bias is not None)
            m, rs = number(stats[:, :1]), number(stats[:, 1:])
            wantg = ref.layer_norm_grad(sn, dyn, m, rs, None if weight is None else wn,
                                        None if r is None else dsn)
            close(got[0], *wantg["dx"], dtype)
            for g, on, name in ((got[1], weight is not None, "dw"), (got[2], bias is not None, "db")):
                assert (g is not None) == on
                if on:
                    close(g, *wantg[name], "fp32")
            again = binding.layer_norm_backward(s, dy, stats, weight, past, want_db=bias is not None)
            assert all(p is q or p.equal(q) for p, q in zip(got, again))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [64, 200, 2048, 8192])
def test_strides_and_in_place(torch, D, dtype):  # noqa: F811
    """Rows of a wider tensor; outputs over the inputs."""
    from gated_delta_rule_49_gb300 import binding
    rng = np.random.default_rng(D)
    x, _, w, _, b, _ = problem(torch, rng, 3 * 11, D, dtype)
    x = x.view(3, 11, D)
    res = torch.randn(3, 11, D, device="cuda").to(x.dtype)
    y, s, stats = binding.layer_norm(x, w, b, res, want_stats=True)
    wide = torch.full((3, 11, 2 * D + 8), float("nan"), dtype=x.dtype, device="cuda")
    wide[..., :D], wide[..., D + 8:] = res, x
    got = binding.layer_norm(wide[..., D + 8:], w, b, wide[..., :D], want_stats=True)
    assert all(p.equal(q) for p, q in zip(got, (y, s, stats)))
    for out in ((x.clone(), res.clone()), (res.clone(), x.clone())):
        a, c = (out[0], out[1]) if out[0].equal(x) else (out[1], out[0])
        binding.layer_norm(a, w, b, c, out=out)
        assert out[0].equal(y) and out[1].equal(s)
    only = x.clone()
    binding.layer_norm(only, w, b, out=(only, None))
    assert only.equal(binding.layer_norm(x, w, b)[0])
    dy, ds = (torch.randn(3, 11, D, device="cuda").to(x.dtype) for _ in range(2))
    want = binding.layer_norm_backward(s, dy, stats, w, ds, want_db=True)
    wide[..., 8:D + 8] = s
    got = binding.layer_norm_backward(wide[..., 8:D + 8], dy, stats, w, ds, want_db=True)
    assert all(p.equal(q) for p, q in zip(got, want))
    ws = torch.empty(binding.gdn_layer_norm_backward_workspace_size(33, D), dtype=torch.uint8,
                     device="cuda")
    for name in ("dy", "ds"):
        over = {"dy": dy.clone(), "ds": ds.clone()}
        dw, db = torch.empty_like(w), torch.empty_like(w)
        binding.gdn_layer_norm_backward(s, over["dy"], stats, w, over["ds"], over[name], dw, db, 33,
                                        D, D, binding._dtype_code(x), ws, ws.numel())
        assert over[name].equal(want[0]) and dw.equal(want[1]) and db.equal(want[2])


def test_far_means(torch):  # noqa: F811
    """Rows about a mean of a thousand deviations keep theirs: the mean is taken off first."""
    from gated_delta_rule_49_gb300 import binding
    for D in (64, 200, 2048, 16384):
        x, xn = tensor(torch, 1000 + np.random.default_rng(D).standard_normal((5, D)))
        y, _, stats = binding.layer_norm(x, want_stats=True)
        want, err, m, r, dm, dr = ref.layer_norm(xn, None, None, 1e-5)
        close(y, want, err, "fp32")
        close(stats[:, 1:], r, dr * r, "fp32")


def test_rows_of_one_value(torch):  # noqa: F811
    """No deviation: zero, or with eps = 0 what 0 / 0 is; other rows are as they are."""
    from gated_delta_rule_49_gb300 import binding
    x = torch.randn(9, 72, device="cuda")
    x[4] = 2.5
    y, _, stats = binding.layer_norm(x, want_stats=True)
    assert (y[4].abs() <= 1e-3).all() and stats[4, 0] == 2.5
    y, _, stats = binding.layer_norm(x, eps=0.0, want_stats=True)
    rest = [i for i in range(9) if i != 4]
    assert y[rest].isfinite().all() and not y[4].isfinite().any()
    x[2, 7] = float("nan")
    y = binding.layer_norm(x)[0]
    assert y[2].isnan().all() and y[[0, 1, 3, 4, 5, 6, 7, 8]].isfinite().all()


def test_nothing(torch):  # noqa: F811
    from gated_delta_rule_49_gb300 import binding
    x, w = torch.zeros(0, 64, device="cuda"), torch.ones(64, device="cuda")
    y, _, stats = binding.layer_norm(x, w, want_stats=True)
    assert y.shape == (0, 64) and stats.shape == (0, 2)
    dx, dw, db = binding.layer_norm_backward(x, x, stats, w, want_db=True)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_offsets_beyond_32_bits(torch):  # noqa: F811
    from gated_delta_rule_49_gb300 import binding
    N, D = (1 << 31) // 128 + 77, 128
    x = torch.empty(N, D, dtype=torch.bfloat16, device="cuda").normal_()
    w, b = torch.randn(2, D, device="cuda")
    y, _, stats = binding.layer_norm(x, w, b, want_stats=True)
    last = x[-500:].contiguous()
    want, _, wstats = binding.layer_norm(last, w, b, want_stats=True)
    assert y[-500:].equal(want) and stats[-500:].equal(wstats)
    dx = binding.layer_norm_backward(x, y, stats, w)[0]
    assert dx[-500:].equal(binding.layer_norm_backward(last, want, wstats, w)[0])


def test_streams_and_graphs(torch):  # noqa: F811
    from gated_delta_rule_49_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(6)
    for N, D in ((700, 2048), (5, 128), (300, 5000)):
        x, res, dy = (torch.randn(N, D, generator=g, device="cuda").bfloat16() for _ in range(3))
        w, b = torch.randn(2, D, generator=g, device="cuda")

        def both(s=None):
            y, z, stats = binding.layer_norm(x, w, b, res, want_stats=True, stream=s)
            return [y, z, stats, *binding.layer_norm_backward(z, dy, stats, w, y, True, stream=s)]

        want = both()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = both(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(p.equal(q) for p, q in zip(got, want))
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = both()
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert all(p.equal(q) for p, q in zip(out, want))
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
            want = both()
