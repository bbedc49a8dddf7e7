"""Many rows of the layer norm, where CTAs take over others' rows: every row is
formed once, whichever CTA forms it."""
import pytest
from test_gpu_scan import status, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def problem(torch, N, D, dtype, seed):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, res = (torch.randn(N, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    w, b = torch.randn(2, D, generator=g, device="cuda")
    return x, res, w, b


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,D", [(3041, 2048), (3040, 2048), (40000, 2048), (200001, 128), (99999, 200),
                                 (300000, 8), (30001, 1000), (9000, 4096), (5001, 8192), (1777, 16384)])
def test_rows(torch, N, D, dtype):  # noqa: F811
    """Bit for bit what calls of few rows give; what is beside the outputs is left."""
    from gated_delta_rule_49_gb300 import binding
    x, res, w, b = problem(torch, N, D, torch.float32 if dtype == "fp32" else torch.bfloat16, N)
    for r in (res, None):
        want = [torch.empty_like(x), None if r is None else torch.empty_like(x),
                torch.empty(N, 2, device="cuda")]
        few = 150 * (2 if D <= 256 else 1)  # rows of calls that deal them out evenly
        for i in range(0, N, few * 32):
            part = slice(i, min(N, i + few))
            got = binding.layer_norm(x[part], w, b, None if r is None else r[part], want_stats=True)
            for p, q in zip(want, got):
                if p is not None:
                    p[part] = q
        for _ in range(3):
            y = torch.full((N + 2, D), 7.0, dtype=x.dtype, device="cuda")
            s = torch.full((N + 2, D), 7.0, dtype=x.dtype, device="cuda")
            stats = torch.full((N, 2), float("nan"), device="cuda")
            binding.gdn_layer_norm(x, r, w, b, y[1:-1], None if r is None else s[1:-1], stats, N, D, D,
                                   D, 1e-5, binding._dtype_code(x))
            assert (y[0] == 7).all() and (y[-1] == 7).all()
            assert stats.isfinite().all()
            for i in range(0, N, few * 32):
                part = slice(i, min(N, i + few))
                out = slice(part.start + 1, part.stop + 1)
                assert y[out].equal(want[0][part]) and stats[part].equal(want[2][part])
                assert r is None or s[out].equal(want[1][part])
            if r is not None:
                assert s[1:-1].equal((x.float() + r.float()).to(x.dtype))
                assert (s[0] == 7).all() and (s[-1] == 7).all()
            # the rows between: their mean from y, by the formula
            z = (x if r is None else s[1:-1]).float()
            assert (stats[:, 0] - z.mean(-1)).abs().max() <= 2.0 ** -24 * 200 * z.abs().mean(-1).max()
            n = (z - stats[:, :1]) * stats[:, 1:] * w + b
            step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -22
            assert ((y[1:-1].float() - n).abs() <= step * (n.abs() + b.abs() + 1e-3)).all()
    assert status() == binding.GDN_OK


def test_streams_and_graphs_of_many_rows(torch):  # noqa: F811
    """Two such calls at once on two streams, in place, and captured and replayed."""
    from gated_delta_rule_49_gb300 import binding
    a, c = problem(torch, 30000, 2048, torch.bfloat16, 1), problem(torch, 150000, 512, torch.bfloat16, 2)
    want = [binding.layer_norm(x, w, b, r)[:2] for x, r, w, b in (a, c)]
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [binding.layer_norm(x, w, b, r, stream=s)[:2] for (x, r, w, b), s in zip((a, c), sides)]
        torch.cuda.synchronize()
        assert all(p.equal(q) for z, v in zip(got, want) for p, q in zip(z, v))
    x, r, w, b = a
    over = x.clone(), r.clone()
    binding.layer_norm(over[0], w, b, over[1], out=over)
    assert over[0].equal(want[0][0]) and over[1].equal(want[0][1])
    with torch.cuda.stream(sides[0]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=sides[0]):
            out = [binding.layer_norm(x, w, b, r)[:2] for x, r, w, b in (a, c)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(p.equal(q) for z, v in zip(out, want) for p, q in zip(z, v))
    assert status() == binding.GDN_OK
