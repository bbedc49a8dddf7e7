"""Further calls of the recurrence and the layer norm: many packed sequences with
bad offsets among them, workspaces of other streams and of two graphs, gates
that are not numbers."""
import numpy as np
import pytest
from test_gpu_scan import close, number, status, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def taken(offsets, T):
    """The sequences that the offsets give: (first, end), empty where they are bad; and whether
    one is."""
    out, upto, bad = [], 0, False
    for a, b in zip(offsets[:-1], offsets[1:]):
        fits = a >= 0 and b >= a and b <= T
        good = fits and a >= upto
        out.append((a, b) if good else (0, 0))
        upto = max(upto, b) if fits else upto
        bad |= not good
    return out, bad


@pytest.mark.parametrize("seed", range(12))
def test_many_sequences(torch, seed):  # noqa: F811
    """Thousands of sequences, more than the table's threads, from well-formed to random offsets."""
    from gated_delta_rule_49_gb300 import binding
    rng = np.random.default_rng(seed)
    B = int(rng.choice([1, 40, 1023, 1024, 1025, 3000]))
    lens = rng.choice([0, 0, 1, 1, 2, 3, 17], B)
    off = np.cumsum(np.concatenate([[rng.integers(0, 3)], lens]))
    T, D = int(off[-1] + rng.integers(0, 9)), 64
    if T == 0:
        T = 1
    for _ in range(int(rng.choice([0, 0, 1, 5, B]))):
        off[rng.integers(0, B + 1)] += int(rng.choice([-40, -3, 2, 1000, 2 ** 30]))
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, gate, dh = (torch.randn(T, D, generator=g, device="cuda") for _ in range(3))
    h0, dhT = torch.randn(2, B, D, generator=g, device="cuda")
    offt = torch.from_numpy(off.astype(np.int32)).cuda()
    seqs, bad = taken(off.tolist(), T)
    h, hT, kept = binding.scan_prefill(x, gate, h0, offsets=offt, keep_states=True)
    assert status() == (binding.GDN_ERR_DEVICE_BOUNDS if bad else binding.GDN_OK)
    dx, dg, dh0 = binding.scan_backward(x, gate, dh, h0, dhT, kept, offsets=offt)
    assert status() == (binding.GDN_ERR_DEVICE_BOUNDS if bad else binding.GDN_OK)
    # by the recurrence in float64, all sequences a token at a time
    a = 1 / (1 + np.exp(-number(gate)))
    xn, dn, s, u = number(x), number(dh), number(h0), number(dhT)
    first, n = np.array([q[0] for q in seqs]), np.array([q[1] - q[0] for q in seqs])
    want, wdx, wdg = np.zeros((T, D)), np.zeros((T, D)), np.zeros((T, D))
    past = np.zeros((T, D))
    for t in range(n.max()):
        i = n > t
        at = first[i] + t
        past[at] = s[i]
        s[i] = a[at] * s[i] + (1 - a[at]) * xn[at]
        want[at] = s[i]
    for t in reversed(range(n.max())):
        i = n > t
        at = first[i] + t
        G = dn[at] + u[i]
        wdx[at] = (1 - a[at]) * G
        wdg[at] = G * (past[at] - xn[at]) * a[at] * (1 - a[at])
        u[i] = a[at] * G
    mine = np.zeros(T, bool)
    for q, e in seqs:
        mine[q:e] = True
    # at most 40 tokens of a few float32 steps each, of values below 30
    for got, ref in ((h, want), (dx, wdx), (dg, wdg)):
        close(got[mine], ref[mine], 1e-4, "fp32")
    close(hT, s, 1e-4, "fp32")
    close(dh0, u, 1e-4, "fp32")


def test_scratch_of_another_stream(torch):  # noqa: F811
    """A workspace taken for a call on another stream is not given to this one's tensors while
    that call runs: every call's result is as on one stream."""
    from gated_delta_rule_49_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(7)
    x, gate, dh = (torch.randn(60000, 512, generator=g, device="cuda").bfloat16() for _ in range(3))
    off = torch.arange(0, 60001, 1000, dtype=torch.int32, device="cuda")
    w = torch.randn(512, generator=g, device="cuda")
    y, _, stats = binding.layer_norm(x, w, want_stats=True)
    calls = (lambda s: binding.scan_prefill(x, gate, offsets=off, stream=s)[:2],
             lambda s: binding.scan_backward(x, gate, dh, offsets=off, want_dh0=True, stream=s),
             lambda s: binding.layer_norm_backward(x, dh, stats, w, want_db=True, stream=s))
    side = torch.cuda.Stream()
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        got = []
        for _ in range(4):
            got.append(call(side))
            torch.full((60000 * 4,), 0x7f, dtype=torch.uint8, device="cuda")  # where scratch was
        torch.cuda.synchronize()
        assert all(p.equal(q) for z in got for p, q in zip(z, want))


def test_one_workspace_in_two_graphs(torch):  # noqa: F811
    """Nothing is kept in a workspace from one call for another: two captured calls take turns on
    one."""
    from gated_delta_rule_49_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(8)
    T, D = 900, 128
    sets = []
    for lens in ([300, 0, 600], [1, 449, 450]):
        x, gate, dh = (torch.randn(T, D, generator=g, device="cuda") for _ in range(3))
        off = torch.tensor(np.cumsum([0] + lens).astype(np.int32), device="cuda")
        sets.append((x, gate, dh, off))
    size = binding.gdn_scan_backward_workspace_size(3, T, D, True, False)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def run(s, workspace):
        x, gate, dh, off = s
        return (*binding.scan_prefill(x, gate, offsets=off, workspace=workspace)[:2],
                *binding.scan_backward(x, gate, dh, offsets=off, want_dh0=True, workspace=workspace))

    want = [run(s, None) for s in sets]
    side, graphs = torch.cuda.Stream(), []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            run(s, ws)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = run(s, ws)
            graphs.append((graph, out))
    torch.cuda.current_stream().wait_stream(side)
    for i in (0, 1, 1, 0, 1, 0):
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert all(p.equal(q) for p, q in zip(graphs[i][1], want[i]))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_gates_that_are_not_numbers(torch, dtype):  # noqa: F811
    """They reach the states of their channel from their token on and the gradients of its inputs
    before it; other channels keep their bits."""
    from gated_delta_rule_49_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(9)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    x, gate, dh = (torch.randn(2, 700, 64, generator=g, device="cuda").to(dt) for _ in range(3))
    h, hT, _ = binding.scan_prefill(x, gate)
    dx, _, _ = binding.scan_backward(x, gate, dh)
    bad = gate.clone()
    bad[1, 333, 5] = float("nan")
    hb, hTb, _ = binding.scan_prefill(x, bad)
    dxb, dgb, _ = binding.scan_backward(x, bad, dh)
    hit = torch.zeros_like(h, dtype=torch.bool)
    hit[1, 333:, 5] = True
    assert hb[hit].isnan().all() and hb[~hit].equal(h[~hit]) and hTb[1, 5].isnan()
    hit = torch.zeros_like(h, dtype=torch.bool)
    hit[1, :334, 5] = True
    assert dxb[hit].isnan().all() and dxb[~hit].equal(dx[~hit])
    assert dgb[1, 333, 5].isnan() and dgb[0].isfinite().all()


def test_more_sequences_than_a_grid_row(torch):  # noqa: F811
    """Short dense sequences by the ten thousand, alone and beside a wide batch."""
    from gated_delta_rule_49_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(10)
    for B, T, D in ((70000, 1, 8), (70001, 3, 8), (9001, 64, 16), (5000, 65, 8)):
        x, gate, dh = (torch.randn(B, T, D, generator=g, device="cuda") for _ in range(3))
        h0 = torch.randn(B, D, generator=g, device="cuda")
        h, hT, kept = binding.scan_prefill(x, gate, h0, keep_states=True)
        dx, dg, dh0 = binding.scan_backward(x, gate, dh, h0, states=kept)
        for i in (0, 1, B // 2, B - 1):
            one = slice(i, i + 1)
            w = binding.scan_prefill(x[one], gate[one], h0[one])
            v = binding.scan_backward(x[one], gate[one], dh[one], h0[one])
            # 65 tokens of a few float32 steps of values below 30, twice over
            for p, q in ((h[one], w[0]), (hT[one], w[1]), (dx[one], v[0]), (dg[one], v[1]),
                         (dh0[one], v[2])):
                assert (p - q).abs().max() < 2e-4


@pytest.mark.parametrize("kind", ["sigmoid", "decay"])
@pytest.mark.parametrize("T", [500, 3000])
def test_states_as_exact_as_float32(torch, T, kind):  # noqa: F811
    """End states and start gradients of bf16 runs are float32 results: off by at most twice what the
    recurrence token by token in float32 is, of the norm (a bias of the gates, small beside bf16,
    grows with every token)."""
    from gated_delta_rule_49_gb300 import binding
    rng = np.random.default_rng(T)
    B, D = 2, 512
    x, dh = (torch.from_numpy(rng.standard_normal((B, T, D)).astype(np.float32)).cuda().bfloat16()
             for _ in range(2))
    g = rng.standard_normal((B, T, D)) + np.linspace(0, 7.5, D)
    if kind == "decay":
        gate = torch.from_numpy((1 / (1 + np.exp(-g))).astype(np.float32)).cuda()
    else:
        gate = torch.from_numpy(g.astype(np.float32)).cuda().bfloat16()
    h0, dhT = (torch.from_numpy(rng.standard_normal((B, D)).astype(np.float32)).cuda() for _ in range(2))
    hT = binding.scan_prefill(x, gate, h0, kind)[1]
    dh0 = binding.scan_backward(x, gate, dh, h0, dhT, kind=kind)[2]

    def ends(t):
        """In type t, from the same inputs."""
        gn, xn, dn = (number(z).astype(t) for z in (gate, x, dh))
        a = gn if kind == "decay" else 1 / (1 + np.exp(-gn))
        b = t(1) if kind == "decay" else 1 / (1 + np.exp(gn))
        s, u, bx = number(h0).astype(t), number(dhT).astype(t), b * xn
        for i in range(T):
            s = a[:, i] * s + bx[:, i]
        for i in reversed(range(T)):
            u = a[:, i] * (dn[:, i] + u)
        return s, u

    for got, f32, f64 in zip((hT, dh0), ends(np.float32), ends(np.float64)):
        off, may = np.linalg.norm(number(got) - f64), np.linalg.norm(f32 - f64)
        assert off <= 2 * may, (off / np.linalg.norm(f64), may / np.linalg.norm(f64))
