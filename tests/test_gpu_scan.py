"""The gated linear recurrence on the GPU against float64, value by value."""
import numpy as np
import pytest
import scan_ref as ref

pytestmark = pytest.mark.gpu
KINDS, DTYPES = ["decay", "sigmoid"], ["fp32", "bf16"]


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    from gated_delta_rule_49_gb300 import binding
    binding.load()
    return torch


def tensor(torch, x, dtype="fp32"):
    """(tensor on the GPU, the float64 values that it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    if dtype == "bf16":
        t = t.bfloat16()
    return t, t.double().cpu().numpy()


def gates(rng, shape, kind):
    """Horizons from one token to thousands, by channel; every sixteenth gate far out."""
    g = rng.standard_normal(shape) + np.linspace(-2, 8, shape[-1])
    g[rng.random(shape) < 1 / 16] *= 6
    return 1 / (1 + np.exp(-g)) if kind == "decay" else g


def inputs(torch, rng, shape, kind, dtype):
    x, xn = tensor(torch, rng.standard_normal(shape), dtype)
    g, gn = tensor(torch, gates(rng, shape, kind), "fp32" if kind == "decay" else dtype)
    return x, xn, g, gn


def number(t):
    return t.double().cpu().numpy()


def close(got, want, err, dtype):
    off, u = np.abs(number(got) - want), ref.U[dtype]
    bound = u * np.abs(want) + (1 + u) * err
    assert got.shape == want.shape and (off <= bound).all(), (off - bound).max()


def status():
    from gated_delta_rule_49_gb300 import binding
    return binding.gdn_get_last_device_status()


SHAPES = [(1, 1, 8), (3, 2, 64), (1, 63, 72), (2, 64, 128), (3, 65, 40), (2, 127, 136), (1, 129, 64),
          (1, 1000, 200), (5, 257, 24), (2, 2051, 64), (70, 3, 16), (1, 4500, 64), (1, 300, 1000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(torch, shape, kind, dtype):
    from gated_delta_rule_49_gb300 import binding
    B, T, D = shape
    rng = np.random.default_rng(T * D)
    x, xn, g, gn = inputs(torch, rng, shape, kind, dtype)
    dh, dhn = tensor(torch, rng.standard_normal(shape), dtype)
    for start in (False, True):
        h0, h0n = tensor(torch, rng.standard_normal((B, D))) if start else (None, None)
        dhT, dhTn = tensor(torch, rng.standard_normal((B, D))) if start else (None, None)
        h, hT, states = binding.scan_prefill(x, g, h0, kind, keep_states=True)
        want, err, _ = ref.scan(xn, gn, h0n, kind)
        close(h, want, err, dtype)
        close(hT, want[:, -1], err[:, -1], "fp32")
        close(states, ref.before(want, h0n)[:, ::64], ref.before(err, None)[:, ::64], "fp32")
        assert binding.scan_prefill(x, g, h0, kind, want_h=False)[1].equal(hT)
        assert binding.scan_prefill(x, g, h0, kind, want_state=False)[0].equal(h)
        wantg = ref.scan_grad(xn, gn, dhn, h0n, dhTn, kind)
        for kept in (states, None):
            dx, dg, dh0 = binding.scan_backward(x, g, dh, h0, dhT, kept, kind, want_dh0=True)
            close(dx, *wantg["dx"], dtype)
            close(dg, *wantg["dgate"], "fp32" if kind == "decay" else dtype)
            close(dh0, *wantg["dh0"], "fp32")
    assert status() == binding.GDN_OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_parts_of_a_projection(torch, kind, dtype):
    """x and the gate with token strides of their own, at the end of their memory too."""
    from gated_delta_rule_49_gb300 import binding
    rng = np.random.default_rng(1)
    B, T, D = 2, 131, 72
    x, xn, g, gn = inputs(torch, rng, (B, T, D), kind, dtype)
    wide = torch.full((B, T, 3 * D), float("nan"), dtype=x.dtype, device="cuda")
    gwide = torch.full((B, T, 2 * D + 8), float("nan"), dtype=g.dtype, device="cuda")
    wide[..., 2 * D:], gwide[..., 8:D + 8] = x, g
    xs, gs = wide[..., 2 * D:], gwide[..., 8:D + 8]
    dh = torch.randn(B, T, D, device="cuda").to(x.dtype)
    for a, b in ((x, gs), (xs, g), (xs, gs), (xs[:1], gs[:1]), (xs[:, :1], gs[:, :1])):
        d = dh[:a.shape[0], :a.shape[1]].contiguous()
        got = binding.scan_prefill(a, b, kind=kind)
        want = binding.scan_prefill(a.contiguous(), b.contiguous(), kind=kind)
        assert got[0].equal(want[0]) and got[1].equal(want[1])
        got = binding.scan_backward(a, b, d, kind=kind)
        want = binding.scan_backward(a.contiguous(), b.contiguous(), d, kind=kind)
        assert got[0].equal(want[0]) and got[1].equal(want[1])


def packed_reference(xn, gn, dhn, h0n, dhTn, off, kind):
    """Sequence by sequence: values, errors, gradients in the packed layout."""
    n, D = len(off) - 1, xn.shape[-1]
    h, err = np.zeros(xn.shape), np.zeros(xn.shape)
    hT, eT = (np.zeros((n, D)) if h0n is None else h0n.copy()), np.zeros((n, D))
    grads = {k: (np.zeros(xn.shape), np.zeros(xn.shape)) for k in ("dx", "dgate")}
    dh0 = ((np.zeros((n, D)) if dhTn is None else dhTn.copy()), np.zeros((n, D)))
    for i in range(n):
        s = slice(off[i], off[i + 1])
        if off[i] >= off[i + 1]:
            continue
        pick = lambda z: None if z is None else z[i:i + 1]  # noqa: E731
        h[s], err[s], _ = (z[0] for z in ref.scan(xn[None, s], gn[None, s], pick(h0n), kind))
        hT[i], eT[i] = h[off[i + 1] - 1], err[off[i + 1] - 1]
        got = ref.scan_grad(xn[None, s], gn[None, s], dhn[None, s], pick(h0n), pick(dhTn), kind)
        for k in ("dx", "dgate"):
            for j in range(2):
                grads[k][j][s] = got[k][j][0]
        for j in range(2):
            dh0[j][i] = got["dh0"][j][0]
    return (h, err), (hT, eT), grads["dx"], grads["dgate"], dh0


PACKED = [[3], [1, 1, 1], [0, 0, 5, 0], [64, 64], [63, 2, 63, 1], [130, 0, 1, 500, 64, 7, 0],
          [1] * 200, [1300, 1, 900, 2100], [0, 0], [16, 16, 17, 15, 8, 8, 128, 256]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens", PACKED, ids=lambda n: ",".join(map(str, n[:8])))
def test_packed(torch, lens, kind, dtype):
    """Sequences one after another; tokens before the first and behind the last are left as they were."""
    from gated_delta_rule_49_gb300 import binding
    rng = np.random.default_rng(len(lens) + sum(lens))
    D = 72
    for lead, tail, start in ((0, 0, True), (5, 70, False)):
        off = np.cumsum([lead] + lens).astype(np.int32)
        T = int(off[-1]) + tail
        if T == 0:
            continue
        x, xn, g, gn = inputs(torch, rng, (T, D), kind, dtype)
        dh, dhn = tensor(torch, rng.standard_normal((T, D)), dtype)
        n = len(lens)
        h0, h0n = tensor(torch, rng.standard_normal((n, D))) if start else (None, None)
        dhT, dhTn = tensor(torch, rng.standard_normal((n, D))) if start else (None, None)
        offt = torch.from_numpy(off).cuda()
        want = packed_reference(xn, gn, dhn, h0n, dhTn, off, kind)
        mine = np.zeros(T, bool)
        mine[off[0]:off[-1]] = True
        h, hT, states = binding.scan_prefill(x, g, h0, kind, offt, keep_states=True)
        close(h[mine], want[0][0][mine], want[0][1][mine], dtype)
        close(hT, *want[1], "fp32")
        held = torch.full((T, D), 7.0, dtype=x.dtype, device="cuda")
        code = binding._dtype_code(x)
        ws = torch.empty(binding.gdn_scan_prefill_workspace_size(n, T, D, True), dtype=torch.uint8,
                         device="cuda")
        binding.gdn_scan_prefill(x, g, h0, held, None, None, offt, n, T, D, D, D,
                                 binding.SCANS[kind], code, ws, ws.numel())
        assert held[mine].equal(h[mine]) and (held[~mine] == 7).all()
        gcode = "fp32" if kind == "decay" else dtype
        for kept in (states, None):
            dx, dg, dh0 = binding.scan_backward(x, g, dh, h0, dhT, kept, kind, offt, want_dh0=True)
            close(dx[mine], want[2][0][mine], want[2][1][mine], dtype)
            close(dg[mine], want[3][0][mine], want[3][1][mine], gcode)
            close(dh0, *want[4], "fp32")
        heldx, heldg = torch.full_like(x, 7.0), torch.full_like(g, 7.0)
        binding.gdn_scan_backward(x, g, dh, h0, dhT, states, heldx, heldg, None, offt, n, T, D, D,
                                  D, binding.SCANS[kind], code, ws, ws.numel())
        assert heldx[mine].equal(dx[mine]) and (heldx[~mine] == 7).all()
        assert heldg[mine].equal(dg[mine]) and (heldg[~mine] == 7).all()
    assert status() == binding.GDN_OK


@pytest.mark.parametrize("bad,good", [
    ([0, 5, 3, 9], [(0, 5), (0, 0), (0, 0)]),      # falls; the next starts before an earlier end
    ([0, 5, 12, 9], [(0, 5), (0, 0), (0, 0)]),     # passes the end, then falls
    ([-2, 4, 6, 10], [(0, 0), (4, 6), (6, 10)]),   # starts before the first token
    ([0, 10, 10, 99], [(0, 10), (0, 0), (0, 0)]),
    ([8, 3, 3, 10], [(0, 0), (0, 0), (3, 10)])])
def test_bad_offsets(torch, bad, good):
    """They are empty sequences and set the status; the others are as they are."""
    from gated_delta_rule_49_gb300 import binding
    T, D = 10, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    x, gate, dh = (torch.randn(T, D, generator=g, device="cuda") for _ in range(3))
    h0, dhT = torch.randn(2, 3, D, generator=g, device="cuda")
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    h, hT, _ = binding.scan_prefill(x, gate, h0, offsets=off)
    assert status() == binding.GDN_ERR_DEVICE_BOUNDS
    dx, dg, dh0 = binding.scan_backward(x, gate, dh, h0, dhT, offsets=off)
    assert status() == binding.GDN_ERR_DEVICE_BOUNDS
    for i, (a, b) in enumerate(good):
        if a == b:
            assert hT[i].equal(h0[i]) and dh0[i].equal(dhT[i])
            continue
        w = binding.scan_prefill(x[None, a:b], gate[None, a:b], h0[i:i + 1])
        close(h[a:b], number(w[0][0]), 1e-6, "fp32")
        close(hT[i], number(w[1][0]), 1e-6, "fp32")
        w = binding.scan_backward(x[None, a:b], gate[None, a:b], dh[None, a:b], h0[i:i + 1], dhT[i:i + 1])
        close(dx[a:b], number(w[0][0]), 1e-5, "fp32")
        close(dg[a:b], number(w[1][0]), 1e-5, "fp32")
        close(dh0[i], number(w[2][0]), 1e-5, "fp32")
    assert status() == binding.GDN_OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_steps(torch, kind, dtype):
    """Token by token, from slices of a projection, in place and not."""
    from gated_delta_rule_49_gb300 import binding
    for B, D in ((1, 8), (3, 200), (64, 2048), (70000, 8)):
        rng = np.random.default_rng(B)
        T = 3
        x, xn, g, gn = inputs(torch, rng, (B, T, D), kind, dtype)
        h0, h0n = tensor(torch, rng.standard_normal((B, D)))
        want, err, _ = ref.scan(xn, gn, h0n, kind)
        state = h0.clone()
        for t in range(T):
            out = torch.empty_like(state)
            y2 = torch.empty_like(x[:, 0].contiguous())
            binding.scan_decode_step(x[:, t], g[:, t], state, kind, h_out=out, y=y2)
            y = binding.scan_decode_step(x[:, t], g[:, t], state, kind)
            assert out.equal(state) and y2.equal(y)
            close(y, want[:, t], err[:, t], dtype)
            close(state, want[:, t], err[:, t], "fp32")


def test_in_place_and_carried(torch):
    """End states over start states, and a sequence in two calls."""
    from gated_delta_rule_49_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(2)
    for B, T, D in ((2, 40, 64), (300, 40, 64), (1, 3000, 64), (2, 700, 72)):
        x, gate = (torch.randn(B, T, D, generator=g, device="cuda") for _ in range(2))
        h0 = torch.randn(B, D, generator=g, device="cuda")
        h, hT, kept = binding.scan_prefill(x, gate, h0, keep_states=True)
        state = h0.clone()
        over = binding.scan_prefill(x, gate, state, out_state=state, keep_states=True)
        assert over[0].equal(h) and over[2].equal(kept) and state.equal(hT)
        cut = T // 3
        first = binding.scan_prefill(x[:, :cut].contiguous(), gate[:, :cut].contiguous(), h0)
        last = binding.scan_prefill(x[:, cut:].contiguous(), gate[:, cut:].contiguous(), first[1])
        both = torch.cat([first[0], last[0]], 1)
        # each within 20 half steps a token of a state of about one, twice over
        assert (both - h).abs().max() <= 2 * 2.0 ** -24 * 20 * 64 and \
            (last[1] - hT).abs().max() <= 2 * 2.0 ** -24 * 20 * 64


def test_nothing(torch):
    from gated_delta_rule_49_gb300 import binding
    h0 = torch.randn(3, 64, device="cuda")
    empty = torch.zeros(3, 0, 64, device="cuda")
    h, hT, states = binding.scan_prefill(empty, empty, h0, keep_states=True)
    assert h.shape == (3, 0, 64) and hT.equal(h0) and states.shape == (3, 0, 64)
    assert (binding.scan_prefill(empty, empty)[1] == 0).all()
    dx, dg, dh0 = binding.scan_backward(empty, empty, empty, h0, dh_T=h0)
    assert dh0.equal(h0) and dx.shape == dg.shape == (3, 0, 64)
    none = torch.zeros(0, 5, 64, device="cuda")
    assert binding.scan_prefill(none, none)[0].shape == (0, 5, 64)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    tok = torch.zeros(0, 64, device="cuda")
    assert binding.scan_prefill(tok, tok, h0, offsets=off)[1].equal(h0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite(torch, bad, kind):
    """They reach their own channel from their token on, and within its sequence only."""
    from gated_delta_rule_49_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(4)
    T, D = 400, 64
    x = torch.randn(T, D, generator=g, device="cuda")
    gate = torch.randn(T, D, generator=g, device="cuda").sigmoid()  # a decay, or a gate near 1/2
    dh = torch.randn(T, D, generator=g, device="cuda")
    off = torch.tensor([0, 100, 250, 400], dtype=torch.int32, device="cuda")
    clean = binding.scan_prefill(x, gate, kind=kind, offsets=off, keep_states=True)
    cgrad = binding.scan_backward(x, gate, dh, kind=kind, offsets=off)
    y = x.clone()
    y[170, 9] = bad
    h, hT, states = binding.scan_prefill(y, gate, kind=kind, offsets=off, keep_states=True)
    hit = torch.zeros(T, D, dtype=torch.bool, device="cuda")
    hit[170:250, 9] = True
    assert (~h[hit].isfinite()).all() and h[~hit].equal(clean[0][~hit])
    assert not hT[1, 9].isfinite() and hT[0].equal(clean[1][0]) and hT[2].equal(clean[1][2])
    for kept in (states, None):
        dx, dg, _ = binding.scan_backward(y, gate, dh, states=kept, kind=kind, offsets=off)
        assert dx.equal(cgrad[0])  # dx has none of x
        hit = torch.zeros(T, D, dtype=torch.bool, device="cuda")
        hit[(171 if kind == "decay" else 170):250, 9] = True
        assert (~dg[hit].isfinite()).all() and dg[~hit].equal(cgrad[1][~hit])
    d = dh.clone()
    d[170, 9] = bad
    dx, dg, _ = binding.scan_backward(x, gate, d, kind=kind, offsets=off)
    hit = torch.zeros(T, D, dtype=torch.bool, device="cuda")
    hit[100:171, 9] = True
    for got, want in ((dx, cgrad[0]), (dg, cgrad[1])):
        assert got[~hit].equal(want[~hit])
    assert (~dx[hit].isfinite()).all()
    # the dense form, across sequences of a batch and tokens that a tile reads beyond its own
    xb, gb = torch.stack([y[:170], y[170:340]]), torch.stack([gate[:170], gate[170:340]])
    hb = binding.scan_prefill(xb, gb, kind=kind)
    assert hb[0][0].isfinite().all() and hb[1][0].isfinite().all()
    assert hb[0][0].equal(binding.scan_prefill(xb[:1], gb[:1], kind=kind)[0][0])
    back = binding.scan_backward(xb, gb, torch.zeros_like(xb), kind=kind)
    assert (back[0] == 0).all() and (back[1][0] == 0).all()


def test_gates_far_out(torch):
    """Saturated gates switch: all of the state or all of the input, and their gradients vanish."""
    from gated_delta_rule_49_gb300 import binding
    for dtype in (torch.float32, torch.bfloat16):
        for g in (-300.0, -100.0, -90.0, 90.0, 100.0, 300.0, float("inf"), float("-inf")):
            x = torch.randn(1, 70, 64, device="cuda").to(dtype)
            gate = torch.full_like(x, g)
            h0 = torch.randn(1, 64, device="cuda")
            h, hT, _ = binding.scan_prefill(x, gate, h0)
            dx, dg, dh0 = binding.scan_backward(x, gate, torch.ones_like(x), h0)
            # what is left is at most 2^-120 of a value
            if g > 0:
                assert (hT - h0).abs().max() < 1e-30 and dx.abs().max() < 1e-30
                assert dh0.equal(torch.full_like(dh0, 70.0))
            else:
                assert h.equal(x) and dx.equal(torch.ones_like(x)) and dh0.abs().max() < 1e-30
            assert dg.abs().max() < 1e-30


def test_offsets_beyond_32_bits(torch):
    """The last tokens of a tensor of more than 2^31 elements: decays of at most 0.9 forget all but
    the last 300 tokens (0.9^300 = 2e-14)."""
    from gated_delta_rule_49_gb300 import binding
    T, D = (1 << 31) // 4096 + 700, 4096
    x = torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").normal_()
    gate = torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").normal_().clamp_(-2, 2)
    dh = torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").normal_()
    cut = slice(T - 900, T)
    h, hT, states = binding.scan_prefill(x, gate, keep_states=True)
    w = binding.scan_prefill(x[:, cut].contiguous(), gate[:, cut].contiguous())
    # equal to float32 steps of a state below 8, then rounded to bf16: one step of that at most
    assert (hT - w[1]).abs().max() < 1e-4
    assert (h[:, -600:].float() - w[0][:, -600:].float()).abs().max() <= 2.0 ** -5
    assert (h[:, -600:] != w[0][:, -600:]).float().mean() < 0.01
    del h
    dx, dg, _ = binding.scan_backward(x, gate, dh, states=states)
    w = binding.scan_backward(x[:, cut].contiguous(), gate[:, cut].contiguous(), dh[:, cut].contiguous())
    for got, want in ((dx, w[0]), (dg, w[1])):
        assert (got[:, -600:] != want[:, -600:]).float().mean() < 0.01
        assert (got[:, -600:].float() - want[:, -600:].float()).abs().max() <= 2.0 ** -3


def test_streams_and_graphs(torch):
    """On another stream, and captured and replayed with new inputs; equal bits every time."""
    from gated_delta_rule_49_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(5)
    for T, D, off in ((900, 200, None), (5000, 64, None), (700, 72, [0, 3, 3, 400, 690])):
        lead = (2, T) if off is None else (T,)
        x, gate, dh = (torch.randn(*lead, D, generator=g, device="cuda").bfloat16() for _ in range(3))
        offt = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
        n = 2 if off is None else 4
        real = slice(None) if off is None else slice(0, 690)
        h0 = torch.randn(n, D, generator=g, device="cuda")

        def both(s=None):
            h, hT, st = binding.scan_prefill(x, gate, h0, offsets=offt, keep_states=True, stream=s)
            return [h[real], hT] + [z if i == 2 else z[real] for i, z in enumerate(
                binding.scan_backward(x, gate, dh, h0, hT, st, offsets=offt, stream=s))]

        want = both()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = both(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(a.equal(b) for a, b in zip(got, want))
        with torch.cuda.stream(side):
            both()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = both()
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert all(a.equal(b) for a, b in zip(out, want))
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
            want = both()
    assert status() == binding.GDN_OK
