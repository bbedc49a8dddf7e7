"""Linear attention with a decay for each head on the GPU against the float64
token recurrence (tests/linear_ref.py).

Every bound is relative to the same recurrence on the magnitudes of the inputs,
so that it holds value by value whatever cancels: `steps` roundings on the way
and half a step of the output's type at the end."""
import linear_ref as ref
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

KV = [(32, 32), (64, 64), (64, 128), (128, 128)]
DECAYS = [1.0, 0.0, 0.3, 0.9, 0.999, 0.75]


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    from gated_delta_rule_49_gb300 import binding
    binding.load()
    return torch


@pytest.fixture(autouse=True)
def clean_status(torch):
    from gated_delta_rule_49_gb300 import binding
    yield
    assert binding.gdn_get_last_device_status() == binding.GDN_OK


def tensor(torch, rng, shape, dtype):
    """A random CUDA tensor of the type and the float64 values that it holds."""
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return x.cuda(), x.double().numpy()


def host(x):
    return x.double().cpu().numpy()


def close(got, want, mag, rel, dtype, what):
    got = host(got)
    assert got.shape == want.shape, what
    out = ref.U[dtype]
    bound = out * np.abs(want) + rel * (1 + out) * mag + 1e-30
    off = np.abs(got - want) / bound
    assert np.isfinite(got).all(), what
    assert off.max(initial=0) <= 1, (what, float(off.max()), float(np.abs(got - want).max()))


class Problem:
    def __init__(self, torch, seed, B, T, Hq, H, K, V, dtype, start=True, lens=None):
        rng = np.random.default_rng(seed)
        lead = (B, T) if lens is None else (sum(lens),)
        self.dtype, self.lens, self.K, self.V = dtype, lens, K, V
        self.q, self.qn = tensor(torch, rng, lead + (Hq, K), dtype)
        self.k, self.kn = tensor(torch, rng, lead + (Hq, K), dtype)
        self.v, self.vn = tensor(torch, rng, lead + (H, V), dtype)
        self.do, self.don = tensor(torch, rng, lead + (H, V), dtype)
        N = B if lens is None else len(lens)
        self.S0, self.S0n = tensor(torch, rng, (N, H, V, K), "fp32")
        self.dST, self.dSTn = tensor(torch, rng, (N, H, V, K), "fp32")
        if not start:
            self.S0 = self.dST = self.S0n = self.dSTn = None
        self.an = np.resize(np.float32(DECAYS), H).astype(np.float64)
        self.a = torch.from_numpy(self.an.astype(np.float32)).cuda()
        self.offsets = None
        if lens is not None:
            at = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
            self.offsets = torch.from_numpy(at).cuda()

    def sequences(self):
        """(q, k, v, do, S0, dST) of each sequence, with a leading axis of 1; dense: all at once."""
        z = lambda x, i: None if x is None else x[i:i + 1]  # noqa: E731
        if self.lens is None:
            yield self.qn, self.kn, self.vn, self.don, self.S0n, self.dSTn
            return
        t = 0
        for i, n in enumerate(self.lens):
            yield (*(x[None, t:t + n] for x in (self.qn, self.kn, self.vn, self.don)),
                   z(self.S0n, i), z(self.dSTn, i))
            t += n

    def join(self, parts, tokens):
        if self.lens is None:
            return parts[0]
        return np.concatenate([p[0] for p in parts]) if tokens else np.concatenate(parts)

    def forward(self, scale):
        """((o, S), (o, S) of the magnitudes)."""
        both = []
        for f in (lambda x: x, lambda x: None if x is None else np.abs(x)):
            r = [ref.linear(f(q), f(k), f(v), self.an, f(S0), scale)
                 for q, k, v, _, S0, _ in self.sequences()]
            both.append((self.join([x[0] for x in r], True), self.join([x[1] for x in r], False)))
        return both

    def backward(self, scale):
        both = []
        for f in (lambda x: x, lambda x: None if x is None else np.abs(x)):
            r = [ref.linear_grad(f(q), f(k), f(v), self.an, f(do), f(S0), f(dST), scale)
                 for q, k, v, do, S0, dST in self.sequences()]
            both.append(tuple(self.join([x[i] for x in r], i < 3) for i in range(4)))
        return both

    @property
    def longest(self):
        return max(self.lens) if self.lens else self.v.shape[1]

    def check_forward(self, o, S, scale):
        (o64, S64), (om, Sm) = self.forward(scale)
        if o is not None:
            close(o, o64, om, ref.steps(self.dtype, self.longest, self.K) +
                  (ref.U["bf16"] if self.dtype == "bf16" else 0), self.dtype, "o")
        if S is not None:
            close(S, S64, Sm, ref.state_steps(self.dtype, self.longest), "fp32", "S_T")

    def check_backward(self, got, scale):
        want, mag = self.backward(scale)
        group = self.v.shape[-2] // self.q.shape[-2]
        rel = ref.steps(self.dtype, self.longest, self.K + self.V + group) + \
            (ref.U["bf16"] if self.dtype == "bf16" else 0)
        for i, name in enumerate(("dq", "dk", "dv")):
            close(got[i], want[i], mag[i], rel, self.dtype, name)
        if got[3] is not None:
            close(got[3], want[3], mag[3], ref.state_steps(self.dtype, self.longest), "fp32", "dS0")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K,V", KV)
@pytest.mark.parametrize("T", [1, 2, 63, 127, 128, 129, 300])
def test_prefill(torch, K, V, T, dtype):
    from gated_delta_rule_49_gb300 import binding
    for start in (True, False):
        p = Problem(torch, T + K, 2, T, 3, 6, K, V, dtype, start)
        o, S = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, scale=0.25)
        p.check_forward(o, S, 0.25)
    # outputs alone and end states alone
    o2, none = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, scale=0.25, want_state=False)
    assert none is None and torch.equal(o2, o)
    none, S2 = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, scale=0.25, want_o=False)
    assert none is None and torch.equal(S2, S)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K,V", KV)
@pytest.mark.parametrize("T", [1, 130, 257])
@pytest.mark.parametrize("Hq,H", [(6, 6), (2, 6)])
def test_backward(torch, K, V, T, Hq, H, dtype):
    from gated_delta_rule_49_gb300 import binding
    for start in (True, False):
        p = Problem(torch, T + V, 2, T, Hq, H, K, V, dtype, start)
        got = binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST, scale=0.5,
                                      want_dS0=True)
        p.check_backward(got, 0.5)


LENS = [1, 0, 64, 200, 128, 0, 3, 129, 0]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K,V", KV)
def test_packed(torch, K, V, dtype):
    from gated_delta_rule_49_gb300 import binding
    for lens in (LENS, [5], [0, 0, 2], list(range(40))):
        p = Problem(torch, len(lens), 0, 0, 1, 2, K, V, dtype, True, lens)
        o, S = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, offsets=p.offsets)
        p.check_forward(o, S, 1.0)
        got = binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST, offsets=p.offsets)
        p.check_backward(got, 1.0)


@pytest.mark.parametrize("dtype,K,V", [("fp32", 32, 32), ("fp32", 64, 128), ("bf16", 128, 128),
                                       ("bf16", 64, 64), ("bf16", 64, 128)])
@pytest.mark.parametrize("packed", [False, True])
def test_long_sequences_are_cut(torch, K, V, dtype, packed):
    """Few long sequences run in segments; end states may replace the start states."""
    from gated_delta_rule_49_gb300 import binding
    lens = [3001, 0, 2500, 17] if packed else None
    p = Problem(torch, 5, 1, 6001, 1, 5, K, V, dtype, True, lens)
    T = sum(lens) if packed else 6001
    B = len(lens) if packed else 1
    dt = binding.GDN_BF16 if dtype == "bf16" else binding.GDN_FP32
    assert binding.gdn_linear_prefill_workspace_size(B, T, 5, K, V, packed, dt) > 0
    S = p.S0.clone()
    o, S1 = binding.linear_prefill(p.q, p.k, p.v, p.a, S, offsets=p.offsets, out_state=S)
    assert S1 is S
    p.check_forward(o, S, 1.0)
    got = binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST, offsets=p.offsets)
    p.check_backward(got, 1.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K,V", KV)
@pytest.mark.parametrize("B", [1, 5])
def test_steps_follow_the_prompt(torch, K, V, B, dtype):
    """A prompt, then single tokens, in place and into another state."""
    from gated_delta_rule_49_gb300 import binding
    T = 70
    p = Problem(torch, B, B, T, 3, 6, K, V, dtype)
    o, S = binding.linear_prefill(p.q[:, :T - 3], p.k[:, :T - 3], p.v[:, :T - 3], p.a, p.S0,
                                  scale=0.5) if B == 1 else binding.linear_prefill(
        *(x[:, :T - 3].contiguous() for x in (p.q, p.k, p.v)), p.a, p.S0, scale=0.5)
    outs = [o]
    for t in range(T - 3, T):
        x = [y[:, t].contiguous() for y in (p.q, p.k, p.v)]
        before = S.clone()
        S2 = torch.full_like(S, float("nan"))
        o2 = binding.linear_decode_step(*x, p.a, S, scale=0.5, S_out=S2)
        assert torch.equal(S, before)
        outs.append(binding.linear_decode_step(*x, p.a, S, scale=0.5)[:, None])
        assert torch.equal(S, S2) and torch.equal(outs[-1][:, 0], o2)
    p.check_forward(torch.cat(outs, 1), S, 0.5)


def test_parts_of_a_projection(torch):
    """q, k and v as slices of one projection's output."""
    from gated_delta_rule_49_gb300 import binding
    for dtype, K, V in (("bf16", 128, 128), ("fp32", 64, 128)):
        p = Problem(torch, 9, 2, 150, 2, 4, K, V, dtype)
        w = [x.shape[-2] * x.shape[-1] for x in (p.q, p.k, p.v)]
        whole = torch.cat([x.flatten(-2) for x in (p.q, p.k, p.v)], -1)
        q, k, v = (x.unflatten(-1, y.shape[-2:]) for x, y in
                   zip(whole.split(w, -1), (p.q, p.k, p.v)))
        assert not q.is_contiguous()
        a = binding.linear_prefill(q, k, v, p.a, p.S0)
        b = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        a = binding.linear_backward(q, k, v, p.a, p.do, p.S0, p.dST)
        b = binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_not_a_number_stays_in_its_sequence(torch, dtype):
    from gated_delta_rule_49_gb300 import binding
    lens = [100, 60, 200]
    p = Problem(torch, 3, 0, 0, 2, 2, 128, 128, dtype, False, lens)
    o, S = binding.linear_prefill(p.q, p.k, p.v, p.a, offsets=p.offsets)
    g = binding.linear_backward(p.q, p.k, p.v, p.a, p.do, offsets=p.offsets, want_dS0=True)
    for x in (p.q, p.k, p.v, p.do):
        x[100:160] = float("nan")
    x = binding.linear_prefill(p.q, p.k, p.v, p.a, offsets=p.offsets)
    y = binding.linear_backward(p.q, p.k, p.v, p.a, p.do, offsets=p.offsets, want_dS0=True)
    for a, b in [(x[0], o)] + list(zip(y[:3], g[:3])):
        assert torch.equal(a[:100], b[:100]) and torch.equal(a[160:], b[160:])
        assert a[100:160].isnan().any()
    for a, b in ((x[1], S), (y[3], g[3])):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_bad_offsets_are_reported(torch, dtype):
    """An offset that falls or passes the end: that sequence is empty, the others are right."""
    from gated_delta_rule_49_gb300 import binding
    p = Problem(torch, 4, 0, 0, 1, 2, 64, 128, dtype, True, [40, 30, 50])
    good = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, offsets=p.offsets)
    for at, bad in ((3, 121), (3, 60), (0, -1)):
        off = p.offsets.clone()
        off[at] = bad
        i = 2 if at == 3 else 0
        o, S = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, offsets=off)
        assert binding.gdn_get_last_device_status() == binding.GDN_ERR_DEVICE_BOUNDS
        for s in range(3):
            assert torch.equal(S[s], p.S0[s] if s == i else good[1][s])
        assert torch.equal(o[40:70], good[0][40:70])


def test_empty_calls(torch):
    from gated_delta_rule_49_gb300 import binding
    p = Problem(torch, 4, 2, 0, 1, 2, 128, 128, "bf16")
    o, S = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0)
    assert o.shape == (2, 0, 2, 128) and torch.equal(S, p.S0)
    dq, dk, dv, dS0 = binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST)
    assert dq.numel() == 0 and torch.equal(dS0, p.dST)
    _, S = binding.linear_prefill(p.q, p.k, p.v, p.a)
    assert not S.any()


def test_other_streams_and_graphs(torch):
    """The same bits on another stream, again, and from a captured graph."""
    from gated_delta_rule_49_gb300 import binding
    p = Problem(torch, 8, 1, 2100, 1, 2, 128, 128, "bf16")

    def both():
        o, S = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0)
        g = binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST)
        x = [y[:, 0].contiguous() for y in (p.q, p.k, p.v)]
        return (o, S, *g, binding.linear_decode_step(*x, p.a, S.clone()))

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = both()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for x in got:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_many_sequences(torch):
    """More sequences than the device holds at once, of a length that fills no block."""
    from gated_delta_rule_49_gb300 import binding
    p = Problem(torch, 2, 60, 33, 6, 6, 64, 64, "bf16")
    o, S = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0)
    p.check_forward(o, S, 1.0)
