"""Values of linear attention that are not finite, on the GPU: they reach what
the definition says and nothing else."""
import linear_ref as ref
import numpy as np
import pytest
from test_gpu_linear import Problem, clean_status, torch  # noqa: F401

pytestmark = pytest.mark.gpu
WIDTHS = [("bf16", 128, 128), ("bf16", 64, 64), ("bf16", 64, 128), ("bf16", 32, 32),
          ("fp32", 64, 128)]
CUT = {True: 3000, False: 300}


def spread(torch, clean, got, want, bound):  # noqa: F811
    """Clean values where the float64 ones are finite (the bits, or the bound that they are held to:
    outputs that share a block with the value are formed again), no finite value where not."""
    finite = np.isfinite(want)
    a, b = (x.double().cpu().numpy() for x in (clean, got))
    assert (np.abs(a - b)[finite] <= 2 * bound[finite]).all()
    assert not np.isfinite(b[~finite]).any()
    assert (a == b)[finite].mean() > 0.9


def bounds(p, scale=1.0):
    """What o, S, dq, dk, dv and dS0 of finite inputs are held to (as in Problem.check_*)."""
    (_, fwd), (_, back) = p.forward(scale), p.backward(scale)
    u, T = ref.U[p.dtype], p.longest
    operand = ref.U["bf16"] if p.dtype == "bf16" else 0
    out = [u * fwd[0] + (ref.steps(p.dtype, T, p.K) + operand) * (1 + u) * fwd[0],
           ref.state_steps(p.dtype, T) * fwd[1]]
    group = p.v.shape[-2] // p.q.shape[-2]
    rel = ref.steps(p.dtype, T, p.K + p.V + group) + operand
    return out + [u * m + rel * (1 + u) * m for m in back[:3]] + \
        [ref.state_steps(p.dtype, T) * back[3]]


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,K,V", WIDTHS)
@pytest.mark.parametrize("cut", [False, True])
def test_not_finite_values_reach_what_follows(torch, K, V, dtype, cut, bad):  # noqa: F811
    from gated_delta_rule_49_gb300 import binding
    T = CUT[cut]
    p = Problem(torch, 12, 1, T, 2, 2, K, V, dtype, True)
    p.an = np.float32([0.9, 1.0]).astype(np.float64)
    p.a = torch.tensor([0.9, 1.0], device="cuda")

    def calls():
        with np.errstate(invalid="ignore"):
            want = ref.linear(p.qn, p.kn, p.vn, p.an, p.S0n) + ref.linear_grad(
                p.qn, p.kn, p.vn, p.an, p.don, p.S0n, p.dSTn)
        o, S = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0)
        only, _ = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, want_state=False)
        return want, (o, S) + binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST), only

    _, clean, _ = calls()
    held = bounds(p)
    for at in ((0, 70, 127, 299) if not cut else (1500,)):
        for x, xn in ((p.q, p.qn), (p.k, p.kn), (p.v, p.vn), (p.do, p.don)):
            keep = xn[0, at, 1, 7]
            x[0, at, 1, 7] = xn[0, at, 1, 7] = bad
            want, got, only = calls()
            for a, b, c, d in zip(clean, got, want, held):
                spread(torch, a, b, c, d)
            spread(torch, clean[0], only, want[0], held[0])
            x[0, at, 1, 7] = xn[0, at, 1, 7] = keep


@pytest.mark.parametrize("dtype,K,V", WIDTHS)
def test_not_finite_values_of_packed_sequences(torch, K, V, dtype):  # noqa: F811
    """The rows around one in sequences that start and end anywhere, several at once."""
    from gated_delta_rule_49_gb300 import binding
    lens = [100, 60, 1, 200]
    p = Problem(torch, 13, 0, 0, 1, 2, K, V, dtype, True, lens)
    p.an = np.float32([0.75, 0.999]).astype(np.float64)
    p.a = torch.tensor([0.75, 0.999], device="cuda")
    clean = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, offsets=p.offsets) + \
        binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST, offsets=p.offsets)
    held = bounds(p)
    for t, h, c in ((50, 0, 3), (60, 0, 3), (55, 1, 30), (160, 1, 31), (200, 0, 0), (360, 0, 1)):
        p.v[t, h, c] = p.vn[t, h, c] = float("nan")
        p.do[t, h, c] = p.don[t, h, c] = float("inf")
    with np.errstate(invalid="ignore"):
        (o, S), _ = p.forward(1.0)
        want, _ = p.backward(1.0)
    state = p.S0.clone()  # which the end states replace
    got = binding.linear_prefill(p.q, p.k, p.v, p.a, state, offsets=p.offsets, out_state=state) + \
        binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST, offsets=p.offsets)
    for a, b, c, d in zip(clean, got, (o, S) + want, held):
        spread(torch, a, b, c, d)
