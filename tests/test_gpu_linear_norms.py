"""Linear attention on the GPU held to the norm of the error, head by head.

The bounds of test_gpu_linear.py go by the sum of the terms' magnitudes, which
for states that live long is larger than the outputs themselves; here the error
may not pass a share of the output's own norm.

States of bf16 runs are float32 results: the weighted values go in as three
bf16 pieces that are exact together, and of a chunk's products some 16 meet the
full sum and are cut, not rounded (2^-24 of it on average); the decay's powers
and the addition to the state take four roundings more: 20 x 2^-24 = 1.2e-6.
(Two pieces would be off by 2.7e-6.)  Outputs of bf16 runs carry three roundings
of half a step 2^-8 at most, 2^-8 / sqrt(3) in the mean each (scores, state,
output), independent of one another: 2^-8.  float32 runs round twice a token on
the way, independently: twice sqrt(2 T) 2^-24, and 2^-20 for the decay's powers
between segments."""
import numpy as np
import pytest
from test_gpu_linear import Problem, clean_status, host, torch  # noqa: F401

pytestmark = pytest.mark.gpu
ALPHA = np.float32([1.0, 0.9, 0.999, 0.9999, 0.5])
STATE, OUTPUT = 20 * 2.0 ** -24, 2.0 ** -8


def off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("dtype,K,V", [("bf16", 128, 128), ("bf16", 64, 64), ("bf16", 64, 128),
                                       ("fp32", 64, 128), ("fp32", 32, 32)])
@pytest.mark.parametrize("T,lens", [(128, None), (300, None), (512, None), (6001, None),
                                    (0, [3001, 1, 2500, 130])])
def test_error_norms(torch, T, lens, K, V, dtype):  # noqa: F811
    from gated_delta_rule_49_gb300 import binding
    p = Problem(torch, 21, 1, T, 5, 5, K, V, dtype, True, lens)
    p.an, p.a = ALPHA.astype(np.float64), torch.from_numpy(ALPHA).cuda()
    o, S = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, offsets=p.offsets)
    got = binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST, offsets=p.offsets)
    (want_o, want_S), _ = p.forward(1.0)
    want, _ = p.backward(1.0)
    state, output = STATE, OUTPUT
    if dtype == "fp32":
        state = output = 2 * np.sqrt(2 * p.longest) * 2.0 ** -24 + 2.0 ** -20
    for h in range(5):
        for name, x, y, bound in (("S", S, want_S, state), ("dS0", got[3], want[3], state)):
            for b in range(y.shape[0]):
                assert off(host(x)[b, h], y[b, h]) <= bound, (name, b, h)
        for name, x, y in (("o", o, want_o), ("dq", got[0], want[0]), ("dk", got[1], want[1]),
                           ("dv", got[2], want[2])):
            x, y = (z.reshape(-1, *z.shape[-2:])[:, h] for z in (host(x), y))
            for t in range(0, y.shape[0], 500):  # also far behind a cut
                assert off(x[t:t + 500], y[t:t + 500]) <= output, (name, t, h)
