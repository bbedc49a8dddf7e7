"""Edges of linear attention on the GPU: bad offsets of batches that are cut into
segments, decays that are not a number, workspaces of the caller, sums of few terms."""
import linear_ref as ref
import numpy as np
import pytest
from test_gpu_linear import Problem, clean_status, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,K,V", [("bf16", 128, 128), ("bf16", 64, 128), ("fp32", 64, 128),
                                       ("fp32", 32, 32)])
def test_bad_offsets_of_sequences_that_are_cut(torch, K, V, dtype):  # noqa: F811
    """The second sequence falls, the third starts inside the first: both are empty, the first and
    the last have the bits that they have beside good ones."""
    from gated_delta_rule_49_gb300 import binding
    lens = [2500, 0, 1500, 2001]
    p = Problem(torch, 6, 0, 0, 1, 5, K, V, dtype, True, lens)
    dt = binding.GDN_BF16 if dtype == "bf16" else binding.GDN_FP32
    assert binding.gdn_linear_prefill_workspace_size(4, 6001, 5, K, V, True, dt) > 0
    bad = p.offsets.clone()
    bad[2] = 1000

    def calls(offsets):
        got = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, offsets=offsets)
        status = [binding.gdn_get_last_device_status()]
        got += binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST, offsets=offsets)
        return got, status + [binding.gdn_get_last_device_status()]

    want, status = calls(p.offsets)
    assert status == [binding.GDN_OK] * 2
    got, status = calls(bad)
    assert status == [binding.GDN_ERR_DEVICE_BOUNDS] * 2
    for i in (0, 2, 3, 4):  # o, dq, dk, dv
        assert torch.equal(got[i][:2500], want[i][:2500])
        assert torch.equal(got[i][4000:], want[i][4000:])
    for i, start in ((1, p.S0), (5, p.dST)):
        for s in range(4):
            assert torch.equal(got[i][s], start[s] if s in (1, 2) else want[i][s])


WIDTHS = [("bf16", 128, 128), ("bf16", 64, 64), ("bf16", 64, 128), ("bf16", 32, 32),
          ("fp32", 64, 128)]


@pytest.mark.parametrize("dtype,K,V", WIDTHS)
@pytest.mark.parametrize("T", [5, 300, 3000])
def test_a_decay_that_is_not_a_number(torch, K, V, dtype, T):  # noqa: F811
    """Its head has no number left, the others keep their bits."""
    from gated_delta_rule_49_gb300 import binding
    for start in (True, False):
        p = Problem(torch, 14, 1, T, 3, 3, K, V, dtype, start)
        clean = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0) + binding.linear_backward(
            p.q, p.k, p.v, p.a, p.do, p.S0, p.dST, want_dS0=True)
        p.a[1] = float("nan")
        got = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0) + binding.linear_backward(
            p.q, p.k, p.v, p.a, p.do, p.S0, p.dST, want_dS0=True)
        for i, (a, b) in enumerate(zip(clean, got)):
            heads = 1 if i in (1, 5) else 2  # states, tokens
            for h in (0, 2):
                assert torch.equal(a.select(heads, h), b.select(heads, h))
            bad = b.select(heads, 1)
            # the last token's gradients of k and v come before any decay
            assert (bad[:, :-1] if i in (3, 4) else bad).isnan().all(), i
        x = [y[:, 0].contiguous() for y in (p.q, p.k, p.v)]
        if start:
            S = p.S0.clone()
            o = binding.linear_decode_step(*x, p.a, S)
            assert o[:, 1].isnan().all() and S[:, 1].isnan().all() and S[:, 0].isfinite().all()


@pytest.mark.parametrize("dtype,K,V", WIDTHS)
def test_empty_sequences_keep_their_states_at_any_decay(torch, K, V, dtype):  # noqa: F811
    from gated_delta_rule_49_gb300 import binding
    p = Problem(torch, 15, 0, 0, 2, 2, K, V, dtype, True, [3000, 0, 40])
    p.a[0] = float("nan")
    _, S = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, offsets=p.offsets)
    dS0 = binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST, offsets=p.offsets)[3]
    assert torch.equal(S[1], p.S0[1]) and torch.equal(dS0[1], p.dST[1])


def test_workspaces_of_the_caller(torch):  # noqa: F811
    """One of its own gives the same bits; one on the CPU, in pieces or too small is refused."""
    from gated_delta_rule_49_gb300 import binding
    p = Problem(torch, 16, 1, 3000, 1, 2, 64, 64, "bf16")
    f, pos = torch.ones(32, device="cuda"), torch.zeros(1, 3000, dtype=torch.int64, device="cuda")
    w = torch.ones(64, device="cuda")
    calls = (
        (lambda ws: binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, workspace=ws),
         binding.gdn_linear_prefill_workspace_size(1, 3000, 2, 64, 64, False, binding.GDN_BF16)),
        (lambda ws: binding.linear_backward(p.q, p.k, p.v, p.a, p.do, workspace=ws)[:3],
         binding.gdn_linear_backward_workspace_size(1, 3000, 1, 2, 64, 64, False, binding.GDN_BF16)),
        (lambda ws: binding.qk_norm_rotate_backward(p.q, p.k, pos, f, p.q, p.k, w, w, workspace=ws),
         binding.gdn_qk_norm_rotate_backward_workspace_size(3000, 1, 1, 64)))
    for call, need in calls:
        assert need > 0
        want = call(None)
        got = call(torch.empty(need, dtype=torch.uint8, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for bad, status in ((torch.empty(need, dtype=torch.uint8), binding.GDN_ERR_INVALID_ARG),
                            (torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2],
                             binding.GDN_ERR_INVALID_ARG),
                            (torch.empty(need - 4, dtype=torch.uint8, device="cuda"),
                             binding.GDN_ERR_WORKSPACE)):
            with pytest.raises(binding.GDNError) as e:
                call(bad)
            assert e.value.status == status


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("T", [1, 2, 8])
def test_few_tokens_whose_terms_cancel(torch, T, K, V):  # noqa: F811
    """bf16 outputs of a few tokens: half a step of the output's type, and float32 steps of the
    terms' magnitudes (no rounding of an operand), whatever is left of the terms."""
    from gated_delta_rule_49_gb300 import binding

    def held(got, want, mag, width):
        got = got.double().cpu().numpy()
        bound = ref.U["bf16"] * np.abs(want) + ref.steps("fp32", T, width) * mag * 1.01
        assert (np.abs(got - want) <= bound + 1e-30).all()

    for seed in range(20):
        for packed in (False, True):
            p = Problem(torch, seed, 1, T, 1, 4, K, V, "bf16", seed % 2 == 0, [T] if packed else None)
            o, S = binding.linear_prefill(p.q, p.k, p.v, p.a, p.S0, scale=0.5, offsets=p.offsets)
            (o64, S64), (om, Sm) = p.forward(0.5)
            held(o, o64, om, K)
            assert (np.abs(S.double().cpu().numpy() - S64) <= ref.state_steps("fp32", T) * Sm).all()
            got = binding.linear_backward(p.q, p.k, p.v, p.a, p.do, p.S0, p.dST, scale=0.5,
                                          offsets=p.offsets)
            want, mag = p.backward(0.5)
            for i in range(3):
                held(got[i], want[i], mag[i], K + V + 4)
