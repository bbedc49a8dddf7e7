"""Edges of linear attention on the GPU: bad offsets of batches that are cut into
segments."""
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
