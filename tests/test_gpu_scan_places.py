"""Outputs of the gated linear recurrence in places that they may take: between the rows of a
projection that holds the inputs, and end states over start states, all with the bits of outputs
of their own."""
import pytest

from gated_delta_rule_49_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def test_between_the_rows_of_a_projection(torch):
    B, D = 2, 64
    p = torch.randn(B, 6 * D, device="cuda").bfloat16()  # x, gate, room for h or y, and its rest
    x, gate, h0 = p[:, :D], p[:, D:2 * D], torch.randn(B, D, device="cuda")
    want, end, _ = binding.scan_prefill(x.reshape(B, 1, D), gate.reshape(B, 1, D), h0)
    room, h_T = p[0, 2 * D:4 * D], h0.clone()
    binding.gdn_scan_prefill(x, gate, h_T, room, h_T, None, None, B, 1, D, 6 * D, 6 * D,
                             binding.GDN_SCAN_SIGMOID, binding.GDN_BF16)
    assert room.equal(want.flatten()) and h_T.equal(end)
    room.zero_()
    h = h0.clone()
    binding.gdn_scan_decode_step(x, gate, h, h, room, B, D, 6 * D, 6 * D,
                                 binding.GDN_SCAN_SIGMOID, binding.GDN_BF16)
    # (two roundings of 2^-24 each, of values below 5)
    assert room.equal(want.flatten()) and torch.allclose(h, end, rtol=0, atol=1e-6)
    # one row further the room meets the second row of x
    with pytest.raises(binding.GDNError) as e:
        binding.gdn_scan_decode_step(x, gate, h, h, p.flatten()[5 * D:], B, D, 6 * D, 6 * D,
                                     binding.GDN_SCAN_SIGMOID, binding.GDN_BF16)
    assert e.value.status == binding.GDN_ERR_INVALID_ARG
    assert binding.gdn_get_last_device_status() == binding.GDN_OK
