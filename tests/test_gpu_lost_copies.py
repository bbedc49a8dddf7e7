"""A copy that never comes: every wait of the kernel runs out, its threads leave together, the
status word says so, and the library computes as before."""
import time

import pytest

from gated_delta_rule_49_gb300 import binding

pytestmark = pytest.mark.gpu
LIMIT = 2_000_000  # about 1 ms of SM clocks


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    binding.load()
    return torch


def run(torch, call, rows, T, D, lost):
    size = 24 * rows * T * D + 1536
    buffer = torch.zeros(size, dtype=torch.uint8, device="cuda")
    assert binding.gdn_get_last_device_status() == binding.GDN_OK
    t0 = time.monotonic()
    binding.gdn_selftest_lost_copy(call, LIMIT, lost, buffer, size, rows, T, D)
    assert binding.gdn_get_last_device_status() == binding.GDN_ERR_TIMEOUT
    # the waits, and those for copies in flight before the end
    assert time.monotonic() - t0 < 10
    assert binding.gdn_get_last_device_status() == binding.GDN_OK


# rows, T, D: a CTA a sequence; one sequence by a cluster of 8 and by several clusters; whole
# sequences in a tile.  Tiles: the first, one in the middle, the last.
SCANS = [(256, 700, 64, (0, 2, 5)), (1, 8192, 64, (0, 11, 63)), (1, 8200, 2048, (3, 64)),
         (400, 64, 64, (0,)), (2, 130, 8, (1,))]


@pytest.mark.parametrize("call", [binding.GDN_SELFTEST_SCAN, binding.GDN_SELFTEST_SCAN_BACKWARD],
                         ids=["prefill", "backward"])
@pytest.mark.parametrize("rows,T,D,lost", SCANS)
def test_recurrence(torch, call, rows, T, D, lost):
    g = torch.Generator(device="cuda").manual_seed(0)
    x, gate = (torch.randn(rows, T, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    want = binding.scan_prefill(x, gate, keep_states=True)
    grads = binding.scan_backward(x, gate, want[0], states=want[2])
    for tile in lost:
        run(torch, call, rows, T, D, tile)
        got = binding.scan_prefill(x, gate, keep_states=True)
        assert all(p.equal(q) for p, q in zip(got, want))
        again = binding.scan_backward(x, gate, want[0], states=want[2])
        assert again[0].equal(grads[0]) and again[1].equal(grads[1])
    assert binding.gdn_get_last_device_status() == binding.GDN_OK
