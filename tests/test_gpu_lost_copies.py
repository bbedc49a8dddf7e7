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


# rows, channels: rows by 8 threads to all 512 of a CTA; one block, and so many rows that CTAs
# take over others' (a sum's)
NORMS = [(3, 64), (200_003, 64), (9, 2048), (8193, 2048), (10, 4096), (3000, 4096), (700, 16384)]


@pytest.mark.parametrize("call", [binding.GDN_SELFTEST_NORM, binding.GDN_SELFTEST_NORM_SUM,
                                  binding.GDN_SELFTEST_NORM_BACKWARD], ids=["norm", "sum", "backward"])
@pytest.mark.parametrize("N,D", NORMS)
def test_layer_norm(torch, call, N, D):
    g = torch.Generator(device="cuda").manual_seed(0)
    x, r = (torch.randn(N, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    want = binding.layer_norm(x, residual=r, want_stats=True)
    grads = binding.layer_norm_backward(want[1], r, want[2], ds=x, want_db=True)
    for lost in (0, N // 2, N - 1):
        run(torch, call, N, 1, D, lost)
        got = binding.layer_norm(x, residual=r, want_stats=True)
        assert all(p.equal(q) for p, q in zip(got, want))
        again = binding.layer_norm_backward(want[1], r, want[2], ds=x, want_db=True)
        assert again[0].equal(grads[0]) and again[2].equal(grads[2])
    assert binding.gdn_get_last_device_status() == binding.GDN_OK


@pytest.mark.parametrize("N,D", [(200_003, 64), (8193, 2048), (3000, 4096), (700, 16384)])
def test_answers_that_never_come(torch, N, D):
    """A sum's CTAs ask which others they may take over (fewer rows than CTAs: none asks)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    x, r = (torch.randn(N, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    want = binding.layer_norm(x, residual=r)[0]
    run(torch, binding.GDN_SELFTEST_NORM_ANSWER, N, 1, D, 0)
    assert binding.layer_norm(x, residual=r)[0].equal(want)
    size = 24 * 9 * D + 1536
    buffer = torch.zeros(size, dtype=torch.uint8, device="cuda")
    binding.gdn_selftest_lost_copy(binding.GDN_SELFTEST_NORM_ANSWER, LIMIT, 0, buffer, size, 9, 1, D)
    assert binding.gdn_get_last_device_status() == binding.GDN_OK
