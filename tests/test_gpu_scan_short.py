"""Batches of short dense sequences, whole ones in a tile, of one, two and three tiles a stream
(152 SMs take 304 tiles of 64 channels at once), against float64 value by value."""
import numpy as np
import pytest
import scan_ref as ref
from test_gpu_scan import close, inputs, status, tensor, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,dtype", [("decay", "fp32"), ("sigmoid", "bf16")])
@pytest.mark.parametrize("shape", [(304, 64, 64), (305, 64, 64), (400, 64, 64), (456, 64, 64),
                                   (457, 63, 64), (609, 64, 64), (610, 64, 64), (911, 64, 64),
                                   (915, 33, 64), (1000, 21, 72), (11, 64, 2048), (14, 50, 2048),
                                   (25, 64, 2048)], ids=str)
def test_tiles_of_a_stream(torch, shape, kind, dtype):  # noqa: F811
    from gated_delta_rule_49_gb300 import binding
    B, T, D = shape
    rng = np.random.default_rng(B + T)
    x, xn, g, gn = inputs(torch, rng, shape, kind, dtype)
    dh, dhn = tensor(torch, rng.standard_normal(shape), dtype)
    h0, h0n = tensor(torch, rng.standard_normal((B, D)))
    dhT, dhTn = tensor(torch, rng.standard_normal((B, D)))
    h, hT, states = binding.scan_prefill(x, g, h0, kind, keep_states=True)
    want, err, _ = ref.scan(xn, gn, h0n, kind)
    close(h, want, err, dtype)
    close(hT, want[:, -1], err[:, -1], "fp32")
    assert states[:, 0].equal(h0)
    grads = ref.scan_grad(xn, gn, dhn, h0n, dhTn, kind)
    for kept in (states, None):
        dx, dg, dh0 = binding.scan_backward(x, g, dh, h0, dhT, kept, kind, want_dh0=True)
        close(dx, *grads["dx"], dtype)
        close(dg, *grads["dgate"], "fp32" if kind == "decay" else dtype)
        close(dh0, *grads["dh0"], "fp32")
    # the end states over the start states, and the bits of a pair by itself where it has the
    # same place in a tile (of at most 1, 2, 3 or 6 of these sequences; elsewhere the runs of
    # tokens that are summed first cut the sequence at other tokens)
    h0c = h0.clone()
    assert binding.scan_prefill(x, g, h0c, kind, out_state=h0c)[0].equal(h) and h0c.equal(hT)
    for i in (0, B // 24 * 12, (B - 2) // 12 * 12):
        s = slice(i, i + 2)
        alone = binding.scan_prefill(x[s], g[s], h0[s], kind)
        assert alone[0].equal(h[s]) and alone[1].equal(hT[s])
    assert status() == binding.GDN_OK
