"""The gated linear recurrence refuses outputs that lie over its inputs or over each other,
wholly or in part (no GPU: every call fails its checks before anything is launched)."""
import pytest

from gated_delta_rule_49_gb300 import binding, build

INV = binding.GDN_ERR_INVALID_ARG
B, T, D = 2, 128, 64  # (packed or not, four states are kept)
PLACE = 1 << 20  # each tensor has 1 MB of addresses, never read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def at(*names):
    return {n: PLACE * (i + 1) for i, n in enumerate(names)}


# name: bytes, of bf16 tensors x and sigmoid gates that are parts of one projection
LD = 3 * D
X, STATE, KEPT = ((B * T - 1) * LD + D) * 2, B * D * 4, 4 * D * 4
DENSE = B * T * D * 2
OFF, WS = (B + 1) * 4, 4096


def prefill(lib, packed=False, **kw):
    a = at("x", "gate", "h0", "h", "h_T", "states", "offsets", "workspace")
    a.update(kw)
    off, ws = (a["offsets"], a["workspace"]) if packed else (None, None)
    return lib.gdn_scan_prefill(a["x"], a["gate"], a["h0"], a["h"], a["h_T"], a["states"], off, B,
                                B * T if packed else T, D, LD, LD, 1, 0, ws, WS, None)


def backward(lib, packed=False, **kw):
    a = at("x", "gate", "dh", "h0", "dh_T", "states", "dx", "dgate", "dh0", "offsets", "workspace")
    a.update(kw)
    off, ws = (a["offsets"], a["workspace"]) if packed else (None, None)
    return lib.gdn_scan_backward(a["x"], a["gate"], a["dh"], a["h0"], a["dh_T"], a["states"],
                                 a["dx"], a["dgate"], a["dh0"], off, B, B * T if packed else T, D,
                                 LD, LD, 1, 0, ws, WS, None)


def step(lib, packed=False, **kw):
    a = at("x", "gate", "h", "h_out", "y")
    a.update(kw)
    return lib.gdn_scan_decode_step(a["x"], a["gate"], a["h"], a["h_out"], a["y"], B, D, LD, LD, 1,
                                    0, None)


STEP = ((B - 1) * LD + D) * 2
CALLS = {
    prefill: (dict(x=X, gate=X, h0=STATE, offsets=OFF), dict(h=DENSE, h_T=STATE, states=KEPT,
                                                             workspace=B * T * 4)),
    backward: (dict(x=X, gate=X, dh=DENSE, h0=STATE, dh_T=STATE, states=KEPT, offsets=OFF),
               dict(dx=DENSE, dgate=DENSE, dh0=STATE, workspace=B * T * 4)),
    step: (dict(x=STEP, gate=STEP, h=STATE), dict(h_out=STATE, y=B * D * 2)),
}
PACKED_ONLY = ("offsets", "workspace")
CASES = [(call, out, other) for call, (ins, outs) in CALLS.items() for out in outs
         for other in (*ins, *outs) if other != out]


@pytest.mark.parametrize("call,out,other", CASES, ids=lambda v: getattr(v, "__name__", v))
def test_refused(lib, call, out, other):
    ins, outs = CALLS[call]
    base = at(*{prefill: ("x", "gate", "h0", "h", "h_T", "states", "offsets", "workspace"),
                backward: ("x", "gate", "dh", "h0", "dh_T", "states", "dx", "dgate", "dh0",
                           "offsets", "workspace"),
                step: ("x", "gate", "h", "h_out", "y")}[call])
    size = {**ins, **outs}
    # the whole of it, its last 16 bytes, and 16 bytes of its own end in the other's start
    for shift in (0, size[other] // 16 * 16 - 16, 16 - size[out] // 16 * 16):
        if (out, other) in (("h_T", "h0"), ("h_out", "h")) and shift == 0:
            continue  # in place
        for packed in (False, True):
            if not packed and (out in PACKED_ONLY or other in PACKED_ONLY):
                continue
            assert call(lib, packed, **{out: base[other] + shift}) == INV, (shift, packed)
