"""The layer norm refuses outputs that lie over its inputs or over each other, but for those that
take an input's place (no GPU: every call fails its checks before anything is launched)."""
import pytest

from gated_delta_rule_49_gb300 import binding, build

INV = binding.GDN_ERR_INVALID_ARG
N, D = 40, 64
PLACE = 1 << 20  # each tensor has 1 MB of addresses, never read
ROWS, LINE, STATS, WIDE = N * D * 2, D * 4, N * 2 * 4, ((N - 1) * 2 * D + D) * 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


FORWARD = ("x", "residual", "w", "b", "y", "s", "stats")
BACKWARD = ("s", "dy", "stats", "w", "ds", "dx", "dw", "db", "workspace")


def at(names):
    return {n: PLACE * (i + 1) for i, n in enumerate(names)}


def forward(lib, stride=D, **kw):
    a = {**at(FORWARD), **kw}
    return lib.gdn_layer_norm(*(a[n] for n in FORWARD), N, D, stride, stride, 1e-5, 0, None)


def backward(lib, stride=D, **kw):
    a = {**at(BACKWARD), **kw}
    return lib.gdn_layer_norm_backward(*(a[n] for n in BACKWARD[:8]), N, D, stride, 0,
                                       a["workspace"], 4 * LINE * N, None)


SIZES = dict(x=ROWS, residual=ROWS, w=LINE, b=LINE, y=ROWS, s=ROWS, stats=STATS, dy=ROWS, ds=ROWS,
             dx=ROWS, dw=LINE, db=LINE, workspace=2 * LINE)
IN_PLACE = {("y", "x"), ("y", "residual"), ("s", "x"), ("s", "residual"), ("dx", "dy"),
            ("dx", "ds"), ("dx", "s")}
PAIRS = [(forward, o, i) for o in ("y", "s", "stats") for i in FORWARD if i != o]
PAIRS += [(backward, o, i) for o in ("dx", "workspace") for i in BACKWARD if i != o]
PAIRS += [(backward, "dw", "db")]


@pytest.mark.parametrize("call,out,other", PAIRS, ids=lambda v: getattr(v, "__name__", v))
def test_refused(lib, call, out, other):
    base = at(FORWARD if call is forward else BACKWARD)
    for shift in (0, SIZES[other] - 16, 16 - SIZES[out]):
        if shift == 0 and (out, other) in IN_PLACE:
            continue
        assert call(lib, **{out: base[other] + shift}) == INV, shift


@pytest.mark.parametrize("call,out,other", [(forward, "y", "x"), (forward, "s", "residual"),
                                            (backward, "dx", "s")])
def test_rows_apart_are_not_replaced(lib, call, out, other):
    base = at(FORWARD if call is forward else BACKWARD)
    for stride in (2 * D, 1 << 40, 1 << 62):
        assert call(lib, stride, **{out: base[other]}) == INV
    assert call(lib, 2 * D, **{out: base[other] + WIDE - 16}) == INV
