"""Sizes at the ends of the gated linear recurrence's range: refused, or computed by every
check and plan on the host without an overflow (no GPU: nothing is launched)."""
import pytest

from gated_delta_rule_49_gb300 import binding, build
from test_scan_abi import F, backward, prefill, step

INV = binding.GDN_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("call", [prefill, backward, step])
@pytest.mark.parametrize("D", [(1 << 31) - 1016, (1 << 31) - 56, (1 << 31) - 8])
def test_channels_near_two_to_the_31(lib, call, D):
    # (rounded up to a CTA's 64 channels such a width was negative, and the plan of short
    # sequences divided by a number of streams of 0)
    for B in (1, 2, 32):
        kw = dict(B=B, D=D, ldx=1 << 31, ldg=1 << 31)
        if call is not step:
            kw["T"] = 1
        assert call(lib, **kw) == INV, (B, D)
        assert call(lib, **kw, dt=1, kind=0) == INV, (B, D)
