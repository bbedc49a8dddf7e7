"""Refusals of the self-test that leaves a copy out (no GPU: nothing is launched)."""
import pytest

from gated_delta_rule_49_gb300 import binding, build

F = 0x10000  # aligned, never read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def test_refusals(lib):
    def call(**kw):
        a = dict(call=0, limit=1000, lost=0, buffer=F, bytes=1 << 30, rows=2, T=300, D=64)
        a.update(kw)
        return lib.gdn_selftest_lost_copy(*a.values(), None)

    for kw in (dict(call=-1), dict(call=99), dict(limit=0), dict(limit=1 << 40), dict(lost=-1),
               dict(buffer=None), dict(buffer=F + 8), dict(rows=0), dict(T=0), dict(D=0),
               dict(D=60), dict(D=32768), dict(rows=1 << 20, T=1 << 20)):
        assert call(**kw) == binding.GDN_ERR_INVALID_ARG, kw
    assert call(bytes=2 * 300 * 64 * 24 - 1) == binding.GDN_ERR_WORKSPACE


@pytest.mark.parametrize("call", [2, 3, 4, 5])
def test_norms_of_other_widths(lib, call):
    for D in (8, 72, 128, 2040, 8192):
        assert lib.gdn_selftest_lost_copy(call, 1000, 0, F, 1 << 30, 2, 30, D, None) == \
            binding.GDN_ERR_INVALID_ARG
