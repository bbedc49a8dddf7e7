"""Segments of packed sequences: the device's own index arithmetic, compiled for
the CPU, against the rule of the documentation, for offsets good and bad."""
import math
import os
import random
import subprocess

import pytest

from gated_delta_rule_49_gb300 import binding, build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def items(tmp_path_factory):
    build.build()
    binding.load()
    exe = str(tmp_path_factory.mktemp("items") / "linear_item_host")
    subprocess.run(["g++", "-std=c++20", "-O1", "-pthread", "-I", build.CSRC,
                    os.path.join(HERE, "linear_item_host.cpp"), "-o", exe], check=True)

    def run(B, T, seg_len, n, offsets=None):
        args = [B, T, seg_len, n, int(offsets is not None), *(offsets or [])]
        out = subprocess.run([exe, *map(str, args)], check=True, capture_output=True, text=True)
        lines = [tuple(map(int, x.split())) for x in out.stdout.splitlines()]
        return lines[:-1], lines[-1][0]

    return run


def accepted(offsets, T):
    """Length of each sequence; None: bad, so empty."""
    out, end = [], 0
    for a, b in zip(offsets, offsets[1:]):
        rises = 0 <= a <= b <= T
        out.append(b - a if rises and a >= end else None)
        if rises:
            end = max(end, b)
    return out


def check(items, offsets, T, seg_len, n):
    """All segments of the accepted sequences are there once, within n slots."""
    got, status = items(len(offsets) - 1, T, seg_len, n, offsets)
    lens = accepted(offsets, T)
    want = []
    for seq, length in enumerate(lens):
        m = max(1, math.ceil((length or 0) / seg_len))
        slot = len(want)
        base = 0 if length is None else offsets[seq]
        want += [(seq, base, base, length or 0, j, m, slot) for j in range(m)]
    assert len(want) <= n, (len(want), n, offsets)
    assert got == want + [(-1, 0, 0, 0, 0, 0, 0)] * (n - len(want)), offsets
    assert bool(status) == (None in lens)
    for seq, base, first, length, j, m, slot in got:
        assert slot + m <= n and first + length <= T


def plan(B, T, H, K, V, dt):
    """Slots of the workspace, and each length of a segment that they could stand for."""
    bytes_ = binding.gdn_linear_prefill_workspace_size(B, T, H, K, V, True, dt)
    n = bytes_ // (4 * H * V * K)
    step = 128 if dt == binding.GDN_BF16 and K >= 64 else 16
    return n, [s for s in range(step, T + step, step) if -(-T // s) + B == n]


@pytest.mark.parametrize("T,H,offsets", [
    (12000, 4, [0, 11000, 1000, 12000]),  # falls in the middle: the third starts inside the first
    (6001, 5, [0, 6000, 1, 6001]),
    (6001, 5, [0, 6001, 0, 6001]),
    (6001, 5, [0, 3000, 2999, 6001]),
    (6001, 5, [0, 6001, -1, 6001]),
    (6001, 5, [0, 7000, 100, 6001]),  # one that passes the end takes nothing from the next
    (6001, 5, [5, 3000, 6000, 6001]),
])
def test_bad_offsets_stay_within_the_workspace(items, T, H, offsets):
    for K, V, dt in ((128, 128, binding.GDN_BF16), (64, 128, binding.GDN_BF16),
                     (32, 32, binding.GDN_FP32)):
        n, seg_lens = plan(len(offsets) - 1, T, H, K, V, dt)
        assert n > 0 and seg_lens  # cut
        for seg_len in (seg_lens[0], seg_lens[-1]):
            check(items, offsets, T, seg_len, n)


def test_offsets_at_random(items):
    """More sequences than a warp has lanes, some offsets moved."""
    rng = random.Random(0)
    for trial in range(12):
        T, B = rng.randint(1, 1500), rng.randint(1, 70)
        offsets = sorted(rng.randint(0, T) for _ in range(B + 1))
        for _ in range(rng.randint(0, 4)):
            offsets[rng.randrange(B + 1)] = rng.choice([rng.randint(0, T), -1, T + 1, 0, T])
        seg_len = rng.choice([16, 128, 1000])
        check(items, offsets, T, seg_len, -(-T // seg_len) + B)


def test_dense_items(items):
    got, status = items(3, 300, 128, 9)
    assert got == [(b, 0, 300 * b, 300, j, 3, 3 * b) for b in range(3) for j in range(3)]
    assert status == 0
    got, _ = items(2, 300, 300, 2)
    assert got == [(b, 0, 300 * b, 300, 0, 1, b) for b in range(2)]
