"""The grouped product's walk over tiles, on the CPU: the kernels' own search (p24_f8_groups.hpp) with its wave
instructions emulated.  Every row of every expert is computed once for each row block, and whatever the offsets hold
no tile lies outside the output and no block goes on without end."""
import ctypes
import os
import random
import subprocess

import pytest


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    here = os.path.dirname(os.path.abspath(__file__))
    so = str(tmp_path_factory.mktemp("walk") / "group_walk.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", os.path.join(here, "host_model", "group_walk.cpp"),
                    "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.group_walk.restype = lib.group_few.restype = ctypes.c_long
    i, ip = ctypes.c_int, ctypes.POINTER(ctypes.c_int)
    lib.group_walk.argtypes = [i, ip, i, i, i, i, ip]
    lib.group_few.argtypes = [ip, i, i, ip]

    def call(bn, offsets, rows, nbm=1, fit=None):
        """(what is wrong, how often each row is computed); without `fit` the kernel for few rows."""
        cover = (i * max(rows, 1))()
        at, experts = (i * len(offsets))(*offsets), len(offsets) - 1
        bad = lib.group_few(at, experts, rows, cover) if fit is None else lib.group_walk(bn, at, experts, rows, nbm, fit, cover)
        return bad, list(cover)[:rows]
    return call


def _sums(counts, first=0):
    out = [first]
    for c in counts:
        out.append(out[-1] + c)
    return out


@pytest.mark.parametrize("bn", [32, 64, 192, 256])
@pytest.mark.parametrize("counts,nbm", [([1], 1), ([0, 0, 5], 3), ([300, 0, 257, 1], 9), ([2] * 70 + [0] * 60 + [3] * 5, 2),
                                        ([0] * 130 + [640, 7], 5)])
def test_every_row_once(walk, bn, counts, nbm):
    """Rows of the experts once a row block, others never; one round of blocks, and blocks that go from tile to tile."""
    for first, behind in ((0, 0), (2, 3)):
        rows = first + sum(counts) + behind
        for fit in (8, 256):
            bad, cover = walk(bn, _sums(counts, first), rows, nbm, fit)
            assert bad == 0
            assert cover == [0] * first + [nbm] * sum(counts) + [0] * behind
        if bn == 32:
            bad, cover = walk(bn, _sums(counts, first), rows)
            assert bad == 0 and cover == [0] * first + [1] * sum(counts) + [0] * behind


def test_offsets_outside_the_rows(walk):
    """Clipped to the rows."""
    bad, cover = walk(64, [-5, 20, 20, 1 << 30], 50, 3, 8)
    assert bad == 0 and cover == [3] * 50
    bad, cover = walk(64, [-(1 << 31), -7, 60, (1 << 31) - 1], 50, 3, 8)
    assert bad == 0 and cover == [3] * 50


FALLING = [[0, 3000] * 100 + [0], [0, 3000] + [1500, 2500] * 40, [100, 0, 3000], [0] * 70 + [3000, 0, 3000],
           [3000] * 65 + [0] * 65 + [3000], [(1 << 31) - 1, -(1 << 31)] * 30]


@pytest.mark.parametrize("bn", [64, 256])
@pytest.mark.parametrize("offsets", FALLING, ids=range(len(FALLING)))
def test_falling_offsets_reach_nothing(walk, offsets, bn):
    """Ranges that overlap: more tiles than the launch allows for.  None of them is computed; by the kernel for few rows
    some are, all inside."""
    for fit in (16, 1024):
        bad, cover = walk(bn, offsets, 3000, 1, fit)
        assert bad == 0 and cover == [0] * 3000
    assert walk(32, offsets, 3000)[0] == 0


def test_random_offsets_stay_inside(walk):
    rng = random.Random(1)
    for _ in range(12):
        rows, experts = rng.randint(1, 2000), rng.randint(1, 150)
        offsets = [rng.randint(-100, rows + 100) for _ in range(experts + 1)]
        if rng.random() < 0.5:
            offsets.sort()
        bad, cover = walk(rng.choice([32, 64, 192]), offsets, rows, rng.randint(1, 4), rng.choice([8, 24, 512]))
        assert bad == 0 and max(cover) <= 4
        assert walk(32, offsets, rows)[0] == 0
