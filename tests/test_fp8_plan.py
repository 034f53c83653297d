"""Which kernel the 8-bit products take (bnn_probe_fp8_plan, host only): the sizes that the GPU tests use reach
every kernel and shape on a device of 148 SMs, and the split of k, with it the order of a sum, depends on the
device's SM count as include/bnn.h says."""
import ctypes as C
import os

import pytest

from conftest import ROOT

EMPTY, REGISTERS, LANES, TILES = 0, 1, 2, 3


@pytest.fixture(scope="module")
def probe():
    from ternary_neural_net_b200 import bnn
    f = bnn.lib().bnn_probe_fp8_plan
    f.argtypes = [C.c_int64] * 4 + [C.c_int] + [C.c_void_p] * 4
    f.restype = C.c_int
    return f


@pytest.fixture(scope="module")
def plan(probe):
    def call(rows, n, k, groups=0, sms=148):
        out = (C.c_int * 4)()
        at = [C.addressof(out) + 4 * i for i in range(4)]
        assert probe(rows, n, k, groups, sms, *at) == 0
        return tuple(out)
    return call


# (rows, n, k, groups) -> (kernel, rows of a tile, columns of a tile, split)
PLANS = {
    (5, 300, 0, 0): (EMPTY, 0, 0, 1),
    (1, 1024, 1000, 0): (REGISTERS, 8, 16, 1),
    (8, 4096, 8192, 0): (REGISTERS, 8, 16, 1),
    (1, 28672, 1280, 0): (LANES, 16, 128, 1),
    (5, 28672, 1200, 0): (LANES, 16, 128, 1),
    (9, 131, 260, 0): (LANES, 16, 128, 1),
    (16, 300, 640, 0): (LANES, 16, 128, 2),
    (12, 400, 1024, 0): (LANES, 16, 128, 4),
    (16, 1000, 8192, 0): (LANES, 16, 128, 8),
    (16, 40000, 300, 0): (LANES, 16, 128, 1),
    (30, 40000, 300, 0): (LANES, 32, 128, 1),
    (24, 300, 640, 0): (LANES, 32, 128, 2),
    (24, 400, 1024, 0): (LANES, 32, 128, 4),
    (24, 700, 4100, 0): (LANES, 32, 128, 8),
    (32, 129, 4100, 0): (LANES, 32, 128, 8),
    (20, 500, 8192, 0): (LANES, 32, 128, 8),
    (64, 1000, 8192, 0): (TILES, 128, 32, 1),
    (300, 2000, 4100, 0): (TILES, 128, 64, 1),
    (3000, 9100, 1100, 0): (TILES, 128, 128, 1),
    (1101, 2304, 2000, 0): (TILES, 256, 256, 1),
    (1101, 2307, 2000, 0): (TILES, 256, 256, 1),
    (2048, 4600, 2000, 0): (TILES, 256, 256, 1),
    (200, 300, 2000, 20): (LANES, 16, 128, 1),
    (200, 300, 2000, 8): (LANES, 32, 128, 1),
    (900, 700, 2000, 4): (TILES, 128, 128, 1),
    (4000, 4100, 2000, 4): (TILES, 128, 256, 1),
    (300, 2707, 2000, 8): (TILES, 128, 256, 1),
}


@pytest.mark.parametrize("sizes", list(PLANS))
def test_plans(plan, sizes):
    assert plan(*sizes) == PLANS[sizes]


def test_every_kernel_and_shape_has_a_size():
    dense = {p for s, p in PLANS.items() if s[3] == 0}
    assert dense == {(EMPTY, 0, 0, 1), (REGISTERS, 8, 16, 1), *((LANES, r, 128, s) for r in (16, 32) for s in (1, 2, 4, 8)),
                     *((TILES, 128, c, 1) for c in (32, 64, 128)), (TILES, 256, 256, 1)}
    grouped = {p for s, p in PLANS.items() if s[3] > 0}
    assert grouped == {(LANES, 16, 128, 1), (LANES, 32, 128, 1), (TILES, 128, 128, 1), (TILES, 128, 256, 1)}


def test_the_split_depends_on_the_sm_count(plan):
    assert plan(16, 4700, 8192, sms=148)[3] == 8 and plan(16, 4700, 8192, sms=132)[3] == 4
    text = " ".join(open(os.path.join(ROOT, "include", "bnn.h")).read().replace("*", " ").split())
    assert "sizes alone decide" not in text
    assert "the sizes and the device's number of SMs decide" in text


def test_probe_refusals(probe):
    out = (C.c_int * 4)()
    at = [C.addressof(out) + 4 * i for i in range(4)]
    for bad in ((0, 1, 1, 0, 148), (1, 0, 1, 0, 148), (1, 1, -1, 0, 148), (1, 1, 1, -1, 148), (1, 1, 1, 0, 1),
                (1 << 31, 1, 1, 0, 148), (1, 1 << 31, 1, 0, 148), (1, 1, (1 << 24) + 1, 0, 148), (1, 1, 1, 1025, 148)):
        assert probe(*bad, *at) == 1, bad
    for i in range(4):
        assert probe(1, 1, 1, 0, 148, *[None if j == i else p for j, p in enumerate(at)]) == 1
