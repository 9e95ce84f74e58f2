"""The plans of the tiled Newton-Schulz path, compiled for the host: the sizes
that the GPU tests run reach every kernel instance that any call launches, and
the slices of a cut product lie inside the workspace."""
import ctypes
import math
import os
import random
import subprocess

import pytest

from tests import emulation
from tests.test_gpu_muon import LARGE, SHAPES

SRC = os.path.join(os.path.dirname(os.path.abspath(emulation.__file__)), "muon_plan.cpp")

pytestmark = pytest.mark.skipif(not emulation.available(), reason="no host C++ compiler")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "muon_plan.so")
    subprocess.run([emulation._compiler(), "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared", "-o", so, SRC],
                   check=True)
    lib = ctypes.CDLL(so)
    lib.emu_muon_plan.argtypes = [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_int64)] * 2

    def of(shape):
        out, size = (ctypes.c_int64 * 24)(), ctypes.c_int64(0)
        one = lib.emu_muon_plan(*shape, out, ctypes.byref(size)) == 0
        return None if one else [list(out[8 * i:8 * i + 8]) for i in range(3)], size.value

    return of


def instances(plan, shape):
    """(product, tile, deep, how its tiles are cut) of every launch of a call."""
    products = plan(shape)[0] or ()
    return {(name, p[0], bool(p[1]), "whole" if not p[3] else "cut" if not p[2] else "whole, then cut")
            for name, p in zip(("gram", "poly", "apply"), products)}


def sizes(count):
    rng = random.Random(5)
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return [(rng.choice((1, 1, 1, 2, 3, 4, 6, 8, 30)), log(1, 6000), log(1, 6000)) for _ in range(count)]


def test_the_gpu_tests_reach_every_instance(plan):
    tested = set().union(*(instances(plan, s) for s in SHAPES + LARGE))
    for s in sizes(20000):
        assert instances(plan, s) <= tested, s
    # cuts over several matrices, whose last tiles are not the first matrix's
    for name in ("gram", "poly", "apply"):
        assert any(s[0] > 1 and i[0] == name and "cut" in i[3] for s in LARGE for i in instances(plan, s)), name


def test_slices_cover_k_and_fit_the_workspace(plan):
    for shape in SHAPES + LARGE + sizes(5000) + [(1, 3, 1 << 20), (65535, 33, 40), (1, 16384, 20000)]:
        products, size = plan(shape)
        if products is None:
            assert size == 0
            continue
        n, m = sorted(shape[1:])
        np_, mp = products[2][6], products[2][7]
        assert np_ >= n and mp >= m and np_ % 64 == 0 and mp % 64 == 0
        planes = shape[0] * (4 * np_ * mp + 2 * np_ * np_) * 4
        for (tile, _, full, rest, slices, cut, lp, rp), k in zip(products, (mp, np_, np_)):
            assert lp % tile == 0 and rp % tile == 0 and full >= 0 and rest >= 0
            if rest:
                assert (slices - 1) * cut < k // 32 <= slices * cut  # none empty, none missing
                # a slice's sums: each of 256 threads' accumulators
                assert planes + rest * slices * 256 * (64 if tile < 128 else 256) <= size, shape
