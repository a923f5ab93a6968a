"""The shapes that the GPU tests run reach every form of a product that the choice of tiles knows; no
GPU: the choice (csrc/linear_tiles.h) is compiled by the host compiler and asked."""
import ctypes
import math
import os
import random
import subprocess

import pytest

from tests.linear_forms import SHAPES, forms
from tile_signaled_grouped_gb300 import build as B

SMS = 152


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    d = tmp_path_factory.mktemp("tiles")
    src, lib = d / "tiles.cpp", d / "tiles.so"
    src.write_text(f'''#include "{os.path.join(B.CSRC, "linear_tiles.h")}"
extern "C" void choose(int I, int J, int nk, int b_mn, int aligned, int sms, int* out) {{
  const moe::TileChoice c = moe::choose_tiles(I, J, nk, b_mn != 0, aligned != 0, sms);
  out[0] = c.bn, out[1] = c.splits;
}}
''')
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", str(src), "-o",
                    str(lib)], check=True)
    f, out = ctypes.CDLL(str(lib)).choose, (ctypes.c_int * 2)()

    def ask(I, J, k, b_mn, aligned):
        f(I, J, (k + 63) // 64, int(b_mn), int(aligned), SMS, out)
        return out[0], out[1]

    return ask


def test_the_shapes_reach_every_form(choose):
    reached = set().union(*(forms(choose, *s) for s in SHAPES))
    rng = random.Random(1)
    size = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))  # noqa: E731
    known = set()
    for _ in range(60000):
        M, N, K = size(1, 8192), size(1, 8192), size(1, 8192)
        if rng.random() < 0.5:
            N, K = (N + 7) // 8 * 8, (K + 7) // 8 * 8
        known |= forms(choose, M, N, K)
    assert len(known) > 60
    assert known <= reached, sorted(known - reached)


def test_a_choice_is_one_the_kernels_take(choose):
    """Powers of two: 16 to 256 columns (64 at least where B is read along its rows), parts only of
    up to 128 columns and of two blocks of k or more each."""
    rng = random.Random(2)
    for _ in range(20000):
        I, J, k = (int(math.exp(rng.uniform(0.0, 10.0))) for _ in range(3))
        b_mn = rng.random() < 0.5
        bn, parts = choose(I, J, k, b_mn, rng.random() < 0.5)
        if bn == -1:
            assert parts == 1
            continue
        assert bn in (16, 32, 64, 128, 256) and parts in (1, 2, 4, 8)
        assert bn >= 64 or (not b_mn and bn >= J)
        assert parts == 1 or (bn <= 128 and (k + 63) // 64 >= 2 * parts)
