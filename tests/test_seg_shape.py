"""Which output tile a product by expert or with 4-bit operands gets (host
arithmetic): what holds for every size, and that the sizes of the GPU tests
reach the tiles that they are there for."""
import os
import shutil
import subprocess

import pytest

from tests import test_gpu_grouped as T
from tests.grouped_reference import SQUARE
from tests.test_gpu_grouped_tiles import DEPTH, ROWS, rounded

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "scaled_fp8_gemm_amd", "csrc")


@pytest.fixture(scope="module")
def tile(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = str(tmp_path_factory.mktemp("seg") / "seg_shape_check")
    subprocess.check_call([gxx, "-O1", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
                           os.path.join(HERE, "seg_shape_check.cpp"), "-o", exe])

    def ask(*words):
        r = subprocess.run([exe], input=" ".join(str(int(w) if not isinstance(w, str) else w)
                                                 for w in words),
                           capture_output=True, text=True)
        assert r.returncode == 0, (r.returncode, r.stdout)
        return r.stdout.strip()
    return ask


def by_rows(tile, lengths, n, fp4, more):
    return tile("rows", sum(lengths) + more, n, len(lengths), True, fp4, 0)


def test_all_sizes(tile):
    assert tile() == ""


@pytest.mark.parametrize("name", list(ROWS))
def test_sizes_of_the_tiles(tile, name):
    lengths, n = ROWS[name]
    for more in (0, 3, 8, 9):            # rows in no segment
        for fp4 in (False, True):
            want = "32x64" if name == "16x64" and not fp4 else name
            assert by_rows(tile, lengths, n, fp4, more) == want
            assert by_rows(tile, lengths, rounded(n, SQUARE), fp4, more) == want


@pytest.mark.parametrize("name", list(DEPTH))
def test_sizes_of_the_gradients(tile, name):
    lengths, n, k = DEPTH[name]
    assert tile("depth", n, k, len(lengths)) == name


# the sizes of test_gpu_grouped.py, with 8- and with 4-bit weights
@pytest.mark.parametrize("case,t8,t4", [(T.FEW16, "32x64", "16x64"), (T.FEW32, "32x64", "16x64"),
                                        (T.FEW64, "64x64", "64x64"), (T.WIDE64, "64x64", "64x64"),
                                        (T.MID, "128x128", "128x128"), (T.BIG, "256x256", "256x256")])
def test_sizes_of_the_parity_tests(tile, case, t8, t4):
    for more in (0, 3, 8, 9):
        assert by_rows(tile, *case, False, more) == t8
        assert by_rows(tile, *case, True, more) == t4


def test_dense_and_depths(tile):
    for (lengths, n), want in zip(T.DEEP, ("16x64", "64x64", "64x128", "128x128", "256x256")):
        assert tile("rows", sum(lengths), n, len(lengths), True, True, 0) == want
    for (m, n), want in (((130, 6800), "64x128"), ((300, 10900), "128x128"), ((520, 13907), "256x256")):
        assert tile("rows", m, n, 1, False, True, 0) == want
