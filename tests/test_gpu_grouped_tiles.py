"""Products by expert on the tiles of 64 x 128 and, with 4-bit weights, of 32
rows: segments longer than the tile, shorter ones and empty ones under every
scaling and format; weight gradients on the tile of 256 rows in the formats
that no other test gives it.  test_seg_shape.py holds the sizes to the tiles
that they are meant for."""
import pytest

from tests.grouped_reference import BLOCK, E2M1, MX, SQUARE, TENSOR
from tests.test_gpu_grouped import run_depth, run_rows

pytestmark = pytest.mark.gpu
FORMATS = [(0, 0), (1, 0), (0, 1), (1, 1)]
FP4 = [(0, E2M1), (1, E2M1), (E2M1, E2M1)]

# tile: segment lengths, columns
ROWS = {"16x64": ([3, 0, 20, 1, 40], 70),            # 4-bit weights
        "32x64": ([60, 0, 33, 7, 32], 70),
        "64x64": ([70, 0, 64, 130, 1], 100),
        "64x128": ([70, 0, 64, 130, 1], 2313),
        "128x128": ([600, 1, 0, 300, 128], 3333),
        "256x256": ([700, 90, 513], 5381)}
# weight gradients: segment lengths in units of 128, sizes
DEPTH = {"64x64": ([2, 0, 1, 5], 130, 71),
         "256x256": ([2, 0, 1, 3, 1, 0, 1, 1], 1300, 1616)}


@pytest.fixture(scope="module")
def F():
    from scaled_fp8_gemm_amd import fp8sg
    fp8sg.lib()
    return fp8sg


def rounded(n, scaling):
    return -(-n // 128) * 128 if scaling == SQUARE else n


# fewer steps than stages, a step that ends early, more than 512 K of scales
@pytest.mark.parametrize("k", [112, 272, 1040])
@pytest.mark.parametrize("fa,fb", FORMATS)
def test_64x128_tensor(F, orc, k, fa, fb):
    lengths, n = ROWS["64x128"]
    run_rows(F, orc, lengths, n, k, TENSOR, TENSOR, fa, fb, first=3, after=5)


@pytest.mark.parametrize("k", [128, 384, 1152])
@pytest.mark.parametrize("sb", [BLOCK, SQUARE])
@pytest.mark.parametrize("fa,fb", FORMATS)
def test_64x128_block(F, orc, k, sb, fa, fb):
    lengths, n = ROWS["64x128"]
    run_rows(F, orc, lengths, rounded(n, sb), k, BLOCK, sb, fa, fb, after=9)


# K of 32, 64, 96 modulo 128: the scale bytes come from memory
@pytest.mark.parametrize("k", [96, 256, 288, 832, 1152])
@pytest.mark.parametrize("fa,fb", FORMATS + FP4)
def test_64x128_mx(F, orc, k, fa, fb):
    lengths, n = ROWS["64x128"]
    run_rows(F, orc, lengths, n, k, MX, MX, fa, fb, first=1, after=2)


@pytest.mark.parametrize("k", [96, 256, 288, 832, 1152, 2048])
@pytest.mark.parametrize("fa,fb", FP4)
def test_32x64_with_4_bit_weights(F, orc, k, fa, fb):
    lengths, n = ROWS["32x64"]
    run_rows(F, orc, lengths, n, k, MX, MX, fa, fb, first=1, after=2)


@pytest.mark.parametrize("scaling,fa,fb", [(TENSOR, 0, 1), (TENSOR, 1, 1), (BLOCK, 0, 0), (BLOCK, 1, 0),
                                           (BLOCK, 1, 1), (MX, 1, 0), (MX, 0, 1)])
def test_256x256_weight_gradients(F, orc, scaling, fa, fb):
    lengths, n, k = DEPTH["256x256"]
    run_depth(F, orc, lengths, n, k, scaling, fa, fb, "add", after=1)
