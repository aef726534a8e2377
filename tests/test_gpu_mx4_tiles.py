"""Products whose tiles fill the chip in one round, on the tile shapes that are taken for them: partial tiles
on both edges, partial last slices, fewer slices than stages, stacked problems cut inside a tile.

The bounds are those of the smaller products: a sum's roundings, and one to the output's type."""

import pytest

from tests.test_gpu_mx4 import check_gemm, random_form

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M, N, K", [
    (128, 14344, 416), (100, 13000, 1056), (200, 7000, 2080), (250, 8072, 96), (65, 14344, 1280),   # 128 x 64
    (777, 4104, 800), (129, 16008, 32), (1000, 4096, 1312), (640, 6160, 2304), (385, 8200, 544),     # 128 x 128, one round
])
def test_one_round_of_tiles(M, N, K, dtype):
    a, b = random_form(M, M, K, 119, 126), random_form(N, N, K, 119, 126)
    a[1][M - 1, 0] = b[1][N - 2, -1] = 255
    check_gemm(a, b, dtype, what="one round")


@pytest.mark.parametrize("ends, N", [([140, 140, 260], 4104), ([3, 250], 6152), ([400, 401, 401, 990], 2056), ([600, 900], 3080)])
@pytest.mark.parametrize("K", [288, 1536])
def test_one_round_of_stacked_problems(ends, N, K):
    a, b = random_form(5, ends[-1] + 7, K, 119, 126), random_form(6, N * len(ends), K, 119, 126)
    a[1][ends[0] // 2, 1] = b[1][N + 9, 0] = 255
    check_gemm(a, b, "bf16", ends, what="one round stacked")
