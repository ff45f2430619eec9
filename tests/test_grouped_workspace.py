"""The grouped product's workspace stays within what the header states."""
import pytest

from post_weight_quantization_hessian_b200 import build, slim


@pytest.fixture(scope="module")
def lib():
    build.build()
    return slim._lib()


@pytest.mark.parametrize("E, m, n, group, xdtype, gathered, R", [
    (1, 4096, 4096, 128, 1, 0, 4096), (8, 11008, 4096, 64, 1, 1, 8192), (1024, 8192, 65472, 64, 1, 0, 33 * 1024),
    (1024, 256, 11264, 32, 0, 0, 40000), (60, 140, 65472, 64, 1, 0, 2040), (2, 20000, 16384, 128, 1, 0, 90),
    (3, 100, 128, 128, 0, 1, 40), (1024, 1 << 20, 32, 32, 1, 1, 1 << 20)])
def test_workspace_is_bounded(lib, E, m, n, group, xdtype, gathered, R):
    k, slots = n // group, min(E, R // 33)
    boxes = -(-n // 64) + -(-k // 8)
    tiles = slots * -(-m // 128) * boxes * 128 * 64 * 2
    parts = 16 * R * k + (6 * R * n if xdtype == 0 else 2 * R * n if gathered else 0)
    got = lib.slim_dequant_grouped_gemm_workspace_bytes(E, m, n, group, 2, xdtype, gathered, R)
    assert got <= min(tiles, 1 << 30) + parts + 3 * 256
    assert got >= parts + min(tiles, boxes * 128 * 64 * 2)


@pytest.mark.parametrize("R, xdtype, gathered, want", [(32, 1, 0, 0), (32, 1, 1, 0), (32, 0, 0, 6 * 32 * 4096)])
def test_workspace_of_few_rows(lib, R, xdtype, gathered, want):
    assert lib.slim_dequant_grouped_gemm_workspace_bytes(4, 4096, 4096, 128, 2, xdtype, gathered, R) == want
