"""Which kernel takes a 4-bit product, on the 152 SMs of a GB300."""
import pytest

SMS = 152


@pytest.fixture(scope="module")
def lib():
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops.lib()


@pytest.mark.parametrize("M,N,K,want", [
    (1, 4096, 7168, 0), (128, 57344, 8192, 0), (200, 4096, 7168, 0), (960, 4096, 2048, 0),
    (1900, 4096, 7168, 1), (2000, 5000, 8192, 1), (8192, 8192, 8192, 2), (4096, 8192, 4096, 2),
])
def test_dense(lib, M, N, K, want):
    assert lib.bwg_fp4_kernel(M, N, K, 0, 0, SMS) == want


def test_grouped(lib):
    assert lib.bwg_fp4_kernel(32768, 4096, 4096, 32, 0, SMS) == 2
    assert lib.bwg_fp4_kernel(758, 2040, 2336, 8, 0, SMS) == 1
    assert lib.bwg_fp4_kernel(758, 2048, 2336, 8, 1, SMS) == 2  # SwiGLU pairs a gate block with an up block
    # halves inside a tile of scales: the plain product, then the activation
    for M in (8, 400, 6079, 32768):
        assert lib.bwg_fp4_kernel(M, 2040, 2336, 8, 1, SMS) == lib.bwg_fp4_kernel(M, 2040, 2336, 8, 0, SMS)


def test_few_rows_never_take_pairs(lib):
    for M in (1, 17, 128):
        for N in (8, 5000, 200000):
            for K in (32, 8192):
                assert lib.bwg_fp4_kernel(M, N, K, 0, 0, SMS) == 0


@pytest.mark.parametrize("bad", [(0, 8, 32, 0, 0, SMS), (8, 0, 32, 0, 0, SMS), (8, 8, 0, 0, 0, SMS), (8, 8, 32, -1, 0, SMS),
                                 (8, 8, 32, 0, 0, 1), ((1 << 31) - 1, 8, 32, 0, 0, SMS)])
def test_invalid_arguments(lib, bad):
    assert lib.bwg_fp4_kernel(*bad) == -1
