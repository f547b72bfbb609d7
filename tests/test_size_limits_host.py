"""Sizes next to 2^31, where rounding up to tiles would leave an int: refused
before anything is computed from them.  No GPU."""
import pytest

UNSUPPORTED = 3
P, Q, R, S, T = 4096, 8192, 12288, 16384, 20480  # addresses that are never read
TOP = (1 << 31) - 1
LARGE = [(1 << 31) - 32, (1 << 31) - 256, (1 << 31) - 480]  # multiples of 32: sizes that K may have


@pytest.fixture(scope="module")
def lib():
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops.lib()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,K", [(8, n) for n in LARGE] + [(n, 64) for n in LARGE + [TOP, TOP - 127]])
def test_quantize_and_read_back(lib, M, K, fmt):
    assert lib.quantize_fp4(P, 0, M, K, K, fmt, None, 1, None, 1, Q, R, None) == UNSUPPORTED
    assert lib.dequantize_fp4(Q, R, fmt, None, 1, None, 1, P, 0, M, K, K, None) == UNSUPPORTED
    assert lib.quantize_fp4(P, 0, M, K, K, fmt, None, 1, S, 3, Q, R, None) == UNSUPPORTED
    assert lib.bwg_fp4_scale_bytes(M, K, fmt, 1, 0) == -1
    assert lib.bwg_fp4_scale_bytes(M, K, fmt, 3, 1) == -1


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,N,K", [(8, 64, n) for n in LARGE] + [(n, 64, 64) for n in LARGE + [TOP]]
                         + [(8, n, 64) for n in LARGE + [TOP]])
def test_products(lib, M, N, K, fmt):
    assert lib.gemm_fp4(P, Q, None, R, S, None, fmt, T, M, N, K, N, 0, None) == UNSUPPORTED
    assert lib.grouped_gemm_fp4(P, Q, None, R, S, None, 1, fmt, T, P, 2, M, N, K, N, 0, 0, None, None) == UNSUPPORTED
    if N % 2 == 0:
        assert lib.grouped_gemm_fp4(P, Q, None, R, S, None, 1, fmt, T, P, 2, M, N, K, N, 0, 1, P, None) == UNSUPPORTED


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("H", [TOP, TOP - 1, (1 << 30) + 1])
def test_rows(lib, H, dtype):
    assert lib.moe_dispatch(P, dtype, 1, H, H, 1, Q, R, 4, S, H, None) == UNSUPPORTED
    assert lib.moe_dispatch_grad(P, dtype, 1, H, H, 1, Q, R, 4, S, H, None) == UNSUPPORTED
    assert lib.moe_combine(P, dtype, 1, H, H, 1, Q, R, S, 4, T, H, None) == UNSUPPORTED
    assert lib.moe_combine_grad(P, Q, dtype, 1, H, H, H, 1, R, S, T, 4, P, H, Q, None) == UNSUPPORTED


def test_the_largest_sizes_are_still_counted(lib):
    most = (1 << 31) - 512
    assert lib.bwg_fp4_scale_bytes(most, 64, 0, 1, 0) == most // 128 * 512
    assert lib.bwg_fp4_scale_bytes(128, most, 0, 1, 0) == most // 64 * 512
    assert lib.bwg_fp4_scale_bytes(most, 64, 0, 1, 1) == (most + 127) // 128 * 512
