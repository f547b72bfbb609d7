"""Products over no depth write zeros: rows of more than 2^31 bytes, whole and up
to their end, with what lies between them left as it was."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops


def filled(rows, cols, ld, dtype):
    return torch.full((rows, ld), 7.0, dtype=dtype, device="cuda")


def check(d, cols):
    for row in d:
        assert int(torch.count_nonzero(row[:cols])) == 0 and bool((row[cols:] == 7.0).all())


def test_gradients_of_a_gated_block(ops):
    """dGU of 2 x (2^30 + 16) in 16 bits."""
    M, N = 2, (1 << 30) + 16
    dh = torch.ones(M, N // 2, dtype=torch.bfloat16, device="cuda")
    d = filled(M, N, N + 8, torch.bfloat16)
    assert ops.lib().gemm_swiglu_grad(dh.data_ptr(), None, None, d.data_ptr(), 0, 0, M, N, 0, N // 2, 8, N, N + 8,
                                      torch.cuda.current_stream().cuda_stream) == 0
    check(d, N)
    assert ops.last_device_error() == (0, 0)


def test_a_dense_product(ops):
    """D of 2 x (2^29 + 8) in FP32."""
    M, N = 2, (1 << 29) + 8
    d = filled(M, N, N + 8, torch.float32)
    e = dict(dtype=torch.bfloat16, device="cuda")
    ops.gemm(torch.empty(M, 0, **e), torch.empty(0, N, **e), out=d[:, :N])
    check(d, N)
    assert ops.last_device_error() == (0, 0)
