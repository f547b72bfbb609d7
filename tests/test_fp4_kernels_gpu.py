"""The kernels of the 4-bit products, each at sizes that the library's own rule
gives to it: with many more k-blocks than its ring has stages, several tiles a
CTA or pair, and rows, columns and K off every tile."""
import numpy as np
import pytest
import torch

from test_fp4_gpu import FMTS, dev, random_fp4
from test_fp4_groups_gpu import assert_swiglu, swiglu_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops


def kernel(ops, M, N, K, G=0, swiglu=False):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return ops.lib().bwg_fp4_kernel(M, N, K, G, int(swiglu), sms), sms


# kernel -> sizes: tiles of 128 x 128, of 192 x 256 and of 192 x 512
DENSE = [(0, 1500, 2600, 8000), (0, 475, 6739, 3456), (0, 202, 21794, 2080), (1, 2001, 5003, 7904), (1, 2135, 7972, 2080),
         (2, 1738, 5713, 3872), (2, 2135, 7972, 3616), (2, 2881, 8475, 3360)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("which,M,N,K", DENSE)
def test_dense_products_are_exact(ops, which, M, N, K, fmt):
    picked, sms = kernel(ops, M, N, K)
    assert picked == which
    rows, cols, workers = ((128, 128, sms), (192, 256, sms // 2), (192, 512, sms // 2))[which]
    assert -(-M // rows) * -(-N // cols) > workers and K > 2 * 4 * 256  # the next tile, and the ring's third round
    rng = np.random.default_rng(M)
    a, A = random_fp4(ops, M, K, fmt, rng, integers=True)
    b, B = random_fp4(ops, N, K, fmt, rng, integers=True)
    want = dev(A) @ dev(B).t()  # in 64 bits
    for _ in range(3):
        assert torch.equal(ops.gemm_fp4(a, b, out_dtype=torch.float32).double(), want)
    assert ops.last_device_error() == (0, 0)


COUNTS = [700, 0, 1900, 1, 193, 2500, 385, 400]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("which,counts,N,K", [(2, COUNTS, 2040, 2336), (1, [n // 8 for n in COUNTS], 2040, 2336)])
def test_grouped_products_are_exact(ops, which, counts, N, K, fmt):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M, G = int(off[-1]), len(counts)
    assert kernel(ops, M, N, K, G)[0] == which
    rng = np.random.default_rng(M)
    a, A = random_fp4(ops, M, K, fmt, rng, offsets=off, integers=True)
    b, B = random_fp4(ops, G * N, K, fmt, rng, groups=G, integers=True)
    A, B = dev(A), dev(B)
    want = torch.cat([A[off[e]:off[e + 1]] @ B[e * N:(e + 1) * N].t() for e in range(G)])
    for _ in range(3):
        assert torch.equal(ops.grouped_gemm_fp4(a, b, out_dtype=torch.float32).double(), want)
    assert ops.last_device_error() == (0, 0)


@pytest.mark.parametrize("fmt", FMTS)
def test_fused_swiglu_of_many_tiles(ops, fmt):
    N, K, G = 1536, 2336, len(COUNTS)
    off = np.concatenate([[0], np.cumsum(COUNTS)]).astype(np.int32)
    M = int(off[-1])
    picked, sms = kernel(ops, M, N, K, G, True)
    assert picked == 2 and sum(-(-n // 192) for n in COUNTS) * 3 > sms // 2
    rng = np.random.default_rng(7)
    a, A = random_fp4(ops, M, K, fmt, rng, 2.0 ** -4 if fmt == "nvfp4" else None, offsets=off, integers=True)
    b, B = random_fp4(ops, G * N, K, fmt, rng, groups=G, integers=True)
    if fmt == "mxfp4":
        b.scales -= torch.where(b.scales == 255, 0, 4).to(torch.uint8)
    gate, up = swiglu_reference(dev(A) / 16, dev(B), off, N)
    first = ops.grouped_gemm_fp4(a, b, swiglu=True, out_dtype=torch.float32)
    assert_swiglu(first, gate, up)
    for _ in range(3):
        assert torch.equal(ops.grouped_gemm_fp4(a, b, swiglu=True, out_dtype=torch.float32), first)
    assert ops.last_device_error() == (0, 0)
