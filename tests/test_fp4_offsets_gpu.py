"""Broken group offsets in the grouped 4-bit product: clamped into the rows and
made non-decreasing, the same in every form of it, and reported."""
import numpy as np
import pytest
import torch

from test_fp4_gpu import FMTS, random_fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,swiglu", [(48, False), (512, True), (60, True)])
@pytest.mark.parametrize("offsets", [[0, 2, 5, 3], [0, 2, 5, -1], [0, 5, 2, 9], [0, 4, 8, 40], [0, 7, 300, 2]])
def test_clamped_offsets_give_their_groups(ops, offsets, N, swiglu, fmt):
    M, G, K = 12, 3, 96
    good = np.clip(np.maximum.accumulate(offsets), 0, M).astype(np.int32)
    rng = np.random.default_rng(3)
    a, _ = random_fp4(ops, M, K, fmt, rng, offsets=good, integers=True)
    b, _ = random_fp4(ops, G * N, K, fmt, rng, groups=G, integers=True)
    n_out = N // 2 if swiglu else N
    want, got = (torch.full((M, n_out), 9.0, device="cuda") for _ in range(2))
    ops.grouped_gemm_fp4(a, b, swiglu=swiglu, out=want)
    assert ops.last_device_error() == (0, 0)
    assert bool((want[int(good[-1]):] == 9).all())
    broken = ops.Fp4Matrix(a.codes, a.scales, fmt, None, torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    ops.grouped_gemm_fp4(broken, b, swiglu=swiglu, out=got)
    status, word = ops.last_device_error()
    assert status == 1 and word >> 56 == 2
    assert torch.equal(got, want)
