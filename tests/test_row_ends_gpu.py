"""Rows of D that end inside 16 bytes: a product writes its columns and nothing of
what lies between them and the next row, by every kernel that stores boxes of D.
Integers of magnitude 2: every sum is exact."""
import ctypes

import pytest
import torch

from gpu_util import forced_kernel

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
COLS = [1, 7, 113, 114, 190, 250, 257, 383, 516, 1030]


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops


@pytest.fixture(autouse=True)
def no_device_error(ops):
    yield
    assert ops.last_device_error() == (0, 0)


def ints(rows, cols, dtype, seed, most=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = -(-cols // 8) * 8
    return torch.randint(-most, most + 1, (rows, ld), generator=g, device="cuda").to(dtype)[:, :cols]


def between(M, N, dtype):
    """(buffer, D): rows of 16 bytes with 7s around D, which ends where the last row does."""
    ld = -(-N // 8) * 8
    buf = torch.full((M * ld + 64,), 7.0, dtype=dtype, device="cuda")
    return buf, buf[:M * ld].view(M, ld)[:, :N]


def check(buf, d, want, what):
    assert torch.equal(d.double(), want), what
    d.fill_(7.0)
    assert bool((buf == 7.0).all()), what


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("kind,M", [("2cta_2c", 700), ("2cta", 300), ("1cta", 300), ("2cta_mc", 600), (None, 40), (None, 128)])
def test_dense(ops, kind, M, out):
    dtype = torch.float16 if out == "fp16" else torch.bfloat16
    for transposed in (False, True):
        for N in COLS:
            a, b = ints(M, 200, dtype, N), ints(200, N, dtype, N + 1, 1)
            want = a.double() @ b.double()
            if out != "fp32":
                want = want.to(DT[out]).double()
            w = torch.zeros(N, 200, dtype=dtype, device="cuda").copy_(b.t()) if transposed else b
            buf, d = between(M, N, DT[out])
            with forced_kernel(kind):
                ops.gemm(a, w, out=d, b_transposed=transposed)
            check(buf, d, want, (kind, M, N, out, transposed))


@pytest.mark.parametrize("out", list(DT))
def test_few_rows_of_every_schedule(ops, out, monkeypatch):
    """The small-M kernel: whole tiles (one and several a CTA), cluster split, stream-K, other tile widths."""
    dtype = torch.float16 if out == "fp16" else torch.bfloat16
    for env, N, K in (({}, 113, 4096), ({"BWG_SMALL_M_SPLIT": "0"}, 113, 640), ({}, 19463, 640), ({}, 24999, 128),
                      ({"BWG_STREAMK": "0"}, 24999, 640),
                      ({"BWG_STREAMK": "1"}, 1001, 2048), ({"BWG_SMALL_M_TILE_N": "80"}, 250, 640),
                      ({"BWG_SMALL_M_TILE_N": "48"}, 250, 640)):
        for M in (1, 17, 72):
            for k, v in env.items():
                monkeypatch.setenv(k, v)
            a, b = ints(M, K, dtype, N), ints(K, N, dtype, N + 1, 1)
            want = (a.float() @ b.float()).to(DT[out]).double()  # integers below 2^24
            buf, d = between(M, N, DT[out])
            ops.gemm(a, b, out=d)
            for k in env:
                monkeypatch.delenv(k)
            check(buf, d, want, (env, M, N, K, out))


def test_few_rows_without_allocation(ops):
    L = ctypes.CDLL(ops.LIB_PATH)  # (the Python calls have no such form)
    f, vp, i = L.gemm_bf16_small_m_noalloc, ctypes.c_void_p, ctypes.c_int
    f.argtypes, f.restype = [vp, vp, vp, i, i, i, i, i, i, i, vp], i
    for N in (1, 113, 1001):
        a, b = ints(17, 640, torch.bfloat16, N), ints(640, N, torch.bfloat16, N + 1, 1)
        buf, d = between(17, N, torch.float32)
        assert f(a.data_ptr(), b.data_ptr(), d.data_ptr(), 17, N, 640, 640, b.stride(0), d.stride(0), 1,
                 torch.cuda.current_stream().cuda_stream) == 0
        check(buf, d, a.double() @ b.double(), N)


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("K,M", [(70, 40), (153, 300), (700, 1000), (9000, 300), (100, 4400)])
def test_transposed(ops, K, M, out):
    """Both tile forms, with and without slices."""
    dtype = torch.float16 if out == "fp16" else torch.bfloat16
    for N in COLS + [4397]:
        a, b = ints(K, M, dtype, N), ints(K, N, dtype, N + 1, 1)
        want = (a.float().t() @ b.float()).to(DT[out]).double()
        buf, d = between(M, N, DT[out])
        ops.gemm(a, b, out=d, a_transposed=True)
        check(buf, d, want, (K, M, N, out))


@pytest.mark.parametrize("out", list(DT))
def test_transposed_one_row(ops, out):
    """D of one row, new and in a buffer that ends with it."""
    for N in (1, 113, 257):
        a, b = ints(700, 1, torch.bfloat16, N), ints(700, N, torch.bfloat16, N + 1, 1)
        want = (a.float().t() @ b.float()).to(DT[out]).double()
        assert torch.equal(ops.gemm(a, b, out_dtype=DT[out], a_transposed=True).double(), want)
        buf = torch.full((N + 64,), 7.0, dtype=DT[out], device="cuda")
        d = buf[:N].view(1, N)
        ops.gemm(a, b, out=d, a_transposed=True)
        check(buf, d, want, (N, out))
