"""Refusals of the gated block's calls, of 8-bit matrices and of products with a
transposed left operand: by the library before it looks for a GPU, and by the
Python calls before they reach the library.  No GPU."""
import contextlib
import types

import pytest
import torch

from blackwell_tensor_core_gb300 import ops
from test_ops_host import BIG, cuda, devices, rec, wide  # noqa: F401 - fixtures

OK, INVALID, ALIGNMENT, UNSUPPORTED = 0, 1, 2, 3
A, B, C, D, E = (4096 * i for i in range(1, 6))  # addresses that are never read
TOP = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    from blackwell_tensor_core_gb300 import build
    build.build()
    return ops.lib()


# ------------------------------------------------------------ the library ---

def forward(lib, x=A, w=B, h=C, codes=None, scales=None, dtype=0, nt=0, M=64, N=128, K=64, ldx=64, ldw=128, ldh=64):
    return lib.gemm_swiglu(x, w, h, codes, scales, dtype, nt, M, N, K, ldx, ldw, ldh, None)


def backward(lib, dh=A, x=B, w=C, dgu=D, dtype=0, nt=0, M=64, N=128, K=64, lddh=64, ldx=64, ldw=128, ldd=128):
    return lib.gemm_swiglu_grad(dh, x, w, dgu, dtype, nt, M, N, K, lddh, ldx, ldw, ldd, None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(h=None), INVALID), (dict(dtype=1), INVALID),
    (dict(dtype=7), INVALID), (dict(M=-1), INVALID), (dict(N=-16), INVALID), (dict(K=-1), INVALID),
    (dict(ldx=56), INVALID), (dict(ldw=120), INVALID), (dict(ldh=56), INVALID), (dict(nt=1, ldw=56), INVALID),
    (dict(codes=D), INVALID), (dict(scales=D), INVALID), (dict(x=A + 8), ALIGNMENT), (dict(w=B + 2), ALIGNMENT),
    (dict(h=C + 8), ALIGNMENT), (dict(ldx=68), ALIGNMENT), (dict(ldw=132), ALIGNMENT), (dict(ldh=68), ALIGNMENT),
    (dict(N=120, ldw=128), ALIGNMENT), (dict(codes=D + 8, scales=E), ALIGNMENT), (dict(codes=D, scales=E + 2), ALIGNMENT),
    (dict(M=TOP), UNSUPPORTED), (dict(K=TOP, ldx=TOP), UNSUPPORTED), (dict(N=TOP - 15, ldw=TOP), UNSUPPORTED),
    (dict(M=0), OK), (dict(N=0), OK),
])
def test_forward_refusals(lib, change, status):
    assert forward(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(dh=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(dgu=None), INVALID),
    (dict(dtype=1), INVALID), (dict(lddh=56), INVALID), (dict(ldx=56), INVALID), (dict(ldw=120), INVALID),
    (dict(ldd=120), INVALID), (dict(dh=A + 8), ALIGNMENT), (dict(dgu=D + 8), ALIGNMENT), (dict(lddh=68), ALIGNMENT),
    (dict(ldd=132), ALIGNMENT), (dict(N=120), ALIGNMENT), (dict(M=TOP), UNSUPPORTED), (dict(M=0), OK), (dict(N=0), OK),
])
def test_backward_refusals(lib, change, status):
    assert backward(lib, **change) == status


def test_grouped_refusals(lib):
    p, hold = ops._ptr_array([B, C])
    q, hold2 = ops._ptr_array([B, None])
    odd, hold3 = ops._ptr_array([B, C + 4])

    def keep(w=p, h=D, codes=E, scales=A, off=B, G=2, M=64, N=128, K=64, dtype=0):
        return lib.grouped_gemm_swiglu_keep(A, w, h, codes, scales, off, dtype, 0, G, M, N, K, None)

    def grad(w=p, dh=D, dgu=E, off=B, G=2, M=64, N=128, K=64, dtype=0):
        return lib.grouped_gemm_swiglu_grad(dh, A, w, dgu, off, dtype, 0, G, M, N, K, None)

    for call in (keep, grad):
        assert call(off=None) == call(w=q) == call(G=-1) == call(dtype=1) == INVALID
        assert call(w=odd) == call(N=120) == call(K=60) == ALIGNMENT
        assert call(M=TOP) == UNSUPPORTED
        assert call(G=0) == call(M=0) == call(N=0) == OK
    assert keep(codes=None) == keep(scales=None) == keep(h=None) == INVALID
    assert grad(dh=None) == grad(dgu=None) == INVALID
    del hold, hold2, hold3


def test_int8_refusals(lib):
    def put(x=A, dtype=0, M=8, N=64, ld=64, parts=1, codes=B, scales=C):
        return lib.quantize_int8(x, dtype, M, N, ld, parts, codes, scales, None)

    def back(y=A, dtype=0, M=8, N=64, ld=64, parts=1, codes=B, scales=C):
        return lib.dequantize_int8(codes, scales, parts, y, dtype, M, N, ld, None)

    for call, m in ((put, "x"), (back, "y")):
        assert call(**{m: None}) == call(codes=None) == call(scales=None) == INVALID
        assert call(dtype=3) == call(M=-1) == call(N=-1) == call(ld=63) == INVALID
        assert call(parts=0) == call(parts=3) == call(N=63, parts=2) == INVALID
        assert call(**{m: A + 1}) == call(scales=C + 2) == ALIGNMENT
        assert call(N=TOP, ld=TOP) == UNSUPPORTED
        assert call(M=0) == call(N=0) == OK

    def grad(dh=A, codes=B, scales=C, dgu=D, h=E, dtype=0, M=8, I=64, lddh=64, ldd=128, ldh=64):
        return lib.swiglu_grad_int8(dh, codes, scales, dgu, h, dtype, M, I, lddh, ldd, ldh, None)

    assert grad(dh=None) == grad(codes=None) == grad(scales=None) == grad(dgu=None) == INVALID
    assert grad(dtype=1) == grad(lddh=56) == grad(ldd=120) == grad(ldh=56) == grad(M=-1) == INVALID
    assert grad(I=60) == grad(dh=A + 8) == grad(codes=B + 8) == grad(ldd=132) == grad(lddh=68) == ALIGNMENT
    assert grad(h=E + 8) == grad(ldh=68) == ALIGNMENT
    assert grad(I=1 << 30, lddh=TOP, ldd=TOP, ldh=TOP) == UNSUPPORTED
    assert grad(M=0) == grad(I=0) == OK


def test_transposed_operand_refusals(lib):
    def dense(a=A, b=B, d=C, dtype=0, out=0, M=64, N=128, K=64, lda=64, ldb=128, ldd=128):
        return lib.gemm_tn(a, b, d, dtype, out, M, N, K, lda, ldb, ldd, None, 0, None)

    assert dense(a=None) == dense(b=None) == dense(d=None) == dense(dtype=1) == dense(out=5) == INVALID
    assert dense(lda=56) == dense(ldb=120) == dense(ldd=120) == dense(K=-1) == INVALID
    assert dense(a=A + 8) == dense(d=C + 8) == dense(lda=68) == dense(ldb=132) == dense(ldd=132) == ALIGNMENT
    assert dense(out=1, ldd=130) == ALIGNMENT
    assert dense(M=TOP, lda=TOP) == dense(K=TOP) == dense(N=TOP, ldb=TOP, ldd=TOP) == UNSUPPORTED
    assert dense(M=0) == dense(N=0) == OK

    def grouped(a=A, b=B, d=C, off=D, dtype=0, out=0, G=2, M=64, N=128, K=64):
        return lib.grouped_gemm_tn(a, b, d, off, dtype, out, G, M, N, K, None, 0, None)

    assert grouped(off=None) == grouped(a=None) == grouped(G=-1) == INVALID
    assert grouped(M=60) == grouped(N=124) == ALIGNMENT
    assert grouped(G=0) == grouped(M=0) == OK


# ------------------------------------------------------- the Python calls ---

def int8(rows, cols, parts=1, dev="cuda:0"):
    return ops.Int8Matrix(cuda(rows, cols, dtype=torch.int8, dev=dev),
                          cuda(rows, ops._int8_blocks(cols, parts), dtype=torch.float32, dev=dev), parts)


def calls(dev="cuda:0"):
    """Every call with operands that it takes, and the names that the library is called by."""
    def m(*shape, **k):
        return cuda(*shape, dev=dev, **k)
    off = cuda(3, dtype=torch.int32, dev=dev)
    return {
        "gemm_swiglu": (lambda **s: ops.gemm_swiglu(m(4, 64), m(64, 128), **s), ["gemm_swiglu"]),
        "gemm_swiglu keep": (lambda **s: ops.gemm_swiglu(m(4, 64), m(64, 128), keep_int8=True, **s), ["gemm_swiglu"]),
        "grouped keep": (lambda **s: ops.grouped_gemm(m(4, 64), [m(64, 128)] * 2, off, swiglu=True, keep_int8=True, **s),
                         ["grouped_gemm_swiglu_keep"]),
        "swiglu_grad": (lambda **s: ops.swiglu_grad(m(4, 64), int8(4, 128, 2, dev), **s), ["swiglu_grad_int8"]),
        "grad": (lambda **s: ops.gemm_swiglu_grad(m(4, 64), m(4, 64), m(64, 128), **s),
                 ["gemm_swiglu_grad", "gemm_bf16_nt", "bwg_tn_workspace", "gemm_tn"]),
        "grad nt": (lambda **s: ops.gemm_swiglu_grad(m(4, 64), m(4, 64), m(128, 64), b_transposed=True, **s),
                    ["gemm_swiglu_grad", "gemm_bf16", "bwg_tn_workspace", "gemm_tn"]),
        "grad kept": (lambda **s: ops.gemm_swiglu_grad(m(4, 64), int8(4, 64, 1, dev), m(64, 128),
                                                       kept=int8(4, 128, 2, dev), with_h=True, **s),
                      ["dequantize_int8", "swiglu_grad_int8", "gemm_bf16_nt", "bwg_tn_workspace", "gemm_tn"]),
        "grad dx": (lambda **s: ops.gemm_swiglu_grad(m(4, 64), int8(4, 64, 1, dev), m(64, 128),
                                                     kept=int8(4, 128, 2, dev), need_dw=False, **s),
                    ["swiglu_grad_int8", "gemm_bf16_nt"]),
        "experts grad": (lambda **s: ops.grouped_gemm_swiglu_grad(m(4, 64), m(4, 64), [m(64, 128)] * 2, off, **s),
                         ["grouped_gemm_swiglu_grad", "grouped_gemm_bf16_nt", "bwg_tn_workspace", "grouped_gemm_tn"]),
        "quantize_int8": (lambda **s: ops.quantize_int8(m(4, 65), **s), ["quantize_int8"]),
        "dequantize_int8": (lambda **s: ops.dequantize_int8(int8(4, 65, 1, dev), **s), ["dequantize_int8"]),
        "gemm a_transposed": (lambda **s: ops.gemm(m(4, 64), m(4, 128), a_transposed=True, **s),
                              ["bwg_tn_workspace", "gemm_tn"]),
        "wgrad": (lambda **s: ops.grouped_gemm_wgrad(m(4, 64), m(4, 128), off, **s),
                  ["bwg_tn_workspace", "grouped_gemm_tn"]),
    }


NAMES = ["gemm_swiglu", "gemm_swiglu keep", "grouped keep", "swiglu_grad", "grad",
         "grad nt", "grad kept", "grad dx", "experts grad", "quantize_int8",
         "dequantize_int8", "gemm a_transposed", "wgrad"]


def test_every_call_is_listed(rec):  # noqa: F811
    assert NAMES == list(calls())


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("name", NAMES)
def test_calls_run_on_their_tensors_device(devices, name, index):  # noqa: F811
    call, names = calls("cuda:%d" % index)[name]
    call()
    assert devices == [(n, index) for n in names]
    assert torch._C._cuda_getDevice() == 0


@pytest.mark.parametrize("name", NAMES)
def test_streams_of_another_device_are_refused(devices, name, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    call, names = calls()[name]
    with pytest.raises(ValueError):
        call(stream=types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=7))
    assert [n for n, _ in devices if not n.startswith("bwg_")] == []
    call(stream=types.SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=7))
    assert [n for n, _ in devices][-1] == names[-1]


def test_bad_operands_are_refused(rec):  # noqa: F811
    x, w, dh = cuda(4, 64), cuda(64, 128), cuda(4, 64)
    f, other = cuda(4, 64, dtype=torch.float32), cuda(64, 128, dtype=torch.float16)
    off = cuda(3, dtype=torch.int32)
    ws = [w, w]
    far = cuda(4, 64, dev="cuda:1")
    bad = [
        lambda: ops.gemm_swiglu(f, w), lambda: ops.gemm_swiglu(x, other), lambda: ops.gemm_swiglu(x, cuda(72, 128)),
        lambda: ops.gemm_swiglu(x, cuda(64, 127)), lambda: ops.gemm_swiglu(far, w),
        lambda: ops.gemm_swiglu(x, w, out=cuda(4, 128)), lambda: ops.gemm_swiglu(x.t(), w),
        lambda: ops.gemm_swiglu(x, w, b_transposed=True), lambda: ops.gemm_swiglu(cuda(1, 64).expand(4, 64), w),
        lambda: ops.grouped_gemm(x, ws, off, keep_int8=True),
        lambda: ops.grouped_gemm(x, [cuda(64, 127)] * 2, off, swiglu=True, keep_int8=True),
        lambda: ops.grouped_gemm(x, ws, off, swiglu=True, keep_int8=True, out=cuda(4, 128)),
        lambda: ops.swiglu_grad(dh, int8(4, 128)), lambda: ops.swiglu_grad(dh, int8(4, 136, 2)),
        lambda: ops.swiglu_grad(f, int8(4, 128, 2)), lambda: ops.swiglu_grad(far, int8(4, 128, 2)),
        lambda: ops.gemm_swiglu_grad(cuda(4, 72), x, w), lambda: ops.gemm_swiglu_grad(dh, cuda(5, 64), w),
        lambda: ops.gemm_swiglu_grad(dh, x, w, with_h=True), lambda: ops.gemm_swiglu_grad(dh, f, w),
        lambda: ops.gemm_swiglu_grad(dh, x, other), lambda: ops.gemm_swiglu_grad(dh, far, w),
        lambda: ops.gemm_swiglu_grad(dh, x, w, kept=int8(4, 128)),
        lambda: ops.gemm_swiglu_grad(dh, x, w, kept=int8(5, 128, 2)),
        lambda: ops.gemm_swiglu_grad(dh, int8(4, 64, 2), w),
        lambda: ops.gemm_swiglu_grad(dh, x, w, kept=int8(4, 128, 2, dev="cuda:1")),
        lambda: ops.grouped_gemm_swiglu_grad(dh, x, ws, cuda(4, dtype=torch.int32)),
        lambda: ops.grouped_gemm_swiglu_grad(dh, x, ws, cuda(3, dtype=torch.int64)),
        lambda: ops.grouped_gemm_swiglu_grad(dh, x, [], cuda(1, dtype=torch.int32)),
        lambda: ops.grouped_gemm_swiglu_grad(dh, x, [w, cuda(64, 136)], off),
        lambda: ops.grouped_gemm_swiglu_grad(dh, x, [w, other], off),
        lambda: ops.grouped_gemm_swiglu_grad(wide(4, 64, 72), x, ws, off),
        lambda: ops.grouped_gemm_swiglu_grad(dh, wide(4, 64, 72), ws, off),
        lambda: ops.grouped_gemm_swiglu_grad(dh, x, ws, off, with_h=True),
        lambda: ops.quantize_int8(cuda(4, 63), parts=2), lambda: ops.quantize_int8(x, parts=3),
        lambda: ops.quantize_int8(x.t()), lambda: ops.quantize_int8(cuda(4, 64, dtype=torch.int32)),
        lambda: ops.dequantize_int8(ops.Int8Matrix(cuda(4, 64, dtype=torch.uint8), cuda(4, 1, dtype=torch.float32))),
        lambda: ops.dequantize_int8(ops.Int8Matrix(cuda(4, 65, dtype=torch.int8), cuda(4, 1, dtype=torch.float32))),
        lambda: ops.dequantize_int8(int8(4, 64), out_dtype=torch.int8),
        lambda: ops.dequantize_int8(int8(4, 64), out=cuda(4, 72)),
        lambda: ops.gemm(x, cuda(5, 128), a_transposed=True), lambda: ops.gemm(f, f, a_transposed=True),
        lambda: ops.gemm(x, dh, a_transposed=True, b_transposed=True),
        lambda: ops.gemm(x, far, a_transposed=True),
        lambda: ops.grouped_gemm_wgrad(x, cuda(5, 64), off), lambda: ops.grouped_gemm_wgrad(x, far, off),
        lambda: ops.grouped_gemm_wgrad(wide(4, 64, 72), dh, off),
        lambda: ops.grouped_gemm_wgrad(x, dh, cuda(3, dtype=torch.int64)),
        lambda: ops.grouped_gemm_wgrad(x, dh, off, out=cuda(2, 64, 72)),
        lambda: ops.grouped_gemm_wgrad(x, dh, off, out_dtype=torch.int8),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            print("taken:", i)
    assert [n for n, _ in rec.calls if not n.startswith("bwg_")] == []


def test_sizes_and_strides_past_32_bits_are_refused(rec):  # noqa: F811
    far = BIG + 64
    i32 = dict(dtype=torch.int32)
    for call in (
        lambda: ops.gemm_swiglu(wide(4, 64, far), cuda(64, 128)), lambda: ops.gemm_swiglu(cuda(4, 64), wide(64, 128, far)),
        lambda: ops.gemm_swiglu(cuda(4, 64), cuda(64, 128), out=wide(4, 64, far)),
        lambda: ops.gemm_swiglu(cuda(BIG + 4, 64), cuda(64, 128)), lambda: ops.gemm_swiglu(cuda(4, 64), cuda(64, far)),
        lambda: ops.gemm_swiglu_grad(wide(4, 64, far), cuda(4, 64), cuda(64, 128)),
        lambda: ops.gemm_swiglu_grad(cuda(4, 64), wide(4, 64, far), cuda(64, 128)),
        lambda: ops.quantize_int8(wide(4, 64, far)), lambda: ops.quantize_int8(cuda(1, far)),
        lambda: ops.quantize_int8(cuda(BIG + 4, 8)), lambda: ops.dequantize_int8(int8(4, 64), out=wide(4, 64, far)),
        lambda: ops.dequantize_int8(int8(BIG + 4, 8)),
        lambda: ops.gemm(wide(4, 64, far), cuda(4, 64), a_transposed=True),
        lambda: ops.gemm(cuda(4, 64), wide(4, 64, far), a_transposed=True),
        lambda: ops.gemm(cuda(1, far), cuda(1, 64), a_transposed=True),
        lambda: ops.grouped_gemm_wgrad(cuda(BIG + 4, 8), cuda(BIG + 4, 8), cuda(2, **i32)),
        lambda: ops.grouped_gemm_wgrad(cuda(4, 8), cuda(4, 8), cuda(BIG + 4, **i32)),
    ):
        with pytest.raises(ValueError):
            call()
    assert [n for n, _ in rec.calls if not n.startswith("bwg_")] == []


def test_a_kept_matrix_shares_a_buffer(rec):  # noqa: F811
    """Codes and scales of a call's own matrix are views, the scales on 256 bytes."""
    for parts, blocks in ((1, 3), (2, 4)):
        q = ops.quantize_int8(cuda(5, 130), parts=parts)
        at, scales_at = rec.calls[-1][1][-3:-1]
        assert q.shape == (5, 130) and scales_at - at == 768
        assert q.codes.shape == (5, 130) and q.codes.dtype == torch.int8
        assert q.scales.shape == (5, blocks) and q.scales.dtype == torch.float32
        assert ops._int8_check(q, "q") == (5, 130)
    with pytest.raises(ValueError):
        ops.swiglu_grad(cuda(5, 65), ops.quantize_int8(cuda(5, 130)))


def test_a_single_row_keeps_its_stride(rec):  # noqa: F811
    """One row of 60 columns in a buffer of 64: the TMA engine wants the 64."""
    ops.gemm_swiglu(wide(1, 60, 64), cuda(60, 128))
    ops.gemm(wide(1, 60, 64), cuda(1, 64), a_transposed=True)
    assert rec.calls[0][1][10] == 64 and rec.calls[-1][1][8] == 64
    ops.gemm_swiglu(wide(1, 64, BIG + 64), cuda(64, 128))
    assert rec.calls[-1][1][10] == 64


def test_parts_that_do_not_fit_the_scales(rec):  # noqa: F811
    """Parts that are changed afterwards would have scales read behind their end;
    halves of whole blocks have the same ones."""
    q = ops.quantize_int8(cuda(5, 130))
    q.parts = 2
    odd = ops.quantize_int8(cuda(5, 65))
    odd.parts = 2
    del rec.calls[:]
    for m in (q, odd):
        with pytest.raises(ValueError):
            ops.dequantize_int8(m)
    with pytest.raises(ValueError):
        ops.swiglu_grad(cuda(5, 65), q)
    assert rec.calls == []
    whole = ops.quantize_int8(cuda(5, 128))
    whole.parts = 2
    ops.swiglu_grad(cuda(5, 64), whole)
    assert [n for n, _ in rec.calls] == ["quantize_int8", "swiglu_grad_int8"]


def test_dx_uses_no_workspace_of_the_library(rec, lib):  # noqa: F811
    """The flag goes with every dX; the dense products take it beside a type, no other call does."""
    for transposed, w in ((False, cuda(64, 128)), (True, cuda(128, 64))):
        for dtype, name in ((torch.bfloat16, "gemm_bf16"), (torch.float16, "gemm_fp16")):
            del rec.calls[:]
            ops.gemm_swiglu_grad(cuda(4, 64, dtype=dtype), cuda(4, 64, dtype=dtype), w.to(dtype),
                                 b_transposed=transposed)
            (args,) = [a for n, a in rec.calls if n == name + ("" if transposed else "_nt")]
            assert args[9] == ops._OUT_CODES[dtype] | ops.NO_WORKSPACE

    def dense(fn, out, M=0, a=A):
        return fn(a, B, C, M, 128, 64, 64, 128, 128, out, None)

    for fn in (lib.gemm_bf16, lib.gemm_fp16, lib.gemm_bf16_nt, lib.gemm_fp16_nt):
        assert dense(fn, 0x100) == dense(fn, 0x101) == dense(fn, 0x102) == OK
        assert dense(fn, 0x103) == dense(fn, 0x200) == dense(fn, 0x100, 4, None) == INVALID
        assert dense(fn, 0x100, 4, A + 8) == ALIGNMENT
    assert dense(lib.gemm_bf16_small_m_noalloc, 0x100) == INVALID


def off16(rows, cols):
    """A matrix that starts 2 bytes behind an aligned address."""
    return cuda(rows * cols + 8)[1:rows * cols + 1].view(rows, cols)


def test_gradients_are_refused_before_anything_runs(rec, monkeypatch):  # noqa: F811
    """Sizes and addresses that a later call of the chain would refuse."""
    # fake tensors have no address: the offset in their storage stands for it
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: 4096 + 2 * t.storage_offset())
    off = cuda(3, dtype=torch.int32)
    x8, kept = int8(4, 64), int8(4, 128, 2)
    w, dh, x = cuda(64, 128), cuda(4, 64), cuda(4, 64)
    for call in (
        # K no multiple of 8
        lambda: ops.grouped_gemm_swiglu_grad(dh, int8(4, 60), [cuda(60, 128)] * 2, off, kept=kept),
        lambda: ops.grouped_gemm_swiglu_grad(dh, cuda(4, 60), [cuda(60, 128)] * 2, off),
        lambda: ops.grouped_gemm_swiglu_grad(dh, cuda(4, 60), [cuda(128, 60)] * 2, off, b_transposed=True),
        lambda: ops.gemm_swiglu_grad(dh, int8(4, 60), cuda(60, 128), kept=kept),
        # halves of w that start off 16 bytes
        lambda: ops.gemm_swiglu_grad(cuda(4, 60), x8, cuda(64, 120), kept=int8(4, 120, 2)),
        lambda: ops.grouped_gemm_swiglu_grad(cuda(4, 60), x8, [cuda(64, 120)] * 2, off, kept=int8(4, 120, 2)),
        # rows of dh that are no rows of its experts' matrix
        lambda: ops.grouped_gemm_swiglu_grad(wide(4, 64, 72), x8, [w, w], off, kept=kept),
        # addresses and row strides off 16 bytes
        lambda: ops.gemm_swiglu_grad(dh, x8, off16(64, 128), kept=kept),
        lambda: ops.gemm_swiglu_grad(dh, x8, wide(64, 128, 132), kept=kept),
        lambda: ops.gemm_swiglu_grad(dh, off16(4, 64), w, kept=kept),
        lambda: ops.gemm_swiglu_grad(dh, wide(4, 64, 68), w, kept=kept),
        lambda: ops.gemm_swiglu_grad(off16(4, 64), x8, w, kept=kept),
        lambda: ops.gemm_swiglu_grad(wide(4, 64, 68), x8, w, kept=kept),
        lambda: ops.grouped_gemm_swiglu_grad(dh, x8, [w, off16(64, 128)], off, kept=kept),
        lambda: ops.grouped_gemm_swiglu_grad(dh, off16(4, 64), [w, w], off, kept=kept),
        lambda: ops.grouped_gemm_swiglu_grad(off16(4, 64), x8, [w, w], off, kept=kept),
    ):
        with pytest.raises((ValueError, ops.BwgError)):
            call()
        assert [n for n, _ in rec.calls if not n.startswith("bwg_")] == []
    # what is not read may lie anywhere, and so may matrices without rows
    del rec.calls[:]
    ops.gemm_swiglu_grad(dh, off16(4, 64), w, kept=kept, need_dw=False)
    ops.gemm_swiglu_grad(dh, x, off16(64, 128), kept=kept, need_dx=False, need_dw=False)
    ops.grouped_gemm_swiglu_grad(dh, off16(4, 60), [off16(60, 128)] * 2, off, kept=kept, need_dx=False, need_dw=False)
    assert [n for n, _ in rec.calls] == ["swiglu_grad_int8", "gemm_bf16_nt", "swiglu_grad_int8", "swiglu_grad_int8"]
    ops.gemm_swiglu_grad(cuda(0, 60), cuda(0, 64), off16(64, 120), need_dw=False)
    ops.grouped_gemm_swiglu_grad(cuda(0, 64), cuda(0, 60), [cuda(60, 128)] * 2, off)


def test_a_kept_input_is_read_back_into_whole_16_bytes(rec):  # noqa: F811
    """x of 60 columns kept in 8 bits: its rows come back 64 apart, and dw is taken as
    it is of the x that it was kept from."""
    for kept in (None, int8(4, 128, 2)):
        del rec.calls[:]
        ops.gemm_swiglu_grad(cuda(4, 64), int8(4, 60), cuda(60, 128), kept=kept, need_dx=False)
        args = dict(rec.calls)
        assert args["dequantize_int8"][5:8] == (4, 60, 64)
        assert args["gemm_tn"][5:9] == (60, 128, 4, 64)
        if kept is None:
            assert args["gemm_swiglu_grad"][6:11] == (4, 128, 60, 64, 64)


def test_a_single_row_has_a_stride_that_fits(rec):  # noqa: F811
    """One row may come with any stride, or with none that the TMA engine takes: its
    end rounded up to 16 bytes stands for it."""
    for ld in (61, 60, 1, 4099):
        ops.gemm_swiglu(wide(1, 60, ld), cuda(60, 128))
        assert rec.calls[-1][1][10] == 64
        ops.gemm(wide(1, 64, ld), wide(1, 128, ld), a_transposed=True)
        assert rec.calls[-1][1][8:10] == (64, 128)
        ops.swiglu_grad(wide(1, 64, ld), int8(1, 128, 2))
        assert rec.calls[-1][1][8] == 64


def test_a_result_of_one_row_has_a_stride_that_fits(rec):  # noqa: F811
    """D of one row of 113 columns: rows of 16 bytes are of no matter to it."""
    for out in (None, wide(1, 113, 120), wide(1, 113, 113)):
        ops.gemm(wide(4, 1, 8), wide(4, 113, 120), out=out, a_transposed=True)
        assert rec.calls[-1][1][10] == 120
    ops.gemm(wide(4, 2, 8), wide(4, 113, 120), out=wide(2, 113, 128), a_transposed=True)
    assert rec.calls[-1][1][10] == 128
