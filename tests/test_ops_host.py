"""The Python calls' own checks, without a GPU: tensors of torch's fake mode
stand for CUDA tensors, and a recorder for the library, so that what would
reach a kernel is seen and nothing is launched."""
import ctypes
import types
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from blackwell_tensor_core_gb300 import ops

BIG = 1 << 32  # what a 32-bit argument loses


class Recorder:
    """Takes the place of the C library; keeps (name, arguments)."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(ops, "lib", lambda: r)
    # where there is a GPU, fake tensors would set up their device's context, which may not exist
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")  # fake tensors have no data pointer
        with FakeTensorMode(allow_non_fake_inputs=True):
            yield r


def cuda(*shape, dtype=torch.bfloat16, dev="cuda:0"):
    return torch.empty(shape, dtype=dtype, device=dev)


def routing(T, k, E, dev="cuda:0"):
    i = dict(dtype=torch.int32, dev=dev)
    return ops.Routing(cuda(E + 1, **i), cuda(T * k, **i), cuda(T, k, **i))


def fp4(rows, K, groups=1, offsets=None, dev="cuda:0"):
    u = dict(dtype=torch.uint8, dev=dev)
    G = groups if offsets is None else offsets.shape[0] - 1
    size = ops._fp4_scale_bytes(rows, K, 0, G, offsets is not None)
    return ops.Fp4Matrix(cuda(rows, K // 2, **u), cuda(size, **u), "nvfp4", None, offsets, groups)


def wide(rows, cols, ld, dtype=torch.bfloat16):
    """[rows, cols] with `ld` elements from row to row."""
    return cuda(8, dtype=dtype).as_strided((rows, cols), (ld, 1))


def test_the_wrapped_argument_is_what_the_checks_are_for():
    assert ctypes.c_int(BIG + 64).value == 64


WIDE_CALLS = [
    ("moe_dispatch", lambda m: ops.moe_dispatch(m(4, 64), routing(4, 2, 3))),
    ("moe_dispatch out", lambda m: ops.moe_dispatch(cuda(4, 64), routing(4, 2, 3), out=m(8, 64))),
    ("moe_dispatch_grad", lambda m: ops.moe_dispatch_grad(m(8, 64), routing(4, 2, 3))),
    ("moe_combine", lambda m: ops.moe_combine(m(8, 64), routing(4, 2, 3), cuda(4, 2, dtype=torch.float32))),
    ("moe_combine_grad rows", lambda m: ops.moe_combine_grad(cuda(4, 64), m(8, 64), routing(4, 2, 3),
                                                             cuda(4, 2, dtype=torch.float32))),
    ("moe_combine_grad d_out", lambda m: ops.moe_combine_grad(m(4, 64), cuda(8, 64), routing(4, 2, 3),
                                                              cuda(4, 2, dtype=torch.float32))),
    ("quantize_fp4", lambda m: ops.quantize_fp4(m(4, 64))),
    ("dequantize_fp4", lambda m: ops.dequantize_fp4(fp4(4, 64), out=m(4, 64))),
    ("gemm_fp4", lambda m: ops.gemm_fp4(fp4(4, 64), fp4(64, 64), out=m(4, 64))),
    ("grouped_gemm_fp4", lambda m: ops.grouped_gemm_fp4(fp4(4, 64, offsets=cuda(3, dtype=torch.int32)),
                                                        fp4(128, 64, groups=2), out=m(4, 64))),
    ("gemm A", lambda m: ops.gemm(m(4, 64), cuda(64, 64))),
    ("gemm B", lambda m: ops.gemm(cuda(4, 64), m(64, 64))),
    ("gemm out", lambda m: ops.gemm(cuda(4, 64), cuda(64, 64), out=m(4, 64))),
]


@pytest.mark.parametrize("call", [c for _, c in WIDE_CALLS], ids=[n for n, _ in WIDE_CALLS])
def test_row_strides_past_32_bits_are_refused(rec, call):
    """2^32 + 64 would arrive as 64, a row stride that the kernels take."""
    with pytest.raises(ValueError):
        call(lambda rows, cols: wide(rows, cols, BIG + 64))
    assert rec.calls == []
    call(lambda rows, cols: wide(rows, cols, (1 << 31) - 8))
    assert len(rec.calls) == 1


def test_a_single_row_has_no_stride(rec):
    ops.moe_dispatch(wide(1, 64, BIG + 64), routing(1, 2, 3))
    (name, args), = rec.calls
    assert name == "moe_dispatch" and args[4] == 64


def test_sizes_past_32_bits_are_refused(rec):
    i = torch.int32
    thin = cuda(8, dtype=i)
    for call in (
        lambda: ops.moe_sort(cuda(BIG + 4, 1, dtype=i), 4),
        lambda: ops.moe_sort(cuda(4, 2, dtype=i), BIG + 4),
        lambda: ops.moe_dispatch(cuda(BIG + 4, 8), routing(BIG + 4, 1, 3)),
        lambda: ops.moe_dispatch(cuda(1, 8), routing(1, BIG + 4, 3)),
        lambda: ops.moe_dispatch(cuda(4, 8), ops.Routing(cuda(BIG + 4, dtype=i), thin, cuda(4, 2, dtype=i))),
        lambda: ops.moe_dispatch(cuda(1, BIG + 8), routing(1, 1, 3)),
        lambda: ops.quantize_fp4(cuda(BIG + 32, 32)),
        lambda: ops.quantize_fp4(cuda(1, BIG + 32)),
        lambda: ops.quantize_fp4(cuda(4, 32), group_offsets=cuda(BIG + 5, dtype=i)),
        lambda: ops.dequantize_fp4(fp4(BIG + 4, 32)),
        lambda: ops.dequantize_fp4(fp4(4, BIG + 32)),
        lambda: ops.gemm_fp4(fp4(4, 32), fp4(BIG + 4, 32)),
        lambda: ops.gemm(cuda(BIG + 4, 32), cuda(32, 8)),
        lambda: ops.gemm(cuda(4, 32), cuda(32, BIG + 8)),
        lambda: ops.grouped_gemm(cuda(BIG + 4, 32), [cuda(32, 8)], cuda(2, dtype=i)),
        lambda: ops.grouped_gemm(cuda(4, 32), [cuda(32, BIG + 8)], cuda(2, dtype=i)),
    ):
        with pytest.raises(ValueError):
            call()
    assert rec.calls == []


# ------------------------------------------------------------- devices ---

def _every_call(dev):
    f32 = dict(dtype=torch.float32, dev=dev)
    i32 = dict(dtype=torch.int32, dev=dev)
    r = routing(4, 2, 3, dev)
    off = cuda(3, **i32)
    return {
        "moe_sort": lambda **s: ops.moe_sort(cuda(4, 2, **i32), 3, **s),
        "moe_dispatch": lambda **s: ops.moe_dispatch(cuda(4, 64, dev=dev), r, **s),
        "moe_dispatch_grad": lambda **s: ops.moe_dispatch_grad(cuda(8, 64, dev=dev), r, **s),
        "moe_combine": lambda **s: ops.moe_combine(cuda(8, 64, dev=dev), r, cuda(4, 2, **f32), **s),
        "moe_combine_grad": lambda **s: ops.moe_combine_grad(cuda(4, 64, dev=dev), cuda(8, 64, dev=dev), r,
                                                             cuda(4, 2, **f32), **s),
        "quantize_fp4": lambda **s: ops.quantize_fp4(cuda(4, 64, dev=dev), **s),
        "dequantize_fp4": lambda **s: ops.dequantize_fp4(fp4(4, 64, dev=dev), **s),
        "gemm_fp4": lambda **s: ops.gemm_fp4(fp4(4, 64, dev=dev), fp4(64, 64, dev=dev), **s),
        "grouped_gemm_fp4": lambda **s: ops.grouped_gemm_fp4(fp4(4, 64, offsets=off, dev=dev),
                                                             fp4(512, 64, groups=2, dev=dev), **s),
        "gemm_bf16": lambda **s: ops.gemm(cuda(4, 64, dev=dev), cuda(64, 64, dev=dev), **s),
        "gemm_bf16_nt": lambda **s: ops.gemm(cuda(4, 64, dev=dev), cuda(64, 64, dev=dev), b_transposed=True, **s),
        "grouped_gemm_bf16": lambda **s: ops.grouped_gemm(cuda(4, 64, dev=dev), [cuda(64, 64, dev=dev)] * 2, off, **s),
        "grouped_gemm_swiglu_bf16": lambda **s: ops.grouped_gemm(cuda(4, 64, dev=dev), [cuda(64, 64, dev=dev)] * 2,
                                                                 off, swiglu=True, **s),
    }


CALLS = ["moe_sort", "moe_dispatch", "moe_dispatch_grad", "moe_combine", "moe_combine_grad", "quantize_fp4",
         "dequantize_fp4", "gemm_fp4", "grouped_gemm_fp4", "gemm_bf16", "gemm_bf16_nt", "grouped_gemm_bf16",
         "grouped_gemm_swiglu_bf16"]


@pytest.fixture
def devices(rec, monkeypatch):
    """Which device is current, as torch.cuda.device would make it, and which
    one was at each call of the library."""
    now = [0]
    seen = []

    class Device:
        def __init__(self, device):
            self.index = device if isinstance(device, int) else device.index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *exc):
            now[0] = self.before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    inner = Recorder.__getattr__

    def __getattr__(self, name):
        call = inner(self, name)

        def with_device(*args):
            seen.append((name, now[0]))
            return call(*args)
        return with_device

    monkeypatch.setattr(Recorder, "__getattr__", __getattr__)
    return seen


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("index", [0, 1])
def test_calls_run_on_their_tensors_device(devices, name, index):
    """The library launches on the current device: on the tensors' one during
    the call, and on the caller's again after it."""
    _every_call("cuda:%d" % index)[name]()
    assert devices == [(name, index)]
    assert torch._C._cuda_getDevice() == 0


@pytest.mark.parametrize("name", CALLS)
def test_streams_of_another_device_are_refused(devices, name, monkeypatch):
    import contextlib
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    with pytest.raises(ValueError):
        _every_call("cuda:0")[name](stream=types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=7))
    assert devices == []
    _every_call("cuda:0")[name](stream=types.SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=7))
    assert devices == [(name, 0)]


def test_stacked_weights_without_columns(rec):
    q = ops.quantize_fp4(cuda(3, 8, 0))
    assert q.shape == (24, 0) and q.groups == 3
    (name, args), = rec.calls
    assert name == "quantize_fp4" and args[2:4] == (24, 0) and args[9] == 3


def test_a_single_column_has_no_column_stride(rec):
    """[4, 1] with strides (1, 4), as the transpose of a row is: torch calls it contiguous."""
    x = cuda(1, 4).t()
    assert x.is_contiguous() and x.stride() == (1, 4)
    ops.moe_dispatch(x, routing(4, 2, 3))
    (name, args), = rec.calls
    assert name == "moe_dispatch" and args[3:5] == (1, 1)
    with pytest.raises(ValueError):
        ops.moe_dispatch(cuda(2, 4).t(), routing(4, 2, 3))
