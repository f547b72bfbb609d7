"""Thin Python binding over libbwgemm.so (ctypes).

Argument marshalling only: every function here converts torch tensors to
device pointers, sizes and leading dimensions, calls the C ABI entry point of
the same name and raises on a non-zero status.  All arithmetic runs in the
library's CUDA kernels; if the library is missing or fails to load, every call
raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbwgemm.so")

OUT_BF16 = 0
OUT_FP32 = 1
OUT_FP16 = 2
_OUT_CODES = {torch.bfloat16: OUT_BF16, torch.float32: OUT_FP32, torch.float16: OUT_FP16}

KERNEL_NONE, KERNEL_ZERO, KERNEL_1CTA, KERNEL_2CTA, KERNEL_SMALL_M, KERNEL_2CTA_MC, KERNEL_2CTA_2C = range(7)

STATUS_NAMES = {0: "BWG_OK", 1: "BWG_ERR_INVALID_ARG", 2: "BWG_ERR_ALIGNMENT",
                3: "BWG_ERR_UNSUPPORTED", 4: "BWG_ERR_CUDA", 5: "BWG_ERR_TIMEOUT",
                6: "BWG_ERR_SCRATCH_LIMIT"}

_lock = threading.Lock()
_lib = None


class BwgError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s failed: %s (%s)" % (what, STATUS_NAMES.get(status, status), status_string(status)))
        self.status = status


class PlanInfo(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("tile_k", ctypes.c_int), ("mma_m", ctypes.c_int), ("mma_n", ctypes.c_int),
                ("stages", ctypes.c_int), ("tiles", ctypes.c_int), ("k_blocks", ctypes.c_int),
                ("coverage", ctypes.c_double), ("smem_input_per_cta", ctypes.c_int),
                ("smem_total", ctypes.c_int), ("grid", ctypes.c_int), ("tx_bytes", ctypes.c_uint32),
                ("idesc", ctypes.c_uint32), ("units", ctypes.c_int), ("streamk", ctypes.c_int),
                ("workers", ctypes.c_int), ("dynamic", ctypes.c_int), ("sk_tiles", ctypes.c_int),
                ("sk_segs", ctypes.c_int), ("split", ctypes.c_int), ("staging_in_ring", ctypes.c_int),
                ("bt_loads", ctypes.c_int), ("pair_loads", ctypes.c_int)]


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libbwgemm.so is not built (%s); run __graft_entry__.build(). "
                                   "There is no fallback implementation." % LIB_PATH)
            L = ctypes.CDLL(LIB_PATH)
            vp, i, u32, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64
            for name in ("gemm_bf16", "gemm_fp16", "gemm_bf16_nt", "gemm_fp16_nt"):
                f = getattr(L, name)
                f.argtypes = [vp, vp, vp, i, i, i, i, i, i, i, vp]
                f.restype = i
            for name in ("grouped_gemm_bf16", "grouped_gemm_fp16", "grouped_gemm_swiglu_bf16",
                         "grouped_gemm_swiglu_fp16", "grouped_gemm_bf16_nt", "grouped_gemm_fp16_nt",
                         "grouped_gemm_swiglu_bf16_nt", "grouped_gemm_swiglu_fp16_nt"):
                f = getattr(L, name)
                f.argtypes = [vp, ctypes.POINTER(vp), vp, vp, i, i, i, i, vp]
                f.restype = i
            for name, args in (("moe_sort", [vp, i, i, i, vp, vp, vp, vp]),
                               ("moe_dispatch", [vp, i, i, i, i, i, vp, vp, i, vp, i, vp]),
                               ("moe_dispatch_grad", [vp, i, i, i, i, i, vp, vp, i, vp, i, vp]),
                               ("moe_combine", [vp, i, i, i, i, i, vp, vp, vp, i, vp, i, vp]),
                               ("quantize_fp4", [vp, i, i, i, i, i, vp, i, vp, i, vp, vp, vp]),
                               ("dequantize_fp4", [vp, vp, i, vp, i, vp, i, vp, i, i, i, i, vp]),
                               ("gemm_fp4", [vp, vp, vp, vp, vp, vp, i, vp, i, i, i, i, i, vp]),
                               ("grouped_gemm_fp4", [vp, vp, vp, vp, vp, vp, i, i, vp, vp, i, i, i, i, i, i, i, vp,
                                                     vp]),
                               ("moe_combine_grad", [vp, vp, i, i, i, i, i, i, vp, vp, vp, i, vp, i, vp, vp])):
                f = getattr(L, name)
                f.argtypes = args
                f.restype = i
            L.gemm_bf16_host.argtypes = [vp, vp, vp, i, i, i, i, vp, vp, vp, vp]
            L.gemm_bf16_host.restype = i
            L.bwg_status_string.argtypes = [i]
            L.bwg_status_string.restype = ctypes.c_char_p
            L.bwg_last_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_ulonglong)]
            L.bwg_last_device_error.restype = i
            for name, args in (("bwg_probe_cluster_pair", [vp, vp, vp, i, vp]),
                               ("bwg_probe_tma_swizzle", [vp, vp, vp]),
                               ("bwg_probe_mma", [vp, vp, vp, i, i, vp]),
                               ("bwg_probe_grouped_tables", [vp, i, i, i, i, i, i, vp, vp])):
                f = getattr(L, name)
                f.argtypes = args
                f.restype = i
            L.bwg_debug_set_trace.argtypes = [vp]
            L.bwg_debug_set_trace.restype = None
            L.bwg_set_watchdog_ns.argtypes = [ctypes.c_ulonglong]
            L.bwg_set_watchdog_ns.restype = None
            L.bwg_debug_set_tx_extra.argtypes = [ctypes.c_uint]
            L.bwg_debug_set_tx_extra.restype = None
            L.bwg_plan.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(PlanInfo)]
            L.bwg_plan.restype = i
            L.bwg_check_gemm_args.argtypes = [vp, vp, vp, i, i, i, i, i, i, i]
            L.bwg_check_gemm_args.restype = i
            L.bwg_idesc_f16.argtypes = [i, i, i, i, i]
            L.bwg_idesc_f16.restype = u32
            L.bwg_smem_desc.argtypes = [u32, u32, u32, i]
            L.bwg_smem_desc.restype = u64
            L.bwg_swizzle128_offset.argtypes = [u32, u32]
            L.bwg_swizzle128_offset.restype = u32
            L.bwg_raster_tile.argtypes = [i, i, i, i, ctypes.POINTER(i), ctypes.POINTER(i)]
            L.bwg_raster_tile.restype = None
            ip = ctypes.POINTER(i)
            L.bwg_grouped_schedule.argtypes = [ip, i, i, i, i, ip, ip, ip]
            L.bwg_grouped_schedule.restype = i
            L.bwg_grouped_tile.argtypes = [i, i, ip, ip, ip, i, ip, ip, ip, ip]
            L.bwg_grouped_tile.restype = None
            L.bwg_tail_split.argtypes = [i, i]
            L.bwg_tail_split.restype = i
            L.bwg_unit_tile.argtypes = [i, i, i, i, ip, ip, ip]
            L.bwg_unit_tile.restype = None
            L.bwg_streamk_begin.argtypes = [i, ctypes.c_longlong, i]
            L.bwg_streamk_begin.restype = ctypes.c_longlong
            L.bwg_streamk_tile_workers.argtypes = [i, i, ctypes.c_longlong, i, ip, ip]
            L.bwg_streamk_tile_workers.restype = None
            L.bwg_grouped_swap_rows.argtypes = [i, i, i]
            L.bwg_grouped_swap_rows.restype = i
            L.bwg_tail_split_f.argtypes = [i, i, i, ip]
            L.bwg_tail_split_f.restype = i
            L.bwg_streamk_tiles.argtypes = [i, i, i, i, ip]
            L.bwg_streamk_tiles.restype = i
            L.bwg_unit_part.argtypes = [i, i, i, i, ip, ip, ip]
            L.bwg_unit_part.restype = None
            L.bwg_fp4_scale_bytes.argtypes = [i, i, i, i, i]
            L.bwg_fp4_scale_bytes.restype = ctypes.c_longlong
            L.bwg_fp4_scale_offset.argtypes = [ctypes.c_longlong, i, i, i]
            L.bwg_fp4_scale_offset.restype = ctypes.c_longlong
            L.bwg_fp4_kernel.argtypes = [i, i, i, i, i, i]
            L.bwg_fp4_kernel.restype = i
            L.bwg_idesc_fp4.argtypes = [i, i, i, i]
            L.bwg_idesc_fp4.restype = u32
            L.bwg_version.argtypes = []
            L.bwg_version.restype = ctypes.c_char_p
            _lib = L
    return _lib


def version() -> str:
    """bwg_version(): library version and the hash of the sources it was built from."""
    return lib().bwg_version().decode()


def status_string(status: int) -> str:
    try:
        return lib().bwg_status_string(int(status)).decode()
    except Exception:  # noqa: BLE001 - only used to format an error
        return "?"


def _check(status: int, what: str) -> None:
    if status != 0:
        raise BwgError(status, what)


def _stream_handle(stream, device) -> int:
    if stream is None:
        # the handle of torch.cuda.current_stream(device), without the Stream
        # object around it (7 us of a 20 us call)
        index = device if isinstance(device, int) else device.index
        return torch._C._cuda_getCurrentRawStream(index)
    if not isinstance(device, int):
        of = getattr(stream, "device", device)
        if of != device:
            raise ValueError("the stream is of %s, the tensors are on %s" % (of, device))
    return int(stream.cuda_stream)


def _on(device, fn, *args):
    """fn(*args) with `device` current: the library launches on the current
    device, and the default stream of every device has the same handle."""
    if device.index == torch._C._cuda_getDevice():
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _new(shape, dtype, dev, stream) -> torch.Tensor:
    """A tensor for the kernels on `stream`, taken from that stream's memory:
    what the allocator hands out may still be in use on the current one."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


# The library takes sizes and row strides as 32-bit ints.  ctypes keeps the
# low 32 bits of what does not fit, so that 2^32 + 64 would pass for 64: every
# size that a caller gives is checked here first.
_INT_MAX = (1 << 31) - 1


def _fits(what: str, *sizes: int) -> None:
    if max(sizes) > _INT_MAX:
        raise ValueError("%s: %d is past 2^31 - 1" % (what, max(sizes)))


def _matrix(t: torch.Tensor, name: str) -> int:
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    if t.stride(1) != 1:
        raise ValueError("%s must be row-major with unit column stride" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    ld = t.stride(0)
    if ld > _INT_MAX:
        raise ValueError("row stride of %s: %d is past 2^31 - 1" % (name, ld))
    return ld


def gemm(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor | None = None,
         out_dtype: torch.dtype = torch.bfloat16, stream=None, b_transposed: bool = False) -> torch.Tensor:
    """D = A @ B through gemm_bf16 / gemm_fp16 (chosen by A's dtype); with
    ``b_transposed`` B is given as [N, K] and D = A @ B.T (gemm_*_nt)."""
    if A.dtype != B.dtype or A.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("A and B must both be bfloat16 or both float16")
    M, K = A.shape
    N, K2 = B.shape if b_transposed else (B.shape[1], B.shape[0])
    if K2 != K:
        raise ValueError("inner dimensions differ: %s x %s" % (tuple(A.shape), tuple(B.shape)))
    if M > _INT_MAX or N > _INT_MAX or K > _INT_MAX:
        raise ValueError("M, N or K is past 2^31 - 1: %d, %d, %d" % (M, N, K))
    dev = A.device
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    if out.dtype not in _OUT_CODES:
        raise TypeError("output dtype must be bfloat16, float16 or float32")
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [%d, %d], got %s" % (M, N, tuple(out.shape)))
    if not (dev == B.device == out.device):
        raise ValueError("A, B and out must be on the same device")
    lda, ldb, ldd = _matrix(A, "A"), _matrix(B, "B"), _matrix(out, "out")
    if b_transposed:
        fn = gemm_bf16_nt if A.dtype == torch.bfloat16 else gemm_fp16_nt
    else:
        fn = gemm_bf16 if A.dtype == torch.bfloat16 else gemm_fp16
    _on(dev, fn, A.data_ptr(), B.data_ptr(), out.data_ptr(), M, N, K, lda, ldb, ldd, _OUT_CODES[out.dtype],
        _stream_handle(stream, dev))
    return out


def gemm_bf16(A_ptr: int, B_ptr: int, D_ptr: int, M: int, N: int, K: int, lda: int, ldb: int,
              ldd: int, out_dtype: int, stream: int) -> None:
    _check(lib().gemm_bf16(A_ptr, B_ptr, D_ptr, M, N, K, lda, ldb, ldd, out_dtype, stream), "gemm_bf16")


def gemm_fp16(A_ptr: int, B_ptr: int, D_ptr: int, M: int, N: int, K: int, lda: int, ldb: int,
              ldd: int, out_dtype: int, stream: int) -> None:
    _check(lib().gemm_fp16(A_ptr, B_ptr, D_ptr, M, N, K, lda, ldb, ldd, out_dtype, stream), "gemm_fp16")


def gemm_bf16_nt(A_ptr: int, B_ptr: int, D_ptr: int, M: int, N: int, K: int, lda: int, ldb: int,
                 ldd: int, out_dtype: int, stream: int) -> None:
    """D = A x B^T with B stored [N, K] (ldb >= K)."""
    _check(lib().gemm_bf16_nt(A_ptr, B_ptr, D_ptr, M, N, K, lda, ldb, ldd, out_dtype, stream),
           "gemm_bf16_nt")


def gemm_fp16_nt(A_ptr: int, B_ptr: int, D_ptr: int, M: int, N: int, K: int, lda: int, ldb: int,
                 ldd: int, out_dtype: int, stream: int) -> None:
    _check(lib().gemm_fp16_nt(A_ptr, B_ptr, D_ptr, M, N, K, lda, ldb, ldd, out_dtype, stream),
           "gemm_fp16_nt")


def grouped_gemm(A: torch.Tensor, Bs: list, group_offsets: torch.Tensor,
                 out: torch.Tensor | None = None, stream=None, swiglu: bool = False,
                 b_transposed: bool = False) -> torch.Tensor:
    """Grouped expert product through grouped_gemm_bf16 / grouped_gemm_fp16.

    With ``swiglu`` each weight is [gate | up] ([K, N]) and the result is
    silu(gate) * up, [M_total, N/2], through grouped_gemm_swiglu_bf16/_fp16.
    With ``b_transposed`` every weight is given as [N, K] (the *_nt entry points)."""
    if A.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("A must be bfloat16 or float16")
    M_total, K = A.shape
    G = len(Bs)
    N = (Bs[0].shape[0] if b_transposed else Bs[0].shape[1]) if G else 0
    want = (N, K) if b_transposed else (K, N)
    for b in Bs:
        if b.shape != want or b.dtype != A.dtype or not b.is_contiguous():
            raise ValueError("every weight matrix must be a contiguous %s tensor of A's dtype"
                             % ("[N, K]" if b_transposed else "[K, N]"))
    if group_offsets.dtype != torch.int32 or group_offsets.numel() != G + 1 or not group_offsets.is_cuda:
        raise ValueError("group_offsets must be a CUDA int32 tensor with G+1 entries")
    if not A.is_contiguous():
        raise ValueError("A must be dense [M_total, K]")
    _fits("rows, columns or groups", M_total, K, N, G)
    n_out = N // 2 if swiglu else N
    if out is None:
        out = torch.empty((M_total, n_out), dtype=A.dtype, device=A.device)
    elif out.shape != (M_total, n_out) or out.dtype != A.dtype or not out.is_contiguous():
        raise ValueError("out must be a dense [M_total, %d] tensor of A's dtype" % n_out)
    bf = A.dtype == torch.bfloat16
    if swiglu and b_transposed:
        fn = grouped_gemm_swiglu_bf16_nt if bf else grouped_gemm_swiglu_fp16_nt
    elif swiglu:
        fn = grouped_gemm_swiglu_bf16 if bf else grouped_gemm_swiglu_fp16
    elif b_transposed:
        fn = grouped_gemm_bf16_nt if bf else grouped_gemm_fp16_nt
    else:
        fn = grouped_gemm_bf16 if bf else grouped_gemm_fp16
    _on(A.device, fn, A.data_ptr(), [b.data_ptr() for b in Bs], out.data_ptr(), group_offsets.data_ptr(), G,
        M_total, N, K, _stream_handle(stream, A.device))
    return out


def _ptr_array(ptrs):
    arr = (ctypes.c_void_p * max(len(ptrs), 1))(*[ctypes.c_void_p(p) for p in ptrs])
    return ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)), arr


def grouped_gemm_bf16(A_ptr: int, B_ptrs: list, D_ptr: int, offsets_ptr: int, G: int, M_total: int,
                      N: int, K: int, stream: int) -> None:
    p, keep = _ptr_array(B_ptrs)
    _check(lib().grouped_gemm_bf16(A_ptr, p, D_ptr, offsets_ptr, G, M_total, N, K, stream),
           "grouped_gemm_bf16")
    del keep


def grouped_gemm_fp16(A_ptr: int, B_ptrs: list, D_ptr: int, offsets_ptr: int, G: int, M_total: int,
                      N: int, K: int, stream: int) -> None:
    p, keep = _ptr_array(B_ptrs)
    _check(lib().grouped_gemm_fp16(A_ptr, p, D_ptr, offsets_ptr, G, M_total, N, K, stream),
           "grouped_gemm_fp16")
    del keep


def gemm_bf16_host(A_host: torch.Tensor, B_host: torch.Tensor, D_host: torch.Tensor,
                   dA: torch.Tensor, dB: torch.Tensor, dD: torch.Tensor, stream=None) -> None:
    """Host-buffer form: copies in, multiplies, copies out; `stream` completes
    after the last copy back (the library pipelines over row chunks)."""
    M, K = A_host.shape
    N = B_host.shape[1]
    if D_host.dtype not in _OUT_CODES:
        raise TypeError("output dtype must be bfloat16, float16 or float32")
    if A_host.dtype != torch.bfloat16 or B_host.dtype != torch.bfloat16:
        raise TypeError("A_host and B_host must be bfloat16")
    if B_host.shape[0] != K or tuple(D_host.shape) != (M, N):
        raise ValueError("shapes must be A [M, K], B [K, N], D [M, N]; got %s, %s, %s"
                         % (tuple(A_host.shape), tuple(B_host.shape), tuple(D_host.shape)))
    for name, t in (("A_host", A_host), ("B_host", B_host), ("D_host", D_host)):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("%s must be a dense host tensor" % name)
        _fits("size of " + name, *t.shape)
    need = {"dA": M * K * 2, "dB": K * N * 2, "dD": M * N * D_host.element_size()}
    for name, t in (("dA", dA), ("dB", dB), ("dD", dD)):
        if not t.is_cuda or not t.is_contiguous() or t.numel() * t.element_size() < need[name]:
            raise ValueError("%s must be a dense CUDA buffer of at least %d bytes" % (name, need[name]))
    _check(_on(dA.device, lib().gemm_bf16_host, A_host.data_ptr(), B_host.data_ptr(), D_host.data_ptr(), M, N, K,
               _OUT_CODES[D_host.dtype], dA.data_ptr(), dB.data_ptr(), dD.data_ptr(),
               _stream_handle(stream, dA.device)), "gemm_bf16_host")


def last_device_error(stream=None) -> tuple[int, int]:
    """(status, raw error word) of the current device; clears the word."""
    info = ctypes.c_ulonglong(0)
    handle = _stream_handle(stream, torch.cuda.current_device()) if torch.cuda.is_available() else 0
    st = lib().bwg_last_device_error(handle, ctypes.byref(info))
    return st, info.value


def set_watchdog_ns(ns: int) -> None:
    lib().bwg_set_watchdog_ns(int(ns))


def debug_set_trace(buffer: "torch.Tensor | None") -> None:
    """Profiling hook: per-CTA unit timestamps into `buffer` (int64 CUDA
    tensor of at least grid * 64 * 3 entries), or None to switch off."""
    lib().bwg_debug_set_trace(None if buffer is None else buffer.data_ptr())


def debug_set_tx_extra(nbytes: int) -> None:
    lib().bwg_debug_set_tx_extra(int(nbytes))


def plan(M: int, N: int, K: int, out_dtype: int = OUT_BF16, sm_count: int = 152,
         force_kernel: int = 0, force_stages: int = 0) -> PlanInfo:
    info = PlanInfo()
    _check(lib().bwg_plan(M, N, K, out_dtype, sm_count, force_kernel, force_stages, ctypes.byref(info)),
           "bwg_plan")
    return info


def check_gemm_args(A: int, B: int, D: int, M: int, N: int, K: int, lda: int, ldb: int, ldd: int,
                    out_dtype: int) -> int:
    return int(lib().bwg_check_gemm_args(A, B, D, M, N, K, lda, ldb, ldd, out_dtype))


def grouped_gemm_swiglu_bf16(A_ptr: int, B_ptrs: list, H_ptr: int, offsets_ptr: int, G: int,
                             M_total: int, N: int, K: int, stream: int) -> None:
    p, keep = _ptr_array(B_ptrs)
    _check(lib().grouped_gemm_swiglu_bf16(A_ptr, p, H_ptr, offsets_ptr, G, M_total, N, K, stream),
           "grouped_gemm_swiglu_bf16")
    del keep


def grouped_gemm_swiglu_fp16(A_ptr: int, B_ptrs: list, H_ptr: int, offsets_ptr: int, G: int,
                             M_total: int, N: int, K: int, stream: int) -> None:
    p, keep = _ptr_array(B_ptrs)
    _check(lib().grouped_gemm_swiglu_fp16(A_ptr, p, H_ptr, offsets_ptr, G, M_total, N, K, stream),
           "grouped_gemm_swiglu_fp16")
    del keep


def _grouped_call(name: str, A_ptr: int, B_ptrs: list, D_ptr: int, offsets_ptr: int, G: int,
                  M_total: int, N: int, K: int, stream: int) -> None:
    p, keep = _ptr_array(B_ptrs)
    _check(getattr(lib(), name)(A_ptr, p, D_ptr, offsets_ptr, G, M_total, N, K, stream), name)
    del keep


def grouped_gemm_bf16_nt(A_ptr, B_ptrs, D_ptr, offsets_ptr, G, M_total, N, K, stream) -> None:
    """Grouped product with every B[g] stored [N, K]."""
    _grouped_call("grouped_gemm_bf16_nt", A_ptr, B_ptrs, D_ptr, offsets_ptr, G, M_total, N, K, stream)


def grouped_gemm_fp16_nt(A_ptr, B_ptrs, D_ptr, offsets_ptr, G, M_total, N, K, stream) -> None:
    _grouped_call("grouped_gemm_fp16_nt", A_ptr, B_ptrs, D_ptr, offsets_ptr, G, M_total, N, K, stream)


def grouped_gemm_swiglu_bf16_nt(A_ptr, B_ptrs, H_ptr, offsets_ptr, G, M_total, N, K, stream) -> None:
    _grouped_call("grouped_gemm_swiglu_bf16_nt", A_ptr, B_ptrs, H_ptr, offsets_ptr, G, M_total, N, K,
                  stream)


def grouped_gemm_swiglu_fp16_nt(A_ptr, B_ptrs, H_ptr, offsets_ptr, G, M_total, N, K, stream) -> None:
    _grouped_call("grouped_gemm_swiglu_fp16_nt", A_ptr, B_ptrs, H_ptr, offsets_ptr, G, M_total, N, K,
                  stream)


# ------------------------------------------------------------ routed rows ---

# Like every call here these are outside automatic differentiation: the
# gradients are calls of their own, and an output never requires one.


class Routing(NamedTuple):
    """What moe_sort makes of the experts' ids: the order of the rows that the
    grouped products read, and the way back."""

    offsets: torch.Tensor   # int32 [E + 1]: first row of each expert, then the rows that have one
    order: torch.Tensor     # int32 [T * k]: the pair t * k + j at each row
    position: torch.Tensor  # int32 [T, k]: the row of each pair


def moe_sort(expert_ids: torch.Tensor, num_experts: int, stream=None) -> Routing:
    """Stable sort of the (token, expert) pairs by expert.  ``expert_ids`` is a
    CUDA int32 or int64 tensor [T, k]; an id outside 0 .. num_experts - 1 marks
    a pair without an expert, sorted behind all others.

    With such pairs the offsets end before T * k: grouped_gemm_fp4 takes them so,
    grouped_gemm reports it (its contract wants the last offset to be the rows
    of A, so give it the first offsets[-1] rows)."""
    if expert_ids.dim() != 2 or expert_ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("expert_ids must be an int32 or int64 tensor [T, k]")
    if not expert_ids.is_cuda or not expert_ids.is_contiguous():
        raise ValueError("expert_ids must be a dense CUDA tensor")
    num_experts = int(num_experts)
    if num_experts < 1:
        raise ValueError("num_experts must be at least 1")
    dev = expert_ids.device
    pairs = expert_ids.numel()
    if pairs > _INT_MAX or num_experts > _INT_MAX:
        raise ValueError("%d pairs of %d experts are past 2^31 - 1" % (pairs, num_experts))
    offsets = _new((num_experts + 1,), torch.int32, dev, stream)
    order = _new((pairs,), torch.int32, dev, stream)
    position = _new(expert_ids.shape, torch.int32, dev, stream)
    _check(_on(dev, lib().moe_sort, expert_ids.data_ptr(), expert_ids.element_size(), pairs, num_experts,
               offsets.data_ptr(), order.data_ptr(), position.data_ptr(), _stream_handle(stream, dev)), "moe_sort")
    return Routing(offsets, order, position)


def _routing(r: Routing, dev) -> tuple[int, int, int]:
    """(T, k, E) of a routing whose tensors the kernels can read on `dev`."""
    offsets, _, position = r
    if not (position.dtype is torch.int32 and offsets.dtype is torch.int32 and position.is_contiguous()
            and offsets.is_contiguous() and position.device == dev and offsets.device == dev):
        raise ValueError("routing must hold dense int32 tensors on %s" % dev)
    ps, os_ = position.shape, offsets.shape
    if len(ps) != 2 or len(os_) != 1 or os_[0] < 2 or ps[1] < 1:
        raise ValueError("routing must hold offsets [E + 1] and position [T, k]")
    if ps[0] * ps[1] > _INT_MAX or os_[0] > _INT_MAX:
        raise ValueError("routing has more than 2^31 - 1 pairs or experts")
    return ps[0], ps[1], os_[0] - 1


def _rows(t: torch.Tensor, name: str, rows: int) -> int:
    """Leading dimension of a row matrix with `rows` rows."""
    if t.dtype not in _OUT_CODES:
        raise TypeError("%s must be bfloat16, float16 or float32" % name)
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError("%s must be a 2-D CUDA tensor" % name)
    have, cols = t.shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError("%s must be row-major with unit column stride" % name)
    if have != rows:
        raise ValueError("%s must have %d rows, got %d" % (name, rows, have))
    if rows <= 1:
        ld = cols  # torch gives a single row any stride
    elif ld < cols:
        raise ValueError("%s must not be a broadcast view: its rows overlap" % name)
    if ld > _INT_MAX or rows > _INT_MAX:
        raise ValueError("%s: %d rows with a row stride of %d are past 2^31 - 1" % (name, rows, ld))
    return ld


def _out_rows(out, rows: int, cols: int, dtype, dev, stream) -> tuple:
    """(output matrix, leading dimension): a new one, or the caller's checked."""
    if out is None:
        return _new((rows, cols), dtype, dev, stream), cols
    if out.shape != (rows, cols) or out.dtype is not dtype or out.device != dev:
        raise ValueError("out must be a [%d, %d] %s tensor on %s" % (rows, cols, dtype, dev))
    return out, _rows(out, "out", rows)


def _pair_weights(w: torch.Tensor, T: int, k: int, dev) -> None:
    if w.dtype is not torch.float32 or w.shape != (T, k) or not w.is_contiguous() or w.device != dev:
        raise ValueError("weights must be a dense float32 tensor [%d, %d] on %s" % (T, k, dev))


def moe_dispatch(x: torch.Tensor, routing: Routing, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Token rows [T, H] in expert order, [T * k, H]; zeros in the rows of
    pairs without an expert (from row routing.offsets[-1] on)."""
    T, k, E = _routing(routing, x.device)
    ldx = _rows(x, "x", T)
    H, dtype, dev = x.shape[1], x.dtype, x.device
    out, ldo = _out_rows(out, T * k, H, dtype, dev, stream)
    _check(_on(dev, lib().moe_dispatch, x.data_ptr(), _OUT_CODES[dtype], T, H, ldx, k, routing.position.data_ptr(),
               routing.offsets.data_ptr(), E, out.data_ptr(), ldo, _stream_handle(stream, dev)), "moe_dispatch")
    return out


def moe_dispatch_grad(d_rows: torch.Tensor, routing: Routing, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Gradient of moe_dispatch: [T * k, H] -> [T, H], each token's rows summed."""
    T, k, E = _routing(routing, d_rows.device)
    ldr = _rows(d_rows, "d_rows", T * k)
    H, dtype, dev = d_rows.shape[1], d_rows.dtype, d_rows.device
    out, ldo = _out_rows(out, T, H, dtype, dev, stream)
    _check(_on(dev, lib().moe_dispatch_grad, d_rows.data_ptr(), _OUT_CODES[dtype], T, H, ldr, k,
               routing.position.data_ptr(), routing.offsets.data_ptr(), E, out.data_ptr(), ldo,
               _stream_handle(stream, dev)), "moe_dispatch_grad")
    return out


def moe_combine(rows: torch.Tensor, routing: Routing, weights: torch.Tensor, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Rows in expert order [T * k, H] back to token order [T, H], each token's
    rows summed with its float32 weights [T, k]."""
    T, k, E = _routing(routing, rows.device)
    ldr = _rows(rows, "rows", T * k)
    H, dtype, dev = rows.shape[1], rows.dtype, rows.device
    _pair_weights(weights, T, k, dev)
    out, ldo = _out_rows(out, T, H, dtype, dev, stream)
    _check(_on(dev, lib().moe_combine, rows.data_ptr(), _OUT_CODES[dtype], T, H, ldr, k, weights.data_ptr(),
               routing.position.data_ptr(), routing.offsets.data_ptr(), E, out.data_ptr(), ldo,
               _stream_handle(stream, dev)), "moe_combine")
    return out


def moe_combine_grad(d_out: torch.Tensor, rows: torch.Tensor, routing: Routing, weights: torch.Tensor,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of moe_combine: (d_rows [T * k, H], d_weights float32 [T, k])."""
    T, k, E = _routing(routing, rows.device)
    ldr, ldy = _rows(rows, "rows", T * k), _rows(d_out, "d_out", T)
    if d_out.dtype != rows.dtype or d_out.shape[1] != rows.shape[1] or d_out.device != rows.device:
        raise ValueError("d_out must have the dtype, columns and device of rows")
    _pair_weights(weights, T, k, rows.device)
    d_rows = _new((T * k, rows.shape[1]), rows.dtype, rows.device, stream)
    d_weights = _new((T, k), torch.float32, rows.device, stream)
    _check(_on(rows.device, lib().moe_combine_grad, d_out.data_ptr(), rows.data_ptr(), _OUT_CODES[rows.dtype], T,
               rows.shape[1], ldy, ldr, k, weights.data_ptr(), routing.position.data_ptr(),
               routing.offsets.data_ptr(), E, d_rows.data_ptr(), rows.shape[1], d_weights.data_ptr(),
               _stream_handle(stream, rows.device)), "moe_combine_grad")
    return d_rows, d_weights


# ------------------------------------------------- 4-bit floating point ---

_FP4_CODES = {"nvfp4": 0, "mxfp4": 1}


class Fp4Matrix:
    """A matrix [rows, K] in microscaled 4-bit floating point.

    codes         uint8 [rows, K / 2], two e2m1 values a byte
    scales        uint8, in tiles of 128 rows x 4 blocks (see the C header)
    format        "nvfp4" (blocks of 16, e4m3 scales) or "mxfp4" (blocks of 32, e8m0)
    global_scale  float32 [1] or [groups] (nvfp4), or None
    group_offsets int32 [groups + 1] of ragged groups of rows, or None
    groups        without offsets: the number of equal groups of rows
    """

    __slots__ = ("codes", "scales", "format", "global_scale", "group_offsets", "groups")

    def __init__(self, codes, scales, format, global_scale=None, group_offsets=None, groups=1):
        self.codes = codes
        self.scales = scales
        self.format = format
        self.global_scale = global_scale
        self.group_offsets = group_offsets
        self.groups = groups if group_offsets is None else group_offsets.shape[0] - 1

    @property
    def shape(self):
        return self.codes.shape[0], self.codes.shape[1] * 2

    @property
    def device(self):
        return self.codes.device


def _fp4_format(fmt: str) -> int:
    if fmt not in _FP4_CODES:
        raise ValueError("format must be 'nvfp4' or 'mxfp4', got %r" % (fmt,))
    return _FP4_CODES[fmt]


def _fp4_global(g, fmt: int, groups: int, dev) -> tuple:
    if g is None:
        return None, 1
    if fmt == 1:
        raise ValueError("mxfp4 has no global scale")
    if g.dtype != torch.float32 or not g.is_contiguous() or g.device != dev or g.numel() not in (1, groups):
        raise ValueError("global_scale must be a dense float32 tensor of 1 or %d values on %s" % (groups, dev))
    return g.data_ptr(), g.numel()


def _fp4_offsets(off, dev):
    if off is None:
        return None
    if off.dtype != torch.int32 or off.dim() != 1 or off.shape[0] < 2 or not off.is_contiguous() or off.device != dev:
        raise ValueError("group_offsets must be a dense int32 tensor [groups + 1] on %s" % dev)
    if off.shape[0] > _INT_MAX:
        raise ValueError("group_offsets has more than 2^31 - 1 groups")
    return off.data_ptr()


def _fp4_scale_bytes(M: int, K: int, fmt: int, G: int, ragged: bool) -> int:
    """bwg_fp4_scale_bytes without the call."""
    if ragged:
        tile_rows = (M + 127 * min(G, M)) // 128
    elif G < 1 or M % G:
        return -1
    else:
        tile_rows = G * (-(-(M // G) // 128))
    return tile_rows * -(-K // (64 if fmt == 0 else 128)) * 512


def _fp4_check(q: Fp4Matrix, name: str) -> int:
    """Format code of an Fp4Matrix whose buffers are as large as the kernels take them."""
    fmt = _fp4_format(q.format)
    codes, scales, ragged = q.codes, q.scales, q.group_offsets is not None
    if codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_contiguous() or not codes.is_cuda:
        raise ValueError("%s.codes must be a dense CUDA uint8 tensor [rows, K / 2]" % name)
    rows, half = codes.shape
    if rows > _INT_MAX or 2 * half > _INT_MAX or q.groups > _INT_MAX:
        raise ValueError("%s: rows, columns or groups past 2^31 - 1" % name)
    need = _fp4_scale_bytes(rows, 2 * half, fmt, q.groups, ragged)
    if need < 0:
        raise ValueError("%s: %d rows do not make %d equal groups" % (name, rows, q.groups))
    if scales.dtype != torch.uint8 or not scales.is_contiguous() or scales.device != codes.device \
            or scales.numel() < need:
        raise ValueError("%s.scales must be a dense uint8 tensor of at least %d bytes on %s"
                         % (name, need, codes.device))
    return fmt


def quantize_fp4(x: torch.Tensor, format: str = "nvfp4", global_scale: torch.Tensor | None = None,
                 group_offsets: torch.Tensor | None = None, groups: int = 1, stream=None) -> Fp4Matrix:
    """x [rows, K] (or stacked weights [groups, N, K]) into 4 bits.  For the
    routed rows of a grouped product give the routing's offsets."""
    fmt = _fp4_format(format)
    if x.dim() == 3:
        if group_offsets is not None or not x.is_contiguous():
            raise ValueError("stacked weights must be dense [groups, N, K], without group_offsets")
        groups = x.shape[0]
        x = x.reshape(groups * x.shape[1], x.shape[2])
    if x.dtype not in _OUT_CODES:
        raise TypeError("x must be bfloat16, float16 or float32")
    rows, K = x.shape
    ldx = _rows(x, "x", rows)
    dev = x.device
    if K % 32:
        raise ValueError("K must be a multiple of 32, got %d" % K)
    off = _fp4_offsets(group_offsets, dev)
    if off is not None:
        groups = group_offsets.shape[0] - 1
    elif groups < 1 or rows % groups:
        raise ValueError("%d rows do not make %d equal groups" % (rows, groups))
    g, n_global = _fp4_global(global_scale, fmt, groups, dev)
    codes = _new((rows, K // 2), torch.uint8, dev, stream)
    scales = _new((_fp4_scale_bytes(rows, K, fmt, groups, off is not None),), torch.uint8, dev, stream)
    _check(_on(dev, lib().quantize_fp4, x.data_ptr(), _OUT_CODES[x.dtype], rows, K, ldx, fmt, g, n_global, off,
               groups, codes.data_ptr(), scales.data_ptr(), _stream_handle(stream, dev)), "quantize_fp4")
    return Fp4Matrix(codes, scales, format, global_scale, group_offsets, groups)


def dequantize_fp4(q: Fp4Matrix, out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """The values of q, [rows, K], computed in FP32 and rounded once."""
    fmt = _fp4_check(q, "q")
    dev = q.codes.device
    rows, K = q.shape
    off = _fp4_offsets(q.group_offsets, dev)
    g, n_global = _fp4_global(q.global_scale, fmt, q.groups, dev)
    out, ldo = _fp4_out(out, out_dtype, rows, K, dev, stream)
    _check(_on(dev, lib().dequantize_fp4, q.codes.data_ptr(), q.scales.data_ptr(), fmt, g, n_global, off, q.groups,
               out.data_ptr(), _OUT_CODES[out.dtype], rows, K, ldo, _stream_handle(stream, dev)), "dequantize_fp4")
    return out


def _fp4_pair(A: Fp4Matrix, B: Fp4Matrix) -> int:
    fmt = _fp4_check(A, "A")
    if _fp4_check(B, "B") != fmt:
        raise ValueError("A and B must have the same format")
    if A.codes.shape[1] != B.codes.shape[1]:
        raise ValueError("inner dimensions differ: %s x %s" % (A.shape, B.shape))
    if A.codes.device != B.codes.device:
        raise ValueError("A and B must be on the same device")
    return fmt


def _fp4_out(out, out_dtype, M: int, N: int, dev, stream) -> tuple:
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in _OUT_CODES:
        raise TypeError("output dtype must be bfloat16, float16 or float32")
    return _out_rows(out, M, N, out_dtype, dev, stream)


def gemm_fp4(A: Fp4Matrix, B: Fp4Matrix, out: torch.Tensor | None = None,
             out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """D = A @ B.T of the values of A [M, K] and B [N, K], FP32 accumulation."""
    fmt = _fp4_pair(A, B)
    if A.group_offsets is not None or B.group_offsets is not None or A.groups != 1 or B.groups != 1:
        raise ValueError("gemm_fp4 takes matrices without groups of rows; see grouped_gemm_fp4")
    dev = A.codes.device
    M, K = A.shape
    N = B.codes.shape[0]
    out, ldo = _fp4_out(out, out_dtype, M, N, dev, stream)
    ga, _ = _fp4_global(A.global_scale, fmt, 1, dev)
    gb, _ = _fp4_global(B.global_scale, fmt, 1, dev)
    _check(_on(dev, lib().gemm_fp4, A.codes.data_ptr(), A.scales.data_ptr(), ga, B.codes.data_ptr(),
               B.scales.data_ptr(), gb, fmt, out.data_ptr(), M, N, K, ldo, _OUT_CODES[out.dtype],
               _stream_handle(stream, dev)), "gemm_fp4")
    return out


def grouped_gemm_fp4(A: Fp4Matrix, B: Fp4Matrix, swiglu: bool = False, out: torch.Tensor | None = None,
                     out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """Grouped expert product in 4 bits: rows of A's group g (its group_offsets)
    times B's group g ([groups * N, K], equal groups) transposed.  With
    ``swiglu`` each B[g] is [gate; up] along N and the result silu(gate) * up."""
    fmt = _fp4_pair(A, B)
    if A.group_offsets is None or B.group_offsets is not None:
        raise ValueError("A must have ragged groups (group_offsets), B equal ones")
    if A.groups != B.groups:
        raise ValueError("A has %d groups, B %d" % (A.groups, B.groups))
    dev = A.codes.device
    off = _fp4_offsets(A.group_offsets, dev)
    M, K = A.shape
    G = B.groups
    N = B.codes.shape[0] // G
    if swiglu and N % 2:
        raise ValueError("swiglu needs an even number of weight rows, got %d" % N)
    n_out = N // 2 if swiglu else N
    out, ldo = _fp4_out(out, out_dtype, M, n_out, dev, stream)
    ga, na = _fp4_global(A.global_scale, fmt, 1, dev)
    gb, n_global = _fp4_global(B.global_scale, fmt, G, dev)
    work = _new((M, N), torch.float32, dev, stream) if swiglu and N % 256 else None
    _check(_on(dev, lib().grouped_gemm_fp4, A.codes.data_ptr(), A.scales.data_ptr(), ga, B.codes.data_ptr(),
               B.scales.data_ptr(), gb, n_global, fmt, out.data_ptr(), off, G, M, N, K, ldo, _OUT_CODES[out.dtype],
               1 if swiglu else 0, None if work is None else work.data_ptr(), _stream_handle(stream, dev)),
           "grouped_gemm_fp4")
    return out
