"""4-bit floating point without a GPU: the scale layout's helpers, the
instruction descriptor's fields and the entry points' argument checks."""
import numpy as np
import pytest

import fp4_util as f4

INVALID, ALIGNMENT, UNSUPPORTED = 1, 2, 3
P, Q, R, S, T = 4096, 8192, 12288, 16384, 20480  # addresses that are never read


@pytest.fixture(scope="module")
def lib():
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops.lib()


@pytest.mark.parametrize("fmt,K", [(0, 32), (0, 64), (0, 4096), (0, 1056), (1, 32), (1, 128), (1, 160), (1, 7168)])
def test_scale_offset_is_the_layouts(lib, fmt, K):
    blocks = K // (16 if fmt == 0 else 32)
    rows = [0, 1, 31, 32, 96, 127, 128, 300, 70000]
    want = f4.scale_places(rows, blocks)
    for i, r in enumerate(rows):
        for b in {0, 1, blocks // 2, blocks - 1}:
            if b < blocks:
                assert lib.bwg_fp4_scale_offset(r, b, K, fmt) == want[i, b]
    # every byte of a whole tile is used once
    all_rows = f4.scale_places(np.arange(256), -(-blocks // 4) * 4).reshape(-1)
    assert sorted(all_rows.tolist()) == list(range(lib.bwg_fp4_scale_bytes(256, K, fmt, 1, 0)))


def test_scale_bytes_hold_every_grouping(lib):
    rng = np.random.default_rng(0)
    for _ in range(200):
        G = int(rng.integers(1, 40))
        counts = rng.integers(0, 300, G) * (rng.random(G) < 0.7)
        M = int(counts.sum())
        need = int(sum(-(-c // 128) for c in counts)) * 512 * 3  # K = 160 in nvfp4: three tiles
        assert need <= lib.bwg_fp4_scale_bytes(M, 160, 0, G, 1) <= (M // 128 + min(G, M)) * 512 * 3 + 511
    assert lib.bwg_fp4_scale_bytes(600, 128, 1, 3, 0) == 3 * 2 * 512
    from blackwell_tensor_core_gb300 import ops
    for M, K, fmt, G, ragged in ((0, 64, 0, 1, 0), (7, 96, 1, 1, 0), (600, 1056, 0, 3, 0), (10, 64, 0, 3, 0),
                                 (5, 64, 1, 900, 1), (1000, 4096, 0, 32, 1), (0, 32, 0, 4, 1)):
        assert ops._fp4_scale_bytes(M, K, fmt, G, bool(ragged)) == lib.bwg_fp4_scale_bytes(M, K, fmt, G, ragged)
    for bad in ((-1, 64, 0, 1, 0), (8, -32, 0, 1, 0), (8, 64, 2, 1, 0), (8, 64, 0, 0, 0), (8, 64, 0, 3, 0)):
        assert lib.bwg_fp4_scale_bytes(*bad) == -1


def test_instruction_descriptor_fields(lib):
    for fmt in (0, 1):
        for n in (16, 96, 192, 256):
            for m in (128, 256):
                for sid in (0, 2):
                    d = lib.bwg_idesc_fp4(fmt, m, n, sid)
                    assert (d >> 4) & 3 == sid and (d >> 29) & 3 == sid
                    assert (d >> 7) & 7 == 1 and (d >> 10) & 3 == 1   # both operands e2m1
                    assert ((d >> 17) & 63) * 8 == n and ((d >> 27) & 3) * 128 == m
                    assert (d >> 23) & 1 == fmt                       # e4m3 or e8m0 scales
                    assert (d >> 15) & 3 == 0 and d >> 31 == 0        # K-major, K = 64


@pytest.mark.parametrize("change,status", [
    (dict(dtype=5), INVALID), (dict(fmt=2), INVALID), (dict(M=-1), INVALID), (dict(K=-32), INVALID),
    (dict(G=0), INVALID), (dict(G=3), INVALID), (dict(K=48), ALIGNMENT), (dict(fmt=1, g=R), INVALID),
    (dict(g=R, ng=2), INVALID), (dict(G=1025, off=R), UNSUPPORTED), (dict(x=None), INVALID), (dict(codes=None), INVALID),
    (dict(scales=None), INVALID), (dict(ldx=63), INVALID), (dict(x=P + 1), ALIGNMENT), (dict(codes=Q + 8), ALIGNMENT),
    (dict(scales=R + 4), ALIGNMENT), (dict(M=0, x=None), 0), (dict(K=0, x=None), 0),
])
def test_quantize_and_dequantize_refuse(lib, change, status):
    a = dict(x=P, dtype=0, M=8, K=64, ldx=64, fmt=0, g=None, ng=1, off=None, G=1, codes=Q, scales=R)
    a.update(change)
    assert lib.quantize_fp4(a["x"], a["dtype"], a["M"], a["K"], a["ldx"], a["fmt"], a["g"], a["ng"], a["off"], a["G"],
                            a["codes"], a["scales"], None) == status
    assert lib.dequantize_fp4(a["codes"], a["scales"], a["fmt"], a["g"], a["ng"], a["off"], a["G"], a["x"], a["dtype"],
                              a["M"], a["K"], a["ldx"], None) == status


GEMM = dict(A=P, As=Q, ga=None, B=R, Bs=S, gb=None, ng=1, fmt=0, D=T, off=P, G=2, M=8, N=64, K=64, ldd=64, out=0,
            swiglu=0, work=None)


def _gemm(lib, a):
    return lib.gemm_fp4(a["A"], a["As"], a["ga"], a["B"], a["Bs"], a["gb"], a["fmt"], a["D"], a["M"], a["N"], a["K"],
                        a["ldd"], a["out"], None)


def _grouped(lib, a):
    return lib.grouped_gemm_fp4(a["A"], a["As"], a["ga"], a["B"], a["Bs"], a["gb"], a["ng"], a["fmt"], a["D"], a["off"],
                                a["G"], a["M"], a["N"], a["K"], a["ldd"], a["out"], a["swiglu"], a["work"], None)


@pytest.mark.parametrize("change,status", [
    (dict(out=3), INVALID), (dict(fmt=-1), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID),
    (dict(K=-32), INVALID), (dict(K=40), ALIGNMENT), (dict(D=None), INVALID), (dict(ldd=63), INVALID),
    (dict(fmt=1, ga=P), INVALID), (dict(fmt=1, gb=P), INVALID), (dict(D=T + 1), ALIGNMENT),
    (dict(D=T + 2, out=1), ALIGNMENT), (dict(A=None), INVALID), (dict(As=None), INVALID), (dict(B=None), INVALID),
    (dict(Bs=None), INVALID), (dict(A=P + 8), ALIGNMENT), (dict(As=Q + 8), ALIGNMENT), (dict(B=R + 8), ALIGNMENT),
    (dict(Bs=S + 8), ALIGNMENT), (dict(M=0, A=None, D=None), 0), (dict(N=0, ldd=0, B=None, D=None), 0),
])
def test_products_refuse(lib, change, status):
    a = dict(GEMM)
    a.update(change)
    assert _gemm(lib, a) == status
    assert _grouped(lib, a) == status


@pytest.mark.parametrize("change,status", [
    (dict(off=None), INVALID), (dict(G=-1), INVALID), (dict(gb=P, ng=3), INVALID), (dict(G=1025), UNSUPPORTED),
    (dict(swiglu=1, N=63), INVALID), (dict(swiglu=1), INVALID), (dict(swiglu=1, work=P + 4), ALIGNMENT),
    (dict(swiglu=1, N=256, ldd=127), INVALID), (dict(G=0, off=None), 0),
])
def test_grouped_product_refuses(lib, change, status):
    a = dict(GEMM)
    a.update(change)
    assert _grouped(lib, a) == status
