"""4-bit operators over many groups of rows: group tables are built 32 groups
at a time, with rows, tiles and scale rows carried from one pass to the next."""
import numpy as np
import pytest
import torch

import fp4_util as f4
from test_fp4_gpu import FMTS, dev, random_fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops


def many_groups(G, seed):
    """Group sizes: most of them empty or short, sizes next to a scale tile's and
    a row tile's ends at the first and last groups of each 32."""
    rng = np.random.default_rng(seed)
    counts = rng.choice([0, 0, 0, 1, 2, 17], G)
    for g in range(0, G, 32):
        for at, n in zip((g - 2, g - 1, g, g + 1), rng.permutation([0, 1, 128, 129, 193, 384])):
            if 0 <= at < G:
                counts[at] = n
    counts[G - 1] = 5
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


GROUPS = [33, 64, 65, 257, 1024]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G", GROUPS)
def test_quantize_and_read_back(ops, G, fmt):
    off = many_groups(G, G)
    M, K = int(off[-1]) + 3, 160
    rng = np.random.default_rng(G + 1)
    x = rng.standard_normal((M, K)).astype(np.float32)
    g = None if fmt == "mxfp4" else (rng.random(G) * 0.01 + 0.001).astype(np.float32)
    q = ops.quantize_fp4(dev(x), fmt, global_scale=None if g is None else dev(g), group_offsets=dev(off))
    scale = f4.untile(q.scales.cpu().numpy(), M, K // f4.BLOCK[fmt], off)
    codes = f4.unpack(q.codes.cpu().numpy())
    out = torch.full((M, K), 7.0, device="cuda")
    ops.dequantize_fp4(q, out=out)
    assert ops.last_device_error() == (0, 0)
    got = out.cpu().numpy()
    for e in range(G):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        ge = np.float32(1) if g is None else g[e]
        c, s = f4.quantize(x[lo:hi], fmt, ge)
        assert np.array_equal(codes[lo:hi], c) and np.array_equal(scale[lo:hi], s), e
        assert np.array_equal(got[lo:hi], f4.values(c, s, fmt).astype(np.float32) * ge), e
    assert (got[off[-1]:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G", GROUPS)
def test_stacked_groups(ops, G, fmt):
    """Equal groups, as weights are held: 130 rows each."""
    w = torch.randn(G, 130, 96, device="cuda")
    y = ops.dequantize_fp4(ops.quantize_fp4(w, fmt), torch.float32).view(G, 130, 96)
    for e in (0, 31, 32, G // 2, G - 1):
        assert torch.equal(y[e], ops.dequantize_fp4(ops.quantize_fp4(w[e], fmt), torch.float32))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K", [(72, 96), (600, 352)])
@pytest.mark.parametrize("G", GROUPS)
def test_grouped_product_is_exact(ops, G, N, K, fmt):
    off = many_groups(G, G + 2)
    M = int(off[-1]) + 5
    rng = np.random.default_rng(G + N)
    a, A = random_fp4(ops, M, K, fmt, rng, offsets=off, integers=True)
    b, B = random_fp4(ops, G * N, K, fmt, rng, groups=G, integers=True)
    D = torch.full((M, N), 9.0, device="cuda")
    ops.grouped_gemm_fp4(a, b, out=D)
    assert ops.last_device_error() == (0, 0)
    A, B = dev(A), dev(B)  # in 64 bits
    for e in range(G):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            assert torch.equal(D[lo:hi].double(), A[lo:hi] @ B[e * N:(e + 1) * N].t()), e
    assert bool((D[off[-1]:] == 9).all())


def swiglu_reference(A, B, off, N):
    """(gate, up) of every row, exact in 64 bits."""
    d = torch.cat([A[off[e]:off[e + 1]] @ B[e * N:(e + 1) * N].t() for e in range(len(off) - 1)])
    return d[:, :N // 2], d[:, N // 2:]


def assert_swiglu(H, gate, up):
    """gate and up are integers over a power of two and exact.  The fast
    exponential is within 2 + 1.173 |gate| units in the last place (its share
    of 1 + e^-gate is sigmoid(-gate)); the sum, the reciprocal and two
    products add at most five.  A gate below -87 may give 0, where |silu| is
    below 1e-36."""
    ref = gate * torch.sigmoid(gate) * up
    rel = ((2 + 1.173 * gate.abs()) * torch.sigmoid(-gate) + 5) * 2.0 ** -23
    assert bool(((H.double() - ref).abs() <= rel * ref.abs() + 1e-30 * up.abs()).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N", [512, 84])
@pytest.mark.parametrize("G", GROUPS)
def test_grouped_swiglu(ops, G, N, fmt):
    """Fused (halves that start a tile of scales) and in two steps."""
    off = many_groups(G, G + 3)
    M, K = int(off[-1]), 96
    rng = np.random.default_rng(G + N + 1)
    a, A = random_fp4(ops, M, K, fmt, rng, 2.0 ** -4 if fmt == "nvfp4" else None, offsets=off, integers=True)
    b, B = random_fp4(ops, G * N, K, fmt, rng, groups=G, integers=True)
    if fmt == "mxfp4":  # gates of a size where silu bends
        b.scales -= torch.where(b.scales == 255, 0, 4).to(torch.uint8)
    H = ops.grouped_gemm_fp4(a, b, swiglu=True, out_dtype=torch.float32)
    assert ops.last_device_error() == (0, 0)
    assert_swiglu(H, *swiglu_reference(dev(A) / 16, dev(B), off, N))
