"""4-bit floating point on the GPU: quantising and reading back against the
definition in numpy, the dense and the grouped product against 64-bit sums."""
import numpy as np
import pytest
import torch

import fp4_util as f4

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.bfloat16, torch.float16, torch.float32]
FMTS = ["nvfp4", "mxfp4"]


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def scale_bytes(ops, M, K, fmt, groups=1, ragged=False):
    return ops.lib().bwg_fp4_scale_bytes(M, K, 0 if fmt == "nvfp4" else 1, groups, int(ragged))


def random_fp4(ops, M, K, fmt, rng, g=None, offsets=None, groups=1, integers=False):
    """A random matrix in 4 bits with NaN scales in the rows that hold nothing:
    (Fp4Matrix, its values in 64 bits)."""
    codes = rng.integers(0, 16, (M, K)).astype(np.uint8)
    blocks = K // f4.BLOCK[fmt]
    if integers:  # values 0, 1, 2, 3, 4, 6 and their negatives with scales 1 and 2: products and sums are exact
        codes = np.where((codes & 7) % 2 == 1, np.where((codes & 7) < 4, codes & 8, codes), codes).astype(np.uint8)
        scale = (rng.integers(0, 2, (M, blocks)) + 127 if fmt == "mxfp4" else
                 rng.choice([0x38, 0x40], (M, blocks))).astype(np.uint8)
    elif fmt == "mxfp4":
        scale = rng.integers(120, 131, (M, blocks)).astype(np.uint8)
    else:
        scale = rng.integers(0x20, 0x58, (M, blocks)).astype(np.uint8)
    G = groups if offsets is None else len(offsets) - 1
    buf = f4.tiles(scale, scale_bytes(ops, M, K, fmt, G, offsets is not None), offsets, groups,
                   fill=0x7F if fmt == "nvfp4" else 0xFF)
    q = ops.Fp4Matrix(dev(f4.pack(codes)), dev(buf), fmt, None if g is None else dev(np.array(g, np.float32).reshape(-1)),
                      None if offsets is None else dev(np.asarray(offsets, np.int32)), groups)
    return q, f4.values(codes, scale, fmt)


def assert_product(got, A, B, K, dtype, what, alpha=1.0):
    """FP32 accumulation: one instruction adds 64 products to the accumulator;
    its rounding is taken as at most 2^-22 of the sum of magnitudes, K / 64
    instructions one after the other, then alpha and one rounding."""
    ref, S = (A @ B.T) * alpha, (np.abs(A) @ np.abs(B).T) * abs(alpha)
    tol = (K / 64 + 3) * 2.0 ** -22 * S + U[dtype] * np.abs(ref) + (6e-8 if dtype == torch.float16 else 0)
    err = np.abs(got.double().cpu().numpy() - ref)
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d outside the bound, first at %s: got %r want %r" % (
        what, bad.sum(), bad.size, tuple(np.argwhere(bad)[0]), float(got[tuple(np.argwhere(bad)[0])]),
        ref[tuple(np.argwhere(bad)[0])])


# ------------------------------------------------------------- quantising ---

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (5, 96), (130, 160), (33, 1056), (257, 4096)])
def test_quantize_equals_the_definition(ops, M, K, dtype, fmt):
    rng = np.random.default_rng(M * K)
    x = dev(rng.standard_normal((M, K)) * np.exp2(rng.integers(-12, 8, (M, K // 32)).repeat(32, 1))).to(dtype)
    x[0, :32] = 0
    x[-1, -1] = -0.0
    g = 0.003 if fmt == "nvfp4" else None
    q = ops.quantize_fp4(x, fmt, global_scale=None if g is None else torch.tensor([g], device="cuda"))
    codes, scale = f4.quantize(x.float().cpu().numpy(), fmt, np.float32(g or 1))
    assert np.array_equal(f4.untile(q.scales.cpu().numpy(), M, K // f4.BLOCK[fmt]), scale)
    assert np.array_equal(f4.unpack(q.codes.cpu().numpy()), codes)
    # and the padding of the tiles along K is zero
    blocks = K // f4.BLOCK[fmt]
    if blocks % 4:
        full = f4.untile(q.scales.cpu().numpy(), M, -(-blocks // 4) * 4)
        assert (full[:, blocks:] == 0).all()
    for out_dtype in TYPES:
        y = ops.dequantize_fp4(q, out_dtype)
        v = f4.values(codes, scale, fmt).astype(np.float32) * np.float32(g or 1)  # exact, then one rounding
        want = torch.from_numpy(v.astype(np.float32)).to(out_dtype)
        assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_ties_and_extremes(ops, fmt):
    """Every tie between two values, saturation, zero and tiny blocks, and
    magnitudes at both ends of FP32."""
    base = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -2.5, -5.0, 0.0, -0.0, 4.0])
    near = np.concatenate([np.nextafter(base[:8].astype(np.float32), np.float32(9)),
                           np.nextafter(base[:8].astype(np.float32), np.float32(0))])
    rows = [np.concatenate([base, near]), np.zeros(32), np.full(32, 1e-42), np.full(32, 3.4e38),
            np.linspace(-3.4e38, 3.4e38, 32), np.linspace(0, 1e-38, 32), np.full(32, 2.0 ** -130),
            np.array([2.0 ** -20] * 31 + [1.0]), np.array([1.9999999] * 16 + [2.0] * 16), np.linspace(-7, 7, 32)]
    x = np.stack(rows).astype(np.float32)
    q = ops.quantize_fp4(dev(x), fmt)
    codes, scale = f4.quantize(x, fmt)
    assert np.array_equal(f4.untile(q.scales.cpu().numpy(), x.shape[0], 32 // f4.BLOCK[fmt]), scale)
    assert np.array_equal(f4.unpack(q.codes.cpu().numpy()), codes)
    if fmt == "nvfp4":
        for g in (1e-33, 2.0 ** -10, 0.1, 1e30):  # steps outside the fast quotient's range, and ties of a power of two
            q = ops.quantize_fp4(dev(x), fmt, global_scale=torch.tensor([g], device="cuda"))
            codes, scale = f4.quantize(x, fmt, np.float32(g))
            assert np.array_equal(f4.untile(q.scales.cpu().numpy(), x.shape[0], 2), scale), g
            assert np.array_equal(f4.unpack(q.codes.cpu().numpy()), codes), g


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nans_mark_their_block_alone(ops, fmt, dtype):
    b = f4.BLOCK[fmt]
    x = torch.randn(4, 128, device="cuda").to(dtype)
    x[0, 3], x[1, 40], x[2, 127] = float("nan"), float("inf"), float("-inf")
    y = ops.dequantize_fp4(ops.quantize_fp4(x, fmt), torch.float32)
    bad = torch.zeros(4, 128, dtype=torch.bool, device="cuda")
    for r, c in ((0, 3), (1, 40), (2, 127)):
        bad[r, c // b * b:(c // b + 1) * b] = True
    assert torch.equal(torch.isnan(y), bad)
    clean = ops.dequantize_fp4(ops.quantize_fp4(torch.where(bad, torch.zeros_like(x), x), fmt), torch.float32)
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_error_is_half_a_step(ops, fmt):
    """In 64 bits: what is read back is within half the local step of x."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((64, 512)).astype(np.float32)
    y = ops.dequantize_fp4(ops.quantize_fp4(dev(x), fmt), torch.float32).double().cpu().numpy()
    s = np.abs(x.reshape(64, -1, f4.BLOCK[fmt])).max(2)
    # steps are at most 2 units of the scale, units at most amax / 4 (mxfp4: amax is in [4, 8) units, saturating
    # at 6) or amax / 6 times one rounding of e4m3 (2^-4)
    unit = s / 4 if fmt == "mxfp4" else s / 6 * (1 + 2.0 ** -4)
    most = (2.0 if fmt == "mxfp4" else 1.0 + 6 * 2.0 ** -4) * unit + 1e-9
    assert (np.abs(y - x).reshape(64, -1, f4.BLOCK[fmt]) <= most[:, :, None]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (5, 3)])
def test_quantize_strided(ops, fmt, dtype, pad, shift):
    M, K = 37, 160
    flat = torch.full((M * (K + pad) + shift,), float("nan"), dtype=dtype, device="cuda")
    x = flat[shift:].view(M, K + pad)[:, :K]
    x.copy_(torch.randn(M, K, device="cuda"))
    a, b = ops.quantize_fp4(x, fmt), ops.quantize_fp4(x.contiguous(), fmt)
    assert torch.equal(a.codes, b.codes)
    blocks = K // f4.BLOCK[fmt]
    sa, sb = (f4.untile(q.scales.cpu().numpy(), M, blocks) for q in (a, b))
    assert np.array_equal(sa, sb)
    out = torch.full((M * (K + pad) + shift,), 3.0, dtype=dtype, device="cuda")
    y = out[shift:].view(M, K + pad)[:, :K]
    ops.dequantize_fp4(a, out=y)
    assert torch.equal(y, ops.dequantize_fp4(b, dtype))
    assert bool((out[shift:].view(M, K + pad)[:, K:] == 3.0).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_ragged_and_stacked_groups(ops, fmt):
    K = 96
    offsets = np.array([0, 0, 130, 131, 131, 400, 528], np.int32)
    M = 540  # the last rows belong to no group
    x = torch.randn(M, K, device="cuda")
    G = len(offsets) - 1
    g = None if fmt == "mxfp4" else torch.rand(G, device="cuda") * 0.01 + 0.001
    q = ops.quantize_fp4(x, fmt, global_scale=g, group_offsets=dev(offsets))
    blocks = K // f4.BLOCK[fmt]
    scale = f4.untile(q.scales.cpu().numpy(), M, blocks, offsets)
    codes = f4.unpack(q.codes.cpu().numpy())
    for e in range(G):
        lo, hi = offsets[e], offsets[e + 1]
        c, s = f4.quantize(x[lo:hi].cpu().numpy(), fmt, 1 if g is None else np.float32(g[e].item()))
        assert np.array_equal(codes[lo:hi], c) and np.array_equal(scale[lo:hi], s)
    out = torch.full((M, K), 7.0, device="cuda")
    ops.dequantize_fp4(q, out=out)
    assert bool((out[528:] == 7.0).all())
    assert ops.last_device_error() == (0, 0)
    w = torch.randn(3, 200, K, device="cuda")
    g = None if fmt == "mxfp4" else torch.rand(3, device="cuda") * 0.01 + 0.001
    q = ops.quantize_fp4(w, fmt, global_scale=g)
    y = ops.dequantize_fp4(q, torch.float32).view(3, 200, K)
    for e in range(3):
        one = ops.quantize_fp4(w[e], fmt, global_scale=None if g is None else g[e:e + 1])
        assert torch.equal(y[e], ops.dequantize_fp4(one, torch.float32))


def test_broken_offsets_are_clamped_and_reported(ops):
    x = torch.randn(100, 64, device="cuda")
    off = torch.tensor([0, 60, 40, 150], dtype=torch.int32, device="cuda")
    q = ops.quantize_fp4(x, "nvfp4", group_offsets=off)
    assert ops.last_device_error()[0] == 1
    w = ops.quantize_fp4(torch.randn(3, 128, 64, device="cuda"), "nvfp4")
    ops.grouped_gemm_fp4(q, w)
    assert ops.last_device_error()[0] == 1
    assert ops.last_device_error() == (0, 0)


def test_quantize_nothing(ops):
    for fmt in FMTS:
        q = ops.quantize_fp4(torch.zeros(0, 64, device="cuda"), fmt)
        assert q.shape == (0, 64) and q.scales.numel() == 0
        assert ops.dequantize_fp4(q).shape == (0, 64)
        w = ops.quantize_fp4(torch.zeros(8, 64, device="cuda"), fmt)
        assert ops.gemm_fp4(q, w).shape == (0, 8)
        assert ops.gemm_fp4(w, q).shape == (8, 0)
        k0 = ops.quantize_fp4(torch.zeros(8, 0, device="cuda"), fmt)
        assert bool((ops.gemm_fp4(k0, k0) == 0).all())


# ---------------------------------------------------------- dense product ---

DENSE = [(1, 8, 32), (1, 128, 64), (16, 128, 256), (17, 200, 96), (64, 256, 512), (72, 520, 1056), (128, 130, 320),
         (129, 256, 256), (192, 512, 768), (193, 513, 544), (300, 1000, 416), (385, 1024, 2048), (1000, 300, 7168),
         (1, 2048, 7168), (5, 300, 7168), (128, 1024, 4096), (97, 4100, 2080), (33, 20000, 512), (100, 19600, 256),
         (1150, 5000, 544), (1150, 5000, 1792)]  # two weight blocks a CTA


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", DENSE)
def test_gemm_integers_are_exact(ops, M, N, K, fmt):
    rng = np.random.default_rng(M + N + K)
    a, A = random_fp4(ops, M, K, fmt, rng, integers=True)
    b, B = random_fp4(ops, N, K, fmt, rng, integers=True)
    D = ops.gemm_fp4(a, b, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert ops.last_device_error() == (0, 0)
    assert np.array_equal(D.double().cpu().numpy(), A @ B.T)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("M,N,K", DENSE[3:])
def test_gemm_within_bound(ops, M, N, K, fmt, out_dtype):
    rng = np.random.default_rng(M + N + K + 1)
    ga, gb = (0.02, 0.5) if fmt == "nvfp4" else (None, None)
    a, A = random_fp4(ops, M, K, fmt, rng, ga)
    b, B = random_fp4(ops, N, K, fmt, rng, gb)
    alpha = float(np.float32(0.02) * np.float32(0.5)) if ga else 1.0
    if out_dtype == torch.float16 and not ga:  # keep the sums inside FP16
        a.scales -= torch.where(a.scales == 255, 0, 8).to(torch.uint8)
        A = A / 256
    D = ops.gemm_fp4(a, b, out_dtype=out_dtype)
    torch.cuda.synchronize()
    assert ops.last_device_error() == (0, 0)
    assert_product(D, A, B, K, out_dtype, "%dx%dx%d %s" % (M, N, K, fmt), alpha)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(2000, 5000, 8192), (1500, 2600, 8000)])
def test_many_tiles_are_exact(ops, M, N, K, fmt):
    """Several tiles a CTA pair and many k-blocks: scales and operands of one
    stage are overwritten by the next while the tensor cores run."""
    rng = np.random.default_rng(M)
    a, A = random_fp4(ops, M, K, fmt, rng, integers=True)
    b, B = random_fp4(ops, N, K, fmt, rng, integers=True)
    want = dev(A) @ dev(B).t()  # in 64 bits
    for _ in range(5):
        assert torch.equal(ops.gemm_fp4(a, b, out_dtype=torch.float32).double(), want)


# tiles of 128 rows whose k-blocks 1 to 8 CTAs share, up to one tile for each SM; two rounds of them; pairs of CTAs
# with one and with two weight blocks
SHARED = [(129, 130, 2304), (200, 512, 8192), (257, 301, 4992), (1000, 128, 2080), (513, 1024, 7168), (640, 640, 4096),
          (300, 1500, 1792), (260, 1280, 6144), (260, 896, 6144), (129, 9000, 1056), (512, 4096, 1024), (19400, 100, 320),
          (129, 10000, 544), (193, 9800, 416), (385, 5000, 1184),
          (385, 5001, 2592), (770, 7600, 5024), (580, 6001, 3104), (1151, 2999, 544)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHARED)
def test_shared_tiles_are_exact(ops, M, N, K, fmt):
    rng = np.random.default_rng(M + N + K + 2)
    a, A = random_fp4(ops, M, K, fmt, rng, integers=True)
    b, B = random_fp4(ops, N, K, fmt, rng, integers=True)
    want = dev(A) @ dev(B).t()  # in 64 bits
    for _ in range(3):
        D = ops.gemm_fp4(a, b, out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert ops.last_device_error() == (0, 0)
        assert torch.equal(D.double(), want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (4, 4), (2, 0), (1, 3)])
def test_shared_tiles_into_a_wider_matrix(ops, fmt, dtype, pad, shift):
    """Rows of D that start on 16 bytes and rows that do not."""
    rng = np.random.default_rng(9)
    M, N, K = 150, 260, 4096
    a, _ = random_fp4(ops, M, K, fmt, rng)
    b, _ = random_fp4(ops, N, K, fmt, rng)
    if dtype == torch.float16:  # keep the sums inside FP16
        a.scales -= torch.where(a.scales == 255, 0, 8).to(torch.uint8)
    buf = torch.full((M, shift + N + pad), -5.0, device="cuda", dtype=dtype)
    ops.gemm_fp4(a, b, out=buf[:, shift:shift + N])
    assert torch.equal(buf[:, shift:shift + N], ops.gemm_fp4(a, b, out_dtype=torch.float32).to(dtype))
    assert bool((buf[:, :shift] == -5.0).all()) and bool((buf[:, shift + N:] == -5.0).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_gemm_into_a_wider_matrix(ops, fmt):
    rng = np.random.default_rng(8)
    M, N, K = 200, 300, 192
    a, A = random_fp4(ops, M, K, fmt, rng, integers=True)
    b, B = random_fp4(ops, N, K, fmt, rng, integers=True)
    buf = torch.full((M, N + 7), -5.0, device="cuda")
    ops.gemm_fp4(a, b, out=buf[:, 3:3 + N])
    assert np.array_equal(buf[:, 3:3 + N].double().cpu().numpy(), A @ B.T)
    assert bool((buf[:, :3] == -5.0).all()) and bool((buf[:, 3 + N:] == -5.0).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_a_nan_block_reaches_its_row_alone(ops, fmt):
    M, N, K = 70, 140, 512
    x = torch.randn(M, K, device="cuda")
    x[33, 100] = float("nan")
    w = ops.quantize_fp4(torch.randn(N, K, device="cuda"), fmt)
    D = ops.gemm_fp4(ops.quantize_fp4(x, fmt), w, out_dtype=torch.float32)
    assert bool(torch.isnan(D[33]).all())
    assert bool(torch.isfinite(torch.cat([D[:33], D[34:]])).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantised_linear_layer(ops, fmt, dtype):
    """Quantise and multiply, against the definition in 64 bits."""
    rng = np.random.default_rng(12)
    M, N, K = 45, 384, 1024
    x = dev(rng.standard_normal((M, K))).to(dtype)
    w = rng.standard_normal((N, K)).astype(np.float32) * 0.02
    gx, gw = (np.float32(np.abs(x.float().cpu().numpy()).max() / 2688), np.float32(np.abs(w).max() / 2688)) \
        if fmt == "nvfp4" else (None, None)
    tg = [None if g is None else torch.tensor([g], device="cuda") for g in (gx, gw)]
    D = ops.gemm_fp4(ops.quantize_fp4(x, fmt, global_scale=tg[0]), ops.quantize_fp4(dev(w), fmt, global_scale=tg[1]),
                     out_dtype=dtype)
    A = f4.values(*f4.quantize(x.float().cpu().numpy(), fmt, gx or 1), fmt)
    B = f4.values(*f4.quantize(w, fmt, gw or 1), fmt)
    assert_product(D, A, B, K, dtype, fmt, 1.0 if gx is None else float(gx) * float(gw))


def test_repeated_products_are_identical(ops):
    rng = np.random.default_rng(77)
    a, _ = random_fp4(ops, 700, 1536, "nvfp4", rng)
    b, _ = random_fp4(ops, 2100, 1536, "nvfp4", rng)
    first = ops.gemm_fp4(a, b)
    for _ in range(40):
        assert torch.equal(ops.gemm_fp4(a, b), first)


# -------------------------------------------------------- grouped product ---

GROUPS = [[5], [0, 0, 3], [300, 0, 256, 1, 0, 191, 37, 193, 530], [192, 384], [128, 64, 129, 1], [0, 0]]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", GROUPS)
@pytest.mark.parametrize("N,K", [(200, 96), (512, 512), (768, 1120), (2600, 352)])
def test_grouped_integers_are_exact(ops, counts, N, K, fmt):
    rng = np.random.default_rng(sum(counts) + N)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M, G = int(off[-1]) + 5, len(counts)  # five rows of no group
    a, A = random_fp4(ops, M, K, fmt, rng, offsets=off, integers=True)
    b, B = random_fp4(ops, G * N, K, fmt, rng, groups=G, integers=True)
    D = torch.full((M, N), 9.0, device="cuda")
    ops.grouped_gemm_fp4(a, b, out=D)
    torch.cuda.synchronize()
    assert ops.last_device_error() == (0, 0)
    got = D.double().cpu().numpy()
    for e in range(G):
        lo, hi = off[e], off[e + 1]
        assert np.array_equal(got[lo:hi], A[lo:hi] @ B[e * N:(e + 1) * N].T)
    assert (got[off[-1]:] == 9.0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N", [512, 256, 1280, 416, 30])
@pytest.mark.parametrize("out_dtype", TYPES)
def test_grouped_swiglu(ops, N, fmt, out_dtype):
    """silu(gate) up with per-group scales.  gate and up carry the product's
    bound e_g, e_u; silu has slope at most 1.1, so the result is within
    1.1 e_g |up| + |silu(gate)| e_u + 1.1 e_g e_u, plus 2^-20 relative for the
    approximate exponential and reciprocal, plus one rounding."""
    rng = np.random.default_rng(N)
    counts = [300, 0, 33, 1, 193]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M, G, K = int(off[-1]), len(counts), 352
    gb = None if fmt == "mxfp4" else rng.random(G).astype(np.float32) * 0.1 + 0.05
    ga = None if fmt == "mxfp4" else np.float32(0.01)
    a, A = random_fp4(ops, M, K, fmt, rng, ga, offsets=off)
    b, B = random_fp4(ops, G * N, K, fmt, rng, gb, groups=G)
    if fmt == "mxfp4":  # keep gates of a size where silu bends
        b.scales -= torch.where(b.scales == 255, 0, 9).to(torch.uint8)
        B = B / 512
    H = ops.grouped_gemm_fp4(a, b, swiglu=True, out_dtype=out_dtype)
    torch.cuda.synchronize()
    assert ops.last_device_error() == (0, 0)
    got = H.double().cpu().numpy()
    for e in range(G):
        lo, hi = off[e], off[e + 1]
        w = B[e * N:(e + 1) * N]
        al = 1.0 if ga is None else float(ga) * float(gb[e])
        d, S = A[lo:hi] @ w.T * al, np.abs(A[lo:hi]) @ np.abs(w).T * al
        err = (K / 64 + 3) * 2.0 ** -22 * S
        gate, up, eg, eu = d[:, :N // 2], d[:, N // 2:], err[:, :N // 2], err[:, N // 2:]
        with np.errstate(over="ignore"):
            silu = gate / (1 + np.exp(-gate))
        ref = silu * up
        tol = 1.1 * eg * np.abs(up) + np.abs(silu) * eu + 1.1 * eg * eu + (2.0 ** -20 + U[out_dtype]) * np.abs(ref) + 1e-7
        if out_dtype == torch.float16:
            ref = np.clip(ref, -65504, 65504)
            keep = np.abs(ref) < 6e4
        else:
            keep = np.ones_like(ref, bool)
        assert (np.abs(got[lo:hi] - ref)[keep] <= tol[keep]).all()


def test_routed_layer_in_4_bits(ops):
    """Sort, dispatch, quantise, FC1 with SwiGLU, quantise, FC2, combine, with
    dropped pairs and empty experts, against 64 bits of each step's inputs."""
    T, k, E, H, I = 130, 2, 9, 256, 384
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(0, 6, (T, k), generator=g, device="cuda")
    ids[torch.rand(T, k, generator=g, device="cuda") < 0.2] = -1
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = torch.rand(T, k, generator=g, device="cuda")
    w1 = ops.quantize_fp4(torch.randn(E, 2 * I, H, generator=g, device="cuda") * 0.06, "mxfp4")
    w2 = ops.quantize_fp4(torch.randn(E, H, I, generator=g, device="cuda") * 0.06, "mxfp4")
    r = ops.moe_sort(ids, E)
    q1 = ops.quantize_fp4(ops.moe_dispatch(x, r), "mxfp4", group_offsets=r.offsets)
    h = ops.grouped_gemm_fp4(q1, w1, swiglu=True)
    q2 = ops.quantize_fp4(h, "mxfp4", group_offsets=r.offsets)
    rows = ops.grouped_gemm_fp4(q2, w2)
    y = ops.moe_combine(rows, r, w)
    torch.cuda.synchronize()
    assert ops.last_device_error() == (0, 0)
    assert bool(torch.isfinite(y.float()).all())
    n = int(r.offsets[-1])
    off = r.offsets.tolist()
    h64 = ops.dequantize_fp4(q2, torch.float32).double()
    W2 = ops.dequantize_fp4(w2, torch.float32).double().view(E, H, I)
    want = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for e in range(E):
        want[off[e]:off[e + 1]] = h64[off[e]:off[e + 1]] @ W2[e].t()
        mag[off[e]:off[e + 1]] = h64[off[e]:off[e + 1]].abs() @ W2[e].abs().t()
    kept = (r.position < n).double() * w.double()
    ref = (want[r.position.long()] * kept[:, :, None]).sum(1)
    S = (mag[r.position.long()] * kept[:, :, None]).sum(1)
    row_err = (want.abs()[r.position.long()] * kept[:, :, None]).sum(1)  # each row was rounded to bf16
    tol = (I / 64 + 3) * 2.0 ** -22 * S + 2.0 ** -8 * row_err + 2.0 ** -8 * ref.abs() + 2.0 ** -8 * 2.0 ** -8 * row_err
    assert bool(((y.double() - ref).abs() <= tol + 1e-6 * row_err).all())


def test_products_on_a_stream_of_their_own(ops):
    rng = np.random.default_rng(5)
    side = torch.cuda.Stream()
    a, _ = random_fp4(ops, 300, 512, "nvfp4", rng)
    b, _ = random_fp4(ops, 416, 512, "nvfp4", rng)
    want = ops.gemm_fp4(a, b)
    torch.cuda.synchronize()
    got = ops.gemm_fp4(a, b, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", FMTS)
def test_matrices_past_32_bits(ops, fmt):
    """More than 2^31 elements to quantise, to read back and in a product."""
    M, K = 70000, 32768
    assert M * K > 1 << 31
    x = torch.randn(1, K, device="cuda").bfloat16().expand(M, K).contiguous()
    tail = torch.randn(130, K, device="cuda").bfloat16()
    x[-130:] = tail
    q = ops.quantize_fp4(x, fmt)
    assert torch.equal(q.codes[-130:], ops.quantize_fp4(tail, fmt).codes)
    assert torch.equal(q.codes[0], q.codes[-131])
    y = ops.dequantize_fp4(q, out=x)
    assert torch.equal(y[-130:], ops.dequantize_fp4(ops.quantize_fp4(tail, fmt)))
    del q, x, y
    a = ops.quantize_fp4(torch.randn(M, 64, device="cuda"), fmt)
    b = ops.quantize_fp4(torch.randn(K, 64, device="cuda"), fmt)
    D = ops.gemm_fp4(a, b)
    for rows in (slice(0, 200), slice(M - 200, M)):
        part = ops.quantize_fp4(ops.dequantize_fp4(a, torch.float32)[rows].contiguous(), fmt)
        assert torch.equal(D[rows], ops.gemm_fp4(part, b))


def test_captured_into_a_graph(ops):
    """The layer's calls replayed from a CUDA graph on new inputs."""
    T, k, E, H = 64, 2, 8, 256
    ids = torch.randint(0, E, (T, k), device="cuda")
    x = torch.randn(T, H, device="cuda").bfloat16()
    w = torch.rand(T, k, device="cuda")
    w1 = ops.quantize_fp4(torch.randn(E, 512, H, device="cuda") * 0.06, "mxfp4")

    def layer():
        r = ops.moe_sort(ids, E)
        q = ops.quantize_fp4(ops.moe_dispatch(x, r), "mxfp4", group_offsets=r.offsets)
        return ops.moe_combine(ops.grouped_gemm_fp4(q, w1, swiglu=True), r, w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(T, H, generator=g, device="cuda"))
        ids.copy_(torch.randint(-1, E, (T, k), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, layer())


def test_python_refusals(ops):
    x = torch.randn(8, 64, device="cuda")
    q = ops.quantize_fp4(x)
    m = ops.quantize_fp4(x, "mxfp4")
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    ragged = ops.quantize_fp4(x, group_offsets=off)
    one = torch.ones(1, device="cuda")
    for call in (lambda: ops.quantize_fp4(x, "fp4"), lambda: ops.quantize_fp4(x[:, :40]),
                 lambda: ops.quantize_fp4(x, "mxfp4", global_scale=one), lambda: ops.quantize_fp4(x.cpu()),
                 lambda: ops.quantize_fp4(x, global_scale=one.double()), lambda: ops.quantize_fp4(x, groups=3),
                 lambda: ops.quantize_fp4(x, group_offsets=off.long()), lambda: ops.quantize_fp4(x[:1].expand(8, 64)),
                 lambda: ops.gemm_fp4(q, m), lambda: ops.gemm_fp4(ragged, q), lambda: ops.grouped_gemm_fp4(q, q),
                 lambda: ops.gemm_fp4(q, ops.quantize_fp4(torch.randn(8, 32, device="cuda"))),
                 lambda: ops.gemm_fp4(ops.Fp4Matrix(q.codes, q.scales[:-1], "nvfp4"), q),
                 lambda: ops.gemm_fp4(ops.Fp4Matrix(q.codes.t(), q.scales, "nvfp4"), q),
                 lambda: ops.grouped_gemm_fp4(ragged, ops.quantize_fp4(torch.randn(2, 8, 64, device="cuda"))),
                 lambda: ops.grouped_gemm_fp4(ragged, ops.quantize_fp4(torch.randn(1, 7, 64, device="cuda")), swiglu=True),
                 lambda: ops.gemm_fp4(q, q, out=torch.empty(8, 9, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ops.quantize_fp4(x.double()), lambda: ops.gemm_fp4(q, q, out_dtype=torch.float64)):
        with pytest.raises(TypeError):
            call()
