"""The FP32 scales of 4-bit matrices over FP32's range: products whose two
scales multiply past it, and quotients next to a tie for many scales."""
import numpy as np
import pytest
import torch

import fp4_util as f4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops


def matrix(ops, M, K, byte, rng, g, offsets=None, groups=1):
    """Codes of 0, 1, 2, -1, -2, one scale byte everywhere: (Fp4Matrix, values without g)."""
    codes = rng.choice([0, 2, 4, 10, 12], (M, K)).astype(np.uint8)
    scale = np.full((M, K // 16), byte, np.uint8)
    G = groups if offsets is None else len(offsets) - 1
    buf = f4.tiles(scale, ops.lib().bwg_fp4_scale_bytes(M, K, 0, G, int(offsets is not None)), offsets, groups)
    q = ops.Fp4Matrix(torch.from_numpy(f4.pack(codes)).cuda(), torch.from_numpy(buf).cuda(), "nvfp4",
                      torch.tensor(np.atleast_1d(np.float32(g)), device="cuda"),
                      None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda"), groups)
    return q, f4.values(codes, scale, "nvfp4")


# scale byte and the two scales.  The sums are integers times 2^16 (scales 2^8), or times 2^-18 (2^-9), of at most
# 17 bits (K 4096, values up to 2): exact, and so are their products with powers of two down to 2^-149.
RANGE = [(0x78, 2.0 ** -75, 2.0 ** -75), (0x78, 2.0 ** -100, 2.0 ** -48), (0x78, 2.0 ** -149, 2.0 ** 10),
         (0x78, 2.0 ** 12, 2.0 ** -149), (0x01, 2.0 ** 60, 2.0 ** 69), (0x01, 2.0 ** 127, 2.0 ** 2),
         (0x38, 2.0 ** 100, 2.0 ** -100), (0x38, 2.0 ** -126, 1.0), (0x38, 0.5, 2.0 ** 100)]


@pytest.mark.parametrize("M,N,K", [(5, 72, 64), (9, 128, 4096), (150, 200, 1024), (400, 5000, 96), (4000, 4096, 2048)])
@pytest.mark.parametrize("byte,ga,gb", RANGE)
def test_scales_whose_product_leaves_fp32(ops, M, N, K, byte, ga, gb):
    rng = np.random.default_rng(K)
    a, A = matrix(ops, M, K, byte, rng, ga)
    b, B = matrix(ops, N, K, byte, rng, gb)
    want = torch.from_numpy(A).cuda() @ torch.from_numpy(B).cuda().t() * ga * gb  # in 64 bits: exact
    got = ops.gemm_fp4(a, b, out_dtype=torch.float32)
    assert torch.equal(got, want.float())


@pytest.mark.parametrize("N,K", [(72, 64), (2600, 352)])
@pytest.mark.parametrize("byte,ga,gb", RANGE)
def test_grouped_scales_whose_product_leaves_fp32(ops, N, K, byte, ga, gb):
    rng = np.random.default_rng(N)
    off = [0, 3, 3, 200, 331]
    G = len(off) - 1
    gs = np.array([gb, 1, gb / 2 if gb > 2.0 ** -149 else gb, 0.25], np.float32)
    a, A = matrix(ops, off[-1], K, byte, rng, ga, offsets=off)
    b, B = matrix(ops, G * N, K, byte, rng, gs, groups=G)
    got = ops.grouped_gemm_fp4(a, b, out_dtype=torch.float32)
    for e in range(G):
        lo, hi = off[e], off[e + 1]
        want = torch.from_numpy(A[lo:hi] @ B[e * N:(e + 1) * N].T * ga * float(gs[e])).cuda()
        assert torch.equal(got[lo:hi], want.float())


@pytest.mark.parametrize("N", [512, 60])
def test_swiglu_scales_whose_product_leaves_fp32(ops, N):
    """A gate and an up of zero stay zero, and finite ones do not turn into
    NaN, where the scales' product alone would be infinite."""
    rng = np.random.default_rng(N)
    off = [0, 130, 131]
    a, A = matrix(ops, 131, 32, 0x01, rng, 2.0 ** 70, offsets=off)
    b, B = matrix(ops, 2 * N, 32, 0x01, rng, 2.0 ** 60, groups=2)
    b.codes[: N // 2] = 0  # group 0: every gate is 0
    b.codes[N + N // 2:] = 0  # group 1: every up is 0
    H = ops.grouped_gemm_fp4(a, b, swiglu=True, out_dtype=torch.float32)
    assert bool((H == 0).all())


def near_ties(d, thresholds):
    """[n] FP32 -> [n, 5 * thresholds] the FP32 neighbours of t d."""
    mid = (d.double()[:, None] * torch.tensor(thresholds, dtype=torch.float64, device=d.device)).float()
    steps = torch.arange(-2, 3, device=d.device, dtype=torch.int32)
    return (mid.view(torch.int32)[:, :, None] + steps).reshape(d.shape[0], -1).view(torch.float32)


# mantissas of the scales: every one within 64 of a multiple of 2^20 (where quotients come nearest to a tie), the
# rest at random
def mantissas(n):
    rng = np.random.default_rng(1)
    near = (np.arange(0, 9)[:, None] * 2 ** 20 + np.arange(-64, 65)).reshape(-1)
    near = near[(near >= 0) & (near < 1 << 23)]
    m = np.concatenate([near, rng.integers(0, 1 << 23, n - near.size)])
    return torch.from_numpy(((127 - 9) << 23 | m).astype(np.int32)).cuda().view(torch.float32)


CODE_TIES = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]


def test_codes_next_to_a_tie(ops):
    """A block whose scale is 1 has the step g: values next to t g for every
    tie t, against quotients in 64 bits rounded to FP32 (53 bits are enough
    for that to equal the FP32 quotient)."""
    for g in mantissas(1 << 16).split(1024):
        G = g.numel()
        x = torch.zeros(G, 48, device="cuda")
        ties = near_ties(g, CODE_TIES)
        x.view(G, 3, 16)[:, :, 0] = (6 * g)[:, None]
        x.view(G, 3, 16)[:, :, 1:13] = torch.cat([ties, ties[:, :1]], 1).view(G, 3, 12)
        x = torch.cat([x, torch.zeros(G, 16, device="cuda")], 1)
        q = ops.quantize_fp4(x, "nvfp4", global_scale=g, groups=G)
        code = torch.from_numpy(f4.unpack(q.codes.cpu().numpy())).cuda()
        quot = (x.double() / g.double()[:, None]).float().double()
        t = torch.tensor(CODE_TIES, dtype=torch.float64, device="cuda")
        lower_even = torch.tensor([True, False] * 4, device="cuda")[:7]  # a tie goes to the even code
        over = (quot[:, :, None] > t) | ((quot[:, :, None] == t) & ~lower_even)
        want = over.sum(2)
        assert torch.equal(code.long(), want), [float(v).hex() for v in g[(code.long() != want).any(1)][:5]]


SCALE_TIES = [1 + (2 * i + 1) / 16 for i in range(8)]


def test_scales_next_to_a_tie(ops):
    """Largest magnitudes next to t (6 g) for the ties t of e4m3 in [1, 2)."""
    for g in mantissas(1 << 15).split(1024):
        G = g.numel()
        c = (6 * g.double()).float()
        amax = near_ties(c, SCALE_TIES)
        x = torch.zeros(G, 40, 16, device="cuda")
        x[:, :, 3] = amax
        q = ops.quantize_fp4(x.view(G, 640), "nvfp4", global_scale=g, groups=G)
        byte = torch.from_numpy(f4.untile(q.scales.cpu().numpy(), G, 40, groups=G)).cuda()
        quot = (amax.double() / c.double()[:, None]).float().double()
        low = torch.floor(quot * 8)  # 8 .. 15, and 16 for 2
        frac = quot * 8 - low
        want = 0x38 + (low - 8).long() + ((frac > 0.5) | ((frac == 0.5) & (low.long() % 2 == 1))).long()
        assert torch.equal(byte.long(), want), [float(v).hex() for v in g[(byte.long() != want).any(1)][:5]]
