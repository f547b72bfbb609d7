"""Products whose left operand is read transposed (gradients of weights), dense
and by expert, against 64-bit sums: exact on integers, within gated_util's bound
on others, and for FP32 results within the bound of sums of 512 rows joined with
rounding to nearest."""
import pytest
import torch

import gated_util as gu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


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


def draw(rows, cols, dtype, seed, integers=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if integers:
        return torch.randint(-2, 3, (rows, cols), generator=g, device="cuda").to(dtype)
    return torch.randn(rows, cols, generator=g, device="cuda").to(dtype)


def want(a, b, out):
    """The sum and its bound: 512 rows at a time where the result is FP32 (or its
    rows are shared out), else all rows on the tensor cores."""
    a, b = a.double(), b.double()
    d, s = a.t() @ b, a.abs().t() @ b.abs()
    rows = a.shape[0]
    if out == torch.float32:
        joined = -(-rows // 512) + 32  # additions of partial sums, those of shares among them
        e = ((512 / 16 + 2) * 2.0 ** -22 + joined * 2.0 ** -24) * s
    else:
        e = (rows / 16 + 34) * 2.0 ** -22 * s
        e = e + gu.u(out) * (d.abs() + e) + gu.tiny(out)
    return d, e


# one step, ragged k-blocks, ragged tiles, tails of 64 columns, few tiles with many rows (shared out), two consumers
SHAPES = [(1, 64, 64), (7, 8, 8), (63, 72, 136), (64, 128, 256), (65, 200, 64), (511, 264, 520), (513, 1000, 72),
          (3000, 64, 40), (9000, 300, 200), (20011, 104, 264), (200, 4104, 4096), (64, 5000, 4608), (1100, 2304, 2056)]


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K,M,N", SHAPES)
def test_dense(ops, K, M, N, dtype, out):
    ld = -(-M // 8) * 8, -(-N // 8) * 8
    a = draw(K, ld[0], DT[dtype], K + M)[:, :M]
    b = draw(K, ld[1], DT[dtype], K + N + 1)[:, :N]
    d = ops.gemm(a, b, out_dtype=DT[out], a_transposed=True)
    assert d.shape == (M, N) and d.dtype == DT[out]
    gu.assert_close(d, *want(a, b, DT[out]), "D")
    assert torch.equal(d, ops.gemm(a, b, out_dtype=DT[out], a_transposed=True))


@pytest.mark.parametrize("K,M,N", SHAPES)
def test_integers_are_exact(ops, K, M, N):
    """Every partial sum is below 2^24."""
    a, b = draw(K, -(-M // 8) * 8, torch.bfloat16, 1, True), draw(K, -(-N // 8) * 8, torch.bfloat16, 2, True)
    d = ops.gemm(a, b, out_dtype=torch.float32, a_transposed=True)
    assert torch.equal(d.double(), a.double().t() @ b.double())


def test_long_sums_keep_their_bits(ops):
    """65536 rows: a sum that stayed on the tensor cores would be 7e-5 off; joined
    ones are, like sums of FP32 blocks, within 2e-6 (in the 2-norm)."""
    a, b = draw(65536, 128, torch.bfloat16, 3), draw(65536, 128, torch.bfloat16, 4)
    d = ops.gemm(a, b, out_dtype=torch.float32, a_transposed=True).double()
    ref = a.double().t() @ b.double()
    assert float((d - ref).norm() / ref.norm()) < 2e-6


def test_more_elements_than_an_int(ops):
    """560000 rows of 4096: what the last rows add arrives, and nothing else."""
    rows, M = 560000, 4096
    a = torch.zeros(rows, M, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    a[-70:], b[-70:] = draw(70, M, torch.bfloat16, 20, True), draw(70, 64, torch.bfloat16, 21, True)
    want_d = a[-70:].double().t() @ b[-70:].double()
    for out in (torch.float32, torch.bfloat16):
        assert torch.equal(ops.gemm(a, b, out_dtype=out, a_transposed=True), want_d.to(out))
    off = gu.offsets([rows - 70, 70])
    d = ops.grouped_gemm_wgrad(a, b, off)
    assert bool((d[0] == 0).all()) and torch.equal(d[1], want_d.to(torch.bfloat16))


def test_strides_and_what_lies_between_rows(ops):
    K, M, N = 777, 136, 200
    a, b = draw(K, M, torch.bfloat16, 5), draw(K, N, torch.bfloat16, 6)
    pa = torch.full((K, M + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    pb = torch.full((K, N + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    pa[:, :M], pb[:, :N] = a, b
    for out in (torch.float32, torch.bfloat16):
        buf = torch.full((M, N + 16), 7.0, dtype=out, device="cuda")
        ops.gemm(pa[:, :M], pb[:, :N], out=buf[:, :N], a_transposed=True)
        assert torch.equal(buf[:, :N], ops.gemm(a, b, out_dtype=out, a_transposed=True))
        assert bool((buf[:, N:] == 7.0).all())


def test_no_rows(ops):
    e = dict(dtype=torch.bfloat16, device="cuda")
    d = torch.full((24, 40), 7.0, device="cuda")
    ops.gemm(torch.empty(0, 24, **e), torch.empty(0, 40, **e), out=d, a_transposed=True)
    assert bool((d == 0).all())
    assert ops.gemm(torch.empty(5, 0, **e), torch.empty(5, 40, **e), a_transposed=True).shape == (0, 40)


COUNTS = [
    [300, 0, 256, 1, 0, 255, 37, 513, 0],
    [0, 0, 5],
    [64],
    [63, 1, 64, 65, 127, 129],
    [7, 0] * 40,
    [0, 5000, 1],
    [0, 0],
]


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("dtype,M,N", [("bf16", 136, 200), ("fp16", 64, 64), ("bf16", 1032, 264), ("bf16", 2048, 2048)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "x".join(map(str, c[:4])))
def test_experts(ops, counts, dtype, M, N, out):
    """A group's rows, and not its neighbours': those hold NaN at each border in turn."""
    rows = sum(counts)
    a, b = draw(rows, M, DT[dtype], rows + M), draw(rows, N, DT[dtype], rows + N)
    off = gu.offsets(counts)
    d = ops.grouped_gemm_wgrad(a, b, off, out_dtype=DT[out])
    assert d.shape == (len(counts), M, N)
    at = 0
    for g, c in enumerate(counts):
        if c == 0:
            assert bool((d[g] == 0).all())
        elif g < 12:
            gu.assert_close(d[g], *want(a[at:at + c], b[at:at + c], DT[out]), "group %d" % g)
        at += c
    assert torch.equal(d, ops.grouped_gemm_wgrad(a, b, off, out_dtype=DT[out]))


def test_a_groups_neighbours_are_not_read(ops):
    counts = [70, 65, 1, 200]
    a, b = draw(336, 72, torch.bfloat16, 8), draw(336, 136, torch.bfloat16, 9)
    off = gu.offsets(counts)
    clean = ops.grouped_gemm_wgrad(a, b, off)
    at = 0
    for g, c in enumerate(counts):
        x, y = a.clone(), b.clone()
        x[at:at + c], y[at:at + c] = float("nan"), float("inf")
        d = ops.grouped_gemm_wgrad(x, y, off)
        for o in range(len(counts)):
            assert bool(d[o].isnan().all()) if o == g else torch.equal(d[o], clean[o])
        at += c


def test_broken_offsets_are_reported(ops):
    a, b = draw(300, 64, torch.bfloat16, 10), draw(300, 72, torch.bfloat16, 11)
    for bad in ([0, 100, 250], [0, 400, 300], [5, 100, 300], [0, -7, 300], [0, 200, 100, 300]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        d = ops.grouped_gemm_wgrad(a, b, off, out_dtype=torch.float32)
        assert ops.last_device_error()[0] == 1, bad
        assert bool(d.isfinite().all())


@pytest.mark.parametrize("shape", [(600, 256, 256), (20000, 256, 256), (300, 4096, 4864)])
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_stalled_calls_give_up(ops, shape, grouped, out):
    K, M, N = shape
    a, b = draw(K, M, torch.bfloat16, 12, True), draw(K, N, torch.bfloat16, 13, True)
    off = gu.offsets([100, K - 100])

    def run():
        if grouped:
            return ops.grouped_gemm_wgrad(a, b, off, out_dtype=DT[out])
        return ops.gemm(a, b, out_dtype=DT[out], a_transposed=True)

    ops.set_watchdog_ns(50_000_000)  # 50 ms
    ops.debug_set_tx_extra(1024)
    try:
        run()
        st, word = ops.last_device_error()
    finally:
        ops.debug_set_tx_extra(0)
        ops.set_watchdog_ns(0)
    assert st == 5 and (word >> 56) == 1, (st, hex(word))
    d = run()
    ref = a[:100].double().t() @ b[:100].double() if grouped else a.double().t() @ b.double()
    assert torch.equal((d[0] if grouped else d), ref.to(DT[out]))


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("dtype,rows", [("fp16", 8192), ("fp16", 8256), ("fp16", 200000), ("bf16", 65536),
                                        ("bf16", 600000)])
def test_long_sums_of_one_sign(ops, dtype, rows, grouped):
    """16-bit results of wide products.  A sum on the tensor cores is cut towards
    zero at every step of 16 rows, by up to 2^-23 of itself: however many rows, the
    results are on average less than an eighth of a rounding short.  (The roundings
    themselves, over 64 columns of 4096 spread over half a binade, average to less
    than u / 128.)"""
    M, N, dt = 4096, 8192, DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(rows)
    a = torch.empty(rows, M, dtype=dt, device="cuda").uniform_(0.5, 1.5, generator=g)
    a *= torch.empty(M, device="cuda").uniform_(0.5, 1.0, generator=g).to(dt)
    b = torch.empty(rows, N, dtype=dt, device="cuda").uniform_(0.05, 0.15, generator=g)
    if grouped:
        d = ops.grouped_gemm_wgrad(a, b, gu.offsets([0, rows]))[1]
    else:
        d = ops.gemm(a, b, out_dtype=dt, a_transposed=True)
    cols = torch.arange(64, device="cuda") * (N // 64) + 5
    ref = torch.zeros(M, 64, dtype=torch.float64, device="cuda")
    for at in range(0, rows, 50000):
        ref += a[at:at + 50000].double().t() @ b[at:at + 50000, cols].double()
    short = float(((d[:, cols].double() - ref) / ref).mean())
    assert abs(short) <= gu.u(dt) * (1 / 8 + 1 / 128), short


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("counts", [[7, 0] * 40, [64, 1, 0] * 30, [130, 3] * 35], ids=lambda c: "x".join(map(str, c[:3])))
def test_every_one_of_many_groups(ops, counts, out):
    """More groups than a launch takes: each of them within its bound, but for four
    that hold NaN, on both sides of the launches' border, and those alone hold NaN."""
    rows, M, N = sum(counts), 136, 200
    a, b = draw(rows, M, torch.bfloat16, 40), draw(rows, N, torch.bfloat16, 41)
    bounds = gu.offsets(counts).tolist()
    full = [g for g, c in enumerate(counts) if c]
    bad = {full[0], max(g for g in full if g < 64), min(g for g in full if g >= 64), full[-1]}
    for g in bad:
        a[bounds[g]:bounds[g + 1]] = float("nan")
    d = ops.grouped_gemm_wgrad(a, b, gu.offsets(counts), out_dtype=DT[out])
    for g, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if g in bad:
            assert bool(d[g].isnan().all()), g
        elif lo == hi:
            assert bool((d[g] == 0).all()), g
        else:
            gu.assert_close(d[g], *want(a[lo:hi], b[lo:hi], DT[out]), "group %d" % g)
