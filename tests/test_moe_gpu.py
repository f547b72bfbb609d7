"""Routed rows on the GPU against plain implementations in 64 bits: the sort
by expert, dispatch, combine and their gradients."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

# unit roundoff of each type
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops


def make_ids(T, k, E, seed, how="random", dtype=torch.int64):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (T, k))
    if how == "one":
        ids[:] = E - 1
    elif how == "dropped":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[rng.random((T, k)) < 0.1] = E + 5
        if T > 2:
            ids[T // 2] = -1  # a token that lost all its experts
    elif how == "none":
        ids[:] = -1
    return torch.from_numpy(ids).to(dtype).cuda()


def sort_plain(ids, E):
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    key = np.where((flat < 0) | (flat >= E), E, flat)
    order = np.argsort(key, kind="stable")
    position = np.empty_like(order)
    position[order] = np.arange(order.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    return offsets, order, position


@pytest.mark.parametrize("T,k,E,how", [
    (1, 1, 1, "random"), (1, 8, 32, "random"), (16, 8, 32, "random"), (33, 3, 7, "dropped"), (5, 2, 1024, "dropped"),
    (512, 8, 64, "random"), (513, 8, 64, "dropped"), (4096, 8, 32, "random"), (4096, 1, 1, "random"),
    (3001, 6, 1000, "dropped"), (2000, 4, 1024, "random"), (40000, 8, 256, "random"), (7000, 8, 16, "one"),
    (300, 4, 8, "none"), (5000, 4, 8, "none"),
])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort_equals_a_stable_argsort(ops, T, k, E, how, dtype):
    ids = make_ids(T, k, E, 100 + T + k + E, how, dtype)
    r = ops.moe_sort(ids, E)
    offsets, order, position = sort_plain(ids, E)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy(), order)
    assert np.array_equal(r.position.cpu().numpy().reshape(-1), position)


def test_sort_of_no_tokens(ops):
    r = ops.moe_sort(torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 5)
    assert r.offsets.tolist() == [0] * 6 and r.order.numel() == 0 and r.position.shape == (0, 4)


def test_sort_feeds_the_grouped_product(ops):
    """offsets keep the grouped product's contract, empty experts included."""
    T, k, E, K, N = 100, 2, 16, 64, 128
    ids = make_ids(T, k, 5, 7)  # experts 5 .. 15 get nothing
    r = ops.moe_sort(ids, E)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-2, 3, (T, K), generator=g, device="cuda").bfloat16()
    Bs = [torch.randint(-2, 3, (K, N), generator=g, device="cuda").bfloat16() for _ in range(E)]
    rows = ops.grouped_gemm(ops.moe_dispatch(x, r), Bs, r.offsets)
    y = ops.moe_combine(rows.float(), r, torch.ones(T, k, device="cuda"))
    torch.cuda.synchronize()
    assert ops.last_device_error() == (0, 0)
    want = torch.stack([sum((x[t].double() @ Bs[e].double()).bfloat16().double() for e in ids[t].tolist())
                        for t in range(T)])
    assert torch.equal(y.double(), want)  # integers: every step is exact


SHAPES = [(1, 1, 4, 1, "random"), (1, 8, 16, 4096, "random"), (7, 3, 5, 7, "dropped"), (33, 2, 8, 64, "dropped"),
          (20, 8, 16, 2047, "dropped"), (64, 9, 16, 260, "random"), (70, 17, 32, 12, "dropped"), (9, 4, 8, 33, "none"),
          (600, 8, 32, 1024, "random")]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,H,how", SHAPES)
def test_dispatch_copies_and_zeroes(ops, T, k, E, H, how, dtype):
    ids = make_ids(T, k, E, 11 + T + H, how)
    r = ops.moe_sort(ids, E)
    g = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    x[0, 0] = float("nan")
    x[-1, -1] = float("inf")
    out = torch.full((T * k, H), float("nan"), dtype=dtype, device="cuda")
    ops.moe_dispatch(x, r, out=out)
    n = int(r.offsets[-1])
    want = x[(r.order // k).long()]
    want[n:] = 0
    size = torch.int32 if dtype == torch.float32 else torch.int16
    assert torch.equal(out.view(size), want.view(size))


def bound(terms_abs, terms, dtype):
    """A sum of `terms` products in FP32, each product and each addition
    rounded once, then one rounding to `dtype`: (terms + 1) 2^-24 of the sum
    of magnitudes, and u of the result (at most the same sum)."""
    return ((terms + 1) * 2.0 ** -24) * terms_abs + U[dtype] * terms_abs + 1e-7 * (dtype == torch.float16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,H,how", SHAPES)
def test_combine_and_dispatch_grad(ops, T, k, E, H, how, dtype):
    ids = make_ids(T, k, E, 12 + T + H, how)
    r = ops.moe_sort(ids, E)
    n = int(r.offsets[-1])
    g = torch.Generator(device="cuda").manual_seed(H + 1)
    rows = torch.randn(T * k, H, generator=g, device="cuda").to(dtype)
    rows[n:] = float("nan")  # what pairs without an expert hold is never used
    w = torch.randn(T, k, generator=g, device="cuda")
    kept = (r.position < n).double()
    picked = torch.nan_to_num(rows.double(), nan=0.0)[r.position.long()]
    for got, weight in ((ops.moe_combine(rows, r, w), w.double() * kept), (ops.moe_dispatch_grad(rows, r), kept)):
        want = (picked * weight[:, :, None]).sum(1)
        mag = (picked * weight[:, :, None]).abs().sum(1)
        err = (got.double() - want).abs()
        assert bool((err <= bound(mag, k, dtype)).all()), float((err - bound(mag, k, dtype)).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,H,how", SHAPES)
def test_combine_grad_against_its_formula(ops, T, k, E, H, how, dtype):
    ids = make_ids(T, k, E, 13 + T + H, how)
    r = ops.moe_sort(ids, E)
    n = int(r.offsets[-1])
    g = torch.Generator(device="cuda").manual_seed(H + 2)
    rows = torch.randn(T * k, H, generator=g, device="cuda").to(dtype)
    rows[n:] = float("nan")
    dy = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    w = torch.randn(T, k, generator=g, device="cuda")
    d_rows, d_w = ops.moe_combine_grad(dy, rows, r, w)
    kept = (r.position < n).double()
    want = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    want[r.position.reshape(-1).long()] = ((w.double() * kept)[:, :, None] * dy.double()[:, None, :]).reshape(-1, H)
    # the product in FP32, then one rounding (fp16: subnormals lose 2^-25 at most)
    err = (d_rows.double() - want).abs()
    assert bool((err <= (2.0 ** -24 + 1.01 * U[dtype]) * want.abs() + 2.0 ** -25 * (dtype == torch.float16)).all())
    assert bool((d_rows[n:] == 0).all())
    prod = torch.nan_to_num(rows.double(), nan=0.0)[r.position.long()] * dy.double()[:, None, :]
    err = (d_w.double() - prod.sum(2) * kept).abs()
    # H products in FP32, summed along threads and then lanes: H + 16 roundings bound any order of it
    assert bool((err <= (H + 16) * 2.0 ** -24 * prod.abs().sum(2) * kept).all())


def test_no_columns(ops):
    r = ops.moe_sort(make_ids(5, 3, 4, 2), 4)
    w = torch.rand(5, 3, device="cuda")
    x, rows = torch.empty(5, 0, device="cuda"), torch.empty(15, 0, device="cuda")
    assert ops.moe_dispatch(x, r).shape == (15, 0) and ops.moe_combine(rows, r, w).shape == (5, 0)
    d_rows, d_w = ops.moe_combine_grad(x, rows, r, w)
    assert d_rows.shape == (15, 0) and bool((d_w == 0).all())


def test_gradients_against_differences(ops):
    """The combine is linear in rows and in weights, so central differences of
    it with steps of powers of two carry only its FP32 rounding."""
    T, k, E, H = 12, 3, 5, 20
    r = ops.moe_sort(make_ids(T, k, E, 3, "dropped"), E)
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = torch.randn(T * k, H, generator=g, device="cuda")
    w = torch.randn(T, k, generator=g, device="cuda")
    dy = torch.randn(T, H, generator=g, device="cuda")
    d_rows, d_w = ops.moe_combine_grad(dy, rows, r, w)

    def loss(rows, w):
        return float((ops.moe_combine(rows, r, w).double() * dy.double()).sum())

    # each loss carries at most (k + 1) 2^-24 of the sum of |dy w rows|
    mag = float((dy.double().abs()[:, None, :] * w.double().abs()[:, :, None]
                 * rows.double().abs()[r.position.long()]).sum()) + 4.0 * T * H * k
    tol = (k + 2) * 2.0 ** -24 * mag
    for t, j in ((0, 0), (3, 2), (T // 2, 1), (T - 1, 0)):
        hi, lo = w.clone(), w.clone()
        hi[t, j] += 1.0
        lo[t, j] -= 1.0
        step = float(hi[t, j].double() - lo[t, j].double())
        assert abs((loss(rows, hi) - loss(rows, lo)) / step - float(d_w[t, j])) <= 2 * tol
    for i, c in ((0, 0), (7, 19), (T * k - 1, 4)):
        hi, lo = rows.clone(), rows.clone()
        hi[i, c] += 1.0
        lo[i, c] -= 1.0
        step = float(hi[i, c].double() - lo[i, c].double())
        assert abs((loss(hi, w) - loss(lo, w)) / step - float(d_rows[i, c])) <= 2 * tol
    # dispatch: <dispatch(x), d> = <x, dispatch_grad(d)> for every x and d
    x = torch.randn(T, H, generator=g, device="cuda")
    d = torch.randn(T * k, H, generator=g, device="cuda")
    a = (ops.moe_dispatch(x, r).double() * d.double()).sum()
    b = (x.double() * ops.moe_dispatch_grad(d, r).double()).sum()
    assert abs(float(a - b)) <= (k + 1) * 2.0 ** -24 * float((x.abs().sum() * d.abs().max()).double())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (8, 8), (5, 1)])
def test_strided_and_shifted_rows(ops, dtype, pad, shift):
    """Leading dimensions above H and bases off 16 bytes; what lies between
    the rows is neither read into results nor written."""
    T, k, E, H = 19, 3, 6, 96
    r = ops.moe_sort(make_ids(T, k, E, 21, "dropped"), E)
    g = torch.Generator(device="cuda").manual_seed(9)

    def view(rows, fill):
        flat = torch.full((rows * (H + pad) + shift,), fill, dtype=dtype, device="cuda")
        v = flat[shift:].view(rows, H + pad)[:, :H]
        return flat, v

    xf, x = view(T, float("nan"))
    x.copy_(torch.randn(T, H, generator=g, device="cuda"))
    rf, rows = view(T * k, 7.0)
    ops.moe_dispatch(x, r, out=rows)
    assert torch.equal(rows, ops.moe_dispatch(x.contiguous(), r))
    gaps = rf[shift:].view(T * k, H + pad)[:, H:]
    assert bool((gaps == 7.0).all())
    w = torch.rand(T, k, device="cuda")
    yf, y = view(T, 5.0)
    ops.moe_combine(rows, r, w, out=y)
    assert torch.equal(y, ops.moe_combine(rows.contiguous(), r, w))
    assert bool((yf[shift:].view(T, H + pad)[:, H:] == 5.0).all())
    a, b = ops.moe_combine_grad(x, rows, r, w)
    c, d = ops.moe_combine_grad(x.contiguous(), rows.contiguous(), r, w)
    # another vector width adds the inner products in another order
    assert torch.equal(a, c) and torch.allclose(b, d, rtol=0, atol=(H + 16) * 2.0 ** -23 * H * 16)


def test_rows_past_32_bits(ops):
    """More than 2^31 elements in the rows: the last ones are found."""
    T, k, E, H = 36000, 2, 4, 32768
    assert T * k * H > 1 << 31
    r = ops.moe_sort(make_ids(T, k, E, 31), E)
    x = torch.randn(T, 1, device="cuda", dtype=torch.float32).bfloat16().expand(T, H).contiguous()
    rows = ops.moe_dispatch(x, r)
    at = torch.tensor([0, 1, T, 2 * T - 2, 2 * T - 1], device="cuda")
    assert torch.equal(rows[at], x[(r.order[at] // k).long()])
    y = ops.moe_dispatch_grad(rows, r)
    assert torch.equal(y, (x.float() * 2).bfloat16())


def test_on_a_stream_of_its_own(ops):
    side = torch.cuda.Stream()
    T, k, E, H = 512, 4, 16, 512
    ids = make_ids(T, k, E, 41)
    x = torch.randn(T, H, device="cuda").bfloat16()
    w = torch.rand(T, k, device="cuda")
    base = ops.moe_sort(ids, E)
    want = ops.moe_combine(ops.moe_dispatch(x, base), base, w)
    torch.cuda.synchronize()
    r = ops.moe_sort(ids, E, stream=side)
    rows = ops.moe_dispatch(x, r, stream=side)
    y = ops.moe_combine(rows, r, w, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


def test_positions_out_of_range_are_reported_and_not_followed(ops):
    T, k, E, H = 6, 2, 3, 16
    r = ops.moe_sort(make_ids(T, k, E, 51), E)
    bad = r.position.clone()
    bad[2, 1], bad[4, 0] = T * k, -3
    r = ops.Routing(r.offsets, r.order, bad)
    x = torch.ones(T, H, device="cuda")
    out = torch.full((T * k, H), 9.0, device="cuda")
    ops.moe_dispatch(x, r, out=out)
    status, word = ops.last_device_error()
    assert status == 1 and word >> 56 == 2
    assert int((out == 9.0).all(1).sum()) == 2  # the two rows that no pair names
    y = ops.moe_combine(x.repeat(k, 1), r, torch.ones(T, k, device="cuda"))
    assert ops.last_device_error()[0] == 1
    assert y[:, 0].tolist() == [2.0, 2.0, 1.0, 2.0, 1.0, 2.0]
    ops.moe_combine_grad(x, x.repeat(k, 1), r, torch.ones(T, k, device="cuda"))
    assert ops.last_device_error()[0] == 1
    assert ops.last_device_error() == (0, 0)


def test_python_refusals(ops):
    T, k, E, H = 4, 2, 3, 16
    r = ops.moe_sort(make_ids(T, k, E, 61), E)
    x = torch.ones(T, H, device="cuda")
    rows = torch.ones(T * k, H, device="cuda")
    w = torch.ones(T, k, device="cuda")
    for call in (lambda: ops.moe_dispatch(x.double(), r), lambda: ops.moe_dispatch(x.to(torch.int32), r)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: ops.moe_dispatch(x[:3], r), lambda: ops.moe_dispatch(x[:1].expand(T, H), r),
                 lambda: ops.moe_dispatch(x.t().contiguous().t(), r), lambda: ops.moe_dispatch(x, r, out=x),
                 lambda: ops.moe_dispatch(x, r._replace(position=r.position.long())),
                 lambda: ops.moe_dispatch(x, r._replace(offsets=r.offsets.cpu())),
                 lambda: ops.moe_combine(rows, r, w.double()), lambda: ops.moe_combine(rows, r, w[:, :1]),
                 lambda: ops.moe_combine(rows[1:], r, w), lambda: ops.moe_combine_grad(x.half(), rows, r, w),
                 lambda: ops.moe_combine_grad(x[:, :8], rows, r, w), lambda: ops.moe_sort(r.position, 0)):
        with pytest.raises(ValueError):
            call()
