"""The gated feed-forward block on a GPU: its forward pass, gate and up kept in
8 bits, its backward pass, for one weight and for experts, against 64-bit forms
within the bounds of gated_util."""
import pytest
import torch

import gated_util as gu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


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


def data(M, K, N, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    return (randn(M, K) * std).to(dtype), (randn(K, N) * K ** -0.5).to(dtype), randn(M, N // 2).to(dtype)


def padded(t, extra, fill=float("nan")):
    """The same matrix with `extra` more elements from row to row."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf, buf[:, :t.shape[1]]


# rows: one, the small-M kernel's ends, one tile and more, two consumers; columns: a unit's half, ragged
# blocks and tiles; depth: one step, ragged k-blocks
SHAPES = [(1, 64, 128), (1, 4096, 4096), (7, 72, 16), (128, 200, 144), (129, 200, 144), (300, 264, 528), (300, 8, 240),
          (512, 520, 400), (1000, 128, 2048), (2500, 136, 2832), (4200, 192, 4112)]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_forward(ops, M, K, N, dtype, transposed):
    x, w, _ = data(M, K, N, DT[dtype], M + N)
    h = ops.gemm_swiglu(x, w.t().contiguous() if transposed else w, b_transposed=transposed)
    assert h.dtype == x.dtype
    gu.assert_close(h, *gu.forward(*gu.gated(x, w), x.dtype), "h")


def check_kept(kept, gate, up, eg, eu):
    """Every value within half a step of gate and up as the product gave them."""
    v, e = torch.cat([gate, up], 1), torch.cat([eg, eu], 1)
    at, n = gu.blocks(v, 2)
    amax = torch.zeros(v.shape[0], n, dtype=torch.float64, device=v.device)
    amax.scatter_reduce_(1, at.expand(v.shape[0], -1), v.abs(), "amax")
    worst = torch.zeros_like(amax)
    worst.scatter_reduce_(1, at.expand(v.shape[0], -1), e, "amax")
    gu.assert_close(kept.scales, amax / 127, worst / 127 + 2.0 ** -23 * amax, "scales")
    step = (amax + worst)[:, at] / 127
    gu.assert_close(gu.value(kept), v, (0.5 + 127 * 2.0 ** -22) * step + e, "kept")
    assert int(kept.codes.to(torch.int32).abs().max()) <= 127


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_forward_that_keeps_gate_and_up(ops, M, K, N, dtype, transposed):
    x, w, _ = data(M, K, N, DT[dtype], M + N + 1)
    h, kept = ops.gemm_swiglu(x, w.t().contiguous() if transposed else w, b_transposed=transposed, keep_int8=True)
    g = gu.gated(x, w)
    gu.assert_close(h, *gu.forward(*g, x.dtype), "h")
    check_kept(kept, *g)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_backward_from_the_inputs(ops, M, K, N, dtype, transposed):
    x, w, dh = data(M, K, N, DT[dtype], M + N + 2)
    got = ops.gemm_swiglu_grad(dh, x, w.t().contiguous() if transposed else w, b_transposed=transposed)
    assert got.h is None
    d, e = gu.backward(dh, *gu.gated(x, w), x.dtype)
    xd, wd = x.double(), w.double()
    gu.assert_close(got.dx, *gu.through(d, e, wd.t(), 0.0, x.dtype), "dx")
    dw = got.dw.t() if transposed else got.dw
    gu.assert_close(dw, *gu.through(xd.t(), 0.0, d, e, x.dtype), "dw")


@pytest.mark.parametrize("keep_x", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_backward_from_8_bits(ops, M, K, N, dtype, keep_x):
    x, w, dh = data(M, K, N, DT[dtype], M + N + 3)
    _, kept = ops.gemm_swiglu(x, w, keep_int8=True)
    v = gu.value(kept)
    gate, up = v[:, :N // 2], v[:, N // 2:]
    ev = 2.0 ** -23  # a code times its scale, rounded to FP32
    eg, eu = ev * gate.abs(), ev * up.abs()
    given = ops.quantize_int8(x) if keep_x else x
    xv = gu.value(given) if keep_x else x.double()
    ex = gu.u(x.dtype) * xv.abs().t() + gu.tiny(x.dtype) if keep_x else 0.0
    got = ops.gemm_swiglu_grad(dh, given, w, kept=kept, with_h=True)
    gu.assert_close(got.h, *gu.forward(gate, up, eg, eu, x.dtype), "h")
    d, e = gu.backward(dh, gate, up, eg, eu, x.dtype)
    gu.assert_close(got.dx, *gu.through(d, e, w.double().t(), 0.0, x.dtype), "dx")
    gu.assert_close(got.dw, *gu.through(xv.t(), ex, d, e, x.dtype), "dw")
    gu.assert_close(ops.swiglu_grad(dh, kept), d, e, "dgu")


@pytest.mark.parametrize("need_dx,need_dw", [(True, False), (False, True), (False, False)])
def test_only_the_gradients_asked_for(ops, need_dx, need_dw):
    x, w, dh = data(200, 72, 144, torch.bfloat16, 4)
    whole = ops.gemm_swiglu_grad(dh, x, w)
    got = ops.gemm_swiglu_grad(dh, x, w, need_dx=need_dx, need_dw=need_dw)
    assert (got.dx is not None, got.dw is not None) == (need_dx, need_dw)
    assert got.dx is None or torch.equal(got.dx, whole.dx)
    assert got.dw is None or torch.equal(got.dw, whole.dw)


def test_gradients_against_differences(ops):
    """The gradients along a direction against central differences of L = sum(dh * h)
    in 64 bits: the difference's own error is the third derivative's, here below
    1e-4 of the terms' sizes with a step of 1e-3 along unit-size directions; the
    gradients' is their bound's."""
    M, K, N = 37, 40, 80
    x, w, dh = data(M, K, N, torch.bfloat16, 5)
    got = ops.gemm_swiglu_grad(dh, x, w)
    g = torch.Generator(device="cuda").manual_seed(6)
    px = torch.randn(M, K, generator=g, device="cuda", dtype=torch.float64)
    pw = torch.randn(K, N, generator=g, device="cuda", dtype=torch.float64) * K ** -0.5

    def loss(t):
        p = (x.double() + t * px) @ (w.double() + t * pw)
        gate, up = p[:, :N // 2], p[:, N // 2:]
        return dh.double() * gate * torch.sigmoid(gate) * up

    step = 1e-3
    terms = (loss(step) - loss(-step)) / (2 * step)
    want = float(terms.sum())
    have = float((got.dx.double() * px).sum() + (got.dw.double() * pw).sum())
    d, e = gu.backward(dh, *gu.gated(x, w), x.dtype)
    bx = gu.through(d, e, w.double().t(), 0.0, x.dtype)[1]
    bw = gu.through(x.double().t(), 0.0, d, e, x.dtype)[1]
    assert abs(have - want) <= float((bx * px.abs()).sum() + (bw * pw.abs()).sum() + 1e-4 * terms.abs().sum())


def test_strides_and_what_lies_between_rows(ops):
    """Padded rows of every operand: NaN between them is not read into a result, and
    the output's padding stays as it was."""
    for M in (1, 100, 300):
        x, w, dh = data(M, 136, 272, torch.bfloat16, 7 + M)
        xp, wp, dp = padded(x, 16)[1], padded(w, 24)[1], padded(dh, 8)[1]
        buf, out = padded(torch.zeros(M, 136, dtype=torch.bfloat16, device="cuda"), 8, 7.0)
        ops.gemm_swiglu(xp, wp, out=out)
        assert torch.equal(out, ops.gemm_swiglu(x, w)) and bool((buf[:, 136:] == 7.0).all())
        kept, same = ops.gemm_swiglu(xp, wp, keep_int8=True)[1], ops.gemm_swiglu(x, w, keep_int8=True)[1]
        assert torch.equal(kept.codes, same.codes) and torch.equal(kept.scales, same.scales)
        a, b = ops.gemm_swiglu_grad(dp, xp, wp), ops.gemm_swiglu_grad(dh, x, w)
        assert torch.equal(a.dx, b.dx) and torch.equal(a.dw, b.dw)
        assert torch.equal(ops.swiglu_grad(dp, kept), ops.swiglu_grad(dh, kept))


def test_empty_and_depthless(ops):
    e = dict(dtype=torch.bfloat16, device="cuda")
    h, kept = ops.gemm_swiglu(torch.empty(0, 64, **e), torch.empty(64, 128, **e), keep_int8=True)
    assert h.shape == (0, 64) and kept.shape == (0, 128)
    got = ops.gemm_swiglu_grad(torch.empty(0, 64, **e), torch.empty(0, 64, **e), torch.empty(64, 128, **e))
    assert got.dx.shape == (0, 64) and bool((got.dw == 0).all())
    for rows in (5, 300):
        h, kept = ops.gemm_swiglu(torch.empty(rows, 0, **e), torch.empty(0, 128, **e), keep_int8=True)
        assert bool((h == 0).all()) and bool((kept.codes == 0).all()) and bool((kept.scales == 0).all())
        got = ops.gemm_swiglu_grad(torch.ones(rows, 64, **e), torch.empty(rows, 0, **e), torch.empty(0, 128, **e))
        assert got.dx.shape == (rows, 0) and got.dw.shape == (0, 128)


def test_infinities_and_nan(ops):
    """A row with a NaN and one with an infinity: their results are NaN or infinite as
    FP32 makes them, their kept blocks read back as NaN, all other rows are untouched."""
    x, w, dh = data(300, 64, 256, torch.bfloat16, 8)
    clean_h, clean = ops.gemm_swiglu(x, w, keep_int8=True)
    x[17, 3], x[200, 5] = float("nan"), float("inf")
    h, kept = ops.gemm_swiglu(x, w, keep_int8=True)
    rest = torch.ones(300, dtype=torch.bool, device="cuda")
    rest[17] = rest[200] = False
    assert torch.equal(h[rest], clean_h[rest]) and bool(h[17].isnan().all()) and not bool(h[200].isfinite().any())
    assert torch.equal(kept.codes[rest], clean.codes[rest]) and torch.equal(kept.scales[rest], clean.scales[rest])
    back = ops.dequantize_int8(kept)
    assert bool(back[17].isnan().all()) and bool(back[200].isnan().all())
    d = ops.swiglu_grad(dh, kept)
    assert bool(d[17].isnan().all()) and bool(d[rest].isfinite().all())


def test_far_gates(ops):
    """Gates of +-1e4 and next to 0: silu and its slope go to their limits, not to NaN."""
    K, I = 64, 64
    x = torch.zeros(4, K, dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[1, 0], x[2, 0] = 10000.0, -10000.0, 1e-30
    w = torch.zeros(K, 2 * I, dtype=torch.bfloat16, device="cuda")
    w[0, :I] = 1.0
    w[0, I:] = 0.5
    dh = torch.ones(4, I, dtype=torch.bfloat16, device="cuda")
    h = ops.gemm_swiglu(x, w).double()
    gate = x[:, :1].double().expand(4, I)
    up = 0.5 * gate
    assert torch.equal(h[1], torch.zeros_like(h[1])) and torch.allclose(h, gate * torch.sigmoid(gate) * up, rtol=2.0 ** -7)
    got = ops.gemm_swiglu_grad(dh, x, w)
    assert bool(got.dx.isfinite().all()) and bool(got.dw.isfinite().all())
    _, kept = ops.gemm_swiglu(torch.cat([x] * 40), w, keep_int8=True)
    assert bool(ops.swiglu_grad(torch.cat([dh] * 40), kept).isfinite().all())


# ------------------------------------------------------------- experts ---

COUNTS = [
    [300, 0, 256, 1, 0, 255, 37, 513, 0],
    [0, 0, 5],
    [64],
    [3, 31, 32, 33, 63, 64, 65, 127, 129],
    [7] * 70,  # two launches
    [0, 2000, 1, 900],
]


def experts(counts, K, N, dtype, seed):
    M = sum(counts)
    x, _, dh = data(M, K, N, dtype, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    w = (torch.randn(len(counts), K, N, generator=g, device="cuda") * K ** -0.5).to(dtype)
    return x, w, dh, gu.offsets(counts)


def by_expert(counts, *mats):
    at = 0
    for i, c in enumerate(counts):
        yield (i, slice(at, at + c)) + tuple(m[at:at + c] for m in mats)
        at += c


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype,K,N", [("bf16", 200, 400), ("fp16", 64, 128), ("bf16", 136, 2064)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "x".join(map(str, c[:4])))
def test_experts(ops, counts, dtype, K, N, transposed):
    dt = DT[dtype]
    x, w, dh, off = experts(counts, K, N, dt, sum(counts) + K)
    ws = [(m.t() if transposed else m).contiguous() for m in w.unbind(0)]
    h, kept = ops.grouped_gemm(x, ws, off, swiglu=True, b_transposed=transposed, keep_int8=True)
    again = ops.grouped_gemm_swiglu_grad(dh, x, ws, off, b_transposed=transposed)
    from8 = ops.grouped_gemm_swiglu_grad(dh, ops.quantize_int8(x), ws, off, kept=kept, with_h=True,
                                         b_transposed=transposed)
    assert again.dw.shape == (len(counts),) + tuple(ws[0].shape)
    for e, rows, xe, he, dhe in by_expert(counts, x, h, dh):
        we = w[e]
        g = gu.gated(xe, we)
        gu.assert_close(he, *gu.forward(*g, dt), "h of expert %d" % e)
        if xe.shape[0]:
            check_kept(ops.Int8Matrix(kept.codes[rows], kept.scales[rows], 2), *g)
        d, b = gu.backward(dhe, *g, dt)
        gu.assert_close(again.dx[rows], *gu.through(d, b, we.double().t(), 0.0, dt), "dx of expert %d" % e)
        dw = again.dw[e].t() if transposed else again.dw[e]
        gu.assert_close(dw, *gu.through(xe.double().t(), 0.0, d, b, dt), "dw of expert %d" % e)
        v = gu.value(ops.Int8Matrix(kept.codes[rows], kept.scales[rows], 2))
        gate, up = v[:, :N // 2], v[:, N // 2:]
        eg, eu = 2.0 ** -23 * gate.abs(), 2.0 ** -23 * up.abs()
        gu.assert_close(from8.h[rows], *gu.forward(gate, up, eg, eu, dt), "h again")
        d, b = gu.backward(dhe, gate, up, eg, eu, dt)
        gu.assert_close(from8.dx[rows], *gu.through(d, b, we.double().t(), 0.0, dt), "dx from 8 bits")


def test_rows_behind_the_last_group(ops):
    """Offsets that end early break the contract: reported, and those rows of H, of
    the kept matrix and of dgu stay as they were."""
    counts, extra, K, N = [100, 0, 233], 70, 72, 144
    x, w, dh, off = experts(counts + [extra], K, N, torch.bfloat16, 9)
    L, s = ops.lib(), torch.cuda.current_stream().cuda_stream
    M, end = sum(counts) + extra, sum(counts)
    ws = list(w[:3].unbind(0))
    p, hold = ops._ptr_array([m.data_ptr() for m in ws])
    h = torch.full((M, N // 2), 3.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((M, N), 5, dtype=torch.int8, device="cuda")
    scales = torch.full((M, 4), 9.0, device="cuda")
    dgu = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    off = off[:4].contiguous()
    assert L.grouped_gemm_swiglu_keep(x.data_ptr(), p, h.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                      off.data_ptr(), 0, 0, 3, M, N, K, s) == 0
    assert ops.last_device_error()[0] == 1
    assert L.grouped_gemm_swiglu_grad(dh.data_ptr(), x.data_ptr(), p, dgu.data_ptr(), off.data_ptr(), 0, 0, 3, M, N, K,
                                      s) == 0
    assert ops.last_device_error()[0] == 1
    assert bool((h[end:] == 3.0).all()) and bool((codes[end:] == 5).all()) and bool((scales[end:] == 9.0).all())
    assert bool((dgu[end:] == 3.0).all())
    d, b = gu.backward(dh[:100], *gu.gated(x[:100], w[0]), torch.bfloat16)
    gu.assert_close(dgu[:100], d, b, "dgu")
    del hold


def test_the_same_weight_for_every_expert(ops):
    counts, K, N = [130, 0, 77], 64, 128
    x, w, dh, off = experts(counts, K, N, torch.bfloat16, 10)
    one = w[0].contiguous()
    got = ops.grouped_gemm_swiglu_grad(dh, x, [one] * 3, off)
    dense = ops.gemm_swiglu_grad(dh, x, one)
    assert torch.equal(got.dx, dense.dx)
    for e, rows, xe, dhe in by_expert(counts, x, dh):
        d, b = gu.backward(dhe, *gu.gated(xe, one), torch.bfloat16)
        gu.assert_close(got.dw[e], *gu.through(xe.double().t(), 0.0, d, b, torch.bfloat16), "dw")


# ------------------------------------------------- streams, graphs, runs ---

def step(ops, x, w, dh):
    h, kept = ops.gemm_swiglu(x, w, keep_int8=True)
    q = ops.quantize_int8(x)
    g = ops.gemm_swiglu_grad(dh, q, w, kept=kept, with_h=True)
    r = ops.gemm_swiglu_grad(dh, x, w)
    return [h, kept.codes, kept.scales, g.dx, g.dw, g.h, r.dx, r.dw]


def test_a_training_step_captured_twice_and_replayed_at_once(ops):
    """Two graphs of one stream, replayed on two streams without any order between
    them, give what eager calls give: no scratch memory is shared."""
    sets = [data(700, 264, 528, torch.bfloat16, 20 + i) for i in range(2)]
    want = [[t.clone() for t in step(ops, *s)] for s in sets]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    torch.cuda.synchronize()
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step(ops, *s))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_captured_behind_copies_and_on_forked_streams(ops):
    """Kernels that set up while the work before ends, behind a copy, behind each
    other and behind a fork's join, replayed with new inputs each time."""
    x, w, dh = data(300, 264, 528, torch.bfloat16, 25)
    xs, main, side = torch.empty_like(x), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        xs.copy_(x)
        a = ops.gemm_swiglu(xs, w)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            b = ops.gemm_swiglu(xs[:64], w)
            c = ops.gemm(xs, dh, a_transposed=True, out_dtype=torch.float32)
        d = ops.gemm_swiglu_grad(dh, xs, w)
        main.wait_stream(side)
        e = ops.gemm(a, c.to(torch.bfloat16), b_transposed=True)
    for seed in (26, 27, 28):
        x.copy_(data(300, 264, 528, torch.bfloat16, seed)[0])
        g.replay()
        torch.cuda.synchronize()
        want = ops.gemm_swiglu_grad(dh, x, w)
        h = ops.gemm_swiglu(x, w)
        t = ops.gemm(x, dh, a_transposed=True, out_dtype=torch.float32)
        for got, ref in ((a, h), (b, ops.gemm_swiglu(x[:64], w)), (c, t), (d.dx, want.dx), (d.dw, want.dw),
                         (e, ops.gemm(h, t.to(torch.bfloat16), b_transposed=True))):
            assert torch.equal(got, ref)


def test_more_elements_than_an_int(ops):
    """70000 x 32768: 2.3e9 codes and gradients; the first and last rows are right."""
    M, K, N = 70000, 64, 32768
    x, w, _ = data(M, K, N, torch.bfloat16, 33)
    h, kept = ops.gemm_swiglu(x, w, keep_int8=True)
    dgu = ops.swiglu_grad(h, kept)
    from_x = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    assert ops.lib().gemm_swiglu_grad(h.data_ptr(), x.data_ptr(), w.data_ptr(), from_x.data_ptr(), 0, 0, M, N, K, N // 2,
                                      K, N, N, torch.cuda.current_stream().cuda_stream) == 0
    for rows in (slice(0, 40), slice(M - 300, M)):
        g = gu.gated(x[rows], w)
        gu.assert_close(h[rows], *gu.forward(*g, torch.bfloat16), "h")
        part = ops.Int8Matrix(kept.codes[rows], kept.scales[rows], 2)
        check_kept(part, *g)
        gu.assert_close(from_x[rows], *gu.backward(h[rows], *g, torch.bfloat16), "dgu")
        v = gu.value(part)
        gate, up = v[:, :N // 2], v[:, N // 2:]
        e = 2.0 ** -23
        gu.assert_close(dgu[rows], *gu.backward(h[rows], gate, up, e * gate.abs(), e * up.abs(), torch.bfloat16), "dgu")


def test_columns_that_end_inside_16_bytes(ops):
    """x of 100 columns in rows of 104: the block and dw are taken, dx is refused."""
    x, w, dh = data(300, 104, 144, torch.bfloat16, 34)
    x[:, 100:] = float("nan")
    x, w = x[:, :100], w[:100]
    gu.assert_close(ops.gemm_swiglu(x, w), *gu.forward(*gu.gated(x, w), x.dtype), "h")
    gu.assert_close(ops.gemm_swiglu(x[:9], w), *gu.forward(*gu.gated(x[:9], w), x.dtype), "h of few rows")
    with pytest.raises(ValueError):
        ops.gemm_swiglu_grad(dh, x, w)
    got = ops.gemm_swiglu_grad(dh, x, w, need_dx=False)
    d, e = gu.backward(dh, *gu.gated(x, w), x.dtype)
    gu.assert_close(got.dw, *gu.through(x.double().t(), 0.0, d, e, x.dtype), "dw")


def test_a_stream_of_its_own(ops):
    x, w, dh = data(300, 72, 400, torch.bfloat16, 30)
    want = step(ops, x, w, dh)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h, kept = ops.gemm_swiglu(x, w, keep_int8=True, stream=s)
    q = ops.quantize_int8(x, stream=s)
    g = ops.gemm_swiglu_grad(dh, q, w, kept=kept, with_h=True, stream=s)
    r = ops.gemm_swiglu_grad(dh, x, w, stream=s)
    s.synchronize()
    for a, b in zip([h, kept.codes, kept.scales, g.dx, g.dw, g.h, r.dx, r.dw], want):
        assert torch.equal(a, b)


def test_runs_are_equal(ops):
    x, w, dh = data(1500, 520, 1040, torch.bfloat16, 31)
    first = [t.clone() for t in step(ops, x, w, dh)]
    for _ in range(5):
        for a, b in zip(step(ops, x, w, dh), first):
            assert torch.equal(a, b)


# ---------------------------------------------------------- bounded waits ---

@pytest.mark.parametrize("call", ["small", "forward", "two", "keep", "grad", "experts_keep", "experts_grad"])
def test_stalled_calls_give_up(ops, call):
    M = {"small": 64, "two": 4200}.get(call, 600)
    K, N = 1024, (4352 if call == "two" else 512)
    x, w, dh = data(M, K, N, torch.bfloat16, 40)
    off = gu.offsets([100, M - 100])
    ws = [w, w]
    run = {
        "small": lambda: ops.gemm_swiglu(x, w), "forward": lambda: ops.gemm_swiglu(x, w),
        "two": lambda: ops.gemm_swiglu(x, w), "keep": lambda: ops.gemm_swiglu(x, w, keep_int8=True)[0],
        "grad": lambda: ops.gemm_swiglu_grad(dh, x, w, need_dx=False, need_dw=False),
        "experts_keep": lambda: ops.grouped_gemm(x, ws, off, swiglu=True, keep_int8=True)[0],
        "experts_grad": lambda: ops.grouped_gemm_swiglu_grad(dh, x, ws, off, need_dx=False, need_dw=False),
    }[call]
    ops.set_watchdog_ns(50_000_000)  # 50 ms
    ops.debug_set_tx_extra(1024)
    try:
        run()
        st, word = ops.last_device_error()
    finally:
        ops.debug_set_tx_extra(0)
        ops.set_watchdog_ns(0)
    assert st == 5 and (word >> 56) == 1, (st, hex(word))
    h = ops.gemm_swiglu(x, w)
    gu.assert_close(h, *gu.forward(*gu.gated(x, w), x.dtype), "h after the stall")


# few rows and a wide dX: 76 tiles of 2 k-blocks and 160 tiles on 152 SMs, where the product's
# k-blocks would be shared out through a workspace of the stream's
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,K,N", [(72, 9728, 128), (17, 20480, 256)])
def test_captured_steps_of_few_rows(ops, M, K, N, transposed):
    """The first calls of a stream, in captures; the two graphs then run at once."""
    sets = []
    for i in range(2):
        x, w, dh = data(M, K, N, torch.bfloat16, 60 + i)
        sets.append((dh, x, w.t().contiguous() if transposed else w))
    want = []
    for dh, x, w in sets:
        r = ops.gemm_swiglu_grad(dh, x, w, b_transposed=transposed)
        want.append((r.dx.clone(), r.dw.clone()))
        d, e = gu.backward(dh, *gu.gated(x, w.t() if transposed else w), x.dtype)
        gu.assert_close(r.dx, *gu.through(d, e, w.double() if transposed else w.double().t(), 0.0, x.dtype), "dx")
    torch.cuda.synchronize()
    graphs, outs, side = [], [], torch.cuda.Stream()
    for dh, x, w in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(ops.gemm_swiglu_grad(dh, x, w, b_transposed=transposed))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(50):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for r, (dx, dw) in zip(outs, want):
        assert torch.equal(r.dx, dx) and torch.equal(r.dw, dw)


@pytest.mark.parametrize("from_8_bits", [False, True])
@pytest.mark.parametrize("M", [1, 300])
def test_a_kept_input_of_columns_that_end_inside_16_bytes(ops, M, from_8_bits):
    """x of 100 columns in rows of 104, kept in 8 bits: dw is that of the values that were kept."""
    x, w, dh = data(M, 104, 144, torch.bfloat16, 35)
    x, w = x[:, :100], w[:100]
    q = ops.quantize_int8(x)
    kept = ops.gemm_swiglu(x, w, keep_int8=True)[1] if from_8_bits else None
    got = ops.gemm_swiglu_grad(dh, q, w, kept=kept, need_dx=False)
    rows = torch.full((M, 104), float("nan"), dtype=x.dtype, device="cuda")[:, :100]
    want = ops.gemm_swiglu_grad(dh, ops.dequantize_int8(q, out=rows), w, kept=kept, need_dx=False)
    assert torch.equal(got.dw, want.dw) and got.dx is None
    if not from_8_bits:
        d, e = gu.backward(dh, *gu.gated(rows, w), x.dtype)
        gu.assert_close(got.dw, *gu.through(rows.double().t(), 0.0, d, e, x.dtype), "dw")
    with pytest.raises(ValueError):
        ops.gemm_swiglu_grad(dh, q, w, kept=kept)


@pytest.mark.parametrize("K", [64, 60])
def test_a_single_row_of_any_stride(ops, K):
    """One row whose stride is no multiple of 8, or less than the row, gives what a dense one does."""
    x, w, dh = data(1, K, 144, torch.bfloat16, 36)
    want = ops.gemm_swiglu_grad(dh, padded(x, 4 if K == 60 else 8)[1], w, need_dx=K == 64)
    h = ops.gemm_swiglu(padded(x, 4 if K == 60 else 8)[1], w)
    for ld in (61, 1):
        xs, ds = x.as_strided(x.shape, (ld, 1)), dh.as_strided(dh.shape, (ld, 1))
        assert torch.equal(ops.gemm_swiglu(xs, w), h)
        got = ops.gemm_swiglu_grad(ds, xs, w, need_dx=K == 64)
        assert torch.equal(got.dw, want.dw) and (K == 60 or torch.equal(got.dx, want.dx))
        d = ops.gemm(xs, ds, a_transposed=True, out_dtype=torch.float32)
        gu.assert_close(d, x.double().t() @ dh.double(), 2.0 ** -22 * (x.double().abs().t() @ dh.double().abs()), "d")
