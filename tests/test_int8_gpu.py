"""Matrices kept in 8 bits on a GPU: codes and scales bit for bit against the
definition in 64 bits, at every layout that takes a path of its own."""
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


def draw(rows, cols, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(torch.randn(cols, generator=g, device="cuda"))
    return x.to(dtype)


SHAPES = [(1, 1), (1, 64), (3, 8), (5, 16), (4, 24), (9, 63), (7, 65), (33, 100), (130, 128), (17, 200), (66, 264),
          (5, 511), (300, 512), (37, 1000), (2, 4104), (70, 4095), (1, 30001), (1000, 48), (65, 520)]


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_codes_scales_and_back(ops, rows, cols, dtype, parts):
    """The definition's codes and scales, bit for bit; read back, each value is the
    product rounded to FP32 and to the type: 2^-24 + u of it."""
    x = draw(rows, cols * parts, DT[dtype], rows + cols)
    q = ops.quantize_int8(x, parts=parts)
    codes, scales = gu.keep(x.float(), parts)
    assert torch.equal(q.scales, scales)
    assert torch.equal(q.codes.double(), codes)
    for out in DT.values():
        y = ops.dequantize_int8(q, out_dtype=out)
        v = gu.value(q)
        gu.assert_close(y, v, (2.0 ** -24 + gu.u(out)) * v.abs() * (1 + 2.0 ** -8) + gu.tiny(out), str(out))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols,shift,extra", [(64, 0, 8), (200, 0, 16), (200, 4, 4), (200, 1, 3), (77, 0, 1), (512, 8, 8),
                                              (4096, 0, 64)])
def test_strides_and_bases(ops, cols, shift, extra, dtype):
    """Rows apart and starting anywhere; the output's padding stays as it was."""
    x = draw(50, cols, DT[dtype], cols)
    buf = torch.full((50, cols + shift + extra), float("nan"), dtype=DT[dtype], device="cuda")
    view = buf[:, shift:shift + cols]
    view.copy_(x)
    a, b = ops.quantize_int8(view), ops.quantize_int8(x)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    buf.fill_(7.0)
    ops.dequantize_int8(a, out=view)
    assert torch.equal(view, ops.dequantize_int8(a, out_dtype=DT[dtype]))
    view.fill_(7.0)
    assert bool((buf == 7.0).all())


@pytest.mark.parametrize("cols", [64, 128, 200, 77])
def test_special_blocks(ops, cols):
    """Zeros stay zero, a NaN or an infinity makes its block NaN and no other, blocks
    below 2^-121 are zero, the smallest above it and the largest numbers are kept."""
    x = torch.ones(8, cols, device="cuda")
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, 7] = float("-inf")
    x[3] = 2.0 ** -122
    x[4] = 2.0 ** -120
    x[5] = 3.4e38
    x[6, 3] = -0.0
    y = ops.dequantize_int8(ops.quantize_int8(x), out_dtype=torch.float32)
    assert bool((y[0] == 0).all()) and bool((y[3] == 0).all()) and torch.equal(y[7], x[7])
    for r in (1, 2):
        assert bool(y[r, :64].isnan().all()) and torch.equal(y[r, 64:], x[r, 64:])
    for r in (4, 5):
        assert bool(((y[r] - x[r]).abs() <= 2.0 ** -22 * x[r].abs()).all())
    assert bool((y[6, 4:] == 1).all()) and float(y[6, 3]) == 0.0


def test_ties_go_to_the_even_code(ops):
    """The block's largest is 127: the codes are the rounded values themselves."""
    x = torch.zeros(1, 64, device="cuda")
    x[0, :8] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5])
    assert ops.quantize_int8(x).codes[0, :8].tolist() == [127, 0, 2, 2, 0, -2, -2, 126]


def test_empty(ops):
    for shape in ((0, 64), (5, 0)):
        q = ops.quantize_int8(torch.empty(shape, device="cuda"))
        assert ops.dequantize_int8(q).shape == shape


def test_more_elements_than_an_int(ops):
    """2^31 + 512 codes: the last rows are where they belong."""
    rows, cols = (1 << 15) + 1, 1 << 16
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(cols, device="cuda") % 128 - 64.0
    q = ops.quantize_int8(x)
    y = ops.dequantize_int8(q)
    want = gu.value(ops.Int8Matrix(q.codes[-1:], q.scales[-1:]))
    gu.assert_close(y[-1:], want, gu.u(torch.bfloat16) * 1.01 * want.abs(), "last row")
    codes, scales = gu.keep(x[-1:].float())
    assert torch.equal(q.codes[-1:].double(), codes) and torch.equal(q.scales[-1:], scales)
    assert bool((q.scales[:-1] == 0).all())


@pytest.mark.parametrize("cols", [64, 77])
def test_where_a_block_becomes_zero(ops, cols):
    """127 / a passes FP32's range from a = 127 * 2^-128 down: those blocks are zero, the
    next number above is kept (its scale has 21 bits: half a code and 2^-21)."""
    edge = 127 * 2.0 ** -128
    x = torch.zeros(4, cols, device="cuda")
    for r, a in enumerate((edge * (1 - 2.0 ** -20), edge, edge * (1 + 2.0 ** -22), 0.995 * 2.0 ** -121)):
        x[r] = a
        x[r, ::3] = -a / 3
    q = ops.quantize_int8(x)
    y = ops.dequantize_int8(q, out_dtype=torch.float32)
    assert not q.scales[:2].any() and not y[:2].any()
    off = (y[2:].double() - x[2:].double()).abs()
    a = x[2:].double().abs().amax(1, keepdim=True)
    assert bool((off <= (0.5 / 127 + 2.0 ** -20) * a).all())
