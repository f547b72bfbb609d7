"""The example's expert layer: its BF16 forms against plain 64-bit sums of the
same steps, and its 4-bit forms against the BF16 one."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, E, K, H, I = 200, 7, 2, 128, 64


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.fixture(scope="module")
def data():
    g = torch.Generator(device="cuda").manual_seed(4)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    x = randn(T, H)
    w1 = [randn(H, 2 * I, std=H ** -0.5) for _ in range(E)]
    w2 = [randn(I, H, std=I ** -0.5) for _ in range(E)]
    router = torch.randn(H, E, generator=g, device="cuda") * H ** -0.5
    return x, w1, w2, router


def plain(x, ids, weights, w1, w2):
    y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(K):
            e = int(ids[t, j])
            gu = x[t].double() @ w1[e].double()
            h = torch.nn.functional.silu(gu[:I]) * gu[I:]
            y[t] += weights[t, j].double() * (h @ w2[e].double())
    return y


def test_bf16_layer(layer, data):
    """Two 16-bit intermediates and the output are each rounded to 2^-8 once:
    in the norm, three such errors of independent signs stay below 3 x 2^-8."""
    x, w1, w2, router = data
    ids, weights = layer.route(x, router, K)
    y = layer.layer_bf16(x, ids, weights, w1, w2).double()
    ref = plain(x, ids, weights, w1, w2)
    assert float((y - ref).norm() / ref.norm()) < 3 * 2.0 ** -8


@pytest.mark.parametrize("fmt,bound", [("nvfp4", 0.3), ("mxfp4", 0.45)])
def test_fp4_layer_is_near_the_bf16_layer(layer, data, fmt, bound):
    """e2m1 values of a normal distribution are off by 0.09 (nvfp4) to 0.13
    (mxfp4) of their norm; a product of two such operands by sqrt(2) of that,
    SwiGLU's product of two again by sqrt(2), FC2's operands add to it: 0.09 x
    sqrt(4 + 2) = 0.22 and 0.13 x sqrt(6) = 0.32; the bounds leave a third."""
    x, w1, w2, router = data
    ids, weights = layer.route(x, router, K)
    ref = layer.layer_bf16(x, ids, weights, w1, w2).double()
    scale = (x.abs().amax().float() / 2688.0).reshape(1) if fmt == "nvfp4" else None
    y = layer.layer_fp4(x, ids, weights, layer.quantize_experts(w1, fmt), layer.quantize_experts(w2, fmt), fmt, scale,
                        scale).double()
    assert float((y - ref).norm() / ref.norm()) < bound


def test_backward_of_the_linear_layer(layer, data):
    """Gradients against automatic differentiation of the layer in 64 bits;
    the rows in between are rounded to BF16 (2^-8) and so is d_x."""
    x, w1, _, router = data
    w = [m[:, :H].contiguous() for m in w1]
    ids, weights = layer.route(x, router, K)
    g = torch.Generator(device="cuda").manual_seed(9)
    d_y = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    y, d_x, d_w = layer.linear_layer_backward(x, ids, weights, w, d_y)
    xd, wd = x.double().requires_grad_(), weights.double().requires_grad_()
    stack = torch.stack([m.double() for m in w])
    rows = torch.einsum("th,tkhn->tkn", xd, stack[ids])
    out = (rows * wd[:, :, None]).sum(1)
    out.backward(d_y.double())
    for got, want in ((y, out.detach()), (d_x, xd.grad), (d_w, wd.grad)):
        assert float((got.double() - want).norm() / want.norm()) < 3 * 2.0 ** -8
