"""The example's calibration: each product's input has a scale of its own."""
import pytest
import torch

from test_moe_layer_gpu import K, data, layer  # noqa: F401 - fixtures

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2.0 ** -4, 1.0, 8.0])
def test_nvfp4_layer_with_calibrated_scales(layer, data, size):  # noqa: F811
    """FC1's output is size^2 (large gates) to size (small) times as large as x.
    The layer's error stays that of its 4-bit operands: a third more than
    0.09 sqrt(6) of the norm, as for the layer with scales of order one."""
    x, w1, w2, router = data
    w1 = [w * size for w in w1]
    ids, weights = layer.route(x, router, K)
    x_scale, h_scale = layer.calibrated_scales(x, ids, w1, "nvfp4")
    ref = layer.layer_bf16(x, ids, weights, w1, w2).double()
    y = layer.layer_fp4(x, ids, weights, layer.quantize_experts(w1, "nvfp4"), layer.quantize_experts(w2, "nvfp4"), "nvfp4",
                        x_scale, h_scale).double()
    assert float((y - ref).norm() / ref.norm()) < 0.3
    assert layer.calibrated_scales(x, ids, w1, "mxfp4") == (None, None)


def test_the_scale_of_x_does_not_serve_a_larger_input(layer, data):  # noqa: F811
    """What the calibration is for: saturated at x's largest value, FC1's output loses most of its norm."""
    x, w1, w2, router = data
    w1 = [w * 8 for w in w1]
    ids, weights = layer.route(x, router, K)
    x_scale, h_scale = layer.calibrated_scales(x, ids, w1, "nvfp4")
    assert float(h_scale) > 8 * float(x_scale)
    ref = layer.layer_bf16(x, ids, weights, w1, w2).double()
    y = layer.layer_fp4(x, ids, weights, layer.quantize_experts(w1, "nvfp4"), layer.quantize_experts(w2, "nvfp4"), "nvfp4",
                        x_scale, x_scale).double()
    assert float((y - ref).norm() / ref.norm()) > 0.5
