"""A routed expert layer, forward and backward, with its experts in BF16 and in 4 bits.

    python examples/moe_layer.py [--tokens 4096] [--experts 32] [--topk 8] [--hidden 4096] [--inner 2048]

The router's choices are sorted by expert, the tokens' rows dispatched into that
order, multiplied by their experts' weights (FC1 with SwiGLU, then FC2) and
combined back with the router's weights.  With the experts in 4 bits each
product's input rows are quantised on the way.  The backward pass shown is that
of a layer with frozen experts: gradients of the tokens and of the router's
weights through a linear expert.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from blackwell_tensor_core_gb300 import ops  # noqa: E402


def route(x, router, topk):
    """Top-k experts of each token and their softmax weights."""
    top, ids = torch.topk(x.float() @ router, topk, dim=1)
    return ids, torch.softmax(top, dim=1)


def layer_bf16(x, ids, weights, w1, w2):
    """w1: experts' [gate | up] as [H, 2 I], w2: [I, H] (lists of BF16 matrices)."""
    r = ops.moe_sort(ids, len(w1))
    rows = ops.moe_dispatch(x, r)
    h = ops.grouped_gemm(rows, w1, r.offsets, swiglu=True)
    return ops.moe_combine(ops.grouped_gemm(h, w2, r.offsets), r, weights)


def quantize_experts(w, fmt):
    """Experts' [in, out] matrices as one 4-bit stack [experts, out, in]."""
    stack = torch.stack([m.t().contiguous() for m in w])
    g = (stack.abs().amax().float() / 2688.0).reshape(1) if fmt == "nvfp4" else None
    return ops.quantize_fp4(stack, fmt, global_scale=g)


def calibrated_scales(x, ids, w1, fmt):
    """The scales of the two products' inputs, x and FC1's output, from a BF16
    pass over sample tokens.  Each input needs its own: with a scale too small
    for it values saturate, with one too large they lose their bits."""
    if fmt != "nvfp4":
        return None, None
    r = ops.moe_sort(ids, len(w1))
    h = ops.grouped_gemm(ops.moe_dispatch(x, r), w1, r.offsets, swiglu=True)
    return tuple((m.abs().amax().float() / 2688.0).reshape(1) for m in (x, h))


def layer_fp4(x, ids, weights, q1, q2, fmt, x_scale=None, h_scale=None):
    """The same with 4-bit experts; x_scale and h_scale are the nvfp4 scales of
    the two products' inputs (calibrated_scales)."""
    r = ops.moe_sort(ids, q1.groups)
    rows = ops.quantize_fp4(ops.moe_dispatch(x, r), fmt, global_scale=x_scale, group_offsets=r.offsets)
    h = ops.quantize_fp4(ops.grouped_gemm_fp4(rows, q1, swiglu=True), fmt, global_scale=h_scale,
                         group_offsets=r.offsets)
    return ops.moe_combine(ops.grouped_gemm_fp4(h, q2), r, weights)


def linear_layer_backward(x, ids, weights, w, d_y):
    """y = combine(rows W): (y, d_x, d_weights) for frozen experts W [H, H]."""
    r = ops.moe_sort(ids, len(w))
    rows = ops.grouped_gemm(ops.moe_dispatch(x, r), w, r.offsets)
    y = ops.moe_combine(rows, r, weights)
    d_rows, d_weights = ops.moe_combine_grad(d_y, rows, r, weights)
    # d(rows W) / d(rows): the same matrices, read as [out, in]
    d_x = ops.moe_dispatch_grad(ops.grouped_gemm(d_rows, w, r.offsets, b_transposed=True), r)
    return y, d_x, d_weights


def timed(fn, reps=20):
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(reps):
        fn()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / reps * 1e6


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("experts", 32), ("topk", 8), ("hidden", 4096), ("inner", 2048)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    x = randn(a.tokens, a.hidden)
    router = randn(a.hidden, a.experts, std=a.hidden ** -0.5).float()
    w1 = [randn(a.hidden, 2 * a.inner, std=a.hidden ** -0.5) for _ in range(a.experts)]
    w2 = [randn(a.inner, a.hidden, std=a.inner ** -0.5) for _ in range(a.experts)]
    ids, weights = route(x, router, a.topk)
    y = layer_bf16(x, ids, weights, w1, w2)
    print("bf16 experts: %8.1f us" % timed(lambda: layer_bf16(x, ids, weights, w1, w2)))
    for fmt in ("nvfp4", "mxfp4"):
        q1, q2 = quantize_experts(w1, fmt), quantize_experts(w2, fmt)
        scales = calibrated_scales(x, ids, w1, fmt)
        y4 = layer_fp4(x, ids, weights, q1, q2, fmt, *scales)
        err = float((y4.float() - y.float()).norm() / y.float().norm())
        print("%s experts: %8.1f us, relative difference from bf16 %.3f" % (
            fmt, timed(lambda: layer_fp4(x, ids, weights, q1, q2, fmt, *scales)), err))
    w = [m[:, :a.hidden].contiguous() for m in w1] if 2 * a.inner >= a.hidden else None
    if w is not None:
        print("linear experts, forward and backward: %8.1f us" % timed(lambda: linear_layer_backward(x, ids, weights, w, x)))
    status, word = ops.last_device_error()
    if status:
        raise SystemExit("device error word %#x" % word)


if __name__ == "__main__":
    main()
