"""The example's expert layer in training: its forward pass and all its gradients
against 64-bit forms of the same steps at the values that the layer kept, with the
bounds of gated_util carried through, and against differences."""
import pytest
import torch

import gated_util as gu
from test_moe_layer_gpu import data, layer  # noqa: F401 - fixtures

pytestmark = pytest.mark.gpu

T, E, K, H, I = 200, 7, 2, 128, 64
BF = torch.bfloat16


@pytest.fixture(scope="module")
def run(layer, data):  # noqa: F811
    from blackwell_tensor_core_gb300 import ops
    x, w1, w2, router = data
    ids, weights = layer.route(x, router, K)
    g = torch.Generator(device="cuda").manual_seed(9)
    dy = torch.randn(T, H, generator=g, device="cuda").to(BF)
    y, kept = layer.training_forward(x, ids, weights, w1, w2)
    grads = layer.training_backward(kept, weights, w1, w2, dy)
    assert ops.last_device_error() == (0, 0)
    return x, ids, weights, w1, w2, dy, y, kept, grads


def test_the_forward_pass_is_the_layers(layer, run):  # noqa: F811
    x, ids, weights, w1, w2, _, y, kept, _ = run
    from blackwell_tensor_core_gb300 import ops
    r = kept[0]
    rows = ops.moe_dispatch(x, r)
    h, _ = ops.grouped_gemm(rows, w1, r.offsets, swiglu=True, keep_int8=True)
    assert torch.equal(y, ops.moe_combine(ops.grouped_gemm(h, w2, r.offsets), r, weights))
    # the same bits but for the gated kernel: within its bound of layer_bf16's H
    same = ops.grouped_gemm(rows, w1, r.offsets, swiglu=True)
    assert float((h.double() - same.double()).norm() / same.double().norm()) <= 2 * gu.u(BF)


def test_gradients(run):
    x, ids, weights, w1, w2, dy, _, (r, rows8, gate_up, out8), (d_x, d_weights, d_w1, d_w2) = run
    at = r.offsets.tolist()
    pos = r.position.long()
    xv, gv, ov = gu.value(rows8), gu.value(gate_up), gu.value(out8)
    ex = gu.u(BF) * xv.abs() + gu.tiny(BF)
    eo = gu.u(BF) * ov.abs() + gu.tiny(BF)
    # the combine's gradient
    dyd = dy.double()
    flat = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
    flat[pos.reshape(-1)] = (weights.double()[:, :, None] * dyd[:, None, :]).reshape(-1, H)
    e_flat = (gu.u(BF) + 2.0 ** -23) * flat.abs() + gu.tiny(BF)
    rows_t = ov[pos]
    dw_ref = (rows_t * dyd[:, None, :]).sum(2)
    dw_e = (eo[pos] * dyd.abs()[:, None, :]).sum(2) + H * 2.0 ** -23 * (rows_t.abs() * dyd.abs()[:, None, :]).sum(2)
    gu.assert_close(d_weights, dw_ref, dw_e, "d_weights")
    dx_rows = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
    ex_rows = torch.zeros_like(dx_rows)
    for e in range(E):
        s = slice(at[e], at[e + 1])
        w1d, w2d = w1[e].double(), w2[e].double()
        dh, e_dh = gu.through(flat[s], e_flat[s], w2d.t(), 0.0, BF)
        gate, up = gv[s, :I], gv[s, I:]
        eg, eu = 2.0 ** -23 * gate.abs(), 2.0 ** -23 * up.abs()
        dgu, e_dgu = gu.backward(dh, gate, up, eg, eu, BF)
        # linear in dh: its error times the factors, both roundings counted again
        one, e_one = gu.backward(torch.ones_like(dh), gate, up, eg, eu, BF)
        e_dgu = e_dgu + (one.abs() + e_one) * torch.cat([e_dh, e_dh], 1) * (1 + 2.0 ** -7)
        gu.assert_close(d_w1[e], *gu.through(xv[s].t(), ex[s].t(), dgu, e_dgu, BF), "d_w1 of expert %d" % e)
        dx_rows[s], ex_rows[s] = gu.through(dgu, e_dgu, w1d.t(), 0.0, BF)
        h, e_h = gu.forward(gate, up, eg, eu, BF)
        gu.assert_close(d_w2[e], *gu.through(h.t(), e_h.t(), flat[s], e_flat[s], BF), "d_w2 of expert %d" % e)
    want = dx_rows[pos].sum(1)
    bound = ex_rows[pos].sum(1) + K * 2.0 ** -23 * dx_rows[pos].abs().sum(1)
    gu.assert_close(d_x, want, bound + gu.u(BF) * (want.abs() + bound) + gu.tiny(BF), "d_x")


def test_gradients_against_differences(run):
    """Along one direction of all parameters at once, L = sum(dy * y) in 64 bits at the
    unkept values.  What the layer kept differs from them: a value by half a step, at
    most 1/254 of its block's largest, for gate and up, the rows and the experts'
    rows.  Each enters the gradient linearly or through silu and its slope (at most
    1.1 and 0.5 a unit), so that the gradient's terms are off by at most 3 such
    parts of blocks whose largest value is below 5 standard deviations: 3 * 5 / 254 =
    6% of the terms' 2-norm, roundings (2^-8 each) far below."""
    x, ids, weights, w1, w2, dy, _, _, (d_x, d_weights, d_w1, d_w2) = run
    g = torch.Generator(device="cuda").manual_seed(11)

    def like(t):
        return torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) * float(t.double().std())

    dirs = [like(x), like(weights), [like(m) for m in w1], [like(m) for m in w2]]

    def loss(t):
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for e in range(E):
            tok, j = torch.nonzero(ids == e, as_tuple=True)
            a = (x.double() + t * dirs[0])[tok] @ (w1[e].double() + t * dirs[2][e])
            h = a[:, :I] * torch.sigmoid(a[:, :I]) * a[:, I:]
            o = h @ (w2[e].double() + t * dirs[3][e])
            total = total + ((weights.double() + t * dirs[1])[tok, j][:, None] * o * dy.double()[tok]).sum()
        return float(total)

    step = 1e-4
    want = (loss(step) - loss(-step)) / (2 * step)
    terms = [d_x.double() * dirs[0], d_weights.double() * dirs[1]]
    terms += [d_w1[e].double() * dirs[2][e] for e in range(E)] + [d_w2[e].double() * dirs[3][e] for e in range(E)]
    have = sum(float(t.sum()) for t in terms)
    scale = sum(float(t.square().sum()) for t in terms) ** 0.5
    assert abs(have - want) <= 0.06 * max(scale, abs(want))


def test_runs_are_equal(layer, run):  # noqa: F811
    x, ids, weights, w1, w2, dy, y, _, grads = run
    for _ in range(3):
        again, kept = layer.training_forward(x, ids, weights, w1, w2)
        assert torch.equal(again, y)
        for a, b in zip(layer.training_backward(kept, weights, w1, w2, dy), grads):
            assert torch.equal(a, b)
