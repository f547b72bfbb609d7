"""Positions outside the routed rows: each kind alone, in each of the row
operators, is left out of every result and reported."""
import pytest
import torch

pytestmark = pytest.mark.gpu

T, E, H = 6, 3, 16
BAD = {"one past the last": lambda pairs: pairs, "further": lambda pairs: pairs + 7,
       "largest": lambda pairs: 2 ** 31 - 1, "below zero": lambda pairs: -1, "smallest": lambda pairs: -2 ** 31}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops


@pytest.mark.parametrize("value", list(BAD))
@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("k", [1, 2, 5, 9])
@pytest.mark.parametrize("call", ["dispatch", "dispatch_grad", "combine", "combine_grad"])
def test_one_bad_position_is_reported(ops, call, k, dropped, value):
    pairs = T * k
    ids = torch.arange(pairs, device="cuda").view(T, k) % E
    if dropped:
        ids[T - 1, 0] = -1
    good = ops.moe_sort(ids, E)
    bad = good.position.clone()
    bad[2, k - 1] = BAD[value](pairs)
    r = ops.Routing(good.offsets, good.order, bad)
    row = int(good.position[2, k - 1])  # the row that no pair names any more
    n = int(good.offsets[-1])
    keep = torch.ones(T, k, device="cuda")
    keep[2, k - 1] = 0
    keep[good.position >= n] = 0
    x = torch.arange(1, T + 1, device="cuda").float()[:, None].expand(T, H).contiguous()
    rows = torch.arange(1, pairs + 1, device="cuda").float()[:, None].expand(pairs, H).contiguous()
    w = torch.full((T, k), 2.0, device="cuda")
    assert ops.last_device_error() == (0, 0)
    if call == "dispatch":
        out = torch.full((pairs, H), 9.0, device="cuda")
        ops.moe_dispatch(x, r, out=out)
        want = x[(good.order // k).long()]
        want[n:] = 0
        want[row] = 9
        assert torch.equal(out, want)
    elif call in ("dispatch_grad", "combine"):
        got = ops.moe_combine(rows, r, w) if call == "combine" else ops.moe_dispatch_grad(rows, r)
        picked = rows[good.position.long()] * keep[:, :, None] * (2 if call == "combine" else 1)
        assert torch.equal(got, picked.sum(1))  # small integers: exact
    else:
        d_rows, d_w = ops.moe_combine_grad(x, rows, r, w)
        others = [i for i in range(pairs) if i != row]
        want = torch.zeros(pairs, H, device="cuda")
        want[good.position.reshape(-1).long()] = (2 * keep[:, :, None] * x[:, None, :]).reshape(-1, H)
        assert torch.equal(d_rows[others], want[others])
        assert torch.equal(d_w, (rows[good.position.long()] * x[:, None, :]).sum(2) * keep)
    status, word = ops.last_device_error()
    assert status == 1 and word >> 56 == 2, (status, hex(word))
    assert ops.last_device_error() == (0, 0)


@pytest.mark.parametrize("call", ["dispatch", "dispatch_grad", "combine", "combine_grad"])
@pytest.mark.parametrize("k", [1, 2, 5, 9])
def test_good_positions_report_nothing(ops, call, k):
    """With every pair kept, and with none: what fills up a kernel's pairs is
    no position."""
    for how in (lambda ids: ids, lambda ids: ids * 0 - 1):
        ids = how(torch.arange(T * k, device="cuda").view(T, k) % E)
        r = ops.moe_sort(ids, E)
        x, rows = torch.ones(T, H, device="cuda"), torch.ones(T * k, H, device="cuda")
        w = torch.ones(T, k, device="cuda")
        {"dispatch": lambda: ops.moe_dispatch(x, r), "dispatch_grad": lambda: ops.moe_dispatch_grad(rows, r),
         "combine": lambda: ops.moe_combine(rows, r, w), "combine_grad": lambda: ops.moe_combine_grad(x, rows, r, w)}[call]()
        assert ops.last_device_error() == (0, 0)
