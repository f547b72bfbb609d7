"""Argument checks of the routed-row operators that need no GPU: the C entry
points refuse bad arguments before they touch a device."""
import pytest
import torch

INVALID, ALIGNMENT, UNSUPPORTED = 1, 2, 3
P, Q, R, S = 4096, 8192, 12288, 16384  # addresses that are never read


@pytest.fixture(scope="module")
def lib():
    from blackwell_tensor_core_gb300 import build, ops
    build.build()
    return ops.lib()


@pytest.mark.parametrize("args,status", [
    ((P, 2, 8, 4, Q, R, S), INVALID),         # ids of two bytes
    ((P, 4, -1, 4, Q, R, S), INVALID),
    ((P, 4, 8, 0, Q, R, S), INVALID),
    ((P, 4, 8, 4, None, R, S), INVALID),
    ((None, 4, 8, 4, Q, R, S), INVALID),
    ((P, 4, 8, 4, Q, None, S), INVALID),
    ((P, 4, 8, 4, Q, R, None), INVALID),
    ((P, 4, 8, 1025, Q, R, S), UNSUPPORTED),  # more experts than one block's counters
    ((P + 4, 8, 8, 4, Q, R, S), ALIGNMENT),
])
def test_sort_refuses(lib, args, status):
    assert lib.moe_sort(*args, None) == status


def _dispatch(lib, X=P, dtype=0, T=2, H=8, ldx=8, k=2, position=Q, offsets=R, E=4, rows=S, ldr=8):
    return lib.moe_dispatch(X, dtype, T, H, ldx, k, position, offsets, E, rows, ldr, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), INVALID), (dict(T=-1), INVALID), (dict(H=-1), INVALID), (dict(k=0), INVALID),
    (dict(E=0), INVALID), (dict(E=1025), UNSUPPORTED), (dict(T=1 << 30, k=4), UNSUPPORTED),
    (dict(X=None), INVALID), (dict(rows=None), INVALID), (dict(position=None), INVALID),
    (dict(offsets=None), INVALID), (dict(ldx=7), INVALID), (dict(ldr=7), INVALID),
    (dict(X=P + 1), ALIGNMENT), (dict(rows=S + 2, dtype=1), ALIGNMENT),
    (dict(T=0, X=None), 0), (dict(H=0, X=None), 0),
])
def test_dispatch_refuses(lib, change, status):
    assert _dispatch(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(w=None), INVALID), (dict(dtype=9), INVALID), (dict(ldr=3), INVALID), (dict(Y=None), INVALID),
    (dict(rows=None), INVALID), (dict(k=-2), INVALID), (dict(T=0, w=None), 0),
])
def test_combine_refuses(lib, change, status):
    a = dict(rows=P, dtype=0, T=2, H=4, ldr=4, k=2, w=Q, pos=R, off=S, E=4, Y=P, ldy=4)
    a.update(change)
    assert lib.moe_combine(a["rows"], a["dtype"], a["T"], a["H"], a["ldr"], a["k"], a["w"], a["pos"], a["off"], a["E"],
                           a["Y"], a["ldy"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(w=None), INVALID), (dict(dw=None), INVALID), (dict(dr=None), INVALID), (dict(dy=None), INVALID),
    (dict(ldy=3), INVALID), (dict(ldr=3), INVALID), (dict(ldd=3), INVALID), (dict(H=-4), INVALID),
    (dict(dr=P + 1), ALIGNMENT), (dict(T=0), 0),
])
def test_combine_grad_refuses(lib, change, status):
    a = dict(dy=P, rows=Q, dtype=2, T=2, H=4, ldy=4, ldr=4, k=2, w=Q, pos=R, off=S, E=4, dr=P, ldd=4, dw=S)
    a.update(change)
    assert lib.moe_combine_grad(a["dy"], a["rows"], a["dtype"], a["T"], a["H"], a["ldy"], a["ldr"], a["k"], a["w"],
                                a["pos"], a["off"], a["E"], a["dr"], a["ldd"], a["dw"], None) == status


def test_python_refuses_what_is_no_device_tensor():
    from blackwell_tensor_core_gb300 import ops
    with pytest.raises(ValueError):
        ops.moe_sort(torch.zeros(4, 2, dtype=torch.int32), 4)  # on the host
    with pytest.raises(ValueError):
        ops.moe_sort(torch.zeros(8, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        ops.moe_sort(torch.zeros(4, 2), 4)
