"""64-bit forms of the gated feed-forward block's operators, with bounds on how
far the kernels' results may be from them (not collected as tests).

Bounds.  u(t) = eps(t) / 2 is a rounding to type t.
  product of K 16-bit pairs summed in FP32 on the tensor cores: every K = 16 step
    may lose the bits below 2^-23 of the larger of the sum and the step's largest
    product, neither above S = sum |a b|, once for the sum and once for the step:
    |error| <= (K / 16 + 2) 2^-22 S.
  silu, its gradient and their products in FP32: __expf (2 ulp and |x| 2^-22 of its
    argument's scaling), the approximate reciprocal (1 ulp) and up to six products
    and sums: 2^-18 of the result, |gate| below 88.
  |silu'| < 1.1, |silu''| <= 0.5, |silu(x)| <= |x|.
"""
import torch


def u(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the step of the subnormal numbers."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def product(a, b):
    """(a @ b, bound) in 64 bits of matrices given exactly."""
    a, b = a.double(), b.double()
    return a @ b, (a.shape[1] / 16 + 2) * 2.0 ** -22 * (a.abs() @ b.abs())


def gated(x, w):
    """gate, up and their bounds."""
    p, e = product(x, w)
    half = w.shape[1] // 2
    return p[:, :half], p[:, half:], e[:, :half], e[:, half:]


def forward(gate, up, eg, eu, dtype):
    """h and its bound from gate and up and theirs."""
    silu = gate * torch.sigmoid(gate)
    h = silu * up
    e = 1.1 * eg * up.abs() + (silu.abs() + 1.1 * eg) * eu + 2.0 ** -18 * h.abs()
    return h, e + u(dtype) * (h.abs() + e) + tiny(dtype)


def backward(dh, gate, up, eg, eu, dtype):
    """dgu = [dgate | dup] and its bound."""
    dh = dh.double()
    s = torch.sigmoid(gate)
    silu, slope = gate * s, s * (1 + gate * torch.sigmoid(-gate))
    dg, du = dh * up * slope, dh * silu
    # the slope is a sum of two terms, each with its own rounding
    eval_g = 2.0 ** -18 * (dh * up).abs() * (s + silu.abs() * torch.sigmoid(-gate))
    edg = dh.abs() * (1.1 * eu + 0.5 * eg * (up.abs() + eu)) + eval_g
    edu = dh.abs() * 1.1 * eg + 2.0 ** -18 * du.abs()
    d, e = torch.cat([dg, du], 1), torch.cat([edg, edu], 1)
    return d, e + u(dtype) * (d.abs() + e) + tiny(dtype)


def through(a, ea, b, eb, dtype):
    """a @ b and its bound, where a and b are off by ea and eb."""
    v = a @ b
    mag = (a.abs() + ea) @ (b.abs() + eb)
    e = mag - a.abs() @ b.abs() + (a.shape[1] / 16 + 2) * 2.0 ** -22 * mag
    return v, e + u(dtype) * (v.abs() + e) + tiny(dtype)


def blocks(v, parts=1):
    """Each element's block of 64 columns of its part: (index [cols], count)."""
    cols = v.shape[1] // parts
    c = torch.arange(v.shape[1], device=v.device)
    per = -(-cols // 64)
    return (c // cols) * per + (c % cols) // 64, per * parts


def keep(v, parts=1):
    """(codes, scales) of 32-bit v by the definition, in 64 bits after its two rounded quotients."""
    at, n = blocks(v, parts)
    a = torch.zeros(v.shape[0], n, dtype=torch.float32, device=v.device)
    a.scatter_reduce_(1, at.expand(v.shape[0], -1), v.abs().float(), "amax")
    full = torch.full_like(a, 127.0)
    inv = torch.where(a > 0, full / torch.where(a > 0, a, full), torch.zeros_like(a))
    return torch.round(v.double() * inv.double()[:, at]), a / full


def value(q):
    """What an Int8Matrix stands for, in 64 bits."""
    at, _ = blocks(q.codes, q.parts)
    return q.codes.double() * q.scales.double()[:, at]


def assert_close(got, want, bound, what=""):
    got = got.double()
    assert got.shape == want.shape, "%s: shape %s, not %s" % (what, tuple(got.shape), tuple(want.shape))
    off = (got - want).abs() - bound
    bad = ~(off <= 0)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError("%s: %d of %d outside the bound; first %s: got %r want %r bound %r" % (
            what, int(bad.sum()), bad.numel(), i, float(got[i]), float(want[i]), float(bound[i])))


def offsets(counts):
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")
