"""Operators that train a gated feed-forward block, as cases that can be timed and compared.

Four operators: the gated block's forward pass (both projections, the activation and the product in one kernel, with
its projections kept in 8 bits where the backward pass will want them), its backward pass (from the projections kept in
8 bits, or from the inputs alone), matrices kept in 8 bits on their own, and the weight gradient's product, whose left
operand is read transposed.  All but the third run on one matrix or on the routed rows of many experts.  ``run``
computes a case in its plain form (elementary torch operations in 32 bits) or, with ``own``, through the calls that a
user makes of ``blackwell_tensor_core_gb300.ops``.  ``exact`` states each operator in 64 bits.

Definitions (row-major; M rows, K columns in, w = [gate | up] with N = 2 I columns, expert e's rows o[e] .. o[e+1]-1):

  forward   g = x w[:, :I], u = x w[:, I:], h = silu(g) * u with silu(v) = v s(v), s(v) = 1 / (1 + e^-v)
  backward  dg = dh * u * s(g) * (1 + g * (1 - s(g))), du = dh * silu(g), dgu = [dg | du],
            dx = dgu w^T, dw = x^T dgu, and h = silu(g) * u where it was not kept
  8 bits    blocks of 64 columns of a row (of g and of u apart): scale a / 127 and codes rint(v * (127 / a)) with the
            block's largest magnitude a, both quotients rounded to 32 bits; the value is code * scale
  weight    D[m, n] = sum_r A[r, m] B[r, n], over all rows or over each expert's: D[e]
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BLOCK = 64


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step through the block: latency
        dict(name="ffn_1_token", op="ffn", M=1, K=4096, N=4096, E=0, dtype="bf16", keep=False),
        # the benchmark's decode-like shape, its columns as gate and up
        dict(name="ffn_72", op="ffn", M=72, K=7168, N=16384, E=0, dtype="bf16", keep=False),
        # an odd batch, sizes that fill no tile
        dict(name="ffn_odd", op="ffn", M=1000, K=2056, N=2832, E=0, dtype="fp16", keep=False),
        # a training step's forward pass: 8192 tokens, the projections kept in 8 bits
        dict(name="ffn_keep_8192", op="ffn", M=8192, K=4096, N=8192, E=0, dtype="bf16", keep=True),
        # the benchmark's routed expert layer in training: 4096 tokens, top 8 of 32
        dict(name="experts_keep", op="ffn", M=32768, K=4096, N=4096, E=32, dtype="bf16", keep=True),
        # a small odd training step that kept nothing: the projections again, then all gradients
        dict(name="grad_odd", op="grad", M=999, K=1032, N=1520, E=0, dtype="fp16", keep=False, x8=False),
        # a large training step that kept nothing
        dict(name="grad_4096", op="grad", M=4096, K=4096, N=16384, E=0, dtype="bf16", keep=False, x8=False),
        # the routed layer's backward pass, everything that it needs kept in 8 bits
        dict(name="experts_grad_kept", op="grad", M=32768, K=4096, N=4096, E=32, dtype="bf16", keep=True, x8=True),
        # a layer's input kept in 8 bits and read back
        dict(name="keep_32768", op="keep", M=32768, K=4096, dtype="bf16"),
        # the same for a small ragged batch whose rows end inside a block
        dict(name="keep_odd", op="keep", M=333, K=7000, dtype="fp16"),
        # the weight gradient of the benchmark's square, summed up in 32 bits
        dict(name="weight_8192", op="weight", M=8192, K=8192, N=8192, E=0, dtype="bf16", out="fp32"),
        # a small layer's weight gradient over a long odd batch
        dict(name="weight_odd", op="weight", M=20011, K=1000, N=1416, E=0, dtype="fp16", out="fp16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, step):
    return max(lo, _log_int(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["ffn", "ffn", "grad", "grad", "keep", "weight"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "keep":
        K = _log_int(rng, 64, 16384)
        return dict(op=op, M=_log_int(rng, 1, min(65536, (1 << 27) // K)), K=K, dtype=dtype)
    E = rng.choice([0, 0, 8, 16, 32])
    K, N = _mult(rng, 256, 4096, 8), _mult(rng, 256, 8192 if E == 0 else 4096, 16)
    if op == "weight":
        return dict(op=op, M=_log_int(rng, 1, 16384), K=K, N=N, E=E, dtype=dtype, out=rng.choice([dtype, "fp32"]))
    if op == "ffn":
        keep = E > 0 or rng.random() < 0.4
        return dict(op=op, M=_log_int(rng, 1, 8192), K=K, N=N, E=E, dtype=dtype, keep=keep)
    keep = rng.random() < 0.5
    return dict(op=op, M=_log_int(rng, 1, 8192), K=K, N=N, E=E, dtype=dtype, keep=keep,
                x8=keep and rng.random() < 0.5)


def _elt(dtype):
    return 4 if dtype == "fp32" else 2


def _kept_bytes(rows, cols):
    return rows * cols + 4 * rows * -(-cols // _BLOCK)


def work(case):
    c = case
    M, K = c["M"], c["K"]
    if c["op"] == "keep":  # in, kept, read again, out
        return {"bytes": 4 * M * K + 2 * _kept_bytes(M, K), "flops": 2 * M * K}
    N, experts = c["N"], max(1, c["E"])
    busy = experts * (1.0 - (1.0 - 1.0 / experts) ** M)  # experts that rows reach
    product = 2 * M * N * K
    if c["op"] == "weight":
        return {"bytes": 2 * M * (K + N) + experts * K * N * _elt(c["out"]), "flops": product}
    kept = 2 * _kept_bytes(M, N // 2) if c["keep"] else 0
    if c["op"] == "ffn":
        return {"bytes": 2 * M * K + 2 * busy * K * N + M * N + kept, "flops": product}
    x = _kept_bytes(M, K) if c["x8"] else 2 * M * K
    h = M * N if c["keep"] else 0
    return {"bytes": M * N + x + kept + 2 * busy * K * N + 2 * M * K + 2 * experts * K * N + h,
            "flops": product * (2 if c["keep"] else 3)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _activations(rows, cols, g):
    """Normal values with channels of different spread, as activations before a linear layer have."""
    spread = torch.exp(0.3 * torch.randn(cols, generator=g, device=g.device))
    return torch.randn(rows, cols, generator=g, device=g.device) * spread


def _ragged(M, E, g):
    """Offsets of M rows over E experts, as a skewed router deals them out."""
    skew = torch.softmax(0.5 * torch.randn(E, generator=g, device=g.device), 0)
    ids = torch.multinomial(skew, M, replacement=True, generator=g)
    counts = (ids[:, None] == torch.arange(E, device=g.device)).sum(0)
    return torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=_device())
    g.manual_seed(int(seed))
    dt = _DT[c["dtype"]]
    M, K = c["M"], c["K"]
    s = {"c": c}
    if c["op"] == "keep":
        s["x"] = _activations(M, K, g).to(dt)
        return s
    N, E = c["N"], c["E"]
    if E > 0:
        s["offsets"] = _ragged(M, E, g)
        s["bounds"] = s["offsets"].tolist()
    else:
        s["bounds"] = [0, M]
    s["x"] = _activations(M, K, g).to(dt)
    if c["op"] == "weight":
        s["dy"] = (0.1 * _activations(M, N, g)).to(dt)
        return s
    w = [(torch.randn(K, N, generator=g, device=g.device) * K ** -0.5).to(dt) for _ in range(max(1, E))]
    s["w"] = torch.stack(w) if E > 0 else w[0]
    s["experts"] = list(s["w"].unbind(0)) if E > 0 else w  # a program's list of weights
    if c["op"] == "grad":
        s["dh"] = (0.1 * _activations(M, N // 2, g)).to(dt)
        if c["keep"]:
            gate, up = _projections(s["x"].to(torch.float32), s)
            parts = [_plain_keep(gate), _plain_keep(up)]
            s["codes"] = torch.cat([p[0] for p in parts], dim=1)
            s["scales"] = torch.cat([p[1] for p in parts], dim=1)
        if c["x8"]:
            s["x_codes"], s["x_scales"] = _plain_keep(s.pop("x").to(torch.float32))
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _blocks(v):
    rows, cols = v.shape
    n = -(-cols // _BLOCK)
    if n * _BLOCK != cols:
        v = torch.nn.functional.pad(v, (0, n * _BLOCK - cols))
    return v.reshape(rows, n, _BLOCK)


def _plain_keep(v):
    """Codes [rows, cols] and scales [rows, blocks] of 32-bit v."""
    b = _blocks(v)
    amax = b.abs().amax(dim=2)
    scale = amax / 127.0
    inv = torch.where(amax > 0, 127.0 / torch.where(amax > 0, amax, torch.ones_like(amax)), torch.zeros_like(amax))
    # in 64 bits: a product next to a tie must not be rounded onto it first
    codes = torch.round(b.double() * inv.double()[:, :, None]).to(torch.int8)
    return codes.reshape(v.shape[0], -1)[:, : v.shape[1]].contiguous(), scale


def _plain_read(codes, scales):
    v = _blocks(codes.to(torch.float32)) * scales[:, :, None]
    return v.reshape(codes.shape[0], -1)[:, : codes.shape[1]]


def _read_pair(s):
    half, blocks = s["codes"].shape[1] // 2, s["scales"].shape[1] // 2
    return (_plain_read(s["codes"][:, :half], s["scales"][:, :blocks]),
            _plain_read(s["codes"][:, half:], s["scales"][:, blocks:]))


def _rows_by(a, s, product):
    """product(rows of expert e, e) for every expert, or of all rows with the one weight."""
    at = s["bounds"]
    return [product(a[at[e]:at[e + 1]], e) for e in range(len(at) - 1)]


def _projections(x, s):
    p = torch.cat(_rows_by(x, s, lambda a, e: a @ s["experts"][e].to(torch.float32)))
    half = p.shape[1] // 2
    return p[:, :half], p[:, half:]


def _weight_product(a, b, s):
    at = s["bounds"]
    d = [a[at[e]:at[e + 1]].t() @ b[at[e]:at[e + 1]] for e in range(len(at) - 1)]
    return torch.stack(d) if s["c"]["E"] > 0 else d[0]


def _run_plain(s):
    c = s["c"]
    dt = _DT[c["dtype"]]
    if c["op"] == "keep":
        return _plain_read(*_plain_keep(s["x"].to(torch.float32))).to(dt)
    if c["op"] == "weight":
        return _weight_product(s["x"].to(torch.float32), s["dy"].to(torch.float32), s).to(_DT[c["out"]])
    if c["op"] == "ffn":
        gate, up = _projections(s["x"].to(torch.float32), s)
        h = (gate / (1.0 + torch.exp(-gate)) * up).to(dt)
        if not c["keep"]:
            return h
        kept = torch.cat([_plain_read(*_plain_keep(gate)), _plain_read(*_plain_keep(up))], dim=1)
        return {"h": h, "kept": kept.to(dt)}
    x = _plain_read(s["x_codes"], s["x_scales"]) if c["x8"] else s["x"].to(torch.float32)
    gate, up = _read_pair(s) if c["keep"] else _projections(x, s)
    dh = s["dh"].to(torch.float32)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dgu = torch.cat([dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * gate * sig], dim=1)
    dx = torch.cat(_rows_by(dgu, s, lambda a, e: a @ s["experts"][e].to(torch.float32).t()))
    d = {"dx": dx.to(dt), "dw": _weight_product(x, dgu, s).to(dt)}
    if c["keep"]:
        d["h"] = (gate * sig * up).to(dt)
    return d


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    from blackwell_tensor_core_gb300 import ops
    c = s["c"]
    dt = _DT[c["dtype"]]
    if c["op"] == "keep":
        return ops.dequantize_int8(ops.quantize_int8(s["x"]), out_dtype=dt)
    if c["op"] == "weight":
        if c["E"] > 0:
            return ops.grouped_gemm_wgrad(s["x"], s["dy"], s["offsets"], out_dtype=_DT[c["out"]])
        return ops.gemm(s["x"], s["dy"], out_dtype=_DT[c["out"]], a_transposed=True)
    if c["op"] == "ffn":
        if c["E"] > 0:
            got = ops.grouped_gemm(s["x"], s["experts"], s["offsets"], swiglu=True, keep_int8=c["keep"])
        else:
            got = ops.gemm_swiglu(s["x"], s["w"], keep_int8=c["keep"])
        return {"h": got[0], "kept": ops.dequantize_int8(got[1], out_dtype=dt)} if c["keep"] else got
    x = ops.Int8Matrix(s["x_codes"], s["x_scales"]) if c["x8"] else s["x"]
    kept = ops.Int8Matrix(s["codes"], s["scales"], parts=2) if c["keep"] else None
    if c["E"] > 0:
        got = ops.grouped_gemm_swiglu_grad(s["dh"], x, s["experts"], s["offsets"], kept=kept, with_h=c["keep"])
    else:
        got = ops.gemm_swiglu_grad(s["dh"], x, s["w"], kept=kept, with_h=c["keep"])
    d = {"dx": got.dx, "dw": got.dw}
    if c["keep"]:
        d["h"] = got.h
    return d


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_kept(v):
    """What v [rows, cols] (64 bits) is read back as, block by block of 64 columns."""
    out = torch.empty_like(v)
    for at in range(0, v.shape[1], _BLOCK):
        b = v[:, at:at + _BLOCK]
        a = b.abs().max(dim=1, keepdim=True).values.to(torch.float32)
        one = torch.ones_like(a)
        r = torch.where(a > 0, torch.div(127.0 * one, torch.where(a > 0, a, one)), 0.0 * one).double()
        out[:, at:at + _BLOCK] = torch.round(b * r) * torch.div(a, 127.0 * one).double()
    return out


def _exact_values(codes, scales):
    """Every element's code times the scale of the block that it lies in."""
    block = torch.arange(codes.shape[1], device=codes.device) // _BLOCK
    return codes.double() * scales.double()[:, block]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "keep":
        return _exact_kept(s["x"].double())
    E = max(1, c["E"])
    at = s["bounds"]
    if c["op"] == "weight":
        d = torch.zeros(E, c["K"], c["N"], dtype=torch.float64, device=s["x"].device)
        for e in range(E):
            d[e] = torch.mm(s["x"][at[e]:at[e + 1]].double().t(), s["dy"][at[e]:at[e + 1]].double())
        return d if c["E"] > 0 else d[0]
    half = c["N"] // 2
    x = _exact_values(s["x_codes"], s["x_scales"]) if c.get("x8") else s["x"].double()
    if c["op"] == "ffn" or not c["keep"]:
        p = torch.zeros(c["M"], c["N"], dtype=torch.float64, device=x.device)
        for e in range(E):
            p[at[e]:at[e + 1]] = torch.mm(x[at[e]:at[e + 1]], s["experts"][e].double())
        gate, up = p[:, :half], p[:, half:]
    else:
        n = s["scales"].shape[1] // 2
        gate = _exact_values(s["codes"][:, :half], s["scales"][:, :n])
        up = _exact_values(s["codes"][:, half:], s["scales"][:, n:])
    sig = torch.sigmoid(gate)
    h = gate * sig * up
    if c["op"] == "ffn":
        return {"h": h, "kept": torch.cat([_exact_kept(gate), _exact_kept(up)], dim=1)} if c["keep"] else h
    dh = s["dh"].double()
    # d silu(g) / dg = s + g s (1 - s)
    dgu = torch.cat([dh * up * (sig + gate * sig * torch.sigmoid(-gate)), dh * gate * sig], dim=1)
    dx = torch.zeros(c["M"], c["K"], dtype=torch.float64, device=x.device)
    dw = torch.zeros(E, c["K"], c["N"], dtype=torch.float64, device=x.device)
    for e in range(E):
        lo, hi = at[e], at[e + 1]
        dx[lo:hi] = torch.mm(dgu[lo:hi], s["experts"][e].double().t())
        dw[e] = torch.mm(x[lo:hi].t(), dgu[lo:hi])
    d = {"dx": dx, "dw": dw if c["E"] > 0 else dw[0]}
    if c["keep"]:
        d["h"] = h
    return d
