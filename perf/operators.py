"""Operators around the expert layer and its 4-bit products, as cases that can be timed and compared.

Seven operators: the routed rows' way to their experts and back (sort and dispatch, the weighted combine, and the
gradient of each) and microscaled 4-bit floating point (quantise and read back, the dense product, the grouped
expert product).  ``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, with ``own``,
through the calls that a user makes of ``blackwell_tensor_core_gb300.ops``.  ``exact`` states each operator in 64 bits.

Definitions (row-major everywhere; T tokens, k experts a token, E experts, H columns):

  sort      pairs p = t * k + j in stable order of their expert, pairs without an expert (id outside 0 .. E-1) last:
            order[r] = the pair at sorted row r, position[t, j] = the sorted row of pair (t, j),
            offsets[e] = the first row of expert e, offsets[E] = the rows that have an expert
  dispatch  rows[r] = x[order[r] // k], zero for r >= offsets[E]
            gradient: dx[t] = sum_j d_rows[position[t, j]] over the pairs that have an expert
  combine   y[t] = sum_j w[t, j] * rows[position[t, j]] over the pairs that have an expert
            gradient: d_rows[position[t, j]] = w[t, j] * dy[t], dw[t, j] = <dy[t], rows[position[t, j]]>, zero elsewhere
  4 bits    values {0, .5, 1, 1.5, 2, 3, 4, 6} with a sign, two a byte (even column in the low half), and one scale a block:
            nvfp4: blocks of 16, scale s = e4m3(amax / (6 g)), at most 448, values of x / (s g), with one g a matrix;
            mxfp4: blocks of 32, scale 2^(floor(log2 amax) - 2) held as e8m0, g = 1; ties go to the even value
  products  D[i, n] = sum_k A[i, k] B[n, k] of the values that the operands stand for; grouped: the rows of expert e
            with B[e]; with SwiGLU, B[e] = [gate | up] along n and H = silu(gate) * up
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BLOCK = {"nvfp4": 16, "mxfp4": 32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step's tokens on their way to the experts: latency
        dict(name="dispatch_decode", op="dispatch", T=16, k=8, E=32, H=4096, dtype="bf16", drop=0.0),
        # the benchmark's expert layer: 4096 tokens, top 8 of 32
        dict(name="dispatch_4096", op="dispatch", T=4096, k=8, E=32, H=4096, dtype="bf16", drop=0.0),
        # training, an odd batch with dropped pairs: the dispatch's gradient
        dict(name="dispatch_grad_odd", op="dispatch_grad", T=5003, k=6, E=64, H=2056, dtype="fp16", drop=0.1),
        # the experts' answers back to one decode step's tokens
        dict(name="combine_decode", op="combine", T=24, k=4, E=64, H=7168, dtype="bf16", drop=0.0),
        # the benchmark's layer again, back to token order
        dict(name="combine_4096", op="combine", T=4096, k=8, E=32, H=4096, dtype="bf16", drop=0.0),
        # training: the combine's gradient, rows in 32 bits whose length divides into no whole vectors
        dict(name="combine_grad_odd", op="combine_grad", T=2049, k=8, E=32, H=2047, dtype="fp32", drop=0.05),
        # activations of the routed layer put into 4 bits and read back (as a training step does to see the error)
        dict(name="quant_nv_32768", op="quant", M=32768, K=4096, fmt="nvfp4", dtype="bf16"),
        # a small ragged batch in the power-of-two format
        dict(name="quant_mx_odd", op="quant", M=999, K=7168, fmt="mxfp4", dtype="fp16"),
        # one token through a linear layer: quantise the activation, multiply by weights kept in 4 bits
        dict(name="linear_1_token_mx", op="linear", M=1, N=4096, K=7168, fmt="mxfp4", dtype="bf16"),
        # the benchmark's decode-like shape
        dict(name="linear_72_nv", op="linear", M=72, N=16384, K=7168, fmt="nvfp4", dtype="bf16"),
        # the headline square, both operands already in 4 bits
        dict(name="gemm_8192_nv", op="gemm", M=8192, N=8192, K=8192, fmt="nvfp4", dtype="bf16"),
        # the benchmark's expert FC1 with SwiGLU: quantise the routed rows, multiply by each expert's weights
        dict(name="experts_fc1_nv", op="experts", T=4096, k=8, E=32, N=4096, K=4096, fmt="nvfp4", dtype="bf16",
             swiglu=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, step):
    return max(lo, _log_int(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "quant", "linear", "gemm", "experts"])
    fmt = rng.choice(["nvfp4", "mxfp4"])
    half = rng.choice(["bf16", "fp16"])
    if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        k = rng.choice([1, 2, 4, 6, 8])
        E = rng.choice([8, 32, 60, 128, 256])
        H = _log_int(rng, 128, 7168)
        H = H if rng.random() < 0.3 else max(8, H // 8 * 8)
        T = _log_int(rng, 1, min(16384, (1 << 27) // (k * H)))
        return dict(op=op, T=T, k=k, E=E, H=H, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    drop=rng.choice([0.0, 0.0, 0.15]))
    if op == "quant":
        K = _mult(rng, 64, 16384, 32)
        return dict(op=op, M=_log_int(rng, 1, min(65536, (1 << 27) // K)), K=K, fmt=fmt,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 256), N=_mult(rng, 512, 16384, 8), K=_mult(rng, 512, 8192, 32), fmt=fmt,
                    dtype=half)
    if op == "gemm":
        return dict(op=op, M=_log_int(rng, 200, 8192), N=_mult(rng, 512, 8192, 8), K=_mult(rng, 512, 8192, 32),
                    fmt=fmt, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    E = rng.choice([8, 16, 32])
    return dict(op=op, T=_log_int(rng, 1, 2048), k=rng.choice([1, 2, 4, 8]), E=E, N=_mult(rng, 512, 4096, 32),
                K=_mult(rng, 512, 4096, 32), fmt=fmt, dtype=half, swiglu=rng.random() < 0.5)


def _elt(dtype):
    return 4 if dtype == "fp32" else 2


def _fp4_bytes(rows, K, fmt):
    return rows * K // 2 + rows * -(-K // _BLOCK[fmt])


def work(case):
    c = case
    if "H" in c:
        e, pairs = _elt(c["dtype"]), c["T"] * c["k"]
        tok, row = c["T"] * c["H"] * e, pairs * c["H"] * e
        kept = row * (1.0 - c["drop"])
        if c["op"] == "dispatch":  # 64-bit ids in, order and position out
            return {"bytes": tok + row + 16 * pairs, "flops": 0}
        if c["op"] == "dispatch_grad":
            return {"bytes": tok + kept + 4 * pairs, "flops": pairs * c["H"]}
        if c["op"] == "combine":
            return {"bytes": tok + kept + 8 * pairs, "flops": 2 * pairs * c["H"]}
        return {"bytes": tok + kept + row + 12 * pairs, "flops": 3 * pairs * c["H"]}
    if c["op"] == "quant":
        n = c["M"] * c["K"] * _elt(c["dtype"])
        return {"bytes": 2 * n + 2 * _fp4_bytes(c["M"], c["K"], c["fmt"]), "flops": 2 * c["M"] * c["K"]}
    if c["op"] == "experts":
        rows = c["T"] * c["k"]
        busy = c["E"] * (1.0 - (1.0 - 1.0 / c["E"]) ** rows)  # experts that rows reach
        out = c["N"] // 2 if c["swiglu"] else c["N"]
        return {"bytes": rows * c["K"] * 2 + busy * _fp4_bytes(c["N"], c["K"], c["fmt"]) + rows * out * 2,
                "flops": 2 * rows * c["N"] * c["K"]}
    act = c["M"] * c["K"] * 2 if c["op"] == "linear" else _fp4_bytes(c["M"], c["K"], c["fmt"])
    return {"bytes": act + _fp4_bytes(c["N"], c["K"], c["fmt"]) + c["M"] * c["N"] * _elt(c["dtype"]),
            "flops": 2 * c["M"] * c["N"] * c["K"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _route(T, k, E, drop, g):
    """Top-k of skewed router logits: int64 ids, 32-bit weights; dropped pairs have id -1."""
    dev = g.device
    logits = torch.randn(T, E, generator=g, device=dev) + 0.5 * torch.randn(E, generator=g, device=dev)
    top, ids = torch.topk(logits, min(k, E), dim=1)
    weights = torch.softmax(top, dim=1)
    if drop > 0:
        ids = ids.masked_fill(torch.rand(ids.shape, generator=g, device=dev) < drop, -1)
    return ids.contiguous(), weights.contiguous()


def _activations(rows, cols, g):
    """Normal values with channels of different spread, as activations before a linear layer have."""
    spread = torch.exp(0.5 * torch.randn(cols, generator=g, device=g.device))
    return torch.randn(rows, cols, generator=g, device=g.device) * spread


def _plain_sort(ids, E):
    flat = ids.reshape(-1).to(torch.int64)
    key = torch.where((flat < 0) | (flat >= E), torch.full_like(flat, E), flat)
    order = torch.argsort(key, stable=True)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=order.device)
    counts = (key[:, None] == torch.arange(E, device=key.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    return offsets.to(torch.int32), order.to(torch.int32), position.to(torch.int32).reshape(ids.shape)


def _weights_fp4(rows, K, fmt, g, groups=1):
    """Weights in 4 bits as a loaded model holds them: codes, scales in tiles of 128 rows x 4, and g."""
    w = torch.randn(rows, K, generator=g, device=g.device) * 0.02
    gs = w.abs().amax() / 2688.0 if fmt == "nvfp4" else torch.ones((), device=g.device)
    gs = gs.reshape(1).to(torch.float32)
    codes, scales = _plain_quantize(w, fmt, gs)
    return _pack(codes), _to_tiles(scales, fmt, groups), gs


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=_device())
    g.manual_seed(int(seed))
    dt = _DT[c["dtype"]]
    s = {"c": c}
    if "H" in c:
        ids, weights = _route(c["T"], c["k"], c["E"], c["drop"], g)
        s["ids"], s["weights"] = ids, weights
        if c["op"] != "dispatch":
            s["offsets"], s["order"], s["position"] = _plain_sort(ids, c["E"])
        if c["op"] in ("dispatch", "combine_grad"):
            s["x"] = _activations(c["T"], c["H"], g).to(dt)
        if c["op"] != "dispatch":
            s["rows"] = _activations(c["T"] * c["k"], c["H"], g).to(dt)
        return s
    if c["op"] == "quant":
        x = _activations(c["M"], c["K"], g)
    elif c["op"] == "gemm":
        a = _activations(c["M"], c["K"], g)
        s["ag"] = _global(a, c["fmt"])
        codes, scales = _plain_quantize(a, c["fmt"], s["ag"])
        s["a"], s["as"] = _pack(codes), _to_tiles(scales, c["fmt"], 1)
        s["b"], s["bs"], s["bg"] = _weights_fp4(c["N"], c["K"], c["fmt"], g)
        return s
    elif c["op"] == "linear":
        x = _activations(c["M"], c["K"], g)
        s["b"], s["bs"], s["bg"] = _weights_fp4(c["N"], c["K"], c["fmt"], g)
    else:
        ids, _ = _route(c["T"], c["k"], c["E"], 0.0, g)
        s["offsets"] = _plain_sort(ids, c["E"])[0]
        s["bounds"] = s["offsets"].tolist()
        x = _activations(c["T"] * c["k"], c["K"], g)
        s["b"], s["bs"], s["bg"] = _weights_fp4(c["E"] * c["N"], c["K"], c["fmt"], g, c["E"])
    s["ag"] = _global(x, c["fmt"])
    s["x"] = x.to(dt)
    return s


def _global(x, fmt):
    """The scale of a matrix: its largest value, before it was rounded to its type, at the largest product of the two
    small formats."""
    if fmt == "mxfp4":
        return torch.ones(1, device=x.device)
    return (x.abs().amax() / 2688.0).reshape(1).to(torch.float32)


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _e2m1_index(a):
    """Index of the nearest of {0, .5, 1, 1.5, 2, 3, 4, 6} to a >= 0, ties to the even index."""
    n = (a > 0.25).to(torch.uint8)
    n += a >= 0.75
    n += a > 1.25
    n += a >= 1.75
    n += a > 2.5
    n += a >= 3.5
    n += a > 5.0
    return n


def _plain_quantize(x, fmt, g):
    """Codes [M, K] and scale bytes [M, K / block] of 32-bit x, every step rounded to 32 bits."""
    M, K = x.shape
    b = _BLOCK[fmt]
    xb = x.reshape(M, -1, b)
    amax = xb.abs().amax(dim=2)
    if fmt == "nvfp4":
        sb = torch.clamp(amax / (6.0 * g), max=448.0).to(torch.float8_e4m3fn)
        step = sb.to(torch.float32) * g
        q = xb / torch.where(step > 0, step, torch.ones_like(step))[:, :, None]
        q = torch.where((step > 0)[:, :, None], q, torch.zeros_like(q))
        scale = sb.view(torch.uint8)
    else:
        exp = (amax.view(torch.int32) >> 23) - 127 - 2
        scale = torch.clamp(exp + 127, min=0, max=254).to(torch.uint8)
        q = xb * ((254 - scale.to(torch.int32)) << 23).view(torch.float32)[:, :, None]
    codes = _e2m1_index(q.abs()) | (torch.signbit(xb).to(torch.uint8) << 3)
    return codes.reshape(M, K), scale


def _pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()


def _tiles_shape(rows, blocks, groups):
    per = -(-(rows // groups) // 128)
    return per, -(-blocks // 4)


def _to_tiles(scales, fmt, groups):
    """Scale bytes in tiles of 128 rows x 4 blocks: byte (r % 32) * 16 + (r // 32) * 4 + b, tiles along K first; the
    rows of each group padded to whole tiles."""
    rows, blocks = scales.shape
    per, nb = _tiles_shape(rows, blocks, groups)
    full = torch.zeros(groups, per * 128, nb * 4, dtype=torch.uint8, device=scales.device)
    full[:, : rows // groups, :blocks] = scales.reshape(groups, rows // groups, blocks)
    return full.reshape(groups * per, 4, 32, nb, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _from_tiles(tiles, rows, blocks, groups):
    per, nb = _tiles_shape(rows, blocks, groups)
    full = tiles.reshape(groups * per, nb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(groups, per * 128, nb * 4)
    return full[:, : rows // groups, :blocks].reshape(rows, blocks)


def _values(codes, scales, fmt, g):
    """What codes [M, K] and scale bytes stand for, in 32 bits."""
    M, K = codes.shape
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    v = table[(codes & 7).long()] * (1.0 - 2.0 * (codes >> 3).to(torch.float32))
    if fmt == "nvfp4":
        s = scales.view(torch.float8_e4m3fn).to(torch.float32)
    else:
        s = torch.exp2(scales.to(torch.float32) - 127.0)
    return (v.reshape(M, -1, _BLOCK[fmt]) * s[:, :, None]).reshape(M, K) * g


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), dim=2).reshape(packed.shape[0], -1)


def _read(packed, tiles, fmt, g, groups=1):
    rows, K = packed.shape[0], packed.shape[1] * 2
    return _values(_unpack(packed), _from_tiles(tiles, rows, K // _BLOCK[fmt], groups), fmt, g)


def _kept(position, offsets):
    return position < offsets[-1]


def _run_plain(s):
    c = s["c"]
    dt = _DT[c["dtype"]]
    if c["op"] == "dispatch":
        offsets, order, position = _plain_sort(s["ids"], c["E"])
        rows = s["x"][(order // c["k"]).long()]
        has = torch.arange(order.numel(), device=order.device) < offsets[-1]
        rows = torch.where(has[:, None], rows, torch.zeros_like(rows))
        return {"offsets": offsets, "order": order, "position": position, "rows": rows}
    if c["op"] in ("dispatch_grad", "combine", "combine_grad"):
        kept = _kept(s["position"], s["offsets"])
        w = s["weights"] if c["op"] != "dispatch_grad" else torch.ones_like(s["weights"])
        w = torch.where(kept, w, torch.zeros_like(w))
        rows = s["rows"][s["position"].long()].to(torch.float32)
        rows = torch.where(kept[:, :, None], rows, torch.zeros_like(rows))
        if c["op"] != "combine_grad":
            return (rows * w[:, :, None]).sum(1).to(dt)
        dy = s["x"].to(torch.float32)
        d_rows = torch.empty_like(s["rows"])
        d_rows[s["position"].reshape(-1).long()] = (w[:, :, None] * dy[:, None, :]).reshape(-1, c["H"]).to(dt)
        return {"d_rows": d_rows, "d_weights": (rows * dy[:, None, :]).sum(2)}
    fmt = c["fmt"]
    if c["op"] == "gemm":
        return (_read(s["a"], s["as"], fmt, s["ag"]) @ _read(s["b"], s["bs"], fmt, s["bg"]).t()).to(dt)
    codes, scales = _plain_quantize(s["x"].to(torch.float32), fmt, s["ag"])
    a = _values(codes, scales, fmt, s["ag"])
    if c["op"] == "quant":
        return a.to(dt)
    if c["op"] == "linear":
        return (a @ _read(s["b"], s["bs"], fmt, s["bg"]).t()).to(dt)
    w = _read(s["b"], s["bs"], fmt, s["bg"], c["E"]).reshape(c["E"], c["N"], c["K"])
    at = s["bounds"]
    d = torch.cat([a[at[e]:at[e + 1]] @ w[e].t() for e in range(c["E"])])
    if c["swiglu"]:
        gate, up = d[:, : c["N"] // 2], d[:, c["N"] // 2:]
        d = gate / (1.0 + torch.exp(-gate)) * up
    return d.to(dt)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    from blackwell_tensor_core_gb300 import ops
    c = s["c"]
    if c["op"] == "dispatch":
        r = ops.moe_sort(s["ids"], c["E"])
        return {"offsets": r.offsets, "order": r.order, "position": r.position, "rows": ops.moe_dispatch(s["x"], r)}
    if c["op"] in ("dispatch_grad", "combine", "combine_grad"):
        r = ops.Routing(s["offsets"], s["order"], s["position"])
        if c["op"] == "dispatch_grad":
            return ops.moe_dispatch_grad(s["rows"], r)
        if c["op"] == "combine":
            return ops.moe_combine(s["rows"], r, s["weights"])
        d_rows, d_weights = ops.moe_combine_grad(s["x"], s["rows"], r, s["weights"])
        return {"d_rows": d_rows, "d_weights": d_weights}
    fmt, dt = c["fmt"], _DT[c["dtype"]]
    ag = s["ag"] if fmt == "nvfp4" else None
    if c["op"] == "quant":
        return ops.dequantize_fp4(ops.quantize_fp4(s["x"], fmt, global_scale=ag), out_dtype=dt)
    bg = s["bg"] if fmt == "nvfp4" else None
    if c["op"] == "experts":
        q = ops.quantize_fp4(s["x"], fmt, global_scale=ag, group_offsets=s["offsets"])
        w = ops.Fp4Matrix(s["b"], s["bs"], fmt, bg, groups=c["E"])
        return ops.grouped_gemm_fp4(q, w, swiglu=c["swiglu"], out_dtype=dt)
    w = ops.Fp4Matrix(s["b"], s["bs"], fmt, bg)
    if c["op"] == "linear":
        return ops.gemm_fp4(ops.quantize_fp4(s["x"], fmt, global_scale=ag), w, out_dtype=dt)
    return ops.gemm_fp4(ops.Fp4Matrix(s["a"], s["as"], fmt, ag), w, out_dtype=dt)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_values(x, fmt, g):
    """x put into 4 bits and back, by the definition, with numpy-like steps in 64 bits."""
    M, K = x.shape
    x = x.double().reshape(M, -1, _BLOCK[fmt])
    big = x.abs().max(dim=2, keepdim=True).values
    if fmt == "nvfp4":
        t = (big / (6.0 * g.double())).clamp(max=448.0)
        # e4m3: 3 mantissa bits down to 2^-6, then steps of 2^-9
        e = torch.floor(torch.log2(t.clamp(min=2.0 ** -6)))
        quantum = torch.exp2(e - 3)
        step = torch.round(t / quantum) * quantum * g.double()
    else:
        _, e = torch.frexp(big)
        step = torch.exp2((e.double() - 1 - 2).clamp(min=-127, max=127))
    q = torch.where(step > 0, x / torch.where(step > 0, step, torch.ones_like(step)), torch.zeros_like(x))
    mag = q.abs().clamp(max=6.0)
    # e2m1: steps of 1/2 below 2, of 1 below 4, of 2 above; round() goes to the even multiple
    unit = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0)).double()
    v = torch.sign(q) * (torch.round(mag / unit) * unit).clamp(max=6.0)
    return (v * step).reshape(M, K)


def _exact_read(packed, tiles, fmt, g, groups=1):
    """Values of stored codes and scale tiles: every element looked up by the layout's own formula."""
    rows, K = packed.shape[0], packed.shape[1] * 2
    dev = packed.device
    cols = torch.arange(K, device=dev)
    byte = packed[:, cols // 2].to(torch.int16)
    code = torch.where(cols % 2 == 0, byte % 16, byte // 16)
    m, e, neg = code % 2, code // 2 % 4, code // 8
    v = torch.where(e == 0, 0.5 * m.double(), (1.0 + 0.5 * m.double()) * torch.exp2(e.double() - 1.0))
    v = torch.where(neg == 1, -v, v)
    per_group = rows // groups
    r = torch.arange(rows, device=dev)
    r = r // per_group * (-(-per_group // 128) * 128) + r % per_group
    blk = torch.arange(K // _BLOCK[fmt], device=dev)
    nb = -(-blk.numel() // 4)
    at = ((r // 128)[:, None] * nb + (blk // 4)[None, :]) * 512 + ((r % 32) * 16 + r % 128 // 32 * 4)[:, None] + blk % 4
    sb = tiles[at].double()
    if fmt == "nvfp4":
        em, ee = sb % 8, torch.floor(sb / 8)
        s = torch.where(ee == 0, em * 2.0 ** -9, (1.0 + em / 8) * torch.exp2(ee - 7))
    else:
        s = torch.exp2(sb - 127)
    return v * s.repeat_interleave(_BLOCK[fmt], dim=1) * g.double()


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if "H" in c:
        T, k = c["T"], c["k"]
        if c["op"] == "dispatch":
            ids = s["ids"].reshape(-1)
            has = (ids >= 0) & (ids < c["E"])
            token = torch.arange(T * k, device=ids.device) // k
            by_expert = torch.sort(torch.where(has, ids, c["E"]), stable=True).indices
            rows = s["x"].double()[token[by_expert]] * has[by_expert].double()[:, None]
            return {"offsets": None, "order": None, "position": None, "rows": rows}
        pos, n = s["position"].long(), int(s["offsets"][-1])
        rows = s["rows"].double()
        w = s["weights"].double() if c["op"] != "dispatch_grad" else torch.ones_like(s["weights"]).double()
        w = w * (pos < n)
        if c["op"] != "combine_grad":
            y = torch.zeros(T, c["H"], dtype=torch.float64, device=rows.device)
            for j in range(k):
                y += w[:, j:j + 1] * rows[pos[:, j]]
            return y
        dy = s["x"].double()
        d_rows, d_w = torch.zeros_like(rows), torch.zeros_like(w)
        for j in range(k):
            d_rows[pos[:, j]] = w[:, j:j + 1] * dy
            d_w[:, j] = (rows[pos[:, j]] * dy).sum(1) * (pos[:, j] < n)
        return {"d_rows": d_rows, "d_weights": d_w}
    fmt = c["fmt"]
    if c["op"] == "gemm":
        return _exact_read(s["a"], s["as"], fmt, s["ag"]) @ _exact_read(s["b"], s["bs"], fmt, s["bg"]).t()
    a = _exact_values(s["x"], fmt, s["ag"])
    if c["op"] == "quant":
        return a
    if c["op"] == "linear":
        return a @ _exact_read(s["b"], s["bs"], fmt, s["bg"]).t()
    w = _exact_read(s["b"], s["bs"], fmt, s["bg"], c["E"]).reshape(c["E"], c["N"], c["K"])
    out = torch.zeros(a.shape[0], c["N"], dtype=torch.float64, device=a.device)
    for e in range(c["E"]):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        out[lo:hi] = a[lo:hi] @ w[e].t()
    if c["swiglu"]:
        gate, up = out[:, : c["N"] // 2], out[:, c["N"] // 2:]
        out = gate * torch.sigmoid(gate) * up
    return out
