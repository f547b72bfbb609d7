"""Microscaled 4-bit floating point in plain numpy, from its definition (not
collected as tests).  Shares no code with the library."""
import numpy as np

BLOCK = {"nvfp4": 16, "mxfp4": 32}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def e4m3_values():
    """The 127 finite non-negative e4m3 values by byte (0x7f is NaN)."""
    v = np.empty(128)
    for b in range(128):
        e, m = b >> 3, b & 7
        v[b] = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    v[127] = np.nan
    return v


def scale_values(bytes_, fmt):
    b = np.asarray(bytes_).astype(np.int64)
    if fmt == "nvfp4":
        return e4m3_values()[b & 127]
    return np.where(b == 255, np.nan, np.exp2(b.astype(np.float64) - 127))


def nearest_even(x, grid):
    """Index into the increasing grid of the value nearest to x, ties to the even index, saturating."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(grid, x, side="left"), 1, len(grid) - 1)
    lo = hi - 1
    d_lo, d_hi = x - grid[lo], grid[hi] - x
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantize(x, fmt, g=1.0):
    """(codes [M, K], scale bytes [M, K / block]) with the stated FP32 steps."""
    x = np.asarray(x, dtype=np.float32)
    M, K = x.shape
    xb = x.reshape(M, K // BLOCK[fmt], BLOCK[fmt])
    amax = np.abs(xb).max(axis=2) if K else np.zeros((M, 0), np.float32)
    bad = ~np.isfinite(xb).all(axis=2)
    with np.errstate(all="ignore"):
        if fmt == "nvfp4":
            t = np.minimum(amax / (np.float32(6) * np.float32(g)), np.float32(448))
            scale = nearest_even(np.where(bad, 0, t), e4m3_values()[:127]).astype(np.uint8)
            step = (e4m3_values()[scale].astype(np.float32) * np.float32(g))[:, :, None]
            q = np.where(step > 0, xb / np.where(step > 0, step, 1), 0).astype(np.float32)
            scale = np.where(bad, 0x7F, scale).astype(np.uint8)
        else:
            _, e = np.frexp(amax.astype(np.float64))
            e = np.where(amax == 0, -127, np.maximum(e - 1 - 2, -127))
            scale = np.where(bad, 255, e + 127).astype(np.uint8)
            q = xb * np.exp2(-np.where(bad, 0, e).astype(np.float64))[:, :, None]
        q = np.where(bad[:, :, None], 0, q)
        mag = nearest_even(np.minimum(np.abs(q), 6), E2M1)
    neg = np.signbit(xb) & ~bad[:, :, None]
    return (mag + 8 * neg).astype(np.uint8).reshape(M, K), scale


def values(codes, scale, fmt, g=1.0):
    """What codes and scale bytes stand for, in 64 bits."""
    M, K = codes.shape
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return (v.reshape(M, K // BLOCK[fmt], BLOCK[fmt]) * scale_values(scale, fmt)[:, :, None]).reshape(M, K) * g


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], axis=2).reshape(packed.shape[0], -1)


def scale_rows(M, offsets=None, groups=1):
    """Scale row of each matrix row (-1: in no group)."""
    if offsets is None:
        per = M // groups
        r = np.arange(M)
        return r // per * (-(-per // 128) * 128) + r % per if per else r
    out = np.full(M, -1, dtype=np.int64)
    start = 0
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        out[lo:hi] = start + np.arange(hi - lo)
        start += -(-(hi - lo) // 128) * 128
    return out


def scale_places(rows, blocks):
    """Byte of every (row, block) in the tiles, by the layout's formula."""
    nt = -(-blocks // 4)
    r = np.asarray(rows, dtype=np.int64)[:, None]
    b = np.arange(blocks)[None, :]
    return (r // 128 * nt + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4


def tiles(scale, nbytes, offsets=None, groups=1, fill=0):
    """Scale bytes [M, blocks] as a tile buffer; `fill` in the rows that hold nothing."""
    M, blocks = scale.shape
    rows = scale_rows(M, offsets, groups)
    buf = np.full(nbytes, fill, dtype=np.uint8)
    if blocks % 4:  # blocks past K are zero in every row
        nt = -(-blocks // 4)
        full = buf.reshape(-1, nt, 32, 4, 4)
        full[:, nt - 1, :, :, blocks % 4:] = 0
    has = rows >= 0
    buf[scale_places(rows[has], blocks)] = scale[has]
    return buf


def untile(buf, M, blocks, offsets=None, groups=1):
    return buf[scale_places(np.maximum(scale_rows(M, offsets, groups), 0), blocks)]
