"""Plain 64-bit forms of the microscaled 4-bit operators (numpy), for their tests."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def e8m0(b):
    b = np.asarray(b).astype(np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))


def e4m3(b):
    b = np.asarray(b).astype(np.int64) & 0x7F
    m, e = b % 8, b // 8
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * np.ldexp(1.0, e - 7))


def quantize(x):
    """x [M, K] float64 -> (codes [M, K] 0..15, scale bytes [M, K/32])."""
    M, K = x.shape
    v = x.reshape(M, K // 32, 32)
    bad = ~np.isfinite(v).all(axis=2)
    top = np.where(bad, 1.0, np.abs(np.where(np.isfinite(v), v, 0.0)).max(axis=2, initial=0.0))
    e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1.0))[1] - 1 - 2, -127)
    e = np.clip(e, -127, 127)
    a = np.abs(np.where(np.isfinite(v), v, 0.0)) / np.ldexp(1.0, e)[..., None]
    # nearest point of the grid, ties to the even code: the midpoint between
    # codes c and c + 1 belongs to the even one of them
    c = np.zeros(a.shape, np.int64)
    for k in range(7):
        mid = (E2M1[k] + E2M1[k + 1]) / 2
        c += (a > mid) | ((a == mid) & (k % 2 == 1))
    codes = c | (np.signbit(v).astype(np.int64) << 3)
    codes[bad] = 0
    return codes.reshape(M, K), np.where(bad, 255, e + 127).astype(np.uint8)


def unpack(codes):
    """[..., K/2] bytes -> [..., K] codes."""
    c = np.asarray(codes)
    return np.stack([c & 15, c >> 4], axis=-1).reshape(*c.shape[:-1], -1)


def values(codes, scales, fmt):
    """The values of packed codes [R, K/2] with row-major scale bytes [R, K/block]."""
    s = e8m0(scales) if fmt == "mxfp4" else e4m3(scales)
    q = E2M1[unpack(codes)]
    return (q.reshape(*s.shape, -1) * s[..., None]).reshape(q.shape)


def slots(R, offsets=None):
    """(tile row, row in tile) of every row, -1 for rows of no group."""
    if offsets is None:
        r = np.arange(R)
        return r // 128, r % 128
    tr, at = np.full(R, -1), np.full(R, -1)
    for e in range(len(offsets) - 1):
        i = np.arange(offsets[e + 1] - offsets[e])
        tr[offsets[e]:offsets[e + 1]] = offsets[e] // 128 + e + i // 128
        at[offsets[e]:offsets[e + 1]] = i % 128
    return tr, at


def tile(rows, offsets=None, fill=0):
    """Row-major scale bytes [R, C] -> tiles, byte by byte of the layout's definition."""
    R, C = rows.shape
    trows = -(-R // 128) if offsets is None else R // 128 + len(offsets) - 1
    t = np.full((trows, -(-C // 4), 512), fill, np.uint8)
    t_pad = np.zeros((R, -(-C // 4) * 4), np.uint8)
    t_pad[:, :C] = rows
    tr, at = slots(R, offsets)
    for r in range(R):
        if tr[r] < 0:
            continue
        base = (at[r] % 32) * 16 + at[r] // 32 * 4
        for c in range(t_pad.shape[1]):
            t[tr[r], c // 4, base + c % 4] = t_pad[r, c]
    return t


def untile(tiles, R, C, offsets=None):
    tr, at = slots(R, offsets)
    c = np.arange(C)
    got = tiles[tr[:, None], c[None, :] // 4, ((at % 32) * 16 + at // 32 * 4)[:, None] + c[None, :] % 4]
    return np.where(tr[:, None] >= 0, got, 0)


def random_packed(R, K, fmt, seed, spread=10):
    """Uniform code bytes and scale bytes (E8M0: 2^-spread .. 2^spread; E4M3: every finite one)."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (R, K // 2), dtype=np.uint8)
    C = K // BLOCK[fmt]
    s = rng.integers(127 - spread, 127 + spread + 1, (R, C)) if fmt == "mxfp4" else rng.integers(0, 127, (R, C))
    return codes, s.astype(np.uint8)


def product(a, w):
    """(a w^T, the sums of |a| |w|, bound on what fp32 accumulation adds).

    The products of E2M1 values and their block scales are exact; an MMA of 64
    k adds them and the accumulator in at least fp32's 24 bits, truncating, so
    one loses at most 2^-23 of the magnitudes it sums for each of the 64 + 1
    terms it aligns in the worst case, and the accumulator 2^-23 per MMA."""
    y = a @ w.T
    mag = np.abs(a) @ np.abs(w).T
    n = -(-a.shape[1] // 64)
    return y, mag, (n + 65) * 2.0 ** -23 * mag


def silu_mul(y, bound):
    """silu(gate) * up of adjacent columns; |silu'| <= 1.1, a few fp32 roundings of the result."""
    g, u = y[:, 0::2], y[:, 1::2]
    bg, bu = bound[:, 0::2], bound[:, 1::2]
    s = g / (1 + np.exp(-g))
    return s * u, 1.1 * bg * np.abs(u) + (np.abs(s) + 1.1 * bg) * bu + 8 * 2.0 ** -23 * np.abs(s * u)


def check(y, r, bound):
    """y (a torch tensor) against r: the accumulation's bound, and half a step of y's type (subnormals: of the least normal)."""
    t = torch.finfo(y.dtype)
    v = y.double().cpu().numpy()
    allowed = bound + (t.eps / 2) * (np.abs(r) + bound) + t.tiny * t.eps / 2 + 3 * 2.0 ** -24 * np.abs(r)
    over = np.abs(v - r) > allowed
    # beyond the type's range: infinite, or at the border of it
    big = np.abs(r) + bound >= t.max * (1 - t.eps)
    over &= ~(big & (np.abs(v) >= t.max * (1 - t.eps)))
    assert not over.any() and not (np.isnan(v) & ~np.isnan(r)).any(), (
        f"{over.sum()} of {over.size} off, first {np.argwhere(over)[:3].tolist()}, {v[over][:3]} for {r[over][:3]}, allowed {allowed[over][:3]}")
