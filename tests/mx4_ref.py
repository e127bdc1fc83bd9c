"""Plain 64-bit forms of the MX4 operators (CPU), written from the format's
definition: the magnitude table, the block scale and the layout formulas of
include/qgemm.h, with no code shared with the library."""
import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TABLE = np.concatenate([GRID, -GRID])


def quantize(x):
    """x float64 [rows, k] -> (codes uint8 [rows, k] 0..15, scale bytes [rows, k/32])."""
    rows, k = x.shape
    v = x.reshape(rows, k // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    a = np.where(bad[..., None], 0.0, np.abs(v))
    top = a.max(-1)
    e = np.frexp(np.where(top > 0, top, 1.0))[1] - 1          # floor(log2)
    s = np.where(top > 0, np.maximum(e - 2 + 127, 0), 0)
    y = a / np.ldexp(1.0, s - 127)[..., None]
    mids = (GRID[:-1] + GRID[1:]) / 2
    code = np.zeros(v.shape, dtype=np.uint8)
    for i, mid in enumerate(mids):                            # between codes i and i + 1
        code += ((y > mid) if i % 2 == 0 else (y >= mid)).astype(np.uint8)   # ties to even
    code |= np.signbit(v).astype(np.uint8) << 3
    code[bad] = 0
    return code.reshape(rows, k), np.where(bad, 255, s).astype(np.uint8)


def values(codes, scales):
    """Codes [..., k], scale bytes [..., k/32] -> float64 values (NaN for 255)."""
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return TABLE[codes] * np.repeat(f, 32, axis=-1)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def tile(codes, scales):
    """Codes [rows, k] 0..15 and scales [rows, k/32] -> tiled bytes, by the
    header's formulas."""
    rows, k = codes.shape
    R, nw = (rows + 15) // 16 * 16, (k + 511) // 512
    full = np.zeros((R, k), dtype=np.uint8)
    full[:rows] = codes
    r, c = np.meshgrid(np.arange(R), np.arange(k), indexing="ij")
    lane = 16 * ((c % 128) // 32) + r % 16
    byte = ((r // 16) * (k // 128) + c // 128) * 1024 + lane * 16 + (c % 32) // 2
    tc = np.zeros(R * k // 2, dtype=np.uint8)
    np.add.at(tc, byte.ravel(), (full << (4 * (c % 2))).astype(np.uint8).ravel())
    ts = np.zeros((R // 16, nw, 64, 4), dtype=np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(k // 32), indexing="ij")
    ts[r // 16, b // 16, 16 * (b % 4) + r % 16, (b // 4) % 4] = scales
    return tc.reshape(R, k // 2), ts


def rne(x, dtype):
    """float64 -> torch dtype with one rounding (nearest even).  Through fp32
    only where that is exact; the test inputs that need a single rounding are
    exact in fp32."""
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(dtype)


def product_bound(a, w, c, dtype):
    """Largest possible |result - c| of sum_k a w in fp32, in any order, then
    rounded to dtype.  The products are exact in fp32 (at most 11 + 2
    significant bits); each of at most k + 1 additions (the bias among them) is
    off by one unit of 2^-23 of a partial sum, which sum |a w| bounds."""
    k = a.shape[-1]
    mag = np.abs(a) @ np.abs(w).T
    acc = (k + 1) * 2.0 ** -23 * mag
    half = torch.finfo(dtype).eps / 2
    tiny = float(torch.finfo(dtype).smallest_normal) * half * 2
    return acc + (np.abs(c) + acc) * half + tiny
