"""Block-scaled 8-bit floats (F8) in plain 64-bit numpy, from their definition:
e4m3 codes, power-of-two scales, products, the gated block and its gradients."""
import numpy as np


def blocks(x):
    return -(-x // 128)


def decode(codes):
    """uint8 e4m3 codes -> values (0x7F and 0xFF are NaN)."""
    c = np.asarray(codes, dtype=np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * np.exp2(e - 7.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


_GRID = decode(np.arange(0x7F))          # the magnitudes 0 .. 448, in code order


def encode(v):
    """The nearest codes of |v| <= 448, ties to the even code, signs kept."""
    a = np.abs(v)
    lo = np.clip(np.searchsorted(_GRID, a, side="right") - 1, 0, 0x7D)
    mid = (_GRID[lo] + _GRID[lo + 1]) / 2
    up = (a > mid) | ((a == mid) & (lo % 2 == 1))
    return ((lo + up) | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def scale_of(top):
    """Scales of blocks whose largest magnitudes are `top`."""
    top = np.asarray(top, dtype=np.float64)
    m, e = np.frexp(np.where(top > 0, top, 1.0))          # top = m 2^e, m in [0.5, 1)
    e = np.maximum(np.where(m > 448 / 512, e - 8, e - 9), -126)
    return np.where(top == 0, 1.0, np.where(np.isfinite(top), np.exp2(e.astype(np.float64)), np.nan))


def pad_blocks(x, r, k):
    """x [rows, cols] zero-padded to whole r x k blocks -> [R, r, C, k]."""
    R, C = -(-x.shape[0] // r), -(-x.shape[1] // k)
    out = np.zeros((R * r, C * k), dtype=x.dtype)
    out[:x.shape[0], :x.shape[1]] = x
    return out.reshape(R, r, C, k)


def quantize(x, block=1):
    """x [rows, k] -> (codes uint8, scales): by rows [blocks(k), rows], by blocks
    [blocks(rows), blocks(k)]."""
    x = np.asarray(x, dtype=np.float64)
    b = pad_blocks(x, block, 128)
    with np.errstate(invalid="ignore"):
        top = np.abs(b).max(axis=(1, 3))
        s = scale_of(top)
        bad = ~np.isfinite(top)[:, None, :, None]
        v = np.where(bad, 0.0, b / np.where(np.isnan(s), 1.0, s)[:, None, :, None])
    codes = encode(v).reshape(b.shape[0] * block, -1)[:x.shape[0], :x.shape[1]]
    return codes, (s.T.copy() if block == 1 else s)


def spread(scales, rows, k, block=1):
    """Scales as one per value [rows, k]."""
    s = np.asarray(scales, dtype=np.float64)
    if block == 1:
        return np.repeat(s.T, 128, axis=1)[:, :k]
    return np.repeat(np.repeat(s, 128, axis=0)[:rows], 128, axis=1)[:, :k]


def values(codes, scales, block=1):
    return decode(codes) * spread(scales, *codes.shape, block)


def pad16(x):
    """Rows padded with zeros to a multiple of 16 values."""
    return np.pad(x, ((0, 0), (0, -x.shape[1] % 16)))


def gate(g, act):
    """act(g) and act'(g)."""
    y, dy = g, np.ones_like(g)
    if act == "gelu":
        c = np.sqrt(8 / np.pi)
        y, dy = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
    s = 1 / (1 + np.exp(-y))
    return g * s, s + g * s * (1 - s) * dy
