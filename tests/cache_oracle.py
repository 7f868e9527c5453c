"""Plain forms of the paged cache for its tests: the position rotation in 64 bits, the 4-bit codec and the places of new
rows, one row after another."""
import numpy as np

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def rotate(x, row, interleaved):
    """A head's elements x (64 bits), its first ones rotated by row: half cosines, half sines."""
    half = len(row) // 2
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = x[..., a] * row[i] - x[..., b] * row[half + i]
        y[..., b] = x[..., b] * row[i] + x[..., a] * row[half + i]
    return y


def rotate_size(x, row, interleaved):
    """The same over absolute values: what the rotation's roundings are counted against."""
    half = len(row) // 2
    x, row = np.abs(x), np.abs(row)
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = x[..., a] * row[i] + x[..., b] * row[half + i]
        y[..., b] = x[..., b] * row[i] + x[..., a] * row[half + i]
    return y


def encode(x, kind):
    """fp32 rows [.., D] to (codes [.., D/2], scales [.., D/32]) as uint8."""
    x = np.asarray(x, dtype=np.float32)
    y = x.reshape(*x.shape[:-1], -1, 32).astype(np.float64)
    top = np.abs(y).max(-1)
    finite = np.isfinite(y).all(-1)
    m, e = np.frexp(np.where(finite & (top > 0), top, 1.0))         # top = m 2^e, 1/2 <= m < 1
    e = e - 1 - 2 + (m > 0.875)
    e = np.where(top > 0, e, -126)
    e = np.clip(e, -126, 125 if kind == "bf16" else 13)
    a = np.abs(np.where(finite[..., None], y, 0.0)) * 2.0 ** -e[..., None].astype(np.float64)
    # the nearest value; of two as near the one whose code is even
    d = np.abs(a[..., None] - VALUES)
    code = np.zeros(a.shape, dtype=np.int64)
    best = d.min(-1)
    for c in (1, 3, 5, 7, 0, 2, 4, 6):          # the last that is as near as any: even ones come last
        code = np.where(d[..., c] == best, c, code)
    code = code + 8 * np.signbit(y)
    code = np.where(finite[..., None], code, 0).reshape(x.shape)
    return (code[..., 0::2] + 16 * code[..., 1::2]).astype(np.uint8), np.where(finite, e + 127, 255).astype(np.uint8)


def decode(code, scale):
    """What codes and scales stand for, in 64 bits."""
    c = np.stack([code & 15, code >> 4], -1).reshape(*code.shape[:-1], -1)
    y = VALUES[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return y * np.repeat(s, 32, -1)


def places(lens, new, table, page, pages, positions=None):
    """(row, sequence, position, page, place) of every new row that is written."""
    at = 0
    for n, (length, count) in enumerate(zip(lens, new)):
        for j in range(count):
            pos = length - count + j
            if length > 0 and 0 <= pos < table.shape[1] * page and (positions is None or pos < positions):
                p = int(table[n, pos // page])
                if 0 <= p < pages:
                    yield at + j, n, pos, p, pos % page
        at += count
