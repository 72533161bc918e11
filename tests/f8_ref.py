"""Plain 64-bit forms of the block-scaled e4m3 operators and of the sort by expert, on the CPU
(numpy), written from their definitions and sharing nothing with the library."""
import numpy as np

# the value of each e4m3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F, 0xFF NaN
_e, _m = (np.arange(128) >> 3), (np.arange(128) & 7)
_pos = np.where(_e == 0, _m / 8.0 * 2.0 ** -6, (1 + _m / 8.0) * 2.0 ** (_e.astype(float) - 7))
_pos[127] = np.nan
VALUES = np.concatenate([_pos, -_pos])
_FINITE = _pos[:127]                       # ascending, 0 .. 448


def blocks(n):
    return -(-n // 128)


def to_byte(v):
    """Nearest e4m3 byte of each v (fp64), ties to the even byte, +-448 beyond, NaN kept."""
    a = np.minimum(np.abs(v), 448.0)
    hi = np.clip(np.searchsorted(_FINITE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _FINITE[lo], _FINITE[hi] - a
    b = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    b = np.where(np.signbit(v), b | 0x80, b)
    return np.where(np.isnan(v), 0x7F, b).astype(np.uint8)


def quantize(x, block_rows=1):
    """(bytes, scales) of x: the least 2^p >= 2^-126 with max|x| <= 448 * 2^p over finite values."""
    x = np.asarray(x, np.float64)
    R, C = x.shape
    q = np.zeros((R, C), np.uint8)
    s = np.ones((-(-R // block_rows), blocks(C)))
    for r in range(s.shape[0]):
        for b in range(s.shape[1]):
            at = (slice(r * block_rows, (r + 1) * block_rows), slice(b * 128, (b + 1) * 128))
            v = x[at]
            top = np.abs(v[np.isfinite(v)]).max(initial=0.0)
            if top > 0:
                p = -126
                while top > 448.0 * 2.0 ** p:
                    p += 1
                s[r, b] = 2.0 ** p
            with np.errstate(invalid="ignore"):
                q[at] = to_byte(v / s[r, b])
    return q, s


def values(q, s, block_rows=1):
    R, C = q.shape
    return VALUES[q] * np.repeat(np.repeat(np.asarray(s, np.float64), block_rows, 0)[:R], 128, 1)[:, :C]


def matmul(a, sa, w, sw, offsets=None):
    """Exact products; `mag` the same with every factor's magnitude (what rounding errors scale with)."""
    x = values(a, sa)
    if offsets is None:
        v = values(w, sw, 128)
        return x @ v.T, np.abs(x) @ np.abs(v).T
    y = np.zeros((a.shape[0], w.shape[1]))
    mag = np.zeros_like(y)
    for e in range(w.shape[0]):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        v = values(w[e], sw[e], 128)
        y[at], mag[at] = x[at] @ v.T, np.abs(x[at]) @ np.abs(v).T
    return y, mag


def sort(ids, E):
    """(row_slot, slot_row, offsets) of the stable sort by expert."""
    T, k = ids.shape
    rows = [f for e in range(E) for f in np.flatnonzero(ids.reshape(-1) == e)]
    row_slot = np.full(T * k, -1, np.int32)
    row_slot[:len(rows)] = rows
    slot_row = np.full(T * k, -1, np.int32)
    slot_row[rows] = np.arange(len(rows))
    counts = [int((ids == e).sum()) for e in range(E)]
    return row_slot, slot_row.reshape(T, k), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def random_e4m3(rng, shape):
    """Bytes over every finite e4m3 value of ordinary size, zeros and subnormals among them."""
    return to_byte(rng.standard_normal(shape) * 40.0)
