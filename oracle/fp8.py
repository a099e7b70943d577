"""Float64 oracle of the fp8 operators: e4m3 rounding, row and block scales, norm, products, expert FFN.

Plain numpy, from the formulas in include/ftmoe.h; shares nothing with the CUDA path.
"""
import numpy as np

BLOCK = 128
TOP = 448.0
TINY = 2.0 ** -126


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _table():
    """Value of every e4m3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if c & 127 == 127:
            a = np.nan
        v[c] = -a if c & 128 else a
    return v


E4M3 = _table()


def decode(codes):
    return E4M3[np.asarray(codes, dtype=np.uint8)]


def step(v):
    """Spacing of the e4m3 values around |v| (2^-9 below the smallest normal 2^-6)."""
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.abs(v)))
    return 2.0 ** (np.clip(np.where(np.isfinite(e), e, -6), -6, 8) - 3)


def round_e4m3(v):
    """Nearest e4m3 value, ties to even, saturating at +-448."""
    v = np.asarray(v, dtype=np.float64)
    s = step(v)
    return np.clip(np.rint(v / s) * s, -TOP, TOP)


def tie_distance(v):
    """Distance of v from the nearest point where its rounding changes, over |v|."""
    s = step(v)
    f = np.abs(v / s - np.floor(v / s) - 0.5) * s
    return f / np.maximum(np.abs(v), 1e-300)


def row_scales(y):
    """[T][H] -> [T][blocks]: max(max|y| / 448, 2^-126), in float64."""
    T, H = y.shape
    p = np.zeros((T, blocks(H) * BLOCK))
    p[:, :H] = np.abs(y)
    return np.maximum(p.reshape(T, -1, BLOCK).max(2) / TOP, TINY)


def spread(scales, H):
    return np.repeat(np.asarray(scales, dtype=np.float64), BLOCK, axis=1)[:, :H]


def quantize_rows(y):
    """(values of the codes, scales as stored in float32)."""
    s = row_scales(y).astype(np.float32).astype(np.float64)
    return round_e4m3(y / spread(s, y.shape[1])), s


def rmsnorm(r, weight, eps):
    r = np.asarray(r, dtype=np.float64)
    return r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def block_spread(scales, n, k):
    s = np.asarray(scales, dtype=np.float64)
    return np.repeat(np.repeat(s, BLOCK, axis=0)[:n], BLOCK, axis=1)[:, :k]


def product(a, a_scales, w, w_scales):
    """(A W^T, the sum of the magnitudes of its terms): a, w are code values."""
    av = a * spread(a_scales, a.shape[1])
    wv = w * block_spread(w_scales, *w.shape)
    return av @ wv.T, np.abs(av) @ np.abs(wv).T


def product_bound(l1, K):
    """How far an f32 result may be from `product`.  Inside a block of 128 the tensor cores add
    four times 32 exact products to an accumulator; each such sum is taken to be right to
    2^-21 of the terms' magnitudes (f32 with some bits lost to aligning the terms).  Across blocks:
    the two scales' product and one fused multiply-add each, at most blocks + 2 roundings
    of 2^-24."""
    return (4 * 2.0 ** -21 + (blocks(K) + 2) * 2.0 ** -24) * l1 + 1e-37


def silu(a):
    with np.errstate(over="ignore"):   # exp(-a) = inf: the quotient is 0
        return a / (1.0 + np.exp(-a))


def quantize_weight(w):
    """[n][k] float64 -> (e4m3 bytes, float32 block scales)."""
    n, k = w.shape
    p = np.zeros((blocks(n) * BLOCK, blocks(k) * BLOCK))
    p[:n, :k] = w
    b = p.reshape(blocks(n), BLOCK, blocks(k), BLOCK)
    s = np.maximum(np.abs(b).max((1, 3)) / TOP, TINY).astype(np.float32)
    return encode(round_e4m3(w / block_spread(s, n, k))), s


def encode(values):
    """Bytes of exact e4m3 values."""
    order = np.argsort(E4M3[:127])
    v = np.asarray(values, dtype=np.float64)
    c = order[np.searchsorted(E4M3[:127][order], np.abs(v))].astype(np.uint8)
    return np.where(np.signbit(v), c | 0x80, c).astype(np.uint8)


def blob(gate, up, down):
    """Bytes of one expert from its three float64 matrices."""
    q = [quantize_weight(m) for m in (gate, up, down)]
    raw = b"".join(c.tobytes() for c, _ in q) + b"".join(s.tobytes() for _, s in q)
    return np.frombuffer(raw + b"\0" * (-len(raw) % 16), dtype=np.uint8)


def blob_parts(raw, H, I):
    """[(code values, scales)] of gate, up and down."""
    out, n, o = [], H * I, 3 * H * I
    for i, (rows, cols) in enumerate([(I, H), (I, H), (H, I)]):
        cnt = blocks(rows) * blocks(cols)
        out.append((decode(raw[i * n:(i + 1) * n]).reshape(rows, cols),
                    np.frombuffer(raw[o:o + 4 * cnt].tobytes(), dtype=np.float32).reshape(blocks(rows), -1)))
        o += 4 * cnt
    return out
