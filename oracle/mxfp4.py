"""MXFP4 encoding and the products of its values, oracle side (test infrastructure).

OCP microscaling format MXFP4: blocks of 32 consecutive elements of a row share
a scale byte b (E8M0: worth 2**(b - 127), 255 is NaN); an element is an e2m1
code: bit 3 the sign, exponent field e (2 bits, bias 1), mantissa bit m: m / 2
for e = 0, else (1 + m / 2) * 2**(e - 1). Two codes a byte, even element low.

Reading of the quantizer: b = floor(log2(max |w|)) - 2 + 127, at least 0 (2 is
the exponent of the largest element, 6 = 1.5 * 2**2); code = the value nearest
to w / 2**(b - 127), ties to the even code, saturated to +-6, sign of w kept; an
all-zero block stores b = 0; a block with an infinity or a NaN b = 255, codes 0.

All arithmetic is fp64 on exact copies of the fp32/bf16 values.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def e2m1_value(codes) -> np.ndarray:
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 1) & 3, c & 1
    mag = np.where(e == 0, m / 2.0, (1 + m / 2.0) * 2.0 ** (e - 1))
    return np.where(c & 8, -mag, mag)


def e8m0_value(b) -> np.ndarray:
    b = np.asarray(b).astype(np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))


def round_to_e2m1(r) -> np.ndarray:
    """Code of the e2m1 value nearest to each finite fp64 number (ties to the even code).

    The magnitudes are the codes 0..7 in ascending order, so the code is the
    number of midpoints passed; a midpoint belongs to the even one of its two codes.
    """
    a = np.abs(np.asarray(r, dtype=np.float64))
    grid = e2m1_value(np.arange(8))
    code = np.zeros(a.shape, dtype=np.int64)
    for c in range(7):
        mid = (grid[c] + grid[c + 1]) / 2
        code += (a > mid) | ((a == mid) & (c % 2 == 1))
    return np.where(np.signbit(r), code | 8, code).astype(np.uint8)


def quantize(w):
    """w [..., cols] -> (codes uint8 [..., cols/2], scale bytes uint8 [..., cols/32])."""
    w = np.asarray(w, dtype=np.float64)
    blk = w.reshape(*w.shape[:-1], w.shape[-1] // BLOCK, BLOCK)
    bad = ~np.isfinite(blk).all(-1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(blk), blk, 0.0)).max(-1))
    _, e = np.frexp(amax)                                   # amax = m * 2**e, 0.5 <= m < 1
    b = np.where(amax > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    step = np.ldexp(1.0, b - 127)[..., None]
    code = round_to_e2m1(np.where(bad[..., None], 0.0, blk) / step)
    code = code.reshape(*w.shape[:-1], w.shape[-1] // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), np.where(bad, 255, b).astype(np.uint8)


def dequantize(q, s) -> np.ndarray:
    """fp64 [..., cols] values of codes [..., cols/2] and scale bytes [..., cols/32]."""
    q = np.asarray(q, dtype=np.uint8)
    v = np.stack([e2m1_value(q & 15), e2m1_value(q >> 4)], -1).reshape(*q.shape[:-1], q.shape[-1] * 2)
    return v * np.repeat(e8m0_value(s), BLOCK, axis=-1)


def tile(q, s):
    """Row-major codes and scales -> the kernels' tiled layout (same shapes), element by element of its definition.

    Codes: 16 rows x 128 columns are 1 KiB; inside, row r's 32 columns c sit in
    the 16 bytes at 256*c + 16*r. Scales: per 16 rows, four such blocks' bytes
    side by side (fewer at the end of the row).
    """
    q, s = np.asarray(q, dtype=np.uint8), np.asarray(s, dtype=np.uint8)
    cols = q.shape[-1] * 2
    rows, n = q.size * 2 // cols, cols // 128
    pieces = q.reshape(rows, cols // 32, 16)
    sc = s.reshape(rows, cols // 32)
    r, c = np.meshgrid(np.arange(rows), np.arange(cols // 32), indexing="ij")
    rg, k, lane = r // 16, c // 4, 16 * (c % 4) + r % 16
    qt = np.empty((rows * cols // 32, 16), np.uint8)
    qt[(rg * n + k) * 64 + lane] = pieces
    m = np.minimum(4, n - 4 * (k // 4))
    st = np.empty(rows * cols // 32, np.uint8)
    st[rg * n * 64 + 256 * (k // 4) + m * lane + k % 4] = sc
    return qt.reshape(q.shape), st.reshape(s.shape)


def grouped_product(a, w, offsets, rows, w2=None):
    """out[r] = W_e a[rows[r]] (or silu of it times W2_e a[rows[r]]) for r in expert e's segment; fp64.

    a [., d], w and w2 [E, f, d] fp64; rows past the last segment are NaN."""
    out = np.full((len(rows), w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        r = np.arange(offsets[e], offsets[e + 1])
        x = a[rows[r]]
        p = x @ w[e].T
        if w2 is not None:
            p = p / (1 + np.exp(-p)) * (x @ w2[e].T)
        out[r] = p
    return out
