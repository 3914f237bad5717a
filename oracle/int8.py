"""Products of int8 rows and int8 matrices with a scale a row and a scale a channel, oracle side (test infrastructure)."""
from __future__ import annotations

import numpy as np


def grouped_product(a_q, a_s, w_q, w_s, off, rows, w2_q=None, w2_s=None) -> np.ndarray:
    """out[r, n] = a_s * w_s[e, n] * sum_k a_q[rows[r], k] * w_q[e, n, k] in fp64 for the rows r of expert e's
    segment [off[e], off[e+1]); with a second matrix silu of it times the second product. NaN past off[-1]."""
    a = np.asarray(a_q, dtype=np.float64)
    out = np.full((len(rows), w_q.shape[1]), np.nan)
    for e in range(len(off) - 1):
        r = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        src = np.asarray(rows[r])

        def product(q, s):
            # integers below 2^53: exact in fp64
            p = a[src] @ np.asarray(q[e], dtype=np.float64).T
            return p * np.asarray(s[e], dtype=np.float64)[None, :] * np.asarray(a_s, dtype=np.float64)[src][:, None]
        g = product(w_q, w_s)
        if w2_q is not None:
            with np.errstate(over="ignore"):
                g = g / (1.0 + np.exp(-g)) * product(w2_q, w2_s)
        out[r] = g
    return out
