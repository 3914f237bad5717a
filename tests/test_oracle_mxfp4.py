"""Pins of the MXFP4 and norm oracles that do not reuse their formulas (CPU)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import mxfp4 as omx
from oracle import norm as onorm

VALUES = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def test_e2m1_values():
    assert omx.e2m1_value(np.arange(16)).tolist() == VALUES + [-v for v in VALUES]
    assert np.signbit(omx.e2m1_value(np.array([8])))[0]


def test_e8m0_values():
    assert omx.e8m0_value(np.array([0, 1, 127, 254])).tolist() == [2.0 ** -127, 2.0 ** -126, 1.0, 2.0 ** 127]
    assert np.isnan(omx.e8m0_value(np.array([255])))[0]


def test_rounding_against_exact_nearest_search():
    rng = np.random.default_rng(0)
    pts = list(rng.uniform(-7, 7, 400))
    for a, b in zip(VALUES, VALUES[1:]):
        mid = (a + b) / 2
        pts += [mid, -mid, np.nextafter(mid, 0), np.nextafter(mid, 9), a, -b]
    codes = omx.round_to_e2m1(np.array(pts))
    for p, c in zip(pts, codes):
        d = [abs(Fraction(abs(p)) - Fraction(v)) for v in VALUES]
        best = [i for i in range(8) if d[i] == min(d)]
        want = best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0)
        assert (c & 7) == want and bool(c & 8) == bool(np.signbit(p)), p


@pytest.mark.parametrize("amax,byte", [(6.0, 127), (4.0, 127), (3.99, 126), (7.99, 127), (8.0, 128), (1.0, 125),
                                       (2.0 ** -126, 0), (2.0 ** -124, 1), (2.0 ** -149, 0), (0.0, 0),
                                       (3.0e38, 252)])
def test_scale_byte(amax, byte):
    w = np.zeros((1, 32))
    w[0, 7] = -amax
    q, s = omx.quantize(w)
    assert s.tolist() == [[byte]]


def test_round_trip_bound_and_lossless_grid():
    rng = np.random.default_rng(1)
    w = rng.standard_normal((5, 96))
    q, s = omx.quantize(w)
    v = omx.dequantize(q, s)
    step = np.repeat(omx.e8m0_value(s), 32, -1)
    # the widest gap below 6 is 2 (half: 1); past 6 the block's largest is below 8
    assert (np.abs(v - w) <= np.where(np.abs(w) > 6 * step, 2, 1) * step).all()
    grid = np.array(VALUES + [-x for x in VALUES] + VALUES + [-x for x in VALUES]) * 2.0 ** -9
    q, s = omx.quantize(grid[None])
    assert (omx.dequantize(q, s)[0] == grid).all()


def test_non_finite_blocks():
    w = np.ones((1, 96))
    w[0, 3], w[0, 70] = np.inf, np.nan
    q, s = omx.quantize(w)
    assert s.tolist() == [[255, 125, 255]]
    assert not q[0, :16].any() and not q[0, 32:].any()
    v = omx.dequantize(q, s)[0]
    assert np.isnan(v[:32]).all() and (v[32:64] == 1).all() and np.isnan(v[64:]).all()


def test_tiled_layout_by_hand():
    """One element at a time: its byte and its scale's byte, from the header's formulas."""
    rows, cols = 32, 640                      # n = 5: a full scale group of four blocks and one of one
    rng = np.random.default_rng(2)
    q = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
    s = rng.integers(0, 256, (rows, cols // 32), dtype=np.uint8)
    qt, st = (x.reshape(-1) for x in omx.tile(q, s))
    n = cols // 128
    for r, col in [(0, 0), (5, 33), (15, 127), (16, 128), (31, 639), (20, 511), (9, 512)]:
        blk, byte = (r // 16) * n + col // 128, (col % 128) // 2
        assert qt[blk * 1024 + 256 * (byte // 16) + 16 * (r % 16) + byte % 16] == q[r, col // 2]
        c = col // 32
        k = c // 4
        m = min(4, n - 4 * (k // 4))
        assert st[(r // 16) * n * 64 + 256 * (k // 4) + m * (16 * (c % 4) + r % 16) + k % 4] == s[r, c]


def test_grouped_product_against_a_scalar_loop():
    rng = np.random.default_rng(3)
    a, w, w2 = rng.standard_normal((3, 8)), rng.standard_normal((3, 2, 8)), rng.standard_normal((3, 2, 8))
    off, rows = [0, 2, 2, 4], [2, 0, 1, 1, 0]
    out, sw = omx.grouped_product(a, w, off, np.array(rows)), omx.grouped_product(a, w, off, np.array(rows), w2)
    for r, e in enumerate([0, 0, 2, 2]):
        for j in range(2):
            g = sum(a[rows[r], i] * w[e, j, i] for i in range(8))
            u = sum(a[rows[r], i] * w2[e, j, i] for i in range(8))
            assert abs(out[r, j] - g) < 1e-12 and abs(sw[r, j] - g / (1 + np.exp(-g)) * u) < 1e-12
    assert np.isnan(out[4]).all()


def test_norms_against_torch():
    torch.manual_seed(0)
    y, res = torch.randn(6, 64, dtype=torch.float64), torch.randn(6, 64, dtype=torch.float64)
    w, w2, g = (torch.randn(64, dtype=torch.float64) for _ in range(3))
    ref = torch.nn.functional.rms_norm(y, (64,), w, 1e-5)
    assert np.allclose(onorm.rms(y.numpy(), w.numpy(), 1e-5), ref.numpy(), rtol=1e-12)
    gate = torch.stack([g, 2 * g])
    out, nxt = onorm.post(y.numpy(), res.numpy(), w.numpy(), gate.numpy(), 4, 0.5, 2.0, 1e-5, w2.numpy(), 1e-3)
    want = 0.5 * res + 2.0 * ref * torch.cat([g.expand(4, 64), 2 * g.expand(2, 64)])
    assert np.allclose(out, want.numpy(), rtol=1e-12)
    assert np.allclose(nxt, torch.nn.functional.rms_norm(want, (64,), w2, 1e-3).numpy(), rtol=1e-12)
    assert onorm.post(y.numpy(), res.numpy())[1] is None
    assert np.array_equal(onorm.post(y.numpy(), res.numpy())[0], (res + y).numpy())
