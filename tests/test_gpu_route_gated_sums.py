"""What the gated router's ids rest on: the error that its fp32 sums are taken to have, and rows whose squares fp32 loses.

A block of a row is 64 bf16 or 32 fp32 columns. Its sum may be off by 6 (bf16) or 8 (fp32) units of 2^-23 of the sum of its
terms' magnitudes: how the matrix instructions round inside is measured, here too, not documented.
"""
import math
import sys

import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from tests.helpers import np64
from tests.test_gpu_route_gated import DT, _gate

pytestmark = pytest.mark.gpu

UNITS = {"bf16": 6.0, "f32": 8.0}
BLOCK = {"bf16": 64, "f32": 32}


def _say(msg):
    print(f"[gate-sums-test] {msg}", file=sys.stderr, flush=True)


def _patterns(rng, act, T, n):
    """T rows of n numbers whose sum, one after another in fp32, loses the most: one large term and many that lie at the end of its
    bits (of one sign, and of both), terms over 24 bits, terms that cancel, and plain ones; each in any order."""
    v = np.empty((T, n))
    for t in range(T):
        kind = t % 6
        if kind == 0:       # each small term is lost next to the large one, together they are not
            v[t] = 2.0 ** -25 * (1 + rng.random(n))
            v[t, rng.integers(n)] = 1
        elif kind == 1:     # as many large as small ones
            v[t] = np.where(rng.random(n) < 0.5, 1, 2.0 ** -rng.integers(22, 27, n)) * (1 + rng.random(n))
        elif kind == 2:     # over all 24 bits
            v[t] = 2.0 ** -rng.uniform(0, 25, n)
        elif kind == 3:     # both signs
            v[t] = rng.choice([-1, 1], n) * 2.0 ** -rng.uniform(0, 25, n)
        elif kind == 4:     # pairs that cancel but for their last bits
            h = 1 + rng.random(n // 2)
            v[t] = rng.permutation(np.concatenate([h, -h * (1 + rng.choice([-1, 1], n // 2) * 2.0 ** -rng.integers(8, 20, n // 2))]))
        else:
            v[t] = rng.standard_normal(n)
    return torch.from_numpy(v.astype(np.float32)).to(DT[act])


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("seed", range(4))
def test_sums_of_a_block_are_off_by_no_more_than_taken(act, seed):
    """One expert is never looked at again, so its sigmoid is that of the kernel's own sum. With the sum's rounded value taken off
    as the router's bias what is left is the error, l: the weight is 0.5 + l / 4 to 2^-25 and |l|^3 / 48."""
    rng = np.random.default_rng(seed)
    T, n = 768, BLOCK[act]
    x = _patterns(rng, act, T, n)
    w = _patterns(rng, act, 6, n)[seed] if seed else torch.ones(n, dtype=DT[act])
    x = torch.cat([x, torch.zeros(T, 64 - n, dtype=DT[act])], 1)
    w = torch.cat([w, torch.zeros(64 - n, dtype=DT[act])])
    terms = np64(x) * np64(w)                            # exact in fp64
    mag = np.abs(terms).sum(1)
    k = 2.0 ** np.floor(np.log2(2.0 ** 9 / mag))         # magnitudes between 2^8 and 2^9, one token a call: its bias is its own
    worst = 0.0
    for t in range(0, T, 8):
        xt = (x[t:t + 1].float() * float(k[t])).to(DT[act])
        s = math.fsum((np64(xt) * np64(w))[0])
        bias = np.float32(-s)
        _, wt = m.moe_route_gated(xt.cuda(), w[None].cuda(), torch.tensor([bias]).cuda(), 1, _gate(sigmoid=True, renorm=False))
        l = (float(wt[0, 0]) - 0.5) * 4
        off = abs(l - (s + float(bias)))
        unit = 2.0 ** -23 * mag[t] * k[t]
        assert off <= UNITS[act] * unit + 4 * 2.0 ** -25 + abs(l) ** 3 / 12, f"{off / unit:.2f} units (pattern {t % 6})"
        worst = max(worst, off / unit)
    _say(f"{act} seed {seed}: off by {worst:.2f} units at most")


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E", [2, 40])
def test_choices_between_sums_of_another_order(E, sigmoid, act):
    """Experts that take the same terms in another order: the fp32 sums differ by their errors, the true ones by one
    small term a block later. Each token hangs on it, for every size of it down to 2^-34 of the magnitudes."""
    rng = np.random.default_rng(E)
    n, T = BLOCK[act], 600
    half = n // 2
    p = _patterns(rng, act, T, half).float()
    x, wr = torch.zeros(T, 192), torch.zeros(E, 192)
    pos = [rng.permutation(half), half + rng.permutation(half)]
    x[:, pos[0]], x[:, pos[1]] = p, p
    mag = p.abs().sum(1, dtype=torch.float64)
    for e in range(E):
        wr[e, pos[e % 2]] = 1                            # the same sum from either half of the block
        wr[e, 128 + e] = 1
    x[:, 128:128 + E] = torch.from_numpy(rng.choice([-1, 1], (T, E)) * 2.0 ** -rng.integers(17, 35, (T, E)).astype(float)
                                         * (1 + rng.random((T, E)))).float() * 2.0 ** mag.log2().round()[:, None].float()
    x, wr = x.to(DT[act]), wr.to(DT[act])
    K = min(E, 8)
    ids, _ = m.moe_route_gated(x.cuda(), wr.cuda(), None, K, _gate(sigmoid=sigmoid))
    small = np64(x)[:, 128:128 + E]                      # the logits but for what all share
    want = np.argsort(-small, axis=1, kind="stable")[:, :K]
    gap = np.sort(small, axis=1)[:, ::-1]
    gap = (gap[:, :K] - np.append(gap, np.full((T, 1), -np.inf), 1)[:, 1:K + 1]).min(1)
    # what 64-bit sums of 192 terms and scores keep apart (a sigmoid falls off as exp(-l))
    clear = gap > 2.0 ** -48 * (1 + mag.numpy()) * np.exp(np.maximum(np64(p).sum(1), 0) if sigmoid else 0)
    assert clear.sum() > T // 2
    bad = np.argwhere((ids.cpu().numpy() != want).any(1) & clear)[:, 0]
    assert bad.size == 0, f"token {bad[0]} (pattern {bad[0] % 6}): {ids[bad[0]].tolist()}, not {want[bad[0]]} ({bad.size} tokens)"


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 40, 4500])
@pytest.mark.parametrize("d", [64, 8192])
@pytest.mark.parametrize("E", [2, 30, 256])
def test_rows_whose_squares_are_lost(E, d, T, act):
    """Tokens of 1e-23 or 1e-30 (squares below fp32) against weights of 1e19 or 1e30 that cancel in fp32 sums but not in 64 bits, and
    the other way round; among them rows of zeros, whose experts tie."""
    if T * d > 1 << 22:
        pytest.skip("the same kernels as with fewer columns")
    rng = np.random.default_rng(E + T)
    for tiny, huge, swap in ((1e-23, 1e19, False), (1e-30, 1e30, False), (1e-23, 1e19, True), (1e-30, 1e30, True)):
        a = torch.zeros(T, d)
        a[:, :3] = float(torch.tensor(tiny).to(DT[act]))
        w = torch.zeros(E, d)
        big = torch.tensor(huge).to(DT[act]).float()
        for e in range(E // 2, E):                       # the first half's logits are zeros
            w[e, 0], w[e, 1], w[e, 2] = big, float(rng.integers(1, 200)) * 2.0 ** -32 * big, -big
        zero = rng.random(T) < 0.5
        if T == 1:
            zero[:] = False
        a[torch.from_numpy(zero)] = 0
        if swap:                                         # tiny weights, huge tokens
            k = float(big) / float(torch.tensor(tiny).to(DT[act]))
            a, w = a.double() * k, w.double() / k
        a, w = a.to(DT[act]), w.to(DT[act])
        l = np64(a)[:, :1] * np64(w)[None, :, 1][0]      # the first and the third term cancel
        K = min(E, 5)
        want = np.argsort(-l, axis=1, kind="stable")[:, :K]
        assert (want[zero] == np.arange(K)).all() and (want[~zero, 0] >= E // 2).all()
        _say(f"E={E} d={d} T={T} {act} {tiny} {swap}")
        for sigmoid in (False, True):
            for use_workspace in (True, False):
                ids, _ = m.moe_route_gated(a.cuda(), w.cuda(), None, K, _gate(sigmoid=sigmoid), use_workspace=use_workspace)
                got = ids.cpu().numpy()
                bad = np.argwhere((got != want).any(1))[:, 0]
                assert bad.size == 0, f"token {bad[0]}: {got[bad[0]]}, not {want[bad[0]]} ({bad.size} tokens)"
