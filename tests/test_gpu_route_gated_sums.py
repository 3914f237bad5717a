"""What the gated router's ids rest on: rows whose squares fp32 loses."""
import sys

import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from tests.helpers import np64
from tests.test_gpu_route_gated import DT, _gate

pytestmark = pytest.mark.gpu

def _say(msg):
    print(f"[gate-sums-test] {msg}", file=sys.stderr, flush=True)


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
