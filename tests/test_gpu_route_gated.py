"""Gated routing on the GPU against the fp64 oracle.

Ids are those of the values in 64 bits, so they are compared for equality, except
where two evaluations in 64 bits may differ: a sum of d products in any order is off
by at most d * 2^-53 * sum_i |x_i w_i|; a score moves by at most as much as its logits
(softmax: twice the largest), its own evaluation takes some 8 + E/2 roundings of 2^-53,
and the bias one more of the sum. So ids may be exchanged between choice values that differ
by no more than
    tau = 2 * (2 * d * 2^-53 * sum_i |x_i w_i| + (8 + E / 2) * 2^-53 + 2^-53 * (1 + |bias|)).
A logit of the kernel that is not looked at again in 64 bits is a sum of fp32 sums of 32 products: each such sum takes at most 32 additions,
and their sum a few more, each off by at most 2^-23 of the magnitudes (half of
that where it rounds), so a logit is off by at most
    delta = 40 * 2^-23 * sum_i |x_i w_i|.
A weight is a ratio of exponentials (softmax, renormalised or not) or a sigmoid
over a sum of sigmoids: its relative error is at most exp(2 delta) - 1 with the
token's largest delta, plus its rounding to fp32 and that of the scale (2^-24 each) and
2^-23 for the fp32 sum of a softmax over all experts.
"""
import itertools
import sys

import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from oracle import gate as ogate
from tests.helpers import np64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")


def _say(msg):
    print(f"[gate-test] {msg}", file=sys.stderr, flush=True)


def _gate(select=None, sigmoid=False, groups=1, group_topk=1, top2=False, renorm=True, scale=1.0):
    return m.Gate(score=m.MOE_SCORE_SIGMOID if sigmoid else m.MOE_SCORE_SOFTMAX,
                  select_bias=None if select is None else torch.from_numpy(select).cuda(), groups=groups,
                  group_topk=group_topk, group_by=m.MOE_GROUP_TOP2 if top2 else m.MOE_GROUP_MAX, renorm=renorm, scale=scale)


def _check(x, wr, bias, K, select=None, what="", **kw):
    """x [T, d], wr [E, d] CPU tensors of one type; bias, select fp32 arrays or None."""
    _say(f"{what} T={x.shape[0]} d={x.shape[1]} E={wr.shape[0]} K={K} {kw}")
    b = None if bias is None else torch.from_numpy(bias).cuda()
    ids, w = m.moe_route_gated(x.cuda(), wr.cuda(), b, K, _gate(select, **kw))
    okw = {k: v for k, v in kw.items()}
    rid, rw, l = ogate.route(np64(x), np64(wr), bias, K, select_bias=select, **okw)
    got = ids.cpu().numpy()
    bad = np.argwhere((got != rid).any(1))[:, 0]
    if bad.size:
        c = ogate.scores(l, kw.get("sigmoid", False)) + (0 if select is None else np.asarray(select, np.float64))
        c = np.concatenate([c, np.full((len(c), 1), -INF)], 1)      # id -1
        tau = 2 ** -52 * (2 * x.shape[1] * (np.abs(np64(x)) @ np.abs(np64(wr)).T).max(1) + 9 + wr.shape[0] / 2
                          + (0 if select is None else np.abs(select[np.isfinite(select)]).max(initial=0)))
        apart = np.abs(np.take_along_axis(c, got, 1) - np.take_along_axis(c, rid, 1)).max(1)
        distinct = np.array([len(set(i)) == len(i) for i in got.tolist()])
        bad = bad[~((apart <= tau) & distinct)[bad]]
    assert bad.size == 0, f"{what}: ids of token {bad[0]}: {got[bad[0]]}, not {rid[bad[0]]} ({bad.size} tokens)"
    with np.errstate(invalid="ignore"):
        mag = (np.abs(np64(x)) @ np.abs(np64(wr)).T).max(1, initial=0.0)
    delta = 40 * 2.0 ** -23 * mag[:, None]
    bound = np.abs(rw) * (np.expm1(np.minimum(2 * delta, 50)) + 4 * 2.0 ** -24 + 2.0 ** -23) + 1e-37
    err = np.abs(np64(w) - rw)
    assert (err <= bound).all(), f"{what}: weights off by {np.max(err / bound):.3g} of the bound"
    return ids, w


def _draw(rng, T, d, E, act, sigma=0.02):
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(DT[act])
    wr = torch.from_numpy((sigma * rng.standard_normal((E, d))).astype(np.float32)).to(DT[act])
    return x, wr


# (T, d, E, K, groups, group_topk): one token to several tiles, every number of expert blocks, odd sizes
SIZES = [(1, 64, 1, 1, 1, 1), (1, 4096, 16, 2, 1, 1), (2, 128, 3, 3, 1, 1), (15, 192, 17, 4, 1, 1), (16, 576, 60, 4, 4, 2),
         (17, 1088, 64, 6, 8, 3), (63, 8192, 64, 6, 8, 3), (64, 320, 16, 8, 2, 2), (65, 448, 33, 5, 3, 2),
         (100, 256, 72, 8, 4, 1), (31, 1344, 65, 2, 5, 5), (33, 832, 128, 8, 64, 5), (130, 512, 160, 7, 8, 4),
         (70, 704, 250, 8, 5, 2), (513, 2048, 256, 8, 8, 4), (1, 4160, 256, 8, 8, 4), (200, 64, 256, 1, 1, 1),
         (1100, 320, 16, 2, 1, 1), (2050, 256, 48, 3, 6, 3)]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,d,E,K,groups,group_topk", SIZES)
def test_against_oracle(T, d, E, K, groups, group_topk, sigmoid, act):
    rng = np.random.default_rng(T * 7919 + d + E)
    x, wr = _draw(rng, T, d, E, act)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    select = ((0.05 if sigmoid else 0.2 / E) * rng.standard_normal(E)).astype(np.float32)
    _check(x, wr, bias, K, select, "all", sigmoid=sigmoid, groups=groups, group_topk=group_topk,
           top2=E // groups >= 2, renorm=True, scale=2.5)
    _check(x, wr, None, K, None, "bare", sigmoid=sigmoid, groups=groups, group_topk=group_topk, renorm=False)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("E,groups", [(72, 4), (128, 1), (250, 10), (256, 8)])
@pytest.mark.parametrize("T", [4096, 4097, 5000, 8193])
def test_many_tokens_of_many_experts(T, E, groups, act):
    """Two blocks of tokens a workgroup, full and partial, and one: against the oracle, and as in another batch."""
    rng = np.random.default_rng(T + E)
    x, wr = _draw(rng, T, 192, E, act)
    select = (0.05 * rng.standard_normal(E)).astype(np.float32)
    kw = dict(sigmoid=True, groups=groups, group_topk=max(1, groups // 2), top2=True)
    ids, _ = _check(x, wr, None, 6, select, "many", **kw)
    part, _ = m.moe_route_gated(x[-700:].contiguous().cuda(), wr.cuda(), None, 6, _gate(select, **kw))
    assert torch.equal(ids[-700:], part)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("E,groups", [(16, 1), (64, 8), (256, 8), (96, 3)])
def test_values_closer_than_fp32_sums(E, groups, act):
    """Pairs of experts whose rows differ in one element, by its last bit, against an x that is tiny there: their
    logits differ by 1e-7 to 1e-12 of the sums. Both orders occur, in and across groups, with and without a bias."""
    rng = np.random.default_rng(E)
    T, d = 96, 1024
    x, wr = _draw(rng, T, d, E, act)
    perm = rng.permutation(E)
    for a, b in zip(perm[::2], perm[1::2]):
        wr[b] = wr[a]
        i = int(rng.integers(d))
        wr[b, i] = torch.nextafter(wr[a, i], torch.tensor(INF if rng.random() < 0.5 else -INF, dtype=wr.dtype))
        x[:, i] = (x[:, i].float() * 2.0 ** -float(rng.integers(0, 12))).to(x.dtype)
    select = np.zeros(E, np.float32)
    for sigmoid, sel in itertools.product((False, True), (None, select, select + 0.25)):
        _check(x, wr, None, min(E, 8), sel, "close", sigmoid=sigmoid, groups=groups, group_topk=max(1, groups // 2),
               top2=True)


@pytest.mark.parametrize("E,groups,K", [(2, 1, 1), (16, 1, 3), (64, 8, 4), (256, 8, 8)])
@pytest.mark.parametrize("base", [700.0, 3000.0])
def test_logits_whose_fp32_sums_are_off_by_more_than_one(E, groups, K, base):
    """Logits of 5e5 and 9e6 that differ by one or two: an fp32 sum's error there, 0.5 to 8, says nothing about a score."""
    rng = np.random.default_rng(E + K)
    T, d = 64, 128
    x, wr = np.zeros((T, d), np.float32), np.zeros((E, d), np.float32)
    x[:, 0], x[:, 1:17] = base, rng.standard_normal((T, 16))
    wr[:, 0], wr[:, 1:17] = base, 0.3 * rng.standard_normal((E, 16))
    _check(torch.from_numpy(x), torch.from_numpy(wr), None, K, what="coarse sums", groups=groups, group_topk=max(1, groups // 2),
           top2=groups > 1)
    _check(torch.from_numpy(x), torch.from_numpy(wr), None, K, select=(0.1 / E * rng.standard_normal(E)).astype(np.float32),
           what="coarse sums", groups=groups, group_topk=max(1, groups // 2), top2=groups > 1)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_a_bias_against_a_score_step_by_step(sigmoid):
    """An expert without a score (a router bias of -inf) whose bias is another one's score but for a few units of fp32, up
    and down over the tokens."""
    T, d, E = 4096, 64, 3
    x, wr = np.zeros((T, d), np.float32), np.zeros((E, d), np.float32)
    x[:, 0], x[:, 1] = 1, (np.arange(T) - T / 2) * 2.0 ** -32
    wr[0, :2] = 0.75, 1
    score = 1 / (1 + np.exp(-0.75))
    _check(torch.from_numpy(x), torch.from_numpy(wr), np.array([0, 0, -INF], np.float32), 1,
           select=np.array([0, -1, score], np.float32), what="steps", sigmoid=sigmoid)


@pytest.mark.parametrize("E,groups,K", [(2, 1, 1), (16, 1, 3), (64, 8, 4), (256, 8, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_a_bias_against_logits_finer_than_fp32(E, groups, K, sigmoid):
    """Logits about 1000 that differ by less than fp32 holds there (6e-5), and biases of the same size as the scores'
    differences: the scores have to come from the 64-bit logits."""
    rng = np.random.default_rng(E + K)
    T, d = 64, 64
    x, wr = np.zeros((T, d), np.float32), np.zeros((E, d), np.float32)
    x[:, 0], x[:, 1:9] = 1000, rng.standard_normal((T, 8))
    wr[:, 0], wr[:, 1:9] = 0 if sigmoid else 1, 2e-5 * rng.standard_normal((E, 8))
    _check(torch.from_numpy(x), torch.from_numpy(wr), None, K, select=(1e-5 / (4 if sigmoid else E) * rng.standard_normal(E)).astype(np.float32),
           what="fine bias", sigmoid=sigmoid, groups=groups, group_topk=max(1, groups // 2), top2=groups > 1)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("E,groups", [(8, 1), (40, 4), (256, 16)])
def test_exact_ties_go_to_the_lower_index(E, groups, act):
    """Small integers: every logit is exact, and many are equal."""
    rng = np.random.default_rng(E + 1)
    x = torch.from_numpy(rng.integers(-2, 3, (50, 64)).astype(np.float32)).to(DT[act])
    x[3] = 0                                                        # every expert ties
    wr = torch.from_numpy(rng.integers(-1, 2, (E, 64)).astype(np.float32)).to(DT[act])
    wr[E // 2:] = wr[:E - E // 2]                                   # equal rows, in other groups
    for sigmoid, top2 in itertools.product((False, True), (False, True)):
        _check(x, wr, None, min(E, 8), None, "ties", sigmoid=sigmoid, groups=groups, group_topk=max(1, groups // 4 + 1),
               top2=top2)


@pytest.mark.parametrize("E,groups,group_topk", [(8, 1, 1), (64, 8, 3), (200, 5, 2)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_disabled_experts(E, groups, group_topk, sigmoid):
    rng = np.random.default_rng(E + 2)
    x, wr = _draw(rng, 40, 256, E, "bf16")
    K = 6
    n = E // groups
    for case in range(4):
        select = (0.05 * rng.standard_normal(E)).astype(np.float32)
        if case == 0:                                               # a few
            select[rng.permutation(E)[:E // 8]] = -INF
        elif case == 1:                                             # all but K - 2, so two ids are -1 at least
            select[rng.permutation(E)[K - 2:]] = -INF
        elif case == 2:                                             # all
            select[:] = -INF
        else:                                                       # whole groups, and one expert by NaN
            select[:n * (groups // 2)] = -INF
            select[-1] = np.nan
        ids, w = _check(x, wr, None, K, select, f"disabled {case}", sigmoid=sigmoid, groups=groups,
                        group_topk=group_topk, top2=n >= 2)
        if case == 2:
            assert (ids == -1).all() and (w == 0).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("E", [16, 256])
def test_extreme_values(E, act):
    """Logits past exp's range, a router bias of -inf, tokens of zeros, tiny, huge and non-finite numbers."""
    rng = np.random.default_rng(E + 3)
    x, wr = _draw(rng, 12, 128, E, act)
    x[0] = 0
    x[1] = (x[1].float() * 1e-30).to(x.dtype)
    x[2] = (x[2].float() * 1e4).to(x.dtype)                         # |l| up to some 1e4: probabilities underflow
    x[3] = (x[3].float() * 1e36).to(x.dtype)                        # products past the fp32 range, logits too
    x[4] = (x[4].float() * 1e-37).to(x.dtype)
    bias = np.zeros(E, np.float32)
    bias[1] = -INF
    select = (0.1 * rng.standard_normal(E)).astype(np.float32)
    select[2] = 1e6
    select[3] = INF
    for sigmoid, renorm in itertools.product((False, True), (False, True)):
        keep = [0, 1, 2, 4, 5, 6, 7, 8, 9, 10, 11] + ([3] if sigmoid else [])
        _check(x[keep], wr, bias, 4, select, "extreme", sigmoid=sigmoid, renorm=renorm)
        _check(x[keep], wr, None, 4, None, "extreme, no bias", sigmoid=sigmoid, renorm=renorm)
    y = x.clone()
    y[5, 7] = float("nan")
    y[6, 9] = INF
    for sigmoid in (False, True):
        ids, w = m.moe_route_gated(y.cuda(), wr.cuda(), None, 4, _gate(sigmoid=sigmoid))
        assert (ids[5] == -1).all() and (w[5] == 0).all()
        rid, rw = m.moe_route_gated(x.cuda(), wr.cuda(), None, 4, _gate(sigmoid=sigmoid))
        rest = [0, 1, 2, 4, 7, 8, 9, 10, 11]
        assert torch.equal(ids[rest], rid[rest]) and torch.equal(w[rest], rw[rest])
        assert torch.isfinite(w).all()


def test_a_token_does_not_depend_on_its_batch():
    """The same ids and weights, bit for bit, alone, in a small batch and in a large one."""
    rng = np.random.default_rng(9)
    for E, act in ((16, "bf16"), (60, "f32"), (256, "bf16")):
        x, wr = _draw(rng, 600, 512, E, act)
        x, wr = x.cuda(), wr.cuda()
        g = _gate((0.05 * rng.standard_normal(E)).astype(np.float32), sigmoid=True, groups=4, group_topk=2)
        ids, w = m.moe_route_gated(x, wr, None, 3, g)
        for rows in (slice(0, 1), slice(5, 6), slice(100, 140), slice(599, 600), slice(3, 70)):
            i, v = m.moe_route_gated(x[rows].contiguous(), wr, None, 3, g)
            assert torch.equal(i, ids[rows]) and torch.equal(v, w[rows]), (E, rows)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,groups", [(1, 4096, 16, 1), (40, 8192, 64, 8), (700, 256, 60, 4), (4500, 128, 256, 8), (3, 8192, 256, 16)])
def test_padded_batch(T, d, E, groups, act):
    """Rows of zeros, of -0 and of the smallest numbers, and experts without weights: ties that the bias breaks, or the index."""
    rng = np.random.default_rng(T)
    x, wr = _draw(rng, T, d, E, act)
    x[rng.random(T) < 0.7] = 0
    x[T // 2] = -0.0
    if T > 2:
        x[1] = torch.finfo(x.dtype).smallest_normal
    wr[E // 3] = 0
    bias = np.where(rng.random(E) < 0.5, 0, 0.125 * rng.integers(-2, 3, E)).astype(np.float32)
    for sigmoid, b, sel in itertools.product((False, True), (None, bias), (None, bias)):
        _check(x, wr, b, 4, sel, "padded", sigmoid=sigmoid, groups=groups, group_topk=max(1, groups // 2), top2=True)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E", [(1, 8192, 16), (5, 8192, 30), (17, 2048, 64), (33, 1088, 100), (64, 832, 250), (1024, 4096, 64),
                                   (100, 576, 256)])
def test_with_and_without_a_workspace(T, d, E, act):
    """Rows split over workgroups or not, in a workspace of any contents: the same ids, and weights within their bounds."""
    rng = np.random.default_rng(T + d)
    x, wr = _draw(rng, T, d, E, act)
    x[T // 2] = 0
    select = (0.05 * rng.standard_normal(E)).astype(np.float32)
    kw = dict(sigmoid=True, groups=2 if E % 2 == 0 else 1, group_topk=1, top2=E % 2 == 0, scale=2.5)
    ids, w = _check(x, wr, None, 4, select, "split", **kw)
    g = _gate(select, **kw)
    a, b = m.moe_route_gated(x.cuda(), wr.cuda(), None, 4, g, use_workspace=False)
    assert torch.equal(a, ids) and torch.equal(b, w)
    ws = torch.full((16 << 20,), 255, dtype=torch.uint8, device="cuda")
    a, b = m.moe_route_gated(x.cuda(), wr.cuda(), None, 4, g, workspace=ws)
    assert torch.equal(a, ids) and torch.equal(b, w)


def test_streams_graphs_and_outputs():
    rng = np.random.default_rng(10)
    x, wr = _draw(rng, 300, 512, 64, "bf16")
    x, wr = x.cuda(), wr.cuda()
    g = _gate((0.05 * rng.standard_normal(64)).astype(np.float32), sigmoid=True, groups=8, group_topk=3, top2=True)
    ref = m.moe_route_gated(x, wr, None, 6, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = m.moe_route_gated(x, wr, None, 6, g)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, other))
    ids = torch.full((300, 6), 77, dtype=torch.int32, device="cuda")
    w = torch.full((300, 6), 7.0, device="cuda")
    src = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_route_gated(src, wr, None, 6, g, ids=ids, w=w)
    for i in range(3):
        src.copy_(x.roll(i, 0))
        graph.replay()
        torch.cuda.synchronize()
        want = m.moe_route_gated(x.roll(i, 0).contiguous(), wr, None, 6, g)
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
    # no token
    e = m.moe_route_gated(x[:0], wr, None, 6, g)
    assert e[0].shape == (0, 6) and e[1].shape == (0, 6)
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_route_gated(x.t()[:256].t(), wr[:, :256].contiguous(), None, 6, g)
    with pytest.raises(ValueError, match="shape"):
        m.moe_route_gated(x, wr[:, :256].contiguous(), None, 6, g)
    with pytest.raises(TypeError, match="dtype"):
        m.moe_route_gated(x, wr.float(), None, 6, g)
