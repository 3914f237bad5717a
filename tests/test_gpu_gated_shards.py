"""Slots that are not placed: a shard of the routed experts, ids of -1, and the rows behind the last segment."""
import sys

import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd._lib import MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_TILED
from oracle import gate as ogate
from oracle import int8 as oint8
from oracle import quant as oquant
from tests.helpers import np64
from tests.test_gpu_forward_gated import _case, _staged

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[shard-test] {msg}", file=sys.stderr, flush=True)


def _r(v):
    return (v + 255) // 256 * 256


@pytest.mark.parametrize("path", [MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_TILED])
@pytest.mark.parametrize("T,d,f,E,K", [(40, 128, 192, 8, 2), (300, 256, 128, 16, 4), (700, 192, 320, 4, 2)])
def test_rows_behind_the_last_segment_are_not_quantized(T, d, f, E, K, path):
    """The expert FFN of a shard writes what its own rows take of the workspace and of the output, and nothing else."""
    x, wr, ex, _, _ = _case(T, d, f, E)
    ids, _ = m.moe_route_gated(x, wr, None, K, m.Gate())
    full = m.moe_expert_ffn_int8(x, *m.moe_permute(ids, E)[:2], ex, K, path=path)
    ids[torch.arange(T, device="cuda") % 4 != 1] = -1        # a quarter of the slots are placed
    off, slots, s2r = m.moe_permute(ids, E)
    rows = int(off[-1])
    assert 0 < rows < T * K // 3
    S = T * K
    # x's codes and scales, h's codes, h's scales, h: each from a multiple of 256 bytes
    sizes = [(T * d, T * d), (T * 4, T * 4), (S * f, rows * f), (S * 4, rows * 4), (S * f * 2, rows * f * 2)]
    ws = torch.full((sum(_r(n) for n, _ in sizes),), 0xAB, dtype=torch.uint8, device="cuda")
    _say(f"T={T} d={d} f={f} E={E} K={K} path={path} rows={rows}")
    y = m.moe_expert_ffn_int8(x, off, slots, ex, K, path=path, workspace=ws)
    at = 0
    for n, used in sizes:
        assert (ws[at + used:at + n] == 0xAB).all(), f"bytes {at + used} to {at + n} of the workspace"
        assert not (ws[at:at + used] == 0xAB).all()
        at += _r(n)
    # the placed slots' rows are those of the whole call
    ids2, _ = m.moe_route_gated(x, wr, None, K, m.Gate())
    whole = m.moe_permute(ids2, E)[2].view(-1).long()
    mine = s2r.view(-1).long()
    placed = mine >= 0
    assert torch.equal(y[mine[placed]], full[whole[placed]])


@pytest.mark.parametrize("act_int8", [False, True])
@pytest.mark.parametrize("T", [1, 33, 400])
def test_a_block_with_slots_of_no_expert(T, act_int8):
    """Too few experts in service: the block is its staged calls, and a token's missing expert adds nothing."""
    E, K, d = 8, 3, 256
    x, wr, ex, b, _ = _case(T, d, 192, E, disabled=E - K + 1)
    v = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    g = m.Gate(select_bias=b, score=m.MOE_SCORE_SIGMOID, scale=1.5)
    out, nxt, ids, w = m.moe_block_forward_gated(x, wr, None, ex, K, g, act_int8, pre_weight=v, weight=v, next_weight=v)
    assert (ids[:, K - 1] == -1).all() and (w[:, K - 1] == 0).all() and (ids[:, :K - 1] >= 0).all()
    n = m.moe_norm_pre(x, v)
    _, rid, rw, rows, s2r, off, _ = _staged(n, wr, None, ex, K, g, act_int8, MOE_PATH_AUTO)
    assert int(off[-1]) == T * (K - 1)
    ro, rn = m.moe_combine_post(rows, s2r, rw, x, weight=v, next_weight=v)
    assert torch.equal(ids, rid) and torch.equal(w, rw) and torch.equal(out, ro) and torch.equal(nxt, rn)
    assert torch.isfinite(out).all()
    # with none in service the layer adds nothing: the norm of zeros
    b[:] = -float("inf")
    out, _, ids, w = m.moe_block_forward_gated(x, wr, None, ex, K, g, act_int8, pre_weight=v, weight=v)
    assert (ids == -1).all() and (w == 0).all() and torch.equal(out, x)


@pytest.mark.parametrize("T", [5, 130])
def test_256_experts_in_eight_shards(T):
    """Routing by 256 experts, then each shard of 32 permutes ids less its first expert, runs its FFN and combines; the shards'
    parts add up to the layer. Some slots have no expert at all."""
    E, n, K, d, f = 256, 32, 8, 128, 64
    u = 2.0 ** -24
    rng = np.random.default_rng(T)
    t = lambda *s, k=1.0: torch.from_numpy((k * rng.standard_normal(s)).astype(np.float32)).to(torch.bfloat16).cuda()
    x, wr = t(T, d), t(E, d, k=0.05)
    w = [t(E, f, d, k=0.05), t(E, f, d, k=0.05), t(E, d, f, k=0.05)]
    b = (0.05 * rng.standard_normal(E)).astype(np.float32)
    live = rng.permutation(E)[:6 if T == 5 else 200]
    b[np.setdiff1d(np.arange(E), live)] = -np.inf
    g = m.Gate(score=m.MOE_SCORE_SIGMOID, select_bias=torch.from_numpy(b).cuda(), scale=2.5)
    ids, tw = m.moe_route_gated(x, wr, None, K, g)
    rid, rw, _ = ogate.route(np64(x), np64(wr), None, K, True, select_bias=b, scale=2.5)
    assert np.array_equal(ids.cpu().numpy(), rid) and ((rid < 0).any() == (T == 5))
    xq, xs = oquant.quantize_rows(np64(x), "f32")
    codes = [oquant.quantize_rows(np64(v), "bf16") for v in w]
    for act_int8 in (False, True):
        total, seen = np.zeros((T, d)), 0
        for s in range(E // n):
            first = s * n
            ex = m.quantize_experts(*(v[first:first + n].contiguous() for v in w), torch.bfloat16)
            off, slots, s2r = m.moe_permute(ids - first, n)
            mine = (rid >= first) & (rid < first + n)
            rows, count = slots.cpu().numpy(), int(off[-1])
            assert count == mine.sum() and set(rows[:count]) == set(np.flatnonzero(mine.reshape(-1)))
            assert np.array_equal((s2r.cpu().numpy().reshape(T, K) >= 0), mine)
            ffn = m.moe_expert_ffn_int8 if act_int8 else m.moe_expert_ffn
            y_rows = ffn(x, off, slots, ex, K)
            ro, src = off.cpu().numpy(), rows[:count] // K
            c = [(q[first:first + n], sc[first:first + n]) for q, sc in codes]
            if act_int8 and count:
                gq, gs = m.moe_quantize_rows(x, torch.float32)
                h = m.moe_grouped_mm_int8(gq, gs, off, ex.q_gate, ex.s_gate, torch.bfloat16, sorted_slots=slots, K=K,
                                          w2_q=ex.q_up, w2_s=ex.s_up)
                hq, hs = oquant.quantize_rows(np64(h[:count]), "f32")
                ref = oint8.grouped_product(hq, hs, c[2][0], c[2][1], ro, np.arange(count))
                assert (np.abs(np64(y_rows)[:count] - ref) <= 3.01 * u * np.abs(ref) + 1e-37).all()
                p = oint8.grouped_product(xq, xs, c[0][0], c[0][1], ro, src, c[1][0], c[1][1])
                assert np.abs(np64(h)[:count] - p).max() <= 2.0 ** -7 * np.abs(p).max()
            y = m.moe_combine(y_rows, s2r, tw, torch.float32)
            assert (y[torch.from_numpy(~mine.any(1)).cuda()] == 0).all()
            total += np64(y)
            seen += count
        assert seen == (rid >= 0).sum()
        # the whole layer from the definition, in fp64 with dequantized weights
        deq = [q.astype(np.float64) * sc.astype(np.float64)[..., None] for q, sc in codes]
        ref = np.zeros((T, d))
        x64 = np64(x)
        for i, k in np.argwhere(rid >= 0):
            e = rid[i, k]
            a = deq[0][e] @ x64[i]
            ref[i] += rw[i, k] * (deq[2][e] @ (a / (1 + np.exp(-a)) * (deq[1][e] @ x64[i])))
        # bf16 activations: the layer's own tolerance; int8 ones round x and h to 1/254 of their largest element
        err = np.abs(total - ref).max()
        assert err <= (4e-2 if act_int8 else 1e-2) * np.abs(ref).max() + 1e-3, err
