"""MXFP4 calls at the ends of their ranges, on the GPU."""
import pytest
import torch

import int8_weight_moe_amd as m

pytestmark = pytest.mark.gpu

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def values(q, s):
    """fp64 numbers of row-major codes and scale bytes, on their device."""
    grid = torch.tensor([*GRID, *(-v for v in GRID)], dtype=torch.float64, device=q.device)
    v = torch.stack([grid[(q & 15).long()], grid[(q >> 4).long()]], -1).flatten(-2)
    scale = torch.exp2(s.double() - 127)                       # powers of two: exact
    return v * scale.repeat_interleave(32, dim=-1)


def draw(rows, cols, gen, lo=118, hi=124):
    """Random codes, and scales worth 2^-9 .. 2^-4."""
    q = torch.randint(0, 256, (*rows, cols // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s = torch.randint(lo, hi, (*rows, cols // 32), generator=gen, device="cuda", dtype=torch.uint8)
    return q, s


def test_down_rows_past_4_gib():
    """h of 6 GiB: the down pass streams (gate/up, whose x is 8 MiB, stays tiled), rows at both ends of h checked.

    Bound: exact products, fp32 sums of f terms: f * 2^-23 of the sum of magnitudes; and for gate/up that of
    tests/mx_helpers.py with its bf16 rounding.
    """
    T, d, f, E, K = 16384, 256, 24576, 64, 8
    S = T * K
    gen = torch.Generator(device="cuda").manual_seed(1)
    mats = {k: draw((E, r), c, gen) for k, (r, c) in dict(gate=(f, d), up=(f, d), down=(d, f)).items()}
    ex = m.pack_mxfp4_experts(*(mats[k][0] for k in ("gate", "up", "down")), *(mats[k][1] for k in ("gate", "up", "down")))
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * (S // E)
    slots = torch.randperm(S, generator=gen, device="cuda").to(torch.int32)
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    h = m.moe_expert_gate_up(x, off, slots, ex, K)
    assert h.numel() * 2 > 1 << 32
    y = m.moe_expert_down(h, off, ex, T, K)
    per = S // E
    for e in (0, 1, E // 2, E - 1):
        W = {k: values(q[e], s[e]) for k, (q, s) in mats.items()}
        for rows in (slice(e * per, e * per + 40), slice((e + 1) * per - 40, (e + 1) * per)):
            a = x[(slots[rows] // K).long()].double()
            g, u = a @ W["gate"].t().contiguous(), a @ W["up"].t().contiguous()
            mg, mu = a.abs() @ W["gate"].abs().t().contiguous(), a.abs() @ W["up"].abs().t().contiguous()
            eps, silu = 2.0 ** -23, g / (1 + torch.exp(-g))
            ref = silu * u
            bound = d * eps * (1.1 * u.abs() * mg + silu.abs() * mu) + (8 + g.abs()) * 2 * eps * ref.abs()
            bound = bound + 2.0 ** -8 * (ref.abs() + bound) + 1e-37
            assert ((h[rows].double() - ref).abs() <= bound).all(), e
            a = h[rows].double()
            ref, mag = a @ W["down"].t().contiguous(), a.abs() @ W["down"].abs().t().contiguous()
            assert ((y[rows].double() - ref).abs() <= f * eps * mag + 1e-37).all(), e


def test_past_4_gib_schedules_in_the_log(monkeypatch, capfd):
    monkeypatch.setenv("MOE_LOG", "1")
    T, d, f, E, K = 16384, 256, 24576, 64, 8
    ex = m.Int8Experts(*(torch.zeros(E, r, c // 2, dtype=torch.uint8, device="cuda") for r, c in ((f, d), (f, d), (d, f))),
                       *(torch.full((E, r, c // 32), 127, dtype=torch.uint8, device="cuda") for r, c in ((f, d), (f, d), (d, f))),
                       fmt=m.MOE_W_MXFP4)
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * (T * K // E)
    slots = torch.arange(T * K, device="cuda", dtype=torch.int32)
    y = m.moe_expert_ffn(torch.ones(T, d, dtype=torch.bfloat16, device="cuda"), off, slots, ex, K)
    lines = [l for l in capfd.readouterr().err.splitlines() if l.startswith("[moe] moe_expert_ffn")]
    assert "; tiled schedule" in lines[0] and "; stream schedule" in lines[1], lines
    assert (y == 0).all()


def test_norm_outputs_in_place_of_an_input():
    """next may take residual's or y's memory, out the other's: the bits of separate outputs."""
    for dt, d in ((torch.bfloat16, 4096), (torch.float32, 320)):
        g = torch.Generator(device="cuda").manual_seed(d)
        y, res = (torch.randn(70, d, generator=g, device="cuda").to(dt) for _ in range(2))
        w = torch.ones(d, dtype=dt, device="cuda")
        out, nxt = m.moe_norm_post(y, res, weight=w, next_weight=w)
        for swap in (False, True):
            a, b = y.clone(), res.clone()
            o2, n2 = m.moe_norm_post(a, b, weight=w, next_weight=w, out=a if swap else b, next_out=b if swap else a)
            assert torch.equal(o2, out) and torch.equal(n2, nxt)
        with pytest.raises(m.MoeError) as e:
            m.moe_norm_post(y, res, weight=w, next_weight=w, out=out, next_out=out)
        assert e.value.status == 6
