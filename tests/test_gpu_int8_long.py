"""Int8 products whose rows pass 4 GiB: which schedule they take, and their values on both sides of the border."""
import sys

import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd._lib import MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_TILED
from tests.test_gpu_gate_int8_limits import _case, _want

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[int8-long-test] {msg}", file=sys.stderr, flush=True)


def _line(capfd, what):
    lines = [l for l in capfd.readouterr().err.splitlines() if l.startswith("[moe]") and what in l]
    assert len(lines) == 1, lines
    return lines[0]


# 65536 rows of 65536 codes are 4 GiB. Rows as they are: tiles at any size; gathered ones: streamed past 4 GiB.
@pytest.mark.parametrize("rows,gather,path,words", [
    (65535, True, MOE_PATH_AUTO, "tiled schedule"), (65536, False, MOE_PATH_AUTO, "tiled schedule"),
    (66001, False, MOE_PATH_AUTO, "tiled schedule"), (66001, False, MOE_PATH_TILED, "tiled schedule"),
    (66001, False, MOE_PATH_STREAM, "stream schedule"), (65536, True, MOE_PATH_AUTO, "stream schedule"),
    (66001, True, MOE_PATH_TILED, "stream schedule"),
])
@pytest.mark.parametrize("swiglu", [False, True])
def test_rows_past_4_gib(rows, gather, path, words, swiglu, monkeypatch, capfd):
    _say(f"rows={rows} gather={gather} path={path} swiglu={swiglu}")
    E, d, f = 3, 65536, 64
    a, a_s, w, w_s = _case(rows, E, d, f, rows)
    # the last segment starts below 4 GiB and ends past it; five rows behind it
    ends = [0, 1000, 65530, rows - 5] if rows > 65540 else [0, 1000, 40000, rows - 5]
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    slots = None
    if gather:                                           # from the last row to the first
        slots = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda")
    out = torch.full((rows, f), -5.0, device="cuda")
    packed = m.moe_pack_rows(w)
    monkeypatch.setenv("MOE_LOG", "1")
    m.moe_grouped_mm_int8(a, a_s, off, packed, w_s, torch.float32, sorted_slots=slots, K=1, path=path, out=out,
                          w2_q=packed if swiglu else None, w2_s=w_s if swiglu else None)
    torch.cuda.synchronize()
    assert words in _line(capfd, "product")
    assert (out[rows - 5:] == -5).all()
    channels = torch.arange(f, device="cuda")
    for e in range(E):
        for r in sorted({ends[e], ends[e] + 127, ends[e] + 128, ends[e + 1] - 1, 65534, 65535, 65536, 65537}):
            if not ends[e] <= r < ends[e + 1]:
                continue
            src = rows - 1 - r if gather else r
            p = _want(a, a_s, w, w_s, src, e, channels)
            if not swiglu:
                assert torch.equal(out[r], p), (e, r)
                continue
            p = p.double()                               # p is the kernel's own, bit for bit: silu and the product remain
            ref = p * torch.sigmoid(p) * p
            # below p = -88.7 exp(-p) passes fp32 and silu(p) is taken as 0: it is 88.73 * exp(-88.72) = 2.7e-37 at most there
            assert ((out[r] - ref).abs() <= 15 * 2.0 ** -24 * ref.abs() + 2.7e-37 * p.abs() + 1e-37).all(), (e, r)


def test_a_layers_h_past_4_gib(monkeypatch, capfd):
    """The expert FFN's down product of a long prompt takes tiles, as its gate/up does."""
    T, d, f, E, K = 33000, 64, 65536, 4, 2
    _say("expert FFN")
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s, k: (torch.randn(*s, generator=gen, device="cuda") * k).to(torch.bfloat16)
    ex = m.quantize_experts(n(E, f, d, k=0.1), n(E, f, d, k=0.1), n(E, d, f, k=0.01), torch.bfloat16)
    x, wr = n(T, d, k=1.0), n(E, d, k=0.1)
    ids, _ = m.moe_route_gated(x, wr, None, K, m.Gate())
    off, slots, s2r = m.moe_permute(ids, E)
    monkeypatch.setenv("MOE_LOG", "1")
    y = m.moe_expert_ffn_int8(x, off, slots, ex, K)
    torch.cuda.synchronize()
    assert "tiled schedule" in _line(capfd, "down")
    # few tokens at a time: rows far below 4 GiB, the same bits
    s2r = s2r.view(T, K).long()
    for t0 in (0, 16000, T - 300):
        i = ids[t0:t0 + 300].contiguous()
        o, s, r = m.moe_permute(i, E)
        part = m.moe_expert_ffn_int8(x[t0:t0 + 300].contiguous(), o, s, ex, K)
        assert torch.equal(part[r.view(-1).long()], y[s2r[t0:t0 + 300].reshape(-1)])
