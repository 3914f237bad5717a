"""Int8 products and gated routing at the far end: rows, weights and outputs past 32-bit byte offsets, the widest shapes,
two calls at once. Sampled rows and channels, exact where the product is (an int32 sum, to fp32, times two scales)."""
import sys

import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd._lib import MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_TILED
from oracle import gate as ogate
from tests.helpers import np64

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[limits-test] {msg}", file=sys.stderr, flush=True)


def _codes(gen, *shape):
    return torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=gen)


def _case(rows, E, d, f, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    a, w = _codes(gen, rows, d), _codes(gen, E, f, d)
    return a, torch.rand(rows, device="cuda", generator=gen) + 0.5, w, torch.rand(E, f, device="cuda", generator=gen) * 1e-3


def _want(a, a_s, w, w_s, row, e, channels):
    """The sampled channels of a row, from the definition: sum in int64, then fp32 roundings in the stated order."""
    total = (w[e, channels].to(torch.int64) * a[row].to(torch.int64)).sum(1)
    assert total.abs().max() < 2 ** 31
    return total.float() * w_s[e, channels] * a_s[row]


@pytest.mark.parametrize("rows,E,d,f,path,what", [
    (70000, 2, 65536, 64, MOE_PATH_AUTO, "rows of codes past 4 GiB"),
    (70000, 2, 65536, 64, MOE_PATH_TILED, "rows of codes past 4 GiB"),
    (40000, 3, 64, 32768, MOE_PATH_AUTO, "an output past 4 GiB"),
    (40000, 3, 64, 32768, MOE_PATH_STREAM, "an output past 4 GiB"),
    (200, 3, 65536, 32768, MOE_PATH_TILED, "weights past 4 GiB"),
    (40, 3, 65536, 32768, MOE_PATH_STREAM, "weights past 4 GiB"),
    (20, 2, 64, 131072, MOE_PATH_AUTO, "the most channels"),
    (300, 64, 64, 64, MOE_PATH_AUTO, "the most experts"),
])
def test_far_ends(rows, E, d, f, path, what):
    _say(f"{what}: rows={rows} E={E} d={d} f={f} path={path}")
    a, a_s, w, w_s = _case(rows, E, d, f, rows + f)
    counts = [(rows - 7) // E] * (E - 1)
    counts.append(rows - 7 - sum(counts))                # seven rows behind the last segment
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    out = torch.full((rows, f), -5.0, device="cuda")
    m.moe_grouped_mm_int8(a, a_s, off, m.moe_pack_rows(w), w_s, torch.float32, path=path, out=out)
    assert (out[rows - 7:] == -5).all()
    channels = torch.tensor(sorted({0, 1, 15, 16, f // 2, f - 17, f - 1}), device="cuda")
    lo = 0
    for e, n in enumerate(counts):
        for row in sorted({lo, lo + n // 2, lo + n - 1}) if n else []:
            assert torch.equal(out[row, channels], _want(a, a_s, w, w_s, row, e, channels)), (e, row)
        lo += n


@pytest.mark.parametrize("T,d,E", [(40000, 65536, 16), (40000, 65536, 200), (1, 65536, 256), (1024, 65536, 256)])
def test_long_rows_are_routed(T, d, E):
    _say(f"T={T} d={d} E={E}")
    gen = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    wr = torch.empty(E, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) * 0.01
    bias = torch.rand(E, device="cuda", generator=gen) * 0.1
    gate = m.Gate(score=m.MOE_SCORE_SIGMOID, select_bias=bias, groups=4, group_topk=2, group_by=m.MOE_GROUP_TOP2, scale=2.0)
    ids, w = m.moe_route_gated(x, wr, None, 4, gate)
    at = sorted({0, T // 2, T - 1})
    rid, rw, _ = ogate.route(np64(x[at]), np64(wr), None, 4, True, select_bias=bias.cpu().numpy(), groups=4, group_topk=2,
                             top2=True, scale=2.0)
    assert np.array_equal(ids[at].cpu().numpy(), rid)
    # a logit's error: 6 units of 2^-23 of |x| |w| (the kernel's bound); a weight follows its score, s (1 - s) <= s of it each,
    # in numerator and sum, then one rounding
    mag = np.linalg.norm(np64(x[at]), axis=1).max() * np.linalg.norm(np64(wr), axis=1).max()
    assert (np.abs(np64(w[at]) - rw) <= (2.1 * 6 * 2.0 ** -23 * mag + 2.0 ** -23) * rw).all()


def test_two_calls_at_once():
    """Products and routing of two batches on two streams, each with its own memory, over and over."""
    T, d, f, E = 200, 8192, 512, 8
    a, a_s, w, w_s = _case(T, E, d, f, 1)
    q = m.moe_pack_rows(w)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = [torch.empty(n, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for n in (3, 70)]
    wr = torch.empty(E, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) * 0.02
    off = [torch.arange(E + 1, dtype=torch.int32, device="cuda") * n for n in (2, 25)]
    size = lambda t: torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    ws = [size(t) for t in x]

    def run(i, out=None, ids=None, wt=None):
        rows = (16, T)[i]
        out = m.moe_grouped_mm_int8(a[:rows], a_s[:rows], off[i], q, w_s, torch.bfloat16, w2_q=q, w2_s=w_s, out=out)
        ids, wt = m.moe_route_gated(x[i], wr, None, 2, m.Gate(), ids=ids, w=wt, workspace=ws[i])
        return out, ids, wt

    want = [run(0), run(1)]
    got = [[torch.zeros_like(t) for t in v] for v in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                run(i, *got[i])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for g, v in zip(got, want) for p, q in zip(g, v))


def test_the_same_row_many_times():
    """sorted_slots of one token's K slots: every expert reads the same row."""
    K, E, d, f = 8, 8, 320, 192
    a, a_s, w, w_s = _case(1, E, d, f, 3)
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([5, 1, 7, 0, 2, 6, 4, 3], dtype=torch.int32, device="cuda")
    for path in (MOE_PATH_STREAM, MOE_PATH_TILED):
        out = m.moe_grouped_mm_int8(a, a_s, off, m.moe_pack_rows(w), w_s, torch.float32, sorted_slots=slots, K=K, path=path)
        for e in range(E):
            assert torch.equal(out[e], _want(a, a_s, w, w_s, 0, e, torch.arange(f, device="cuda")))
