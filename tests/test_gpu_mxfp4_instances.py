"""Every kernel instance that products with MXFP4 weights are launched as, at sizes that reach it.

Each case names the instance (the log's line has to say it was taken, so a rule that moves cannot drop it from here)
and compares every output with the formula in fp64, computed on the GPU expert by expert. The bounds are those of
tests/mx_helpers.py. Row counts leave every number of 16-row blocks in a last tile, an expert without rows and rows past
the last segment; reductions leave a partial scale group; channels leave a partial last tile where a tile allows it.
"""
import sys

import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd._lib import MOE_PATH_STREAM, MOE_PATH_TILED, MOE_W_MXFP4
from tests.test_gpu_mxfp4_limits import draw, values

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -23
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows(counts, K, gen):
    """(offsets, slots, S): a shuffled slot list over the segments' rows and at least one row past them."""
    last = sum(counts)
    S = last + 1 + -(last + 1) % K
    off = torch.tensor([0, *counts], device="cuda").cumsum(0).to(torch.int32)
    slots = torch.randperm(S, generator=gen, device="cuda").to(torch.int32)
    slots[last:] = -1
    return off, slots, S


def _check(got, a, rows, counts, mats, d, bf16, what):
    """got [S, N] against (W a) or silu(W a) (W2 a), a [., d] fp64, mats the row-major codes and scales."""
    r0 = 0
    for e, n in enumerate(counts):
        if n == 0:
            continue
        x = a[rows[r0:r0 + n].long()]
        p, mag = [], []
        for q, s in mats:
            w = values(q[e], s[e]).t().contiguous()
            p.append(x @ w)
            mag.append(x.abs() @ w.abs_())
            del w
        ref, bound = p[0], d * EPS * mag[0]
        if len(p) == 2:
            silu = p[0] / (1 + torch.exp(-p[0]))
            ref = silu * p[1]
            bound = (d * EPS * (1.1 * p[1].abs() * mag[0] + silu.abs() * mag[1])
                     + (8 + p[0].abs()) * 2 * EPS * ref.abs())
        if bf16:
            bound = bound + 2.0 ** -8 * (ref.abs() + bound)
        worst = ((got[r0:r0 + n].double() - ref).abs() - (bound + 1e-37)).max()
        assert worst <= 0, f"{what}: expert {e}, {worst.item():.3g} past the bound"
        r0 += n
    assert (got[r0:] == 7.0).all(), f"{what}: rows past the last segment were written"


def _say(msg):
    print(f"[mxfp4-instance] {msg}", file=sys.stderr, flush=True)


def _logged(capfd):
    lines = [l.split("; ", 1)[1] for l in capfd.readouterr().err.splitlines() if l.startswith("[moe] ")]
    return lines


class Case:
    """Weights and rows of one product; run(path, workspace) gives out over a buffer of sevens."""

    def __init__(self, kind, counts, N, d, out="f32", seed=0):
        self.kind, self.counts, self.N, self.d = kind, counts, N, d
        E = len(counts)
        gen = torch.Generator(device="cuda").manual_seed(seed + N + d)
        self.two = kind in ("gate_up", "product2")
        self.mx = kind.startswith("product")
        self.K = 1 if kind == "down" else 2
        self.off, self.slots, self.S = _rows(counts, self.K, gen)
        self.T = self.S // self.K
        self.mats = [draw((E, N), d, gen) for _ in range(2 if self.two else 1)]
        packed = [m.moe_pack_mxfp4(*w) for w in self.mats]
        self.out_dtype = DT[out] if self.mx else torch.bfloat16 if kind == "gate_up" else torch.float32
        self.rows = torch.arange(self.S, device="cuda") if kind == "down" else self.slots // self.K
        if self.mx:
            self.a = draw((self.T,), d, gen, 120, 130)
            self.a64 = values(*self.a)
            self.w = packed
        else:
            self.a = torch.randn(self.T, d, generator=gen, device="cuda").to(torch.bfloat16)
            self.a64 = self.a.double()
            none = torch.zeros(E, 0, 0, dtype=torch.uint8, device="cuda")
            if kind == "gate_up":
                (q0, s0), (q1, s1) = packed
                self.ex = m.Int8Experts(q0, q1, none, s0, s1, none, fmt=MOE_W_MXFP4)
            else:   # the sizes are those of the gate matrix: a view of E x d rows without memory of its own
                gate = torch.empty(1, dtype=torch.uint8, device="cuda").expand(E, d, N // 2)
                self.ex = m.Int8Experts(gate, none, packed[0][0], none, none, packed[0][1], fmt=MOE_W_MXFP4)

    def run(self, path, workspace=True):
        out = torch.full((self.S, self.N), 7.0, dtype=self.out_dtype, device="cuda")
        if self.mx:
            w2 = dict(w2_q=self.w[1][0], w2_s=self.w[1][1]) if self.two else {}
            return m.moe_grouped_mm_mxfp4(*self.a, self.off, *self.w[0], self.out_dtype, sorted_slots=self.slots, K=self.K,
                                          path=path, out=out, **w2)
        if self.two:
            return m.moe_expert_gate_up(self.a, self.off, self.slots, self.ex, self.K, path=path, h=out,
                                        use_workspace=workspace)
        return m.moe_expert_down(self.a, self.off, self.ex, self.T, 1, path=path, y_rows=out, split_workspace=workspace)

    def check(self, got, what):
        _check(got, self.a64, self.rows, self.counts, self.mats, self.d, self.out_dtype == torch.bfloat16, what)


def _run(capfd, monkeypatch, case, path, instance):
    _say(f"{case.kind} counts {case.counts} channels {case.N} reduction {case.d}: {instance}")
    monkeypatch.setenv("MOE_LOG", "1")
    capfd.readouterr()
    got = case.run(path)
    lines = _logged(capfd)
    monkeypatch.delenv("MOE_LOG")
    assert lines == [instance]
    case.check(got, instance)
    return got


# ------------------------------------------------------------------ streaming kernel

# up to eight rows an expert on average (one expert has more than a pass of 16), and more than eight
COUNTS = {16: [17, 0, 1, 5], 32: [35, 0, 1, 15]}
# reduction for a number of slices while the items are few: 1, 2, 5 and 9 scale groups, the last one partial
FEW = {1: 384, 2: 896, 4: 2176, 8: 4224}
# (kind, channels of an item) -> {slices: (channels, reduction)}; four experts
STREAM = {
    ("gate_up", 16): {ks: (128, d) for ks, d in FEW.items()},
    ("gate_up", 32): {1: (8320, 384), 2: (8320, 3712), 4: (12416, 7808)},
    ("down", 16): {ks: (128, d) for ks, d in FEW.items()},
    ("down", 32): {ks: (2176, d) for ks, d in FEW.items()},
    ("down", 64): {1: (16512, 384), 2: (16512, 3712), 4: (24704, 7808)},
    ("product", 16): {ks: (128, d) for ks, d in FEW.items()},
    ("product", 32): {1: (32896, 384), 2: (32896, 3712)},
    ("product2", 16): {ks: (128, d) for ks, d in FEW.items()},
}


def _stream_cases():
    for (kind, width), by_slices in STREAM.items():
        for ks, (N, d) in by_slices.items():
            for rows in COUNTS:
                for out in ("bf16", "f32") if kind.startswith("product") else ("",):
                    yield pytest.param(kind, width, rows, ks, N, d, out, id=f"{kind}-{width}ch-{rows}rows-{ks}slices{out}")


@pytest.mark.parametrize("kind,width,rows,slices,N,d,out", _stream_cases())
def test_stream(capfd, monkeypatch, kind, width, rows, slices, N, d, out):
    case = Case(kind, COUNTS[rows], N, d, out)
    _run(capfd, monkeypatch, case, MOE_PATH_STREAM,
         f"stream schedule, {width}-channel items, {rows}-row passes, reduction in {slices} slices")


# ------------------------------------------------------------------ tiled kernel

# last tiles of every class of row blocks, with 128-row tiles and with 64-row ones
MID, SMALL = [257, 0, 43, 90], [64, 0, 65, 1]
MANY = [1100, 0, 700, 301]
STATIC, CLAIMED = "static tile order", "the last tiles of each XCD queue claimed"
TILED = [
    # kind, tile, counts, channels, reduction
    ("gate_up", "64x128", [130, 0, 43, 90], 256, 640),
    ("gate_up", "64x256", [130, 0, 43, 90], 8576, 384),
    ("gate_up", "128x256", [400, 0, 143, 190], 384, 640),
    ("down", "64x128", SMALL, 384, 640),
    ("down", "64x256", SMALL, 32640, 384),             # 32640 = 127 * 256 + 128
    ("down", "128x128", [130, 0, 43, 90], 384, 640),
    ("down", "128x256", [130, 0, 43, 90], 32640, 384),
    ("down", "128x256", MANY, 384, 640),
    ("product", "128x128", MID, 384, 640),
    ("product", "128x256", MID, 32640, 384),
    ("product", "128x256", MID, 32640, 1024),
    ("product2", "128x128", MID, 384, 640),
    ("product2", "128x256", MID, 16384, 384),
    ("product2", "128x256", MID, 16384, 1152),
]


def _tiled_cases():
    for kind, tile, counts, N, d in TILED:
        for out in ("bf16", "f32") if kind.startswith("product") else ("",):
            yield pytest.param(kind, tile, counts, N, d, out, id=f"{kind}-{tile}-{sum(counts)}-{N}-{d}{out}")


@pytest.mark.parametrize("kind,tile,counts,N,d,out", _tiled_cases())
def test_tiled(capfd, monkeypatch, kind, tile, counts, N, d, out):
    case = Case(kind, counts, N, d, out)
    _run(capfd, monkeypatch, case, MOE_PATH_TILED, f"tiled schedule, {tile} tiles, {STATIC}")


# claimed tails: at least 2048 tiles, four row tiles an expert and a reduction of 2048
CLAIMS = [
    ("gate_up", "128x256", MANY, 12544, 2176),
    ("down", "64x256", [500, 0, 300, 301], 23936, 2176),
    ("down", "128x256", MANY, 24960, 2176),
]


@pytest.mark.parametrize("kind,tile,counts,N,d", CLAIMS)
def test_claimed_tail(capfd, monkeypatch, kind, tile, counts, N, d):
    """The claimed order gives the static order's bits, and again when a captured call is replayed."""
    case = Case(kind, counts, N, d)
    got = _run(capfd, monkeypatch, case, MOE_PATH_TILED, f"tiled schedule, {tile} tiles, {CLAIMED}")
    assert torch.equal(case.run(MOE_PATH_TILED, workspace=False), got)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = case.run(MOE_PATH_TILED)
    for i in range(3):
        case.a.copy_(torch.randn(case.T, d, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(case.run(MOE_PATH_TILED, workspace=False), out), i


def test_claimed_tail_with_one_crowded_expert():
    """All rows in one expert of four: the tile count's bound is loose, most queues' ends are empty."""
    case = Case("down", [0, 0, 2100, 0], 24960, 2176)
    got = case.run(MOE_PATH_TILED)
    case.check(got, "crowded")
    assert torch.equal(case.run(MOE_PATH_TILED, workspace=False), got)


# ------------------------------------------------------------------ the borders between the schedules

def _schedules(capfd, monkeypatch, call):
    monkeypatch.setenv("MOE_LOG", "1")
    capfd.readouterr()
    r = call()
    names = [l.split(" schedule")[0] for l in _logged(capfd)]
    monkeypatch.delenv("MOE_LOG")
    return r, names


# (experts, width of d and f): 16384 output channels over all experts, and 18432. Per call the rows an expert on both
# sides of each border, with the schedules of the gate/up and the down pass. 4-bit activations: both borders are one.
FEW_CHANNELS, MORE_CHANNELS = (8, 2048), (16, 1152)
BORDERS = [
    (FEW_CHANNELS, 20, "stream stream", "stream stream"), (FEW_CHANNELS, 21, "tiled stream", "tiled tiled"),
    (FEW_CHANNELS, 32, "tiled stream", "tiled tiled"), (FEW_CHANNELS, 33, "tiled tiled", "tiled tiled"),
    (MORE_CHANNELS, 8, "stream stream", "stream stream"), (MORE_CHANNELS, 9, "tiled stream", "tiled tiled"),
    (MORE_CHANNELS, 16, "tiled stream", "tiled tiled"), (MORE_CHANNELS, 17, "tiled tiled", "tiled tiled"),
]


@pytest.mark.parametrize("size,rows,bf16,mx", BORDERS)
def test_borders_of_the_schedules(capfd, monkeypatch, size, rows, bf16, mx):
    """AUTO on both sides of each border: the schedules taken, the numbers, and the layer made of the same passes.

    Between the borders the gate/up pass is tiled with a workspace that is laid out for a streamed down pass.
    """
    E, n = size
    gen = torch.Generator(device="cuda").manual_seed(rows)
    S = rows * E if rows % 4 == 0 else (rows - 1) * E + 1         # a border is full, or passed by one row
    x = torch.randn(S, n, generator=gen, device="cuda").to(torch.bfloat16)
    wr = (torch.randn(E, n, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    mats = [draw((E, n), n, gen, 116, 121) for _ in range(3)]
    ex = m.pack_mxfp4_experts(*(q for q, _ in mats), *(s for _, s in mats))
    (y, ids, gw), names = _schedules(capfd, monkeypatch, lambda: m.moe_forward(x, wr, None, ex, 1))
    assert " ".join(names) == bf16
    off, slots, s2r = m.moe_permute(ids, E)
    counts = (off[1:] - off[:-1]).tolist()
    y_rows, names = _schedules(capfd, monkeypatch, lambda: m.moe_expert_ffn(x, off, slots, ex, 1))
    assert " ".join(names) == bf16
    assert torch.equal(m.moe_combine(y_rows, s2r, gw, torch.bfloat16), y)
    h = m.moe_expert_gate_up(x, off, slots, ex, 1)
    assert torch.equal(m.moe_expert_down(h, off, ex, S, 1), y_rows)
    _check(h, x.double(), slots, counts, mats[:2], n, True, "gate/up")
    _check(y_rows, h.double(), torch.arange(S, device="cuda"), counts, mats[2:], n, False, "down")
    # with 4-bit activations
    y_rows, names = _schedules(capfd, monkeypatch, lambda: m.moe_expert_ffn_mxfp4(x, off, slots, ex, 1))
    assert " ".join(names) == mx
    hq, hs = m.moe_quantize_mxfp4(m.moe_grouped_mm_mxfp4(*m.moe_quantize_mxfp4(x), off, ex.q_gate, ex.s_gate, torch.bfloat16,
                                                         sorted_slots=slots, w2_q=ex.q_up, w2_s=ex.s_up))
    _check(y_rows, values(hq, hs), torch.arange(S, device="cuda"), counts, mats[2:], n, False, "4-bit down")
