"""Slots that are not placed: the rows behind the last segment."""
import sys

import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd._lib import MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_TILED
from tests.test_gpu_forward_gated import _case

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
