"""The binding's checks of the MXFP4 and block calls (CPU: each call is refused before it reaches the library)."""
import dataclasses
import os
import subprocess
import sys

import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd import ops
from int8_weight_moe_amd import MOE_W_BF16, MOE_W_FP8, MOE_W_INT8, MOE_W_MXFP4, Int8Experts

E, F, D = 3, 256, 128


def _experts(fmt):
    z = lambda dt, *shape: torch.zeros(*shape, dtype=dt)
    dims = dict(gate=(F, D), up=(F, D), down=(D, F))
    if fmt == MOE_W_MXFP4:
        t = {"q_" + k: z(torch.uint8, E, r, c // 2) for k, (r, c) in dims.items()}
        t.update({"s_" + k: z(torch.uint8, E, r, c // 32) for k, (r, c) in dims.items()})
    else:
        code = {MOE_W_INT8: torch.int8, MOE_W_FP8: torch.uint8, MOE_W_BF16: torch.bfloat16}[fmt]
        t = {"q_" + k: z(code, E, r, c) for k, (r, c) in dims.items()}
        t.update({"s_" + k: None if fmt == MOE_W_BF16 else z(torch.bfloat16, E, r) for k, (r, c) in dims.items()})
    return Int8Experts(**t, fmt=fmt)


def _calls(ex):
    x = torch.zeros(4, D, dtype=torch.bfloat16)
    off, srt = torch.zeros(E + 1, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    wr = torch.zeros(E, D, dtype=torch.bfloat16)
    yield lambda: m.moe_block_forward(x, wr, None, ex, 2, pre_weight=x[0])
    if ex.fmt != MOE_W_MXFP4:
        return
    yield lambda: m.moe_expert_ffn_mxfp4(x, off, srt, ex, 2)
    yield lambda: m.moe_expert_ffn(x, off, srt, ex, 2)
    yield lambda: m.moe_forward(x, wr, None, ex, 2)
    yield lambda: m.moe_forward_noalloc(x, wr, None, ex, 2)


@pytest.mark.parametrize("fmt", [MOE_W_INT8, MOE_W_FP8, MOE_W_BF16, MOE_W_MXFP4])
def test_expert_tensors_are_checked_against_each_other(fmt):
    """One tensor too short, or of another type, is named before any pointer is taken (here: before the device check)."""
    good = _experts(fmt)
    names = ["q_up", "q_down"] + ([] if fmt == MOE_W_BF16 else ["s_up", "s_down"])
    for name in names:
        t = getattr(good, name)
        for bad in (t[:, :-16].contiguous(), t[:-1].contiguous(), t.to(torch.float32), None):
            for call in _calls(dataclasses.replace(good, **{name: bad})):
                with pytest.raises(ValueError, match=f"the experts' {name} is"):
                    call()
    for call in _calls(good):
        with pytest.raises(ValueError, match="not on the current HIP device"):
            call()


def test_staged_passes_check_the_matrices_they_read():
    ex = _experts(MOE_W_MXFP4)
    x = torch.zeros(4, D, dtype=torch.bfloat16)
    off, srt = torch.zeros(E + 1, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    for name in ("q_up", "s_gate", "s_up"):
        with pytest.raises(ValueError, match=f"the experts' {name} is"):
            m.moe_expert_gate_up(x, off, srt, dataclasses.replace(ex, **{name: getattr(ex, name)[:, :, :-1].contiguous()}), 2)
    for name in ("q_down", "s_down"):
        with pytest.raises(ValueError, match=f"the experts' {name} is"):
            m.moe_expert_down(torch.zeros(8, F, dtype=torch.bfloat16), off,
                              dataclasses.replace(ex, **{name: getattr(ex, name)[:-1].contiguous()}), 4, 2)
    # a matrix that a pass does not read may be missing
    with pytest.raises(ValueError, match="not on the current HIP device"):
        m.moe_expert_gate_up(x, off, srt, dataclasses.replace(ex, q_down=None, s_down=None), 2)
    one = Int8Experts(*(getattr(ex, k)[:1] for k in ("q_gate", "q_up")), ex.q_down[:1, :-16],
                      *(getattr(ex, k)[:1] for k in ("s_gate", "s_up", "s_down")), fmt=MOE_W_MXFP4)
    with pytest.raises(ValueError, match="the experts' q_down is"):
        m.moe_mlp_forward(x, one)


def test_down_takes_experts_without_their_gate_and_up():
    ex = dataclasses.replace(_experts(MOE_W_MXFP4), q_up=None, s_up=None)
    with pytest.raises(ValueError, match="not on the current HIP device"):
        m.moe_expert_down(torch.zeros(8, F, dtype=torch.bfloat16), torch.zeros(E + 1, dtype=torch.int32), ex, 4, 2)


def test_sizes_past_32_bits_are_not_cut():
    """A size whose low 32 bits are a small valid one is refused (tensors without memory stand for the large ones)."""
    big = (1 << 32) + 128
    w = torch.empty(1, big, dtype=torch.bfloat16, device="meta")
    q, s = torch.empty(1, big // 2, dtype=torch.uint8, device="meta"), torch.empty(1, big // 32, dtype=torch.uint8, device="meta")
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: m.moe_quantize_mxfp4(w), lambda: m.moe_dequantize_mxfp4(q, s, torch.bfloat16),
                 lambda: m.moe_pack_mxfp4(q, s), lambda: m.moe_norm_pre(w, w[0]), lambda: m.moe_norm_post(w, w),
                 lambda: m.moe_grouped_mm_mxfp4(q, s, off, q[None], s[None], torch.float32),
                 lambda: m.moe_grouped_mm_mxfp4(q[:, :64], s[:, :4], off, q[None, :, :64], s[None, :, :4],
                                                torch.float32, sorted_slots=off, K=(1 << 32) + 1)):
        with pytest.raises(ValueError, match="past 2\\^31"):
            call()


@pytest.mark.parametrize("gate_tokens,kept", [(1, 1), (7, 7), ((1 << 32) + 1, 0x7fffffff), (1 << 31, 0x7fffffff),
                                              (0, 0), (-1, 0), (-(1 << 32) + 1, 0)])
def test_gate_tokens_past_32_bits(gate_tokens, kept):
    """Past every token it is the same as T; below 1 it reaches the library as a value that it refuses."""
    assert ops._post(5, 64, torch.float32, None, None, gate_tokens, 1.0, 1.0, 1e-6, None, None).gate_tokens == kept


@pytest.mark.parametrize("fmt", [MOE_W_INT8, MOE_W_BF16, MOE_W_MXFP4])
def test_down_takes_h_in_any_contiguous_form(fmt):
    """h is read as T*K rows of f numbers whatever its shape; one that holds fewer, or other rows, is refused."""
    ex = _experts(fmt)
    off = torch.zeros(E + 1, dtype=torch.int32)
    h = torch.zeros(8, F, dtype=torch.bfloat16)
    down = lambda t: m.moe_expert_down(t, off, ex, 4, 2)
    with pytest.raises(Exception) as plain:
        down(h)                                        # past the checks of the width, to the missing GPU
    for form in (h.view(-1), h.view(4, 2, F), h.view(16, F // 2), torch.zeros(11, F, dtype=torch.bfloat16), torch.zeros(9 * F)):
        with pytest.raises(type(plain.value)) as e:
            down(form)
        assert str(e.value) == str(plain.value)
    for bad in (h[:, :128].contiguous(), torch.zeros(8, 2 * F), h[:7], h.view(-1)[:-1]):
        with pytest.raises(ValueError, match="columns"):
            down(bad)


def test_import_on_a_torch_without_gpu_bindings():
    """The package imports, and says what is missing at the first call, where torch was built without a GPU."""
    code = ("import torch\n"
            "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import int8_weight_moe_amd as m\n"
            "try:\n"
            "    m.moe_norm_pre(torch.zeros(2, 64), torch.ones(64))\n"
            "except ValueError as e:\n"
            "    assert 'not on the current HIP device' in str(e)\n"
            "    print('imported')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr
