"""8-bit weights and products on the host (no GPU): configurations, sizes,
argument refusals, and the float64 reference that the GPU tests use."""
import ctypes as C

import numpy as np
import pytest
import torch

import int8_reference as R
from mixture_experts_layer_41_b200 import _lib as L
from mixture_experts_layer_41_b200 import api

A = 1 << 20      # a non-null, 16-byte aligned address that no refused call touches


def _cfg(**kw):
    base = dict(num_tokens=64, hidden=64, intermediate=128, num_experts=8, top_k=2, weight_dtype="i8_channel")
    base.update(kw)
    return api.make_config(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(), L.MOE_OK),
    (dict(act="relu"), L.MOE_OK),
    (dict(weight_layout="fused_gate_up"), L.MOE_OK),
    (dict(shared_intermediate=64), L.MOE_OK),
    (dict(fused_gather=True), L.MOE_OK),
    (dict(hidden=72), L.MOE_ERR_UNSUPPORTED),
    (dict(intermediate=136), L.MOE_ERR_UNSUPPORTED),
    (dict(hidden=131056), L.MOE_OK),
    (dict(hidden=131072), L.MOE_ERR_UNSUPPORTED),
    (dict(intermediate=131072), L.MOE_ERR_UNSUPPORTED),
    (dict(act_dtype="f32"), L.MOE_ERR_UNSUPPORTED),
])
def test_validate_8_bit(kw, status):
    cfg = _cfg(**kw)
    assert api.moe_validate(cfg) == status
    assert (api.moe_workspace_size(cfg) > 0) == (status == L.MOE_OK)


def test_8_bit_workspace_has_no_row_copy():
    cfg = _cfg()
    assert api.moe_workspace_region(cfg, "x_perm")[1] == 0
    assert api.moe_workspace_region(cfg, "h")[1] == 64 * 2 * 128 * 2


def _weights(**kw):
    w = dict(w1=A, w2=A, w3=A, scale1=A, scale2=A, scale3=A, bias1=0, bias2=0, bias3=0, shared1=0, shared2=0, shared3=0)
    w.update(kw)
    return L.moe_weights(*[w[f] or None for f, _ in L.moe_weights._fields_])


@pytest.mark.parametrize("kw,cfg_kw", [
    (dict(scale1=0), {}), (dict(scale2=0), {}), (dict(scale3=0), {}), (dict(w2=0), {}), (dict(w1=A + 8), {}),
    (dict(scale1=A + 4), {}), (dict(bias1=A), {}), (dict(bias3=A), {}),
    (dict(), dict(weight_layout="fused_gate_up")),
    (dict(w2=0), dict(weight_layout="fused_gate_up")),
])
def test_8_bit_weights_are_checked(kw, cfg_kw):
    cfg = _cfg(**cfg_kw)
    w = _weights(**kw)
    st = L.lib().moe_grouped_ffn(C.byref(cfg), A, A, C.byref(w), A, A, 1 << 40, None)
    assert st == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("args,status", [
    ((A, L.MOE_BF16, -1, 64, A, A), L.MOE_ERR_INVALID_ARG),
    ((A, L.MOE_BF16, 4, 0, A, A), L.MOE_ERR_INVALID_ARG),
    ((A, L.MOE_I8_CHANNEL, 4, 64, A, A), L.MOE_ERR_INVALID_ARG),
    ((A, 9, 4, 64, A, A), L.MOE_ERR_INVALID_ARG),
    ((A, L.MOE_F32, 4, 72, A, A), L.MOE_ERR_UNSUPPORTED),
    ((None, L.MOE_F32, 4, 64, A, A), L.MOE_ERR_INVALID_ARG),
    ((A, L.MOE_F32, 4, 64, A + 8, A), L.MOE_ERR_INVALID_ARG),
    ((A, L.MOE_F32, 4, 64, A, A + 4), L.MOE_ERR_INVALID_ARG),
    ((None, L.MOE_F32, 0, 64, None, None), L.MOE_OK),
])
def test_quantize_rows_refusals(args, status):
    assert L.lib().moe_quantize_rows(*args, None) == status


MM = dict(groups=2, rows=8, n=40, k=64, x=A, xs=A, off=A, w=A, ws=A, dt=L.MOE_BF16, out=A, work=A, bytes=1 << 30)


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0), L.MOE_ERR_INVALID_ARG), (dict(rows=-1), L.MOE_ERR_INVALID_ARG), (dict(n=0), L.MOE_ERR_INVALID_ARG),
    (dict(k=0), L.MOE_ERR_INVALID_ARG), (dict(groups=257), L.MOE_ERR_UNSUPPORTED), (dict(k=72), L.MOE_ERR_UNSUPPORTED),
    (dict(k=131072), L.MOE_ERR_UNSUPPORTED), (dict(n=1 << 30), L.MOE_ERR_UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), L.MOE_ERR_UNSUPPORTED), (dict(off=None), L.MOE_ERR_INVALID_ARG),
    (dict(dt=L.MOE_I8_CHANNEL), L.MOE_ERR_INVALID_ARG), (dict(x=None), L.MOE_ERR_INVALID_ARG),
    (dict(xs=A + 4), L.MOE_ERR_INVALID_ARG), (dict(w=None), L.MOE_ERR_INVALID_ARG), (dict(ws=None), L.MOE_ERR_INVALID_ARG),
    (dict(out=A + 2), L.MOE_ERR_INVALID_ARG), (dict(work=None), L.MOE_ERR_WORKSPACE), (dict(bytes=0), L.MOE_ERR_WORKSPACE),
])
def test_quantized_matmul_refusals(kw, status):
    a = dict(MM, **kw)
    assert L.lib().moe_quantized_matmul(a["groups"], a["rows"], a["n"], a["k"], a["x"], a["xs"], a["off"], a["w"], a["ws"],
                                        a["dt"], a["out"], a["work"], a["bytes"], None) == status


def test_quantized_matmul_workspace_size():
    assert api.moe_quantized_matmul_workspace_size(1, 0, 1, 16) > 0
    assert api.moe_quantized_matmul_workspace_size(256, 100, 3, 131056) > 0
    for bad in ((0, 1, 1, 16), (1, 1, 1, 8), (257, 1, 1, 16), (1, -1, 1, 16)):
        assert api.moe_quantized_matmul_workspace_size(*bad) == 0


def test_wrappers_refuse_wrong_tensors():
    x = torch.zeros((4, 32))
    q, s = torch.zeros((4, 32), dtype=torch.int8), torch.zeros(4)
    for bad in ((x.half(), q, s), (x, q.float(), s), (x, q[:3], s), (x, q, s[:3]), (x, q, s.double()),
                (torch.zeros((32, 4)).t(), q, s)):
        with pytest.raises(ValueError):
            api.moe_quantize_rows(*bad)
    w, ws, out, work = torch.zeros((2, 8, 32), dtype=torch.int8), torch.zeros((2, 8)), torch.zeros((4, 8)), \
        torch.zeros(4096, dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    for bad in ((q[:, :16], s, w, ws, out, work, off), (q, s[:2], w, ws, out, work, off), (q, s, w, ws[:1], out, work, off),
                (q, s, w, ws, out.half(), work, off), (q, s, w, ws, out[:3], work, off), (q, s, w, ws, out, work, off[:2]),
                (q, s, w, ws, out, work, off.long()), (q, s, w.float(), ws, out, work, off),
                (q, s, w.transpose(0, 1), ws, out, work, off)):
        with pytest.raises(ValueError):
            api.moe_quantized_matmul(*bad)


# ---------------------------------------------------------------- the reference itself

def test_reference_bf16_round_matches_torch():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(4000, generator=g, dtype=torch.float64)
    assert np.array_equal(R.bf16_round(x.numpy()), x.to(torch.bfloat16).double().numpy())


def test_reference_quantize_closed_forms():
    q, s = R.quantize(np.array([[0.0, 0.0], [254.0, 127.0], [-3.0, 1.5], [127.0, 0.5]]))
    assert np.array_equal(q, [[0, 0], [127, 64], [-127, 64], [127, 0]])
    assert np.allclose(s, [0.0, 2.0, 3.0 / 127, 1.0])


def test_reference_ffn_follows_the_dense_one():
    """The 8-bit FFN is near the dense one, and on most rows its bound is
    rounding alone: an element lies within 2^-17 of a bf16 border (2^-8 to
    2^-7 of itself apart) with a chance of at most 2^-8, so a row of 48 holds
    none with a chance of 0.83, and then the bound is four fp32 half steps."""
    rng = np.random.default_rng(1)
    x = R.bf16_round(rng.standard_normal((20, 64)))
    dense = {i: rng.standard_normal(sh) * 0.1 for i, sh in (("1", (48, 64)), ("2", (48, 64)), ("3", (64, 48)))}
    w = {}
    for i, m in dense.items():
        w["w" + i], w["s" + i] = R.quantize(m)
    y, bound = R.expert_ffn(x, w, "swiglu")
    ref = (R.silu(x @ dense["1"].T) * (x @ dense["2"].T)) @ dense["3"].T
    rel = np.linalg.norm(y - ref) / np.linalg.norm(ref)
    assert 1e-3 < rel < 3e-2
    rounding = (bound <= 4.01 * R.F32_HALF_STEP * np.abs(y)).all(1)
    assert rounding.sum() >= 10
