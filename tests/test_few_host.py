"""moe_forward_few on the host (no GPU): what it refuses."""
import ctypes as C

import pytest

from mixture_experts_layer_41_b200 import _lib as L
from mixture_experts_layer_41_b200 import api

A = 1 << 20      # a non-null, 16-byte aligned address that no refused call touches


def _cfg(**kw):
    base = dict(num_tokens=16, hidden=64, intermediate=128, num_experts=8, top_k=2)
    base.update(kw)
    return api.make_config(**base)


def call(cfg, x=A, wr=A, bias=None, w=None, out=A, ids=None, wts=None, stats=None, ws=A, n=1 << 40):
    w = w if w is not None else L.moe_weights(A, A, A, A, A, A, A, A, A, None, None, None)
    st = C.byref(stats) if stats is not None else None
    return L.lib().moe_forward_few(C.byref(cfg), x, wr, bias, C.byref(w), out, ids, wts, st, ws, n, None)


def test_few_tokens_constant_matches_header():
    import os
    import re
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")
    assert int(re.search(r"#define MOE_FEW_TOKENS (\d+)", open(header).read()).group(1)) == L.MOE_FEW_TOKENS


@pytest.mark.parametrize("kw,status,word", [
    (dict(num_tokens=17), L.MOE_ERR_UNSUPPORTED, "MOE_FEW_TOKENS"),
    (dict(act_dtype="f32", weight_dtype="f32"), L.MOE_ERR_UNSUPPORTED, "bf16"),
    (dict(num_experts=512), L.MOE_ERR_UNSUPPORTED, ""),
    (dict(top_k=9), L.MOE_ERR_INVALID_TOPK, ""),
])
def test_few_refuses_configurations(kw, status, word):
    assert call(_cfg(**kw)) == status
    text = L.lib().moe_last_error().decode()
    assert word in text if word else text == ""


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=A + 2), dict(wr=None), dict(wr=A + 4), dict(bias=A + 4), dict(out=None), dict(out=A + 8),
    dict(ids=A + 4), dict(wts=A + 4), dict(stats=L.moe_stats(A + 4, A, A, A)), dict(stats=L.moe_stats(A, A, A, A + 8)),
    dict(w=L.moe_weights(None, A, A)), dict(w=L.moe_weights(A, None, A)), dict(w=L.moe_weights(A, A, A + 8)),
])
def test_few_refuses_pointers(kw):
    assert call(_cfg(), **kw) == L.MOE_ERR_INVALID_ARG


def test_few_needs_its_weights_and_workspace():
    assert call(_cfg(shared_intermediate=64)) == L.MOE_ERR_INVALID_ARG
    assert call(_cfg(weight_dtype="i8_channel"), w=L.moe_weights(A, A, A)) == L.MOE_ERR_INVALID_ARG
    assert call(_cfg(weight_dtype="q4_affine_g64"), w=L.moe_weights(A, A, A, A, A, A)) == L.MOE_ERR_INVALID_ARG
    assert call(_cfg(), ws=None) == L.MOE_ERR_WORKSPACE
    assert call(_cfg(), n=api.moe_workspace_size(_cfg()) - 1) == L.MOE_ERR_WORKSPACE


def test_few_wrapper_names_the_reason():
    cfg = _cfg(num_tokens=17)
    import torch
    t = torch.zeros(64)
    with pytest.raises(L.MoEError, match="at most MOE_FEW_TOKENS"):
        api.moe_forward_few(cfg, t, t, None, dict(w1=t, w2=t, w3=t), t, None, None, None, t, stream=0)


def test_workspace_grows_only_for_few_tokens():
    """The one-kernel form's buffers are part of the workspace of layers it can
    run, and of no other."""
    small, large = _cfg(num_tokens=16), _cfg(num_tokens=17)
    assert api.moe_workspace_size(small) > api.moe_workspace_size(large)
