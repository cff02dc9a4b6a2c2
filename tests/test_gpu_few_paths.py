"""moe_forward_few on the GPU: paths and reports that the cases of
test_gpu_few.py do not reach."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import int8_reference as R
import test_gpu_few
from gpu_harness import check_route
from mixture_experts_layer_41_b200 import _lib as L
from mixture_experts_layer_41_b200 import api
from moe_cases import as_f64, oracle_route
from test_gpu_few import ANY, bf, check_few, ds, few, make_run, q4, sw

pytestmark = pytest.mark.gpu

# Rows of more than 2048 bytes go through the eight warps of a group, whose
# results meet; more than eight tokens of an expert are two blocks.  Down
# projections of 8192 bytes a row and more are cut along K in small batches, in
# two parts or (from 16384) four.  Most rows end inside a segment of 64 bytes.
CASES = {
    "bf16_two_blocks": (bf(T=16, d=2056, F=2072, E=2, k=2), "bf16"),
    "bf16_two_blocks_uneven": (bf(T=9, d=2056, F=2072, E=3, k=2), "bf16"),
    "i8_two_blocks": (bf(T=16, d=4112, F=4112, E=2, k=2), "i8"),
    "i8_two_blocks_uneven": (bf(T=9, d=4112, F=4112, E=3, k=2), "i8"),
    "q4_two_blocks": (q4(T=16, d=4160, F=4160, E=2, k=2), "q4"),
    "q4_two_blocks_uneven": (q4(T=9, d=4160, F=4160, E=3, k=2), "q4"),
    "bf16_cut_in_two": (bf(T=1, d=520, F=4104, E=2, k=1), "bf16"),
    "bf16_cut_in_four": (bf(T=2, d=264, F=8200, E=2, k=2), "bf16"),
    "bf16_cut_nine_tokens": (bf(T=9, d=264, F=8200, E=2, k=2), "bf16"),
    "i8_cut_in_two": (bf(T=2, d=528, F=8208, E=2, k=1), "i8"),
    "i8_cut_in_four": (bf(T=1, d=272, F=16400, E=2, k=2), "i8"),
    "i8_cut_sixteen_tokens": (bf(T=16, d=272, F=8208, E=2, k=2), "i8"),
    "q4_cut_in_two": (q4(T=1, d=448, F=16448, E=2, k=1), "q4"),
    "q4_cut_in_four": (q4(T=2, d=192, F=32832, E=2, k=2), "q4"),
    "q4_cut_sixteen_tokens": (q4(T=16, d=192, F=16448, E=2, k=2), "q4"),
    "bf16_relu": (sw(T=11, d=1032, F=1048, E=4, k=2, capacity_factor=0.0), "bf16"),
    "bf16_relu_cut": (sw(T=3, d=1032, F=4104, E=4, k=2, capacity_factor=0.0), "bf16"),
    "i8_relu": (sw(T=16, d=2064, F=2096, E=3, k=2, capacity_factor=1.25), "i8"),
    "bf16_shared": (ds(T=16, d=2056, F=1048, E=16, n_group=4, topk_group=2, k=4, shared_F=1096), "bf16"),
    "i8_shared": (ds(T=10, d=2064, F=2064, E=16, n_group=4, topk_group=2, k=4, shared_F=1112), "i8"),
}



def cut_ffn(x, w, act):
    """int8_reference.expert_ffn where the down projection is cut along K: each
    of at most four partial sums is rounded to fp32, scaled (two roundings) and
    added, which costs at most 4 half steps of the magnitudes of the terms."""
    y, bound = expert_ffn(x, w, act)
    q, s = R.quantize(x)
    gate = (q @ w["w1"].astype(np.float64).T) * s[:, None] * w["s1"][None, :]
    if act == "relu":
        h = np.maximum(gate, 0.0)
    else:
        h = R.silu(gate) * ((q @ w["w2"].astype(np.float64).T) * s[:, None] * w["s2"][None, :])
    hq, hs = R.quantize(R.bf16_round(h))
    terms = (np.abs(hq) @ np.abs(w["w3"].astype(np.float64) * w["s3"][:, None]).T) * hs[:, None]
    return y, bound + 4 * R.F32_HALF_STEP * terms


expert_ffn = R.expert_ffn


@pytest.fixture
def case(monkeypatch):
    def make(name, **kw):
        monkeypatch.setitem(test_gpu_few.CASES, name, CASES[name])
        if "cut" in name:
            monkeypatch.setattr(R, "expert_ffn", cut_ffn)
        return make_run(name, **kw)
    return make


@pytest.mark.parametrize("name", sorted(CASES))
def test_few_paths_match_float64(name, case):
    run = case(name)
    run.fill_canary()
    few(run)
    torch.cuda.synchronize()
    assert run.status() == 0
    assert (run.ws_full[run.ws.numel():] == 0xA5).all()
    for full, rows in run.guarded.values():
        assert (full.view(torch.uint8)[rows:] == 0xA5).all()
    check_route(run, oracle_route(run.w, run.inp), max_unsafe_fraction=ANY)
    check_few(run)
    first = run.out.clone()
    run.fill_canary()
    few(run)
    torch.cuda.synchronize()
    assert torch.equal(run.out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("name", ["bf16_two_blocks", "i8_two_blocks", "q4_two_blocks", "i8_cut_in_four", "q4_cut_in_two",
                                  "bf16_shared"])
def test_few_paths_fused_gate_up(name, case):
    a, b = case(name), case(name, fused=True)
    few(a)
    few(b)
    torch.cuda.synchronize()
    assert a.status() == 0 and b.status() == 0
    assert torch.equal(a.out.view(torch.int16), b.out.view(torch.int16))


@pytest.mark.parametrize("name", ["bf16_two_blocks", "bf16_cut_in_four", "bf16_relu", "i8_two_blocks", "i8_cut_in_two",
                                  "i8_relu", "q4_two_blocks", "q4_cut_in_two"])
def test_few_paths_agree_with_forward(name, case):
    run = case(name)
    few(run)
    torch.cuda.synchronize()
    got, ids, kept = as_f64(run.out), run.ids.clone(), run.stats["kept_counts"].clone()
    run.forward()
    assert torch.equal(ids, run.ids) and torch.equal(kept, run.stats["kept_counts"])
    ref = as_f64(run.out)
    assert np.linalg.norm(got - ref) <= 1e-2 * np.linalg.norm(ref)


@pytest.mark.parametrize("kind", ["bf16", "i8", "q4"])
def test_few_rows_with_one_outlier(kind, case):
    """Tokens with one element 1000 times the rest, as hidden states of a model
    have them.  4-bit experts take a row as integers over its largest element,
    8-bit experts as codes over it: the bounds follow from that."""
    run = case(kind + "_two_blocks")
    x = run.inp["x"]
    x *= 0.1
    for t in range(run.w.T):
        x[t, (37 * t + 5) % run.w.d] = 100.0 if t % 2 else -100.0
    few(run)
    torch.cuda.synchronize()
    assert run.status() == 0
    check_few(run)


def test_few_wait_limit_names_its_kernel():
    """A grid barrier that runs out is reported as the few-token kernel's, not as
    a tensor-core kernel's."""
    run = make_run("long_rows")
    try:
        api.moe_set_wait_timeout_ns(1)
        few(run)
        assert run.status() == L.MOE_ERR_DEVICE
        text = L.lib().moe_last_error().decode()
    finally:
        api.moe_set_wait_timeout_ns(0)
    assert "few-token kernel" in text and "timed out" in text and "tensor-core" not in text, text
    few(run)
    torch.cuda.synchronize()
    assert run.status() == 0
