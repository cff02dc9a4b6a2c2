"""moe_forward_few on the GPU: the whole layer for a few tokens in one kernel,
against float64, for every weight type and router, at the sizes and token
counts where it can go wrong."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import int8_reference as R
from gpu_harness import Run, check_route
from mixture_experts_layer_41_b200 import _lib as L
from mixture_experts_layer_41_b200 import api
from mixture_experts_layer_41_b200.inputs import to_host, workload
from moe_cases import as_f64, oracle_route, router_bias_of
from oracle import moe_oracle as O
from test_gpu_int8 import I8Run

pytestmark = pytest.mark.gpu

bf = lambda **kw: workload("mixtral_prefill", **kw)
q4 = lambda **kw: workload("decode_q4", **kw)
ds = lambda **kw: workload("deepseek_v3", **kw)
sw = lambda **kw: workload("switch_top1", **kw)

# name -> (workload, weights)
CASES = {
    "one_token": (bf(T=1, d=256, F=320, E=8, k=2), "bf16"),
    "two_tokens_k1": (bf(T=2, d=64, F=64, E=2, k=1), "bf16"),
    "three_ragged": (bf(T=3, d=200, F=136, E=6, k=3), "bf16"),
    "five_k_is_e": (bf(T=5, d=512, F=256, E=4, k=4), "bf16"),
    "eight_wide": (bf(T=8, d=1040, F=528, E=40, k=8), "bf16"),
    "nine_tokens_two_blocks": (bf(T=9, d=264, F=200, E=2, k=2), "bf16"),
    "sixteen_all_one_expert": (sw(T=16, d=128, F=264, E=8, k=1, capacity_factor=0.0), "bf16"),
    "sixteen_drops": (sw(T=16, d=256, F=136, E=4, k=2, capacity_factor=1.0), "bf16"),
    "relu_odd_rows": (sw(T=7, d=136, F=72, E=16, k=3, capacity_factor=1.25), "bf16"),
    "no_norm": (bf(T=6, d=128, F=64, E=100, k=5, norm_topk_prob=False), "bf16"),
    "groups_shared": (ds(T=4, d=448, F=256, E=32, n_group=8, topk_group=4, shared_F=256), "bf16"),
    "shared_other_width": (ds(T=16, d=448, F=128, E=256, shared_F=200), "bf16"),
    "k32": (bf(T=16, d=64, F=64, E=64, k=32), "bf16"),
    "long_rows": (bf(T=1, d=7168, F=1024, E=2, k=1), "bf16"),
    "long_reduction": (bf(T=2, d=512, F=14336, E=2, k=2), "bf16"),
    "i8_one_token": (bf(T=1, d=256, F=320, E=8, k=2), "i8"),
    "i8_ragged": (bf(T=3, d=208, F=144, E=6, k=3), "i8"),
    "i8_two_blocks": (bf(T=13, d=272, F=208, E=2, k=2), "i8"),
    "i8_relu_drops": (sw(T=16, d=256, F=144, E=4, k=2, capacity_factor=1.0), "i8"),
    "i8_shared": (ds(T=4, d=448, F=256, E=32, n_group=8, topk_group=4, shared_F=256), "i8"),
    "i8_many_experts": (bf(T=16, d=512, F=192, E=128, k=8), "i8"),
    "i8_long": (bf(T=2, d=4096, F=2048, E=2, k=1), "i8"),
    "q4_one_token": (q4(T=1, d=256, F=320, E=8, k=2), "q4"),
    "q4_smallest": (q4(T=2, d=64, F=64, E=2, k=1), "q4"),
    "q4_odd_groups": (q4(T=5, d=448, F=192, E=16, k=4), "q4"),
    "q4_decode": (q4(T=16, d=2048, F=768, E=128, k=8), "q4"),
    "q4_two_blocks": (q4(T=16, d=320, F=128, E=2, k=2), "q4"),
    "q4_long": (q4(T=1, d=4096, F=8192, E=2, k=1), "q4"),
}
SKEWED = {"sixteen_all_one_expert", "sixteen_drops"}


def make_run(name, seed=41, fused=False):
    w, kind = CASES[name]
    run = I8Run(w, seed=seed, fused=fused) if kind == "i8" else Run(w, seed=seed)
    if fused and kind != "i8":
        for a in ("w", "s", "b"):
            if a + "2" in run.weights:
                run.weights[a + "1"] = torch.cat([run.weights[a + "1"], run.weights.pop(a + "2")], 1).contiguous()
        run.cfg.weight_layout = L.MOE_LAYOUT_FUSED_GATE_UP
    if name in SKEWED:
        run.bias = torch.full((w.E,), 0.0, device="cuda")
        run.bias[1] = 50.0
        run.inp["logit_bias"] = run.bias
    n = api.moe_workspace_size(run.cfg)
    run.ws_full = torch.full((n + (1 << 16),), 0xA5, dtype=torch.uint8, device="cuda")
    run.ws = run.ws_full[:n]
    return run


# Batches this small may lie within the 1e-4 margin altogether (32 of 64
# experts whose probabilities spread 16 % around 1/64 are 2.5 * 0.16 / 64 / 64
# = 1e-4 apart at the cut); such tokens are still checked for a correct choice
# within the margin and for exact weights.
ANY = 1.0


def few(run, stream=None):
    api.moe_forward_few(run.cfg, run.inp["x"], run.inp["w_router"], run.bias, run.weights, run.out, run.ids, run.wts,
                        run.stats, run.ws, stream)


# ---------------------------------------------------------------- reference

def dense(run, e):
    """Expert e's matrices in float64 and their magnitudes term by term."""
    m, a = {}, {}
    inp = run.inp
    for i in "123":
        if inp.get("q" + i) is not None:
            words = inp["q" + i][e].cpu().numpy().view(np.uint32)
            code = ((words[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).reshape(words.shape[0], -1)
            s = np.repeat(as_f64(inp["s" + i][e]), 64, axis=1)
            b = np.repeat(as_f64(inp["b" + i][e]), 64, axis=1)
            m[i], a[i] = s * code + b, np.abs(s) * code + np.abs(b)
        elif inp.get("w" + i) is not None:
            m[i] = as_f64(inp["w" + i][e])
            a[i] = np.abs(m[i])
    return m, a


def ffn(x, m, a, act, fixed=False):
    """(y, bound): the expert in float64 and how far fp32 sums over its products
    and an intermediate of 16 bits may be from it.  A sum over K takes K / 128
    dependent tensor-core additions per warp and 8 + 8 further ones, each off
    by at most 2^-22 of the magnitudes added.  ``fixed`` (4-bit weights): x and
    the intermediate are rounded to integer multiples of their row's largest
    magnitude over 32512, so each element is off by at most half of that (and
    the quotient by 2^-22 of the element, two fp32 roundings)."""
    eps = lambda K: (K / 128 + 24) * 2.0 ** -22
    fix = lambda v: np.abs(v).max(1, keepdims=True) / 65024 + 2.0 ** -22 * np.abs(v) if fixed else 0.0 * v
    ax = np.abs(x)
    g = x @ m["1"].T
    dg = eps(x.shape[1]) * (ax @ a["1"].T) + fix(x) @ a["1"].T
    if act == "relu":
        h, dh = np.maximum(g, 0.0), dg
    else:
        u = x @ m["2"].T
        du = eps(x.shape[1]) * (ax @ a["2"].T) + fix(x) @ a["2"].T
        h = R.silu(g) * u
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(R.silu(g)) * du + 2.0 ** -20 * np.abs(h)    # |silu'| < 1.1
    dh = dh + (fix(np.abs(h) + dh) if fixed else 2.0 ** -16 * np.abs(h))
    y = h @ m["3"].T
    return y, dh @ a["3"].T + eps(h.shape[1]) * ((np.abs(h) + dh) @ a["3"].T)


def check_few(run):
    w = run.w
    x = as_f64(run.inp["x"])
    ids, wts = run.ids.cpu().numpy(), run.wts.cpu().numpy().astype(np.float64)
    cap = O.capacity(w.T, w.k, w.E, float(np.float32(w.capacity_factor)))
    ref = O.dispatch(ids, w.E, cap, wts)
    assert np.array_equal(run.stats["raw_counts"].cpu().numpy(), ref["raw_counts"])
    assert np.array_equal(run.stats["kept_counts"].cpu().numpy(), ref["kept_counts"])
    assert int(run.stats["dropped"][0]) == ref["dropped"]
    out, bound = np.zeros((w.T, w.d)), np.zeros((w.T, w.d))
    for e in range(w.E):
        t, j = np.nonzero((ids == e) & (ref["slot_row"] >= 0))
        if not t.size:
            continue
        if hasattr(run, "host"):
            y, b = R.expert_ffn(x[t], {k: v[e] for k, v in run.host.items()}, w.act)
        else:
            y, b = ffn(x[t], *dense(run, e), w.act, w.weight_format == "q4_affine_g64")
        np.add.at(out, t, y * wts[t, j][:, None])
        # fp32 scales, weights and the sum of k + 1 terms
        np.add.at(bound, t, (b + (w.k + 8) * R.F32_HALF_STEP * (np.abs(y) + b)) * wts[t, j][:, None])
    if w.shared_F:
        m = {i: as_f64(run.weights["ws" + i]) for i in "123"}
        y, b = ffn(x, m, {i: np.abs(v) for i, v in m.items()}, "swiglu")
        out, bound = out + y, bound + b
    bound = bound + R.BF16_HALF_STEP * (np.abs(out) + bound)
    got = as_f64(run.out)
    assert (np.abs(got - out) - bound).max() <= 0.0, (np.abs(got - out) / np.maximum(bound, 1e-30)).max()


# ---------------------------------------------------------------- tests

@pytest.mark.parametrize("name", sorted(CASES))
def test_few_matches_float64(name):
    run = make_run(name)
    run.fill_canary()
    few(run)
    torch.cuda.synchronize()
    assert run.status() == 0
    assert (run.ws_full[run.ws.numel():] == 0xA5).all()
    for full, rows in run.guarded.values():
        assert (full.view(torch.uint8)[rows:] == 0xA5).all()
    check_route(run, oracle_route(run.w, run.inp), max_unsafe_fraction=ANY)
    check_few(run)
    if name == "sixteen_all_one_expert":
        assert int(run.stats["kept_counts"][1]) == 16
    first = run.out.clone()
    run.fill_canary()
    few(run)
    torch.cuda.synchronize()
    assert torch.equal(run.out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("name", ["one_token", "groups_shared", "i8_ragged", "i8_shared", "q4_odd_groups"])
def test_few_fused_gate_up(name):
    a, b = make_run(name), make_run(name, fused=True)
    few(a)
    few(b)
    torch.cuda.synchronize()
    assert a.status() == 0 and b.status() == 0
    assert torch.equal(a.out.view(torch.int16), b.out.view(torch.int16))


@pytest.mark.parametrize("name", ["eight_wide", "sixteen_drops", "groups_shared", "i8_two_blocks", "q4_decode"])
def test_few_agrees_with_forward(name):
    """The one-kernel form and the staged layer: the same choices and counts,
    outputs within both paths' bf16 roundings (the staged one rounds the
    intermediate, every expert output and the sum)."""
    run = make_run(name)
    few(run)
    torch.cuda.synchronize()
    got, ids, kept = as_f64(run.out), run.ids.clone(), run.stats["kept_counts"].clone()
    run.forward()
    assert torch.equal(ids, run.ids) and torch.equal(kept, run.stats["kept_counts"])
    ref = as_f64(run.out)
    assert np.linalg.norm(got - ref) <= 1e-2 * np.linalg.norm(ref)


@pytest.mark.parametrize("T", range(1, 17))
@pytest.mark.parametrize("kind", ["bf16", "i8", "q4"])
def test_few_every_token_count(T, kind):
    w = {"bf16": bf, "i8": bf, "q4": q4}[kind](T=T, d=192, F=128, E=12, k=3)
    CASES["_t"] = (w, kind)
    try:
        run = make_run("_t", seed=T)
    finally:
        del CASES["_t"]
    run.fill_canary()
    few(run)
    torch.cuda.synchronize()
    assert run.status() == 0
    check_route(run, oracle_route(w, run.inp), max_unsafe_fraction=ANY)
    check_few(run)


def test_few_padded_tokens():
    """Rows of zeros (a padded batch) route by ties to the lowest experts and
    give zeros; the other tokens are as they are without them."""
    for name in ("eight_wide", "i8_many_experts", "q4_odd_groups"):
        run = make_run(name)
        few(run)
        torch.cuda.synchronize()
        before = run.out.clone()
        run.inp["x"][2:5] = 0
        few(run)
        torch.cuda.synchronize()
        assert run.status() == 0
        assert (run.out[2:5] == 0).all()
        k = run.w.k
        assert torch.equal(run.ids[2:5].cpu(), torch.arange(k, dtype=torch.int32).expand(3, k))
        keep = [t for t in range(run.w.T) if not 2 <= t < 5]
        assert torch.equal(run.out[keep].view(torch.int16), before[keep].view(torch.int16))


def test_few_nan_token_is_reported():
    """A NaN token chooses nothing (ids -1, a device status) and the others
    keep their outputs."""
    for name in ("eight_wide", "groups_shared", "i8_many_experts"):
        run = make_run(name)
        few(run)
        torch.cuda.synchronize()
        before = run.out.clone()
        run.inp["x"][1, 5] = float("nan")
        few(run)
        torch.cuda.synchronize()
        assert run.status() == L.MOE_ERR_DEVICE
        assert (run.ids[1] == -1).all()
        keep = [t for t in range(run.w.T) if t != 1]
        assert torch.equal(run.out[keep].view(torch.int16), before[keep].view(torch.int16))


def test_few_null_outputs():
    run = make_run("groups_shared")
    few(run)
    torch.cuda.synchronize()
    ref = run.out.clone()
    run.out.zero_()
    api.moe_forward_few(run.cfg, run.inp["x"], run.inp["w_router"], run.bias, run.weights, run.out, None, None, None, run.ws)
    torch.cuda.synchronize()
    assert torch.equal(run.out.view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("name", ["groups_shared", "i8_shared", "q4_decode"])
def test_few_graph_and_streams(name):
    """Captured and replayed on new tokens; two layers on two streams at once."""
    run, other = make_run(name, seed=1), make_run(name, seed=2)
    layer = api.MoELayer(run.cfg, run.inp["w_router"], run.weights, router_bias=run.bias)
    x = run.inp["x"]
    layer.forward_few(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward_few(x)
    g = torch.Generator(device="cuda").manual_seed(3)
    for _ in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16))
        layer.forward_few(x)
        eager = layer.o.out.clone()
        layer.o.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.o.out.view(torch.int16), eager.view(torch.int16))
        assert layer.status() == 0
    few(run)
    few(other)
    torch.cuda.synchronize()
    want = run.out.clone(), other.out.clone()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    run.out.zero_()
    other.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        few(run, streams[0])
        few(other, streams[1])
    torch.cuda.synchronize()
    assert torch.equal(run.out, want[0]) and torch.equal(other.out, want[1])
    assert run.status() == 0 and other.status() == 0


def test_few_refuses_tensors_elsewhere():
    """A tensor left on the host is refused before the launch."""
    run = make_run("groups_shared")
    args = [run.cfg, run.inp["x"], run.inp["w_router"], run.bias, run.weights, run.out, None, None, None, run.ws]
    for i in (1, 2, 3, 5, 9):
        with pytest.raises(ValueError, match="current CUDA device"):
            api.moe_forward_few(*(a.cpu() if j == i else a for j, a in enumerate(args)))
    with pytest.raises(ValueError, match="current CUDA device"):
        api.moe_forward_few(*args[:4], dict(run.weights, w3=run.weights["w3"].cpu()), *args[5:])


def test_few_two_graphs_at_once():
    """Two captured layers, a workspace each, replayed on two streams without
    waiting for one another."""
    layers, want, graphs = [], [], []
    for name, seed in (("groups_shared", 1), ("i8_shared", 2)):
        run = make_run(name, seed=seed)
        layer = api.MoELayer(run.cfg, run.inp["w_router"], run.weights, router_bias=run.bias)
        layer.forward_few(run.inp["x"])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.forward_few(run.inp["x"])
        layers.append((layer, run))
        want.append(layer.o.out.clone())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for layer, _ in layers:
        layer.o.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for (layer, _), out in zip(layers, want):
        assert layer.status() == 0
        assert torch.equal(layer.o.out, out)


@pytest.mark.parametrize("name", ["long_rows", "i8_long", "q4_long", "groups_shared"])
def test_few_wait_timeout_reports_and_recovers(name):
    """With a 1 ns bound the first wait that is not already over gives up: a
    device status, and the context and workspace stay good."""
    run = make_run(name)
    try:
        api.moe_set_wait_timeout_ns(1)
        few(run)
        st = run.status()
        text = L.lib().moe_last_error().decode()
    finally:
        api.moe_set_wait_timeout_ns(0)
    assert st == L.MOE_ERR_DEVICE, st
    assert "timed out" in text, text
    few(run)
    torch.cuda.synchronize()
    assert run.status() == 0
    check_few(run)


def test_few_decoding_steps():
    """A run of steps as a server makes them: the prompt through forward, then
    one-kernel steps whose outputs feed the next step, the router's balancing
    bias updated in between; each step is checked."""
    w = ds(T=3, d=256, F=128, E=32, n_group=8, topk_group=4, shared_F=128)
    CASES["_d"] = (w, "i8")
    try:
        run = make_run("_d", seed=9)
    finally:
        del CASES["_d"]
    layer = api.MoELayer(run.cfg, run.inp["w_router"], run.weights, router_bias=run.bias)
    x = run.inp["x"]
    layer.forward(x)
    for _ in range(4):
        o = layer.forward_few(x)
        torch.cuda.synchronize()
        assert layer.status() == 0
        run.out, run.ids, run.wts = o.out, o.topk_ids, o.topk_w
        run.stats = layer.stats()
        check_few(run)
        layer.update_bias(1e-3)
        y = x.float() + o.out.float()
        x.copy_((y / y.pow(2).mean(1, keepdim=True).sqrt()).to(torch.bfloat16))
