"""8-bit integers on the GPU: row quantisation, the product with scales per
token and channel, and the layer with 8-bit experts, against float64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import int8_reference as R
from gpu_harness import Run, check_dispatch, check_route
from mixture_experts_layer_41_b200 import _lib as L
from mixture_experts_layer_41_b200 import api
from mixture_experts_layer_41_b200.inputs import to_host, workload
from moe_cases import as_f64, oracle_route, router_bias_of

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def quantize(x, stream=None):
    q = torch.full(x.shape, 99, dtype=torch.int8, device="cuda")
    s = torch.full(x.shape[:-1], -1.0, device="cuda")
    api.moe_quantize_rows(x, q, s, stream)
    return q, s


# ---------------------------------------------------------------- row quantisation

def check_quantize(x):
    q, s = quantize(x)
    torch.cuda.synchronize()
    ref_q, ref_s = R.quantize(x.cpu().double().numpy())
    assert np.array_equal(q.cpu().numpy().astype(np.float64), ref_q)
    assert np.array_equal(s.cpu().numpy(), ref_s.astype(np.float32))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (7, 48), (33, 1024), (5, 1040), (3, 4096), (2, 16384), (2, 16400),
                                       (1, 40000), (700, 208), (20000, 16)])
def test_quantize_rows(rows, cols, dt):
    g = torch.Generator(device="cuda").manual_seed(rows * 31 + cols)
    x = torch.randn((rows, cols), generator=g, device="cuda") * torch.exp(
        torch.randn((rows, 1), generator=g, device="cuda"))
    check_quantize(x.to(DT[dt]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_ties_and_near_ties(dt):
    """Rows whose quotients 127 x / a are n + 1/2 exactly for every n, and the
    neighbours of those elements on both sides."""
    x = torch.zeros((4, 400), dtype=torch.float64)
    half = torch.arange(-126.5, 127.0, 1.0, dtype=torch.float64)          # 254 ties
    for i, a in enumerate((127.0, 254.0, 2.0 ** -40 * 127, 1.9921875)):    # 1.9921875 = 255 / 128
        x[i, :half.numel()] = half * (a / 127.0)
        x[i, 300] = a
    x = x.to(DT[dt])
    check_quantize(x.cuda())
    bits = x.view(torch.int16 if dt == "bf16" else torch.int32)
    for step in (-1, 1):
        y = (bits + step * (bits != 0).to(bits.dtype)).view(DT[dt])       # (int16 / int32 throughout)
        y[:, 300] = x[:, 300]
        check_quantize(y.cuda())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_extremes(dt):
    """Rows of zeros, of the largest and of the smallest values (subnormals
    too), one element alone, and rows that hold an infinity or a NaN."""
    x = torch.zeros((8, 64), device="cuda")
    x[1] = torch.linspace(-1, 1, 64) * 3.3e38
    x[2] = torch.linspace(-1, 1, 64) * 1e-37
    x[3] = torch.linspace(-1, 1, 64) * 3e-39       # subnormal
    x[4, 17] = -2.5
    x[5] = torch.linspace(-1, 1, 64) * 2.0 ** 101
    x = x.to(DT[dt])
    check_quantize(x)
    x[6, 3] = float("inf")
    x[7] = 1.0
    x[7, 63] = float("nan")
    q, s = quantize(x)
    torch.cuda.synchronize()
    assert torch.isnan(s[6:]).all() and (q[6:] == 0).all()
    assert torch.isfinite(s[:6]).all()


def test_quantize_no_rows_and_guard():
    x = torch.randn((3, 32), device="cuda")
    q = torch.full((4, 32), 99, dtype=torch.int8, device="cuda")
    s = torch.full((4,), -1.0, device="cuda")
    api.moe_quantize_rows(x[:0], q[:0], s[:0])
    api.moe_quantize_rows(x, q[:3], s[:3])
    torch.cuda.synchronize()
    assert (q[3] == 99).all() and s[3] == -1.0


# ---------------------------------------------------------------- product

def mm_inputs(rows, n, k, groups=1, seed=0):
    rng = np.random.default_rng(seed + rows + 7 * n + 13 * k)
    q = rng.integers(-127, 128, (rows, k)).astype(np.int8)
    wq = rng.integers(-127, 128, (groups, n, k)).astype(np.int8)
    s = np.exp(rng.standard_normal(rows)).astype(np.float32) * 1e-2
    ws = np.exp(rng.standard_normal((groups, n))).astype(np.float32) * 1e-3
    return q, s, wq, ws


def run_mm(q, s, wq, ws, dt, offsets=None, fill=0.0):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    rows, (groups, n, k) = q.shape[0], wq.shape
    full = torch.full((rows + 8, n), fill, dtype=DT[dt], device="cuda")
    size = api.moe_quantized_matmul_workspace_size(groups, rows, n, k)
    w = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    api.moe_quantized_matmul(d(q), d(s), d(wq), d(ws), full[:rows], w[:size], group_offsets=off)
    torch.cuda.synchronize()
    assert (w[size:] == 0xA5).all()
    assert (full[rows:] == fill).all()
    return full[:rows], api.moe_workspace_status(w[:size])


def check_mm(out, ref, dt, fill=0.0):
    """The sum is an exact integer; rounding it, the product of the scales and
    the scaled value cost three fp32 half steps, bf16 output one of its own."""
    got = out.float().cpu().numpy().astype(np.float64)
    none = np.isnan(ref)
    assert np.all(got[none] == fill)
    tol = 3.01 * R.F32_HALF_STEP + (R.BF16_HALF_STEP if dt == "bf16" else 0.0)
    err = np.abs(got - ref)[~none] - tol * np.abs(ref)[~none]
    assert err.size == 0 or err.max() <= 0.0, err.max()


MM = [(1, 64, 64), (1, 4096, 4096), (1, 2051, 1424), (3, 8, 16), (5, 1, 48), (16, 256, 272), (17, 129, 144),
      (31, 520, 2048), (33, 7, 400), (64, 300, 96), (100, 1024, 528), (128, 256, 128), (129, 257, 144), (130, 4100, 64),
      (500, 1000, 1040), (777, 2051, 1424), (1300, 4096, 256), (500, 4100, 1040), (1090, 2310, 1072), (257, 6500, 1024),
      (320, 3200, 2064)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n,k", MM)
def test_quantized_matmul(rows, n, k, dt):
    q, s, wq, ws = mm_inputs(rows, n, k)
    out, st = run_mm(q, s, wq, ws, dt)
    assert st == 0
    check_mm(out, R.matmul(q, s, wq, ws), dt)


def test_quantized_matmul_largest_sums():
    """Every product at its largest magnitude over a long reduction: the
    32-bit sums reach 128 * 128 * 131056 = 2147221504."""
    k = 131056
    q = np.full((3, k), -128, np.int8)
    q[1] = 127
    q[2] = np.where(np.arange(k) % 2, 127, -128)
    wq = np.full((1, 9, k), -128, np.int8)
    wq[0, 4] = 127
    s, ws = np.ones(3, np.float32), np.ones((1, 9), np.float32)
    for rows in (1, 3, 40):
        qq = np.tile(q, (14, 1))[:rows]
        out, st = run_mm(qq, np.ones(rows, np.float32), wq, ws, "f32")
        assert st == 0
        check_mm(out, R.matmul(qq, np.ones(rows), wq, ws), "f32")


GROUPS = [
    (2, 70, 64, 64, [0, 0, 70]),
    (5, 400, 264, 144, [0, 129, 129, 130, 390, 400]),
    (5, 400, 264, 144, [0, 1, 2, 3, 4, 5]),
    (8, 2048, 512, 256, [0, 128, 256, 256, 900, 901, 1500, 1500, 2000]),
    (64, 64, 48, 80, list(range(0, 65))),
    (256, 300, 33, 48, [0] * 128 + list(range(129))),
    (3, 20, 130, 96, [0, 0, 0, 0]),
    (1, 50, 130, 96, [0, 20]),
    (4, 30, 520, 2064, [0, 1, 1, 12, 30]),
    (3, 24, 33, 4112, [0, 8, 17, 24]),
    (8, 32, 200, 2048, [0, 0, 0, 0, 32, 32, 32, 32, 32]),
    (8, 32, 5, 2304, [0, 3, 4, 4, 4, 5, 6, 30, 31]),
    (1, 16, 40, 8208, [0, 13]),
    (3, 900, 2600, 1056, [0, 300, 301, 900]),
    (4, 1000, 1603, 1040, [0, 0, 640, 641, 950]),
    (2, 513, 2500, 1024, [0, 513, 513]),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_quantized_matmul_groups(case, dt):
    groups, rows, n, k, off = GROUPS[case]
    q, s, wq, ws = mm_inputs(rows, n, k, groups)
    out, st = run_mm(q, s, wq, ws, dt, off, fill=-7.0)
    assert st == 0
    check_mm(out, R.matmul(q, s, wq, ws, off), dt, -7.0)


def test_quantized_matmul_repairs_bad_offsets():
    """A step down and an end past the rows: a device status, and every row of
    the repaired (running maximum, clamped) groups as the definition has it."""
    for rows in (12, 300):
        q, s, wq, ws = mm_inputs(rows, 40, 64, 4)
        bad = [0, 7, 3, 9, rows + 50]
        out, st = run_mm(q, s, wq, ws, "f32", bad, fill=-7.0)
        assert st == L.MOE_ERR_DEVICE
        check_mm(out, R.matmul(q, s, wq, ws, [0, 7, 7, 9, rows]), "f32", -7.0)


def test_quantized_matmul_nan_rows_stay_apart():
    """A row quantised from a NaN gives a row of NaN; its neighbours are exact."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((200, 256), generator=g, device="cuda").to(torch.bfloat16)
    x[3, 100] = float("nan")
    x[150, 0] = float("-inf")
    xq, xs = quantize(x)
    wq, ws = quantize(torch.randn((72, 256), generator=g, device="cuda"))
    for rows in (4, 200):
        out = torch.zeros((rows, 72), device="cuda")
        w = torch.empty(api.moe_quantized_matmul_workspace_size(1, rows, 72, 256), dtype=torch.uint8, device="cuda")
        api.moe_quantized_matmul(xq[:rows], xs[:rows], wq, ws, out, w)
        ref = R.matmul(xq[:rows].cpu().numpy(), xs[:rows].cpu().double().numpy(), wq.cpu().numpy()[None],
                       ws.cpu().double().numpy()[None])
        bad = torch.isnan(xs[:rows]).cpu().numpy()
        assert bad.sum() == (1 if rows == 4 else 2)
        assert torch.isnan(out[torch.from_numpy(bad).cuda()]).all()
        check_mm(out[torch.from_numpy(~bad).cuda()], ref[~bad], "f32")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantized_matmul_bits_do_not_depend_on_the_batch(dt):
    """A row's result is the same bits in a batch of one, of sixteen, of a
    hundred and of a thousand rows, which run in different kernels."""
    q, s, wq, ws = mm_inputs(1000, 2312, 1040)
    full, st = run_mm(q, s, wq, ws, dt)
    assert st == 0
    for rows in (1, 16, 100):
        part, st = run_mm(q[:rows], s[:rows], wq, ws, dt)
        assert st == 0 and torch.equal(part, full[:rows])


def test_quantized_matmul_no_rows():
    w = torch.full((256,), 0xA5, dtype=torch.uint8, device="cuda")
    e8 = lambda *s: torch.zeros(s, dtype=torch.int8, device="cuda")
    api.moe_quantized_matmul(e8(0, 64), torch.zeros(0, device="cuda"), e8(8, 64), torch.ones(8, device="cuda"),
                             torch.zeros((0, 8), device="cuda"), w)
    assert api.moe_workspace_status(w) == 0


def test_quantized_matmul_streams_and_graph():
    """The same call on another stream and replayed from a graph with new
    inputs in the same buffers."""
    q, s, wq, ws = mm_inputs(150, 264, 272, 3)
    off = torch.tensor([0, 40, 41, 150], dtype=torch.int32, device="cuda")
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    tq, ts, twq, tws = d(q), d(s), d(wq), d(ws)
    out = torch.zeros((150, 264), device="cuda")
    w = torch.empty(api.moe_quantized_matmul_workspace_size(3, 150, 264, 272), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.moe_quantized_matmul(tq, ts, twq, tws, out, w, group_offsets=off, stream=side)
    side.synchronize()
    check_mm(out, R.matmul(q, s, wq, ws, off.tolist()), "f32")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_quantized_matmul(tq, ts, twq, tws, out, w, group_offsets=off)
    for seed in (1, 2):
        q2, s2, _, _ = mm_inputs(150, 264, 272, 3, seed)
        tq.copy_(d(q2))
        ts.copy_(d(s2))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check_mm(out, R.matmul(q2, s2, wq, ws, off.tolist()), "f32")


# ---------------------------------------------------------------- the layer with 8-bit experts

LAYER = {
    "small_swiglu": workload("mixtral_prefill", T=200, d=256, F=320, E=8, k=2),
    "ragged": workload("mixtral_prefill", T=333, d=208, F=144, E=4, k=3),
    "relu_drops": workload("switch_top1", T=257, d=144, F=272, E=8, k=2, capacity_factor=1.25),
    "top1_skew": workload("switch_top1", T=600, d=128, F=256, E=16, k=1),
    "one_token": workload("mixtral_prefill", T=1, d=128, F=256, E=4, k=2),
    "groups_shared": workload("deepseek_v3", T=300, d=448, F=256, E=32, n_group=8, topk_group=4, shared_F=256),
    "many_experts": workload("mixtral_prefill", T=64, d=512, F=192, E=128, k=8),
    "few_rows": workload("mixtral_prefill", T=9, d=1040, F=528, E=6, k=2),
    "few_long_rows": workload("mixtral_prefill", T=5, d=2320, F=2064, E=4, k=3),
    "large_groups": workload("mixtral_prefill", T=900, d=1040, F=1056, E=4, k=2),
    "large_relu": workload("switch_top1", T=1500, d=1040, F=1040, E=4, k=1, capacity_factor=1.25),
    "few_relu": workload("switch_top1", T=14, d=2064, F=208, E=4, k=1, capacity_factor=1.25),
}


class I8Run(Run):
    """Run with the dense weights replaced by their 8-bit codes."""

    def __init__(self, w, seed=0, fused=False):
        super().__init__(w, seed=seed)
        self.host = {}
        dense = dict(self.weights)
        for i in "123":
            t = dense.pop("w" + i, None)
            if t is not None:
                dense["w" + i], dense["s" + i] = quantize(t)
                self.host["w" + i], self.host["s" + i] = dense["w" + i].cpu().numpy(), dense["s" + i].cpu().numpy()
        if fused:
            dense["w1"] = torch.cat([dense["w1"], dense.pop("w2")], 1).contiguous()
            dense["s1"] = torch.cat([dense["s1"], dense.pop("s2")], 1).contiguous()
        self.weights = dense
        self.cfg.weight_dtype = L.MOE_I8_CHANNEL
        self.cfg.weight_layout = L.MOE_LAYOUT_FUSED_GATE_UP if fused else L.MOE_LAYOUT_SEPARATE
        n = api.moe_workspace_size(self.cfg)
        self.ws_full = torch.full((n + (1 << 16),), 0xA5, dtype=torch.uint8, device="cuda")
        self.ws = self.ws_full[:n]


def check_layer(run):
    """The output against float64 on the GPU's own routing.  y_perm and the
    output are bf16 (half a step each), the combine adds its k terms in fp32."""
    w = run.w
    x = as_f64(run.inp["x"])
    ids, wts = run.ids.cpu().numpy(), run.wts.cpu().numpy().astype(np.float64)
    slot = run.slot_row.cpu().numpy()
    out, bound = np.zeros((w.T, w.d)), np.zeros((w.T, w.d))
    for e in range(w.E):
        t, j = np.nonzero((ids == e) & (slot >= 0))
        if not t.size:
            continue
        y, b = R.expert_ffn(x[t], {k: v[e] for k, v in run.host.items()}, w.act)
        np.add.at(out, t, y * wts[t, j][:, None])
        np.add.at(bound, t, (b + (R.BF16_HALF_STEP + 40 * R.F32_HALF_STEP) * (np.abs(y) + b)) * wts[t, j][:, None])
    if w.shared_F:
        s = {i: as_f64(run.weights["ws" + i]) for i in "123"}
        h = R.silu(x @ s["1"].T) * (x @ s["2"].T)
        y = h @ s["3"].T
        # bf16 intermediate (summed in magnitude), bf16 output, fp32 sums over d and F terms
        b = (R.BF16_HALF_STEP + 1e-4) * (np.abs(h) @ np.abs(s["3"]).T) + R.BF16_HALF_STEP * np.abs(y)
        out, bound = out + y, bound + b
    bound = bound + R.BF16_HALF_STEP * (np.abs(out) + bound)
    got = as_f64(run.out)
    assert (np.abs(got - out) - bound).max() <= 0.0, (np.abs(got - out) / np.maximum(bound, 1e-30)).max()


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("name", sorted(LAYER))
def test_layer_with_8_bit_experts(name, fused):
    w = LAYER[name]
    if fused and w.act == "relu":
        pytest.skip("the fused gate/up layout needs two projections")
    run = I8Run(w, seed=31, fused=fused)
    run.staged()
    assert run.status() == 0
    check_route(run, oracle_route(w, run.inp), max_unsafe_fraction=0.35)
    check_dispatch(run)
    check_layer(run)
    staged = run.out.clone()
    run.fill_canary()
    run.forward()
    assert run.status() == 0
    assert torch.equal(run.out.view(torch.int16), staged.view(torch.int16))
    assert (run.ws_full[run.ws.numel():] == 0xA5).all()


def test_layer_8_bit_ffn_leaves_rows_behind_the_last_group():
    w = LAYER["relu_drops"]
    run = I8Run(w, seed=32).staged()
    n = int(run.offsets[-1])
    assert n < w.T * w.k
    run.fill_canary()
    api.moe_permute(run.cfg, run.inp["x"], run.ids, run.wts, run.offsets, run.perm_token, run.perm_w, run.slot_row,
                    run.x_perm, run.stats, run.ws)
    api.moe_grouped_ffn(run.cfg, run.x_perm, run.offsets, run.weights, run.y_perm, run.ws)
    torch.cuda.synchronize()
    assert run.status() == 0
    full, rows = run.guarded["y_perm"]
    assert (full.view(torch.uint8)[n:] == 0xA5).all()


def test_layer_8_bit_bad_offsets_are_reported():
    w = LAYER["small_swiglu"]
    run = I8Run(w, seed=33).staged()
    bad = run.offsets.clone()
    bad[3] = min(int(bad[5]) + 7, w.T * w.k)
    api.moe_grouped_ffn(run.cfg, run.x_perm, bad, run.weights, run.y_perm, run.ws)
    torch.cuda.synchronize()
    assert run.status() == L.MOE_ERR_DEVICE


def test_layer_8_bit_in_a_graph():
    """MoELayer.forward captured and replayed on new tokens gives the eager bits."""
    w = LAYER["groups_shared"]
    run = I8Run(w, seed=34)
    layer = api.MoELayer(run.cfg, run.inp["w_router"], run.weights, router_bias=router_bias_of(w, run.inp))
    x = run.inp["x"]
    layer.forward(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x)
    g = torch.Generator(device="cuda").manual_seed(3)
    for _ in range(2):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16))
        layer.forward(x)
        eager = layer.o.out.clone()
        layer.o.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.o.out.view(torch.int16), eager.view(torch.int16))
        assert layer.status() == 0


@pytest.mark.parametrize("sizes", [dict(T=700, d=512, F=640), dict(T=900, d=1040, F=1056, E=4)])
def test_layer_8_bit_barrier_timeout_reports_and_recovers(sizes):
    """A 1 ns bound on the barrier waits makes the product give up: a device
    status, and the context and workspace stay good.  On one SM a tile, and on
    pairs of SMs."""
    w = workload("mixtral_prefill", **sizes)
    run = I8Run(w, seed=35).staged()
    try:
        api.moe_set_wait_timeout_ns(1)
        api.moe_grouped_ffn(run.cfg, run.x_perm, run.offsets, run.weights, run.y_perm, run.ws)
        st = run.status()
    finally:
        api.moe_set_wait_timeout_ns(0)
    assert st == L.MOE_ERR_DEVICE
    run.staged()
    assert run.status() == 0
    check_layer(run)


def test_quantized_calls_refuse_tensors_elsewhere():
    """A tensor left on the host is refused before any launch, whichever it is."""
    q = torch.zeros((4, 32), dtype=torch.int8, device="cuda")
    args = [torch.zeros((4, 32), device="cuda"), q, torch.zeros(4, device="cuda")]
    for i in range(3):
        with pytest.raises(ValueError, match="current CUDA device"):
            api.moe_quantize_rows(*(a.cpu() if j == i else a for j, a in enumerate(args)))
    args = [q, torch.zeros(4, device="cuda"), torch.zeros((2, 8, 32), dtype=torch.int8, device="cuda"),
            torch.zeros((2, 8), device="cuda"), torch.zeros((4, 8), device="cuda"),
            torch.zeros(4096, dtype=torch.uint8, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")]
    for i in range(7):
        with pytest.raises(ValueError, match="current CUDA device"):
            api.moe_quantized_matmul(*(a.cpu() if j == i else a for j, a in enumerate(args)))


def test_quantized_matmul_calls_at_once():
    """A large product on one stream and many small ones on another, a
    workspace each: the bits of the calls one after the other."""
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    calls = []
    for rows, n, k in ((1090, 2312, 1040), (5, 520, 2320)):
        q, s, wq, ws = (d(a) for a in mm_inputs(rows, n, k))
        w = torch.empty(api.moe_quantized_matmul_workspace_size(1, rows, n, k), dtype=torch.uint8, device="cuda")
        calls.append((q, s, wq, ws, torch.zeros((rows, n), device="cuda"), w))
    want = []
    for c in calls:
        api.moe_quantized_matmul(*c)
        want.append(c[4].clone())
        c[4].zero_()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        api.moe_quantized_matmul(*calls[0], stream=streams[0])
        for _ in range(5):
            api.moe_quantized_matmul(*calls[1], stream=streams[1])
    torch.cuda.synchronize()
    for c, out in zip(calls, want):
        assert api.moe_workspace_status(c[5]) == 0
        assert torch.equal(c[4], out)
