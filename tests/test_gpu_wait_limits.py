"""Barrier waits that run out at different points of the tensor-core kernels and
of the few-token kernel.

Under a limit between 1 ns and a few tens of us a call gives up early, in the
middle, or not at all.  Whatever it does, it has to say so (a status, or the
right bits), let what it has under way land, and return long before any of its
drains runs out; the next call under the default limit has to be right."""
from __future__ import annotations

import os
import subprocess
import sys
import time

import numpy as np
import pytest
import torch

from gpu_harness import Run
from mixture_experts_layer_41_b200 import _lib as L
from mixture_experts_layer_41_b200 import api
from mixture_experts_layer_41_b200.inputs import workload
from test_gpu_few import make_run
from test_gpu_int8 import I8Run, mm_inputs

pytestmark = pytest.mark.gpu

LIMITS_NS = (1, 200, 1000, 2000, 4000, 8000, 16000, 32000)
DRAIN_S = 0.2          # one drain that runs out takes this long


def i8_product(rows, n, k, groups=1, offsets=None):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    q, s, wq, ws = (d(a) for a in mm_inputs(rows, n, k, groups))
    out = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")
    ws8 = torch.empty(api.moe_quantized_matmul_workspace_size(groups, rows, n, k), dtype=torch.uint8, device="cuda")
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    return lambda: api.moe_quantized_matmul(q, s, wq, ws, out, ws8, group_offsets=off), out, ws8


def ffn(run):
    run.staged()
    assert run.status() == 0
    call = lambda: api.moe_grouped_ffn(run.cfg, run.x_perm, run.offsets, run.weights, run.y_perm, run.ws)
    return call, run.y_perm, run.ws


def route(w):
    run = Run(w, seed=35)
    call = lambda: api.moe_route(run.cfg, run.inp["x"], run.inp["w_router"], run.bias, run.ids, run.wts, run.prob_sum,
                                 run.ws)
    return call, run.wts, run.ws


def gather(w):
    """The whole layer with its rows gathered inside the product (below 512 tokens no router waits)."""
    run = Run(w, seed=35)
    run.cfg.fused_gather = 1
    call = lambda: api.moe_forward(run.cfg, run.inp["x"], run.inp["w_router"], run.bias, run.weights, run.out, run.ids,
                                   run.wts, run.stats, run.ws)
    return call, run.out, run.ws


def few(name):
    """The few-token kernel: a block that gives up goes on with what it finds, in bounds."""
    run = make_run(name)
    call = lambda: api.moe_forward_few(run.cfg, run.inp["x"], run.inp["w_router"], run.bias, run.weights, run.out, run.ids,
                                       run.wts, run.stats, run.ws)
    return call, run.out, run.ws


CALLS = {
    # 8-bit product on pairs of SMs: one group, ragged groups (last tiles of 64 to 256 tokens), SwiGLU
    "i8_pair": lambda: i8_product(1090, 2312, 2320),
    "i8_pair_groups": lambda: i8_product(1100, 1544, 1040, 4, [0, 300, 310, 900, 1100]),
    "i8_pair_swiglu": lambda: ffn(I8Run(workload("mixtral_prefill", T=900, d=1040, F=1056, E=4), seed=35)),
    "bf16_pair": lambda: ffn(Run(workload("mixtral_prefill", T=1100, d=1032, F=1160, E=4), seed=35)),
    "bf16_pair_relu": lambda: ffn(Run(workload("switch_top1", T=1300, d=1032, F=1160, E=4, capacity_factor=0.0), seed=35)),
    # one SM a tile: 256, 128 and 64 columns, fewer K-blocks than stages, and a layer
    "i8_256": lambda: i8_product(1500, 3080, 1008),
    "i8_128": lambda: i8_product(1100, 2312, 1008),
    "i8_64": lambda: i8_product(100, 520, 4112),
    "i8_short": lambda: i8_product(700, 2312, 80),
    "i8_swiglu": lambda: ffn(I8Run(workload("mixtral_prefill", T=700, d=512, F=640), seed=35)),
    "bf16": lambda: ffn(Run(workload("mixtral_prefill", T=1100, d=1032, F=1160, E=4), seed=35)),
    "bf16_short": lambda: ffn(Run(workload("switch_top1", T=700, d=72, F=136, E=4, capacity_factor=0.0), seed=35)),
    "bf16_gather": lambda: gather(workload("mixtral_prefill", T=500, d=1032, F=1160, E=4)),
    "q4_tc": lambda: ffn(Run(workload("decode_q4", T=200, d=2048, F=1024, E=8, k=2), seed=35)),
    "q4_tc_short": lambda: ffn(Run(workload("decode_q4", T=200, d=128, F=128, E=8, k=2), seed=35)),
    "few_bf16": lambda: few("groups_shared"),
    "few_bf16_long": lambda: few("long_reduction"),
    "few_i8": lambda: few("i8_many_experts"),
    "few_q4": lambda: few("q4_decode"),
    "router_i8": lambda: route(workload("deepseek_v3", T=1024, d=2048, F=64, shared_F=0)),
    "router_bf16": lambda: route(workload("deepseek_v3", T=1024, d=2048, F=64, shared_F=0)),
}
OTHER_PROCESS = {"router_bf16"}     # its environment is read once per process

# the environment that selects a kernel
ENV = {"bf16_pair": {"MOE_TC_PAIR": "1"}, "bf16_pair_relu": {"MOE_TC_PAIR": "1"}, "q4_tc": {"MOE_Q4_KERNEL": "tc"},
       "q4_tc_short": {"MOE_Q4_KERNEL": "tc"}, "router_bf16": {"MOE_ROUTER_TC": "bf16"}}


def timed(call, ws):
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    return time.perf_counter() - t0, api.moe_workspace_status(ws)


def check(name):
    bits = lambda t: t.view(torch.int16)
    call, out, ws = CALLS[name]()
    assert timed(call, ws)[1] == 0
    want = out.clone()
    gave_up = slow = 0
    for limit in LIMITS_NS:
        for _ in range(6):
            out.zero_()
            api.moe_set_wait_timeout_ns(limit)
            try:
                seconds, status = timed(call, ws)
            finally:
                api.moe_set_wait_timeout_ns(0)
            slow += seconds >= DRAIN_S
            if status == 0:
                assert torch.equal(bits(out), bits(want)), limit
            else:
                assert status == L.MOE_ERR_DEVICE, (limit, status)
                text = L.lib().moe_last_error().decode()
                assert "timed out" in text, (limit, text)
                gave_up += 1
        assert timed(call, ws)[1] == 0
        assert torch.equal(bits(out), bits(want)), limit
    assert gave_up >= 1
    assert slow <= 1, slow         # (the host may have paused once)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_waits_that_run_out(name, monkeypatch):
    for key, value in ENV.get(name, {}).items():
        monkeypatch.setenv(key, value)
    if name not in OTHER_PROCESS:
        check(name)
        return
    tests = os.path.dirname(os.path.abspath(__file__))
    code = (f"import sys; sys.path[:0] = [{os.path.dirname(tests)!r}, {tests!r}]\n"
            f"import test_gpu_wait_limits as t; t.check({name!r}); print('checked')")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "checked" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
