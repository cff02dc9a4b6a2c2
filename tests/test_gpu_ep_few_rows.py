"""Expert parallelism whose ranks receive few rows: the rows' own workspace need
is below that of the largest batch, for every weight type.  One GPU, both
shards in one process."""
from __future__ import annotations

import pytest
import torch

from gpu_harness import Run
from mixture_experts_layer_41_b200 import api, ep
from mixture_experts_layer_41_b200.inputs import workload
from test_gpu_int8 import I8Run

pytestmark = pytest.mark.gpu

WORLD = 2
CASES = {
    # 9 tokens a rank, one expert each: at most 18 rows, about 9 to a rank
    "bf16": ("bf16", workload("mixtral_prefill", T=9, d=256, F=384, E=8, k=1)),
    "i8": ("i8", workload("mixtral_prefill", T=9, d=256, F=384, E=8, k=1)),
    "q4": ("q4", workload("decode_q4", T=9, d=256, F=384, E=8, k=1)),
    "i8_one_token": ("i8", workload("mixtral_prefill", T=1, d=256, F=384, E=8, k=2)),
    "i8_shared": ("i8", workload("deepseek_v3", T=40, d=256, F=128, E=32, n_group=8, topk_group=4, shared_F=128)),
    "i8_relu_drops": ("i8", workload("switch_top1", T=64, d=256, F=272, E=16, k=2, capacity_factor=1.0)),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_expert_parallel_few_rows(name, monkeypatch):
    """Each shard's output is that of the whole layer on its tokens, bit for
    bit (the rows' products do not depend on the rows beside them)."""
    kind, w = CASES[name]
    monkeypatch.setenv("MOE_Q4_KERNEL", "mma")
    runs = [I8Run(w, seed=r) if kind == "i8" else Run(w, seed=r) for r in range(WORLD)]
    base, e_local = runs[0], w.E // WORLD
    shards = []
    for r in range(WORLD):
        local = {k: v[r * e_local:(r + 1) * e_local] if not k.startswith("ws") else v for k, v in base.weights.items()}
        shards.append(ep.DeviceOps(base.cfg, base.inp["w_router"], local, WORLD, router_bias=base.bias,
                                   device=torch.device("cuda")))
    outs = ep.emulate(shards, [run.inp["x"] for run in runs])
    torch.cuda.synchronize()
    layer = api.MoELayer(base.cfg, base.inp["w_router"], base.weights, router_bias=base.bias)
    for run, shard, out in zip(runs, shards, outs):
        assert shard.status() == 0
        ref = layer.forward(run.inp["x"]).out
        torch.cuda.synchronize()
        assert layer.status() == 0
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
