"""The layer calls refuse tensors that do not fit the config, before the library
reads or writes past their ends or takes one type for another (no GPU)."""
import pytest
import torch

from mixture_experts_layer_41_b200 import _lib as L
from mixture_experts_layer_41_b200 import api

T, D, F, E, K = 16, 64, 128, 8, 2
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
FORMATS = {"bf16": "bf16", "i8": "i8_channel", "q4": "q4_affine_g64"}


class Called(Exception):
    pass


@pytest.fixture(autouse=True)
def library(monkeypatch):
    """A library whose calls only say that the checks were passed."""
    class Stub:
        def __getattr__(self, name):
            def call(*args):
                raise Called(name)
            return call
    monkeypatch.setattr(api, "_have_gpu", lambda: False)
    monkeypatch.setattr(L, "lib", lambda: Stub())


def weights(kind, fused=False, relu=False, shared=0):
    w, rows = {}, {"1": 2 * F if fused else F, "2": F, "3": D}
    for i in "123":
        if i == "2" and (fused or relu):
            continue
        n, k = rows[i], F if i == "3" else D
        if kind == "bf16":
            w["w" + i] = torch.zeros((E, n, k), dtype=BF)
        elif kind == "i8":
            w["w" + i], w["s" + i] = torch.zeros((E, n, k), dtype=torch.int8), torch.zeros((E, n))
        else:
            w["w" + i] = torch.zeros((E, n, k // 8), dtype=I32)
            w["s" + i], w["b" + i] = (torch.zeros((E, n, k // 64), dtype=BF) for _ in "sb")
    if shared:
        w.update(ws1=torch.zeros((shared, D), dtype=BF), ws2=torch.zeros((shared, D), dtype=BF),
                 ws3=torch.zeros((D, shared), dtype=BF))
    return w


def arguments(kind="bf16", **kw):
    cfg = api.make_config(num_tokens=T, hidden=D, intermediate=F, num_experts=E, top_k=K, weight_dtype=FORMATS[kind],
                          weight_layout="fused_gate_up" if kw.get("fused") else "separate",
                          act="relu" if kw.get("relu") else "swiglu", shared_intermediate=kw.get("shared", 0))
    return dict(cfg=cfg, x=torch.zeros((T, D), dtype=BF), w_router=torch.zeros((E, D)), router_bias=torch.zeros(E),
                weights=weights(kind, **kw), out=torch.zeros((T, D), dtype=BF), topk_ids=torch.zeros((T, K), dtype=I32),
                topk_w=torch.zeros((T, K)),
                stats=dict(raw_counts=torch.zeros(E, dtype=I32), kept_counts=torch.zeros(E, dtype=I32),
                           prob_sum=torch.zeros(E), dropped=torch.zeros(4, dtype=I32)),
                ws=torch.zeros(64, dtype=torch.uint8), stream=0)


@pytest.mark.parametrize("kind", sorted(FORMATS))
@pytest.mark.parametrize("kw", [{}, dict(fused=True), dict(relu=True), dict(shared=64)])
def test_fitting_tensors_reach_the_library(kind, kw):
    with pytest.raises(Called, match="moe_forward_few"):
        api.moe_forward_few(**arguments(kind, **kw))
    a = arguments(kind, **kw)
    a.update(router_bias=None, topk_ids=None, topk_w=None, stats=None)
    with pytest.raises(Called, match="moe_forward_few"):
        api.moe_forward_few(**a)
    with pytest.raises(Called, match="moe_forward"):
        api.moe_forward(**arguments(kind, **kw))


@pytest.mark.parametrize("name,bad", [
    ("x", torch.zeros((4, D), dtype=BF)), ("x", torch.zeros((T, D))), ("x", torch.zeros((T, D), dtype=torch.float16)),
    ("x", torch.zeros((T + 1, D), dtype=BF)), ("out", torch.zeros((4, D), dtype=BF)), ("out", torch.zeros((T, D))),
    ("out", torch.zeros((2 * T, D), dtype=BF)), ("w_router", torch.zeros((E, D), dtype=BF)),
    ("w_router", torch.zeros((E - 1, D))), ("router_bias", torch.zeros(E - 1)),
    ("router_bias", torch.zeros(E, dtype=torch.float64)), ("topk_ids", torch.zeros((T, K), dtype=torch.int64)),
    ("topk_ids", torch.zeros((4, K), dtype=I32)), ("topk_w", torch.zeros((T, K), dtype=BF)), ("topk_w", torch.zeros((4, K))),
])
def test_few_refuses_a_tensor_that_does_not_fit(name, bad):
    a = arguments()
    a[name] = bad
    with pytest.raises(ValueError, match=name):
        api.moe_forward_few(**a)


@pytest.mark.parametrize("name,bad", [("raw_counts", torch.zeros(E)), ("kept_counts", torch.zeros(E - 1, dtype=I32)),
                                      ("prob_sum", torch.zeros(E, dtype=I32)), ("dropped", torch.zeros(0, dtype=I32))])
def test_few_refuses_stats_that_do_not_fit(name, bad):
    a = arguments()
    a["stats"][name] = bad
    with pytest.raises(ValueError, match=name):
        api.moe_forward_few(**a)


@pytest.mark.parametrize("kind", sorted(FORMATS))
@pytest.mark.parametrize("fused", [False, True])
def test_few_refuses_weights_that_do_not_fit(kind, fused):
    for name in weights(kind, fused, shared=64):
        for change in (lambda t: t[:-1].contiguous(), lambda t: t.to(torch.float64)):
            a = arguments(kind, fused=fused, shared=64)
            a["weights"][name] = change(a["weights"][name])
            with pytest.raises(ValueError, match=name):
                api.moe_forward_few(**a)
    # weights of another type than the config's
    a = arguments(kind, fused=fused)
    a["weights"] = weights("bf16" if kind != "bf16" else "i8", fused)
    with pytest.raises(ValueError, match="w1"):
        api.moe_forward_few(**a)


@pytest.mark.parametrize("name", ["x", "out"])
def test_forward_refuses_rows_that_do_not_fit(name):
    for bad in (torch.zeros((4, D), dtype=BF), torch.zeros((T, D)), torch.zeros((T, D), dtype=torch.float16)):
        a = arguments()
        a[name] = bad
        with pytest.raises(ValueError, match=name):
            api.moe_forward(**a)
    a = arguments()
    a[name] = torch.zeros((T + 4, D), dtype=BF)         # a larger buffer: its first rows, as ever
    with pytest.raises(Called):
        api.moe_forward(**a)
