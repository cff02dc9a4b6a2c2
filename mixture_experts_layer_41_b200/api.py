"""Python face of the C ABI in include/moe.h: the same calls, same names.

Each function converts torch tensors to raw pointers and forwards to
libmoe.so; every step of the layer runs in the library's kernels.  torch is
used for device memory and streams only.  Output tensors are caller-owned,
as in C; ``MoELayer`` is a convenience holder that allocates them.
"""
from __future__ import annotations

import ctypes as C
import functools
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib as L
from ._lib import check, moe_config, moe_stats, moe_weights

_ROUTERS = {"softmax_topk": L.MOE_ROUTER_SOFTMAX_TOPK, "sigmoid_group": L.MOE_ROUTER_SIGMOID_GROUP}
_ACTS = {"relu": L.MOE_ACT_RELU, "swiglu": L.MOE_ACT_SWIGLU}
_DTYPES = {"f32": L.MOE_F32, "bf16": L.MOE_BF16, "q4_affine_g64": L.MOE_Q4_AFFINE_G64,
           "i8_channel": L.MOE_I8_CHANNEL}
_TORCH_DT = {L.MOE_F32: torch.float32, L.MOE_BF16: torch.bfloat16}
_MOE_DT = {v: k for k, v in _TORCH_DT.items()}
_LAYOUTS = {"separate": L.MOE_LAYOUT_SEPARATE, "fused_gate_up": L.MOE_LAYOUT_FUSED_GATE_UP}


def make_config(*, num_tokens: int, hidden: int, intermediate: int, num_experts: int, top_k: int,
                router: str = "softmax_topk", norm_topk_prob: bool = True, routed_scaling: float = 1.0,
                n_group: int = 1, topk_group: int = 1, capacity_factor: float = 0.0,
                act: str = "swiglu", act_dtype: str = "bf16", weight_dtype: str = "bf16",
                shared_intermediate: int = 0, aux_alpha: float = 0.01,
                weight_layout: str = "separate", fused_gather: bool = False) -> moe_config:
    return moe_config(num_tokens, hidden, intermediate, num_experts, top_k, _ROUTERS[router],
                      1 if norm_topk_prob else 0, routed_scaling, n_group, topk_group,
                      capacity_factor, _ACTS[act], _DTYPES[act_dtype], _DTYPES[weight_dtype],
                      shared_intermediate, aux_alpha, _LAYOUTS[weight_layout], 1 if fused_gather else 0)


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    return t.data_ptr()


# The current stream's handle alone: building torch's Stream object costs 8 us a
# call, this 0.3 us.  Private to torch: None in a release that lacks them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _s(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None and _raw_device is not None and torch.cuda.is_initialized():
            return _raw_stream(_raw_device())
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


@functools.lru_cache(maxsize=None)
def _have_gpu() -> bool:
    return torch.cuda.is_available()


def _on_current(*tensors) -> None:
    """Refuses tensors that are not on the current device: a kernel launched
    there cannot be expected to read them."""
    if not _have_gpu():
        return
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors must be on the current CUDA device (cuda:{dev}); got one on {t.device}")


def _holds(needs) -> None:
    """Refuses tensors of another type than the call takes them for, or with
    fewer elements than it reads or writes: ``needs`` are (name, tensor, type,
    elements).  A missing tensor passes: the library knows which may be."""
    for name, t, dtype, n in needs:
        if t is not None and (t.dtype is not dtype or t.numel() < n):
            raise ValueError(f"{name} must be {dtype} with {n} elements for this config, not {t.dtype} with {t.numel()}")


def _check_rows(cfg, x, out) -> None:
    """The token rows of a layer call: [num_tokens, hidden] of the activations' type."""
    dt, n = _TORCH_DT.get(cfg.act_dtype), cfg.num_tokens * cfg.hidden
    if dt is not None:                                  # (else no valid config: the library says so)
        _holds((("x", x, dt, n), ("out", out, dt, n)))


def _check_few(cfg, x, w_router, router_bias, weights: dict, out, topk_ids, topk_w, stats) -> None:
    """Every tensor of a few-token call (bf16 activations)."""
    T, d, F, E, k, Fs = (cfg.num_tokens, cfg.hidden, cfg.intermediate, cfg.num_experts, cfg.top_k,
                         cfg.shared_intermediate)
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    w, st = weights.get, (stats or {}).get
    n = E * F * d
    n1 = 2 * n if cfg.weight_layout == L.MOE_LAYOUT_FUSED_GATE_UP else n
    relu, fmt = cfg.act == L.MOE_ACT_RELU, cfg.weight_dtype
    w1, w2, w3 = w("w1"), None if relu else w("w2"), w("w3")
    needs = [("x", x, bf16, T * d), ("out", out, bf16, T * d), ("w_router", w_router, f32, E * d),
             ("router_bias", router_bias, f32, E), ("topk_ids", topk_ids, i32, T * k), ("topk_w", topk_w, f32, T * k)]
    if stats is not None:
        needs += [("raw_counts", st("raw_counts"), i32, E), ("kept_counts", st("kept_counts"), i32, E),
                  ("prob_sum", st("prob_sum"), f32, E), ("dropped", st("dropped"), i32, 1)]
    if fmt == L.MOE_BF16:
        needs += [("w1", w1, bf16, n1), ("w2", w2, bf16, n), ("w3", w3, bf16, n)]
    elif fmt == L.MOE_I8_CHANNEL:
        needs += [("w1", w1, torch.int8, n1), ("w2", w2, torch.int8, n), ("w3", w3, torch.int8, n),
                  ("s1", w("s1"), f32, n1 // d), ("s2", None if relu else w("s2"), f32, E * F), ("s3", w("s3"), f32, E * d)]
    else:
        for name, t, codes in (("w1", w1, n1), ("w2", w2, n), ("w3", w3, n)):       # in words of any width
            if t is not None and (t.is_floating_point() or 2 * _nbytes(t) < codes):
                raise ValueError(f"{name} must hold {codes} 4-bit codes in integer words, not {tuple(t.shape)} of {t.dtype}")
        needs += [(p + i, w(p + i), bf16, g // 64) for p in "sb" for i, g in (("1", n1), ("2", n), ("3", n))]
    if Fs > 0:
        needs += [("ws1", w("ws1"), bf16, Fs * d), ("ws2", w("ws2"), bf16, Fs * d), ("ws3", w("ws3"), bf16, Fs * d)]
    _holds(needs)
    for name, t, n in (("x", x, T), ("out", out, T)):
        if t is not None and t.numel() != n * d:
            raise ValueError(f"{name} must be [{n}, {d}] for this config, not {tuple(t.shape)}")


# ---------------------------------------------------------------- host-only calls

def moe_capacity(num_tokens: int, top_k: int, num_experts: int, capacity_factor: float) -> int:
    return L.lib().moe_capacity(num_tokens, top_k, num_experts, capacity_factor)


def moe_validate(cfg: moe_config) -> int:
    return L.lib().moe_validate(C.byref(cfg))


def moe_workspace_size(cfg: moe_config) -> int:
    return L.lib().moe_workspace_size(C.byref(cfg))


def moe_aux_loss(cfg: moe_config, kept_counts_host: torch.Tensor, prob_sum_host: torch.Tensor):
    raw, scaled = C.c_double(), C.c_double()
    kc = kept_counts_host.to(torch.int32).contiguous()
    ps = prob_sum_host.to(torch.float32).contiguous()
    check(L.lib().moe_aux_loss(C.byref(cfg), kc.data_ptr(), ps.data_ptr(), C.byref(raw), C.byref(scaled)),
          "moe_aux_loss")
    return raw.value, scaled.value


def moe_routing_health(cfg: moe_config, kept_counts_host: torch.Tensor, dropped: int) -> dict:
    er, ms, df, col = C.c_double(), C.c_double(), C.c_double(), C.c_int32()
    kc = kept_counts_host.to(torch.int32).contiguous()
    check(L.lib().moe_routing_health(C.byref(cfg), kc.data_ptr(), int(dropped), C.byref(er), C.byref(ms),
                                     C.byref(df), C.byref(col)), "moe_routing_health")
    return dict(entropy_ratio=er.value, max_share=ms.value, dropped_fraction=df.value,
                collapsed=bool(col.value))


def moe_kernel_launches() -> int:
    """Kernels the library has launched in this process so far."""
    return L.lib().moe_kernel_launches()


def moe_set_wait_timeout_ns(ns: int) -> None:
    """Bound on the tensor-core kernels' barrier waits (0: the 2 s default)."""
    check(L.lib().moe_set_wait_timeout_ns(int(ns)), "moe_set_wait_timeout_ns")


def moe_status_string(status: int) -> str:
    return L.lib().moe_status_string(status).decode()


def moe_set_phase_events(events) -> None:
    """Register MOE_PHASE_COUNT torch.cuda.Event objects (or None to turn it off)."""
    if events is None:
        check(L.lib().moe_set_phase_events(None, 0), "moe_set_phase_events")
        return
    for e in events:
        if not e.cuda_event:
            raise ValueError("record each event once before registering it (torch creates it lazily)")
    arr = (C.c_void_p * len(events))(*[e.cuda_event for e in events])
    check(L.lib().moe_set_phase_events(arr, len(events)), "moe_set_phase_events")


def moe_workspace_status(ws: torch.Tensor, stream=None) -> int:
    return L.lib().moe_workspace_status(_p(ws), _s(stream))


_REGIONS = {"offsets": L.MOE_WS_OFFSETS, "perm_token": L.MOE_WS_PERM_TOKEN, "perm_w": L.MOE_WS_PERM_W,
            "slot_row": L.MOE_WS_SLOT_ROW, "x_perm": L.MOE_WS_X_PERM, "h": L.MOE_WS_H, "y_perm": L.MOE_WS_Y_PERM,
            "shared_h": L.MOE_WS_SHARED_H, "shared_out": L.MOE_WS_SHARED_OUT,
            "router_logits": L.MOE_WS_ROUTER_LOGITS}


def moe_workspace_region(cfg: moe_config, region: str):
    """(byte offset, bytes) of one of moe_forward's intermediates inside the workspace."""
    off, n = C.c_size_t(), C.c_size_t()
    check(L.lib().moe_workspace_region(C.byref(cfg), _REGIONS[region], C.byref(off), C.byref(n)),
          "moe_workspace_region")
    return off.value, n.value


def workspace_view(cfg: moe_config, ws: torch.Tensor, region: str, dtype: torch.dtype, cols: int = 1):
    """A tensor view of one workspace region (no copy), [bytes / (cols * itemsize), cols]."""
    off, n = moe_workspace_region(cfg, region)
    return ws[off:off + n].view(dtype).view(-1, cols)


# ---------------------------------------------------------------- device calls

def _weights_struct(w: dict) -> moe_weights:
    g = lambda k: _p(w.get(k))
    return moe_weights(g("w1"), g("w2"), g("w3"), g("s1"), g("s2"), g("s3"), g("b1"), g("b2"), g("b3"),
                       g("ws1"), g("ws2"), g("ws3"))


def _stats_struct(stats: Optional[dict]) -> Optional[moe_stats]:
    if stats is None:
        return None
    g = lambda k: _p(stats.get(k))
    return moe_stats(g("raw_counts"), g("kept_counts"), g("prob_sum"), g("dropped"))


def moe_route(cfg, x, w_router, router_bias, topk_ids, topk_w, prob_sum, ws, stream=None):
    check(L.lib().moe_route(C.byref(cfg), _p(x), _p(w_router), _p(router_bias), _p(topk_ids), _p(topk_w),
                            _p(prob_sum), _p(ws), _nbytes(ws), _s(stream)), "moe_route")


def moe_route_forced(cfg, x, w_router, router_bias, forced_ids, topk_ids, topk_w, prob_sum, ws, stream=None):
    check(L.lib().moe_route_forced(C.byref(cfg), _p(x), _p(w_router), _p(router_bias), _p(forced_ids),
                                   _p(topk_ids), _p(topk_w), _p(prob_sum), _p(ws), _nbytes(ws), _s(stream)),
          "moe_route_forced")


def moe_update_bias(cfg, counts, expert_bias, coeff: float, stream=None):
    check(L.lib().moe_update_bias(C.byref(cfg), _p(counts), _p(expert_bias), coeff, _s(stream)),
          "moe_update_bias")


def moe_route_noalloc(cfg, x, w_router, router_bias, topk_ids, topk_w, prob_sum, stream=None):
    """moe_route for callers that cannot allocate: no workspace argument; the
    router's scratch is a fixed 1 MiB device array inside the library (see
    include/moe.h for the size limit and the rule that overlapping calls race)."""
    st = L.lib().moe_route_noalloc(C.byref(cfg), _p(x), _p(w_router), _p(router_bias), _p(topk_ids),
                                   _p(topk_w), _p(prob_sum), _s(stream))
    if st != L.MOE_OK:
        raise L.MoEError(st, "moe_route_noalloc: " + L.lib().moe_last_error().decode())


def moe_permute(cfg, x, topk_ids, topk_w, expert_offsets, perm_token, perm_w, slot_row, x_perm, stats, ws,
                stream=None):
    st = _stats_struct(stats)
    check(L.lib().moe_permute(C.byref(cfg), _p(x), _p(topk_ids), _p(topk_w), _p(expert_offsets),
                              _p(perm_token), _p(perm_w), _p(slot_row), _p(x_perm),
                              C.byref(st) if st is not None else None, _p(ws), _nbytes(ws), _s(stream)),
          "moe_permute")


def moe_expert_counts(cfg, topk_ids, raw_counts, ws, stream=None):
    check(L.lib().moe_expert_counts(C.byref(cfg), _p(topk_ids), _p(raw_counts), _p(ws), _nbytes(ws),
                                    _s(stream)), "moe_expert_counts")


def moe_permute_shard(cfg, x, topk_ids, topk_w, counts_by_rank, rank, capacity, expert_offsets, perm_token,
                      perm_w, slot_row, x_perm, stats, ws, stream=None):
    """``counts_by_rank``: [world, E] int32 device tensor of every shard's
    moe_expert_counts (``exchange_counts``), or None for a single shard."""
    st = _stats_struct(stats)
    world = 1 if counts_by_rank is None else int(counts_by_rank.shape[0])
    check(L.lib().moe_permute_shard(C.byref(cfg), _p(x), _p(topk_ids), _p(topk_w), _p(counts_by_rank), world,
                                    int(rank), int(capacity), _p(expert_offsets), _p(perm_token), _p(perm_w),
                                    _p(slot_row), _p(x_perm), C.byref(st) if st is not None else None, _p(ws),
                                    _nbytes(ws), _s(stream)),
          "moe_permute_shard")


def exchange_counts(raw_counts: torch.Tensor, group=None) -> torch.Tensor:
    """The sharded layer's one exchange: all-gather every rank's per-expert
    raw counts (an E-int32 message per rank) into a [world, E] tensor on the
    same device.  Token shards must be contiguous and in rank order."""
    import torch.distributed as dist
    world = dist.get_world_size(group)
    n = raw_counts.numel()
    gathered = torch.empty(world * n, dtype=raw_counts.dtype, device=raw_counts.device)
    dist.all_gather_into_tensor(gathered, raw_counts.reshape(-1).contiguous(), group=group)
    return gathered.view(world, n)


def moe_ep_local_ids(recv_counts, rows: int, ids, stream=None):
    """Local expert id of each received row (arrival order) from the
    [world, experts_per_rank] received counts."""
    world, e_local = recv_counts.shape
    check(L.lib().moe_ep_local_ids(_p(recv_counts), int(world), int(e_local), int(rows), _p(ids), _s(stream)),
          "moe_ep_local_ids")


def moe_grouped_ffn(cfg, x_perm, expert_offsets, weights: dict, y_perm, ws, stream=None):
    w = _weights_struct(weights)
    check(L.lib().moe_grouped_ffn(C.byref(cfg), _p(x_perm), _p(expert_offsets), C.byref(w), _p(y_perm),
                                  _p(ws), _nbytes(ws), _s(stream)), "moe_grouped_ffn")


def moe_quantize_rows(x, codes, scales, stream=None):
    """``x`` [..., cols] (bf16 or fp32) to int8 ``codes`` of the same shape and
    fp32 ``scales`` [...], one per row of the last axis."""
    if x.dtype not in _MOE_DT:
        raise ValueError("moe_quantize_rows takes float32 or bfloat16 rows")
    if codes.dtype != torch.int8 or codes.shape != x.shape:
        raise ValueError("codes must be an int8 tensor of x's shape")
    if scales.dtype != torch.float32 or scales.shape != x.shape[:-1]:
        raise ValueError("scales must be a float32 tensor with one element per row of x")
    _on_current(x, codes, scales)
    cols = x.shape[-1]
    check(L.lib().moe_quantize_rows(_p(x), _MOE_DT[x.dtype], scales.numel(), cols, _p(codes), _p(scales), _s(stream)),
          "moe_quantize_rows")


def moe_quantized_matmul_workspace_size(groups: int, rows: int, n: int, k: int) -> int:
    return L.lib().moe_quantized_matmul_workspace_size(groups, rows, n, k)


def moe_quantized_matmul(x_codes, x_scales, w_codes, w_scales, out, ws, group_offsets=None, stream=None):
    """``out[r] = x_scales[r] * w_scales[g] * (w_codes[g] @ x_codes[r])`` for
    the rows of each group.  ``w_codes`` [n, k] or [groups, n, k]; ``out``
    [rows, n] bf16 or fp32; ``group_offsets`` [groups + 1] int32, needed when
    there is more than one group."""
    if w_codes.dim() not in (2, 3):
        raise ValueError(f"w_codes must be [n, k] or [groups, n, k], not {tuple(w_codes.shape)}")
    groups = w_codes.shape[0] if w_codes.dim() == 3 else 1
    n, k = w_codes.shape[-2:]
    rows = x_codes.shape[0]
    if x_codes.dtype != torch.int8 or w_codes.dtype != torch.int8 or x_codes.shape != (rows, k):
        raise ValueError("codes must be int8: x_codes [rows, k], w_codes [n, k] or [groups, n, k]")
    if x_scales.dtype != torch.float32 or w_scales.dtype != torch.float32 or x_scales.numel() != rows \
            or w_scales.numel() != groups * n:
        raise ValueError("scales must be float32: x_scales [rows], w_scales [n] or [groups, n]")
    if out.dtype not in _MOE_DT or out.shape != (rows, n):
        raise ValueError("out must be a float32 or bfloat16 tensor [rows, n]")
    if group_offsets is not None and (group_offsets.dtype != torch.int32 or group_offsets.numel() != groups + 1):
        raise ValueError("group_offsets must be an int32 tensor [groups + 1]")
    _on_current(x_codes, x_scales, w_codes, w_scales, out, ws, group_offsets)
    check(L.lib().moe_quantized_matmul(groups, rows, n, k, _p(x_codes), _p(x_scales), _p(group_offsets), _p(w_codes),
                                       _p(w_scales), _MOE_DT[out.dtype], _p(out), _p(ws), _nbytes(ws), _s(stream)),
          "moe_quantized_matmul")


def moe_shared_expert(cfg, x, weights: dict, shared_out, ws, stream=None):
    w = _weights_struct(weights)
    check(L.lib().moe_shared_expert(C.byref(cfg), _p(x), C.byref(w), _p(shared_out), _p(ws), _nbytes(ws),
                                    _s(stream)), "moe_shared_expert")


def moe_combine(cfg, y_perm, slot_row, topk_w, shared_out, out, stream=None):
    check(L.lib().moe_combine(C.byref(cfg), _p(y_perm), _p(slot_row), _p(topk_w), _p(shared_out), _p(out),
                              _s(stream)), "moe_combine")


def moe_forward(cfg, x, w_router, router_bias, weights: dict, out, topk_ids, topk_w, stats, ws, stream=None):
    _check_rows(cfg, x, out)
    w = _weights_struct(weights)
    st = _stats_struct(stats)
    check(L.lib().moe_forward(C.byref(cfg), _p(x), _p(w_router), _p(router_bias), C.byref(w), _p(out),
                              _p(topk_ids), _p(topk_w), C.byref(st) if st is not None else None, _p(ws),
                              _nbytes(ws), _s(stream)), "moe_forward")


def moe_forward_few(cfg, x, w_router, router_bias, weights: dict, out, topk_ids, topk_w, stats, ws, stream=None):
    """``moe_forward`` for at most ``MOE_FEW_TOKENS`` tokens, in one kernel.
    Tensors whose type or size is not the config's are refused (ValueError):
    a batch of another size needs a config of its own."""
    if cfg.num_tokens <= L.MOE_FEW_TOKENS and cfg.act_dtype == L.MOE_BF16:      # (others are refused below)
        _on_current(x, w_router, router_bias, out, topk_ids, topk_w, ws, *weights.values(), *(stats or {}).values())
        _check_few(cfg, x, w_router, router_bias, weights, out, topk_ids, topk_w, stats)
    w = _weights_struct(weights)
    st = _stats_struct(stats)
    code = L.lib().moe_forward_few(C.byref(cfg), _p(x), _p(w_router), _p(router_bias), C.byref(w), _p(out),
                                   _p(topk_ids), _p(topk_w), C.byref(st) if st is not None else None, _p(ws),
                                   _nbytes(ws), _s(stream))
    if code == L.MOE_ERR_UNSUPPORTED:
        raise L.MoEError(code, "moe_forward_few: " + (L.lib().moe_last_error().decode() or "unsupported"))
    check(code, "moe_forward_few")


def moe_forward_host(cfg, x_host, w_router, router_bias, weights: dict, out_host, kept_counts_host,
                     prob_sum_host, dropped_host, ws, stream=None):
    w = _weights_struct(weights)
    check(L.lib().moe_forward_host(C.byref(cfg), _p(x_host), _p(w_router), _p(router_bias), C.byref(w),
                                   _p(out_host), _p(kept_counts_host), _p(prob_sum_host), _p(dropped_host),
                                   _p(ws), _nbytes(ws), _s(stream)), "moe_forward_host")


# ---------------------------------------------------------------- convenience holder

@dataclass
class Outputs:
    out: torch.Tensor
    topk_ids: torch.Tensor
    topk_w: torch.Tensor
    raw_counts: torch.Tensor
    kept_counts: torch.Tensor
    prob_sum: torch.Tensor
    dropped: torch.Tensor


class MoELayer:
    """Holds a config, device-resident weights, a workspace and output buffers,
    and runs ``moe_forward`` on them."""

    def __init__(self, cfg: moe_config, w_router: torch.Tensor, weights: dict,
                 router_bias: Optional[torch.Tensor] = None, device=None):
        status = moe_validate(cfg)
        check(status, "moe_validate")
        self.cfg = cfg
        self.device = torch.device(device) if device is not None else w_router.device
        self.w_router = w_router
        self.router_bias = router_bias
        self.weights = weights
        self.ws = torch.empty(moe_workspace_size(cfg), dtype=torch.uint8, device=self.device)
        T, k, E, d = cfg.num_tokens, cfg.top_k, cfg.num_experts, cfg.hidden
        dt = _TORCH_DT[cfg.act_dtype]
        i32 = dict(dtype=torch.int32, device=self.device)
        self.o = Outputs(out=torch.empty((T, d), dtype=dt, device=self.device),
                         topk_ids=torch.empty((T, k), **i32),
                         topk_w=torch.empty((T, k), dtype=torch.float32, device=self.device),
                         raw_counts=torch.empty(E, **i32), kept_counts=torch.empty(E, **i32),
                         prob_sum=torch.empty(E, dtype=torch.float32, device=self.device),
                         dropped=torch.empty(4, **i32))

    def stats(self) -> dict:
        o = self.o
        return dict(raw_counts=o.raw_counts, kept_counts=o.kept_counts, prob_sum=o.prob_sum, dropped=o.dropped)

    def forward(self, x: torch.Tensor, stream=None, forced_ids: Optional[torch.Tensor] = None) -> Outputs:
        """One layer forward.  ``forced_ids`` [T, k] int32 replays recorded
        expert choices (router replay): the stages then run one by one, with
        moe_route_forced in place of the router.  Bad recorded ids surface, as
        in moe_forward, through ``status()`` (the dispatch flags them too)."""
        o = self.o
        if forced_ids is None:
            moe_forward(self.cfg, x, self.w_router, self.router_bias, self.weights, o.out, o.topk_ids,
                        o.topk_w, self.stats(), self.ws, stream)
            return o
        cfg = self.cfg
        _check_rows(cfg, x, o.out)
        T, k, d = cfg.num_tokens, cfg.top_k, cfg.hidden
        _holds((("forced_ids", forced_ids, torch.int32, T * k),))
        if not hasattr(self, "_stage"):
            i32 = dict(dtype=torch.int32, device=self.device)
            dt = _TORCH_DT[cfg.act_dtype]
            self._stage = dict(off=torch.empty(cfg.num_experts + 1, **i32), perm_token=torch.empty(T * k, **i32),
                               perm_w=torch.empty(T * k, dtype=torch.float32, device=self.device),
                               slot_row=torch.empty((T, k), **i32),
                               x_perm=torch.empty((T * k, d), dtype=dt, device=self.device),
                               y_perm=torch.empty((T * k, d), dtype=dt, device=self.device),
                               shared=torch.empty((T, d), dtype=dt, device=self.device)
                               if cfg.shared_intermediate > 0 else None)
        st = self._stage
        moe_route_forced(cfg, x, self.w_router, self.router_bias, forced_ids, o.topk_ids, o.topk_w, o.prob_sum,
                         self.ws, stream)
        moe_permute(cfg, x, o.topk_ids, o.topk_w, st["off"], st["perm_token"], st["perm_w"], st["slot_row"],
                    st["x_perm"], self.stats(), self.ws, stream)
        moe_grouped_ffn(cfg, st["x_perm"], st["off"], self.weights, st["y_perm"], self.ws, stream)
        if st["shared"] is not None:
            moe_shared_expert(cfg, x, self.weights, st["shared"], self.ws, stream)
        moe_combine(cfg, st["y_perm"], st["slot_row"], o.topk_w, st["shared"], o.out, stream)
        return o

    def forward_few(self, x: torch.Tensor, stream=None) -> Outputs:
        """One layer forward in a single kernel, for layers of at most
        ``MOE_FEW_TOKENS`` tokens (moe_forward_few)."""
        o = self.o
        moe_forward_few(self.cfg, x, self.w_router, self.router_bias, self.weights, o.out, o.topk_ids, o.topk_w,
                        self.stats(), self.ws, stream)
        return o

    def update_bias(self, coeff: float, stream=None) -> None:
        """Aux-loss-free balancing step on ``router_bias`` from the last
        forward's raw per-expert counts (moe_update_bias)."""
        if self.router_bias is None:
            raise ValueError("update_bias needs a router_bias tensor")
        moe_update_bias(self.cfg, self.o.raw_counts, self.router_bias, coeff, stream)

    def status(self, stream=None) -> int:
        return moe_workspace_status(self.ws, stream)
